"""The example's decode loop: trees give the tokens that single steps give, in
fewer steps, and leave a sound cache.  float32, where near ties of the
target's answers are out of rounding's reach.  GPU."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("seed", [0, 1])
def test_trees_decode_what_single_steps_decode(seed):
    import tree_decode

    a = tree_decode.run(requests=3, document=150, tokens=48, tree=True, dtype=torch.float32, seed=seed)
    b = tree_decode.run(requests=3, document=150, tokens=48, tree=False, dtype=torch.float32, seed=seed)
    assert a["tokens"] == b["tokens"]
    assert a["status"] == b["status"] == (0, 0)
    assert a["steps"] < b["steps"] == 47
    for r in (a, b):
        d = r["decoder"]
        refs = d.cache.refs.tolist()
        # after compaction the pages in use are the lowest ones, and the tables name exactly those
        assert all(refs[:r["used"]]) and not any(refs[r["used"]:])
        held = d.cache.table[d.cache.table >= 0]
        assert sorted(set(held.tolist())) == list(range(r["used"])) and held.numel() == sum(refs)


def test_sixteen_bits():
    import tree_decode

    r = tree_decode.run(requests=4, document=300, tokens=40)
    assert r["status"] == (0, 0) and all(len(t) == 40 for t in r["tokens"])
