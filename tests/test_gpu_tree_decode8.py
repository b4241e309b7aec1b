"""The example with a cache in 8 bits and the rotating calls: that it runs, and leaves the pool in order.  GPU."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("tree", [True, False])
def test_a_cache_in_eight_bits(dtype, tree):
    import tree_decode

    r = tree_decode.run(requests=4, document=300, tokens=40, tree=tree, dtype=dtype, cache8=True)
    assert r["status"] == (0, 0) and all(len(t) == 40 for t in r["tokens"])
    refs = r["decoder"].cache.refs.tolist()
    assert all(refs[:r["used"]]) and not any(refs[r["used"]:])
    scale = r["decoder"].pool.scale
    assert bool((scale > 0).all()) and bool(torch.isfinite(scale).all())
