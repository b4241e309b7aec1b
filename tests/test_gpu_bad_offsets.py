"""A packing offset that falls or lies outside concerns its own request alone:
the requests before and behind it are served.  GPU."""
import numpy as np
import pytest
import torch

import context_lookup_speculative_gb300 as clk
from test_gpu_attend import Prompt
from test_gpu_cache import Both, ints

pytestmark = pytest.mark.gpu


def append_packed(c, slots, off, rows, good):
    """Counts are the requests' rows; those of the positions in `good` are written."""
    counts = [off[b + 1] - off[b] if b in good else 3 for b in range(len(slots))]
    assert c.grow(slots, counts) == []
    marks = np.arange(c.mark, c.mark + rows)
    c.mark += rows
    k, v = (torch.from_numpy(np.stack([c.value(marks, 2 * l + x) for l in range(c.layers)])).to("cuda", c.dt) for x in (0, 1))
    clk.cache_append(c.h, ints(slots), c.pool, k, v, ints(counts), offsets=ints(off, torch.int64))
    c.m.append([slots[b] for b in good], [[int(marks[off[b] + i]) for i in range(counts[b])] for b in good])


@pytest.mark.parametrize("layers", [1, 9])
@pytest.mark.parametrize("off,rows,good", [
    ([0, 1000000, 10, 20], 20, [2]),                            # past the end, then falling
    ([0, 5, 100, 12, 20, 18, 30], 33, [0, 3, 5]),               # valid ones between, two of which share rows
    ([-3, 4, 9, -1, 2, 40, 33, 33, 39], 40, [1, 4, 6, 7]),      # before the start
    ([7, 0, 8, 8, 1 << 40, 8, 20], 25, [1, 2, 5]),
    ([30, 20, 10, 0, 3], 30, [3]),
])
def test_packed_rows_around_a_bad_offset(off, rows, good, layers):
    B = len(off) - 1
    c = Both(B + 2, 5, 60, 16, layers=layers, heads=2)
    slots = list(range(B, 0, -1))
    append_packed(c, slots, off, rows, good)
    c.check(status=clk.EINVAL)
    assert c.h.status()[1] in [slots[b] for b in range(B) if b not in good]


def test_many_packed_requests_around_a_bad_offset():
    """More requests than a CTA has threads, more rows than a CTA moves at once."""
    rng = np.random.default_rng(0)
    n = rng.integers(0, 40, size=600)
    off = np.concatenate([[0], np.cumsum(n)])
    rows = int(off[-1])
    off = off.tolist()
    for at in (3, 250, 599):
        off[at] = rows + 5
    good = [b for b in range(600) if b not in (2, 3, 249, 250, 598, 599)]
    c = Both(600, 3, 2000, 16, heads=1)
    append_packed(c, list(range(600)), off, rows, good)
    c.check(status=clk.EINVAL)


def around(seed, lens, bad, off, G, D, kind, ctx=None, tail=4):
    """Prompts of `lens` rows whose requests `bad` are empty; `off` is what the call is given."""
    p = Prompt(seed, lens, G, 1, D, kind, ctx=ctx, tail=tail)
    good = list(p.off)
    assert all(lens[b] == 0 for b in bad)
    assert all(off[b:b + 2] == good[b:b + 2] for b in range(len(lens)) if b not in bad)
    p.off = off
    p.run()
    torch.cuda.synchronize()
    if p.kw:
        assert p.cache.status()[0] == clk.EINVAL
        p.cache.status_clear()
    p.off = good
    p.check(rows=15)


@pytest.mark.parametrize("kind,D", [("f32", 40), ("f32", 128), ("bf16", 200), ("bf16", 64), ("f16", 128)])
@pytest.mark.parametrize("G", [1, 3, 40])
def test_prompts_around_a_bad_offset(G, kind, D):
    around(1, [0, 0, 10], [0, 1], [0, 1000000, 0, 10], G, D, kind)
    around(2, [5, 0, 0, 7, 0, 0, 8], [1, 2, 4, 5], [0, 5, 1000, 5, 12, -4, 12, 20], G, D, kind)
    around(3, [70, 0, 0, 90, 0, 0, 1], [1, 2, 4, 5], [0, 70, 1 << 40, 70, 160, -1, 160, 161], G, D, kind, ctx=[0, 0, 0, 130, 5, 0, 33])


@pytest.mark.parametrize("kind,D", [("f32", 40), ("bf16", 64)])
def test_many_prompts_around_a_bad_offset(kind, D):
    rng = np.random.default_rng(1)
    lens = rng.integers(0, 30, size=700)
    bad = (0, 1, 99, 100, 400, 401, 698, 699)
    lens[list(bad)] = 0
    off = np.concatenate([[0], np.cumsum(lens)]).tolist()
    T = off[-1] + 4
    for at, x in ((1, T + 3), (100, -1), (401, 1 << 33), (699, -7)):
        off[at] = x
    around(4, lens.tolist(), bad, off, 2, D, kind)
