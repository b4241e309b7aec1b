"""Attention over a cache in 8 bits with rows that end inside a vector of 16 elements, in pools whose rows begin on
one: every row's elements, and nothing behind the last row.  GPU."""
import pytest
import torch

from test_gpu_attend import DT, NAN
from test_gpu_attend8 import Prompt8, Tree8

pytestmark = pytest.mark.gpu
BEHIND = 4096  # elements


def inside(case):
    """The case's out becomes the middle of a larger buffer of sevens; returns a look at what lies around it."""
    n = case.out.numel()
    whole = torch.full((n + 2 * BEHIND,), 7.0, dtype=case.out.dtype, device="cuda")
    case.out = whole[BEHIND:BEHIND + n].view(case.out.shape)
    case.out.fill_(NAN)

    def untouched():
        torch.cuda.synchronize()
        return bool((whole[:BEHIND] == 7).all()) and bool((whole[BEHIND + n:] == 7).all())

    return untouched


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("D", [8, 24, 40, 56, 72, 88, 104, 120])
def test_trees(D, kind):
    """Uncut items, cut ones, and a last request that ends the buffer."""
    assert DT[kind].itemsize == 2
    for seed, ctx, G, nodes in ((1, [70, 0, 129], 2, [5, 3, 5]), (2, [9000, 5], 4, [5, 5]), (3, [300] * 40, 1, [5] * 40)):
        t = Tree8(D + seed, len(ctx), 5, ctx, G, 2, D, 16, kind, nodes=nodes, pad8=8)
        untouched = inside(t)
        t.run().check(only=None if len(ctx) < 9 else [0, 17, 39])
        assert untouched()


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("D", [8, 24, 40, 56, 72, 88, 104, 120])
def test_prompts(D, kind):
    for seed, lens, ctx in ((1, [70, 1, 0, 33], [0, 30, 20, 140]), (2, [40], [5000])):
        p = Prompt8(D + seed, lens, 2, 2, D, kind, ctx=ctx, pad8=8)
        untouched = inside(p)
        p.run().check(rows=12)
        assert untouched()
