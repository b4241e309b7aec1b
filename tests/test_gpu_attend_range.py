"""Attention where scores are large beside their differences, against 64 bits.
Queries and keys are whole numbers, so that every score is exact in float32 and
the softmax of scores in the millions is well defined: the tolerances are
those of cache_model.tolerance.  GPU."""
import math

import pytest
import torch

from test_gpu_attend import Prompt, Tree

pytestmark = pytest.mark.gpu


def whole(x, most, seed, times=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x.copy_((torch.randint(-most, most + 1, x.shape, generator=g, device="cuda") * times).to(x.dtype))


def far(q, k, pools, offset):
    """Every score is the offset and a small whole number; cached keys add the level that `levels` gives them."""
    for x, most in ((q, 1), (k, 1), (pools, 1)):
        whole(x, most, 40)
    q[..., 0], q[..., 1] = 1.0, math.copysign(2048.0, offset)
    k[..., 0], k[..., 1] = 0.0, abs(offset) / 2048
    pools[..., 0], pools[..., 1] = 0.0, abs(offset) / 2048


def levels(cache, pool, slot, n, P, step, tile=128):
    for i in range(-(-n // P)):
        pool[0, cache.table[slot, i].long(), :, :, 0] = step * (i * P // tile)


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("D", [40, 64])
@pytest.mark.parametrize("step", [16.0, 100.0, 240.0])
def test_tiles_that_are_computed_again(step, D, kind):
    """Rows of up to 64 look for a tile's maximum after its weights have grown too large: here in every tile of every
    row, by more than a weight's type can hold, so that each tile's weights are replaced before they are used."""
    t = Tree(38, 3, 5, [1200, 640, 0], 4, 2, D, 32, kind, nodes=[5, 5, 2], scale=1.0)
    far(t.q, t.k, t.pool[0], 0.0)
    for s in range(3):
        levels(t.cache, t.pool, s, t.by_slot[s], 32, step)
    t.run().check()
    p = Prompt(39, [140, 300], 4, 2, D, kind, ctx=[1000, 520], P=32)
    p.scale = 1.0
    far(p.q, p.k, p.pool[0], 0.0)
    for s in range(2):
        levels(p.cache, p.pool, s, p.by_slot[s], 32, step)
    p.run().check(rows=12)
