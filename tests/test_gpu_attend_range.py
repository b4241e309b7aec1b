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


def tree(seed, D, kind, scale, most=2, times=1.0, **kw):
    kw = {**dict(B=2, N=4, ctx=[700, 131], G=2, Hkv=1, P=32, nodes=[4, 3]), **kw}
    t = Tree(seed, D=D, kind=kind, scale=scale, **kw)
    whole(t.q, most, seed, times)
    whole(t.k, most, seed + 1, times)
    whole(t.pool[0], most, seed + 2, times)
    return t


def prompt(seed, D, kind, scale, most=2, times=1.0, lens=(300, 20), ctx=(200, 0)):
    p = Prompt(seed, list(lens), 2, 1, D, kind, ctx=list(ctx), P=32)
    p.scale = scale
    whole(p.q, most, seed, times)
    whole(p.k, most, seed + 1, times)
    whole(p.pool[0], most, seed + 2, times)
    return p


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("D", [64, 128, 40])
@pytest.mark.parametrize("scale", [1e-19, 1e3, 1e6, 1e9, 1e19])
def test_scales_of_every_size(scale, D, kind):
    """Uniform weights at one end, the largest scores alone (ties among them) at the other."""
    tree(30, D, kind, scale).run().check()
    prompt(31, D, kind, scale).run().check(rows=25)


@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("D", [64, 128])
def test_queries_and_keys_in_the_thousands(D, kind):
    tree(32, D, kind, 1.0, times=1000.0).run().check()
    prompt(33, D, kind, 1.0, times=1000.0).run().check(rows=25)


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
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("step", [0.0, 3.0, 9.0, -5.0])
@pytest.mark.parametrize("offset", [2.0 ** 22, -2.0 ** 22, 2.0 ** 14])
def test_maxima_that_rise_far_from_zero(offset, step, D, kind):
    """A reference that changes from tile to tile, between the streams and between the parts of an item."""
    t = Tree(34, 2, 4, [1300, 190], 2, 1, D, 32, kind, nodes=[4, 4], scale=1.0)
    far(t.q, t.k, t.pool[0], offset)
    t.q[:, 1, 0, 0] = -1.0
    t.q[:, 2, 1, 0] = 0.0
    for s in range(2):
        levels(t.cache, t.pool, s, t.by_slot[s], 32, step)
    t.run().check()
    p = Prompt(35, [150, 300], 2, 1, D, kind, ctx=[900, 33], P=32)
    p.scale = 1.0
    far(p.q, p.k, p.pool[0], offset)
    for s in range(2):
        levels(p.cache, p.pool, s, p.by_slot[s], 32, step)
    p.run().check(rows=12)


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("D", [64, 128])
def test_parts_are_joined_far_from_zero(D, kind):
    """One request's keys in many CTAs: the parts' references differ by a few, and lie in the millions."""
    t = Tree(36, 1, 16, [12011], 4, 1, D, 64, kind, nodes=[16], scale=1.0)
    far(t.q, t.k, t.pool[0], 2.0 ** 22)
    levels(t.cache, t.pool, 0, 12011, 64, 1.0, tile=1024)
    t.run().check()
    p = Prompt(37, [5], 4, 1, D, kind, ctx=[9003], P=64)
    p.scale = 1.0
    far(p.q, p.k, p.pool[0], 2.0 ** 22)
    levels(p.cache, p.pool, 0, 9003, 64, 1.0, tile=1024)
    p.run().check()


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
