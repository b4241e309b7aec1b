"""Attention over a cache in 8 bits whose values lie at the end of the inputs' type, or past it: float16 rows at the top
of their range are appended as codes of up to 448 with the scale 256, so that 65,504 stands for 65,536, and rotated keys
for up to 92,681 and more.  Against 64 bits over what the cache holds, with the tolerances of cache_model.tolerance.  GPU."""
import math

import pytest
import torch

import context_lookup_speculative_gb300 as clk
from test_gpu_attend import DT, ints
from test_gpu_attend8 import Prompt8, Tree8

pytestmark = pytest.mark.gpu
TOP = 65504.0


def stands(pool):
    T = pool.data.shape[3] // pool.scale.shape[3]
    return (pool.data.double().unflatten(3, (-1, T)) * pool.scale[..., None, None].double()).flatten(3, 4)


def append_top(case, lens, rotated, seed):
    """Every cached row again, by an append: keys of the size of float16's largest, values of size one and here and there
    the largest.  Scores are of size one with the softmax's scale below."""
    Hkv, D = case.Hkv, case.D
    g = torch.Generator(device="cuda").manual_seed(seed)
    k = torch.randn((sum(lens), Hkv, D), generator=g, device="cuda").mul_(TOP).clamp_(-TOP, TOP).half()
    v = torch.randn((sum(lens), Hkv, D), generator=g, device="cuda")
    pick = torch.rand(v.shape, generator=g, device="cuda")
    v = torch.where(pick < 0.03, TOP * v.sign(), torch.where(pick < 0.06, 63488.0 * v.sign(), v)).half()
    off = [0]
    for n in lens:
        off.append(off[-1] + n)
    rot = clk.Rotary.of(10000.0 ** (-torch.arange(D // 2) / (D // 2)), max(lens) + 1) if rotated else None
    clk.cache_append_rotary(case.cache, ints(case.slots.tolist()), case.pool8, k[None], v[None], ints(lens), rotary=rot,
                            offsets=ints(off, torch.int64))
    case.pool = stands(case.pool8)
    held = torch.cat([case.pool[1][case.cache.table[int(s), :-(-n // case.P)].long()].transpose(1, 2).flatten(0, 1)[:n]
                      for s, n in zip(case.slots, lens)])
    assert float(held.abs().max()) == 65536.0
    case.scale = 1 / (TOP * math.sqrt(D))
    return case


def prompts(kind, D, rotated, pad8, **kw):
    for lens, ctx, P in (([70, 1, 33], [130, 20, 400], 16), ([40], [3000], 64)):
        p = Prompt8(D + P, lens, 2, 2, D, kind, ctx=ctx, P=P, pad8=pad8, **kw)
        append_top(p, ctx, rotated, D).run().check(rows=15)


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("rotated", [False, True])
@pytest.mark.parametrize("D,pad8", [(64, 3), (128, 1), (40, 0), (256, 0)])
def test_rows_at_the_top_in_the_general_kernel(D, pad8, rotated, kind):
    t = Tree8(D, 2, 4, [300, 33], 2, 2, D, 16, kind, nodes=[4, 4], pad8=pad8)
    append_top(t, t.ctx, rotated, D).run().check()
    prompts(kind, D, rotated, pad8)


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("rotated", [False, True])
@pytest.mark.parametrize("D,pad8", [(64, 0), (128, 0), (40, 8), (96, 0)])
def test_trees_over_rows_at_the_top(D, pad8, rotated, kind):
    t = Tree8(D, 2, 4, [300, 33], 2, 2, D, 16, kind, nodes=[4, 4], pad8=pad8)
    append_top(t, t.ctx, rotated, D).run().check()


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("D", [64, 40])
def test_the_general_kernel_does_not_round_what_the_cache_holds(D, kind):
    """Scales that are no powers of two: with products in float32 the tolerances need no term for it."""
    Tree8(1, 3, 6, [300, 20, 129], 3, 2, D, 64, kind, nodes=[6, 6, 6], T=32, odd=True, pad8=3).run().check()
    Prompt8(2, [40, 200], 3, 2, D, kind, ctx=[300, 20], P=64, T=64, odd=True, pad8=1).run().check(rows=15)


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("rotated", [False, True])
@pytest.mark.parametrize("D,pad8", [(64, 0), (128, 0), (40, 8), (96, 0)])
def test_prompts_over_rows_at_the_top(D, pad8, rotated, kind):
    prompts(kind, D, rotated, pad8)


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lens,ctx,P,T", [([200, 3], [700, 129], 32, 32), ([60], [5000], 64, 16), ([300, 20, 7], [257, 1500, 128], 128, 128)])
def test_prompts_over_values_past_the_type(lens, ctx, P, T, D, kind):
    """Blocks of keys and values of up to 229,376 beside blocks of size one, changing from tile to tile, in items that are
    whole and in parts.  Codes are multiples of 2^-9 and scales 2^-8 or more, so that float16 holds the values times 2^-2."""
    p = Prompt8(D + P, lens, 3, 2, D, kind, ctx=ctx, P=P, T=T)
    g = torch.Generator(device="cuda").manual_seed(D)
    pages = p.pool8.scale.shape[1]
    for x in (0, 1):
        big = torch.rand((pages, 1, 1), generator=g, device="cuda") < (0.3 if P < 128 else 0.5)
        high = torch.exp2(torch.randint(7, 10, p.pool8.scale[x].shape, generator=g, device="cuda").float())
        p.pool8.scale[x] = torch.where(big, high, p.pool8.scale[x])
    p.pool = stands(p.pool8)
    assert float(p.pool.abs().max()) > 2 * TOP
    p.scale = 1 / (2.0 ** 9 * 100 * math.sqrt(D))
    p.run().check(rows=15)


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("plane,exponent", [(0, 8), (1, 8), (0, 40)])
def test_keys_or_values_past_the_type(plane, exponent, D, kind):
    """One of the two alone, in one block of a long prefix; keys of 2^40 times the others, whose scores hardly count then."""
    p = Prompt8(D + exponent, [50, 130], 4, 1, D, kind, ctx=[4001, 600], P=64, T=32)
    for slot, n in zip(p.slots, (4001, 600)):
        for page in p.cache.table[int(slot), :-(-n // 64)].tolist()[1::7]:
            p.pool8.scale[plane, page, :, 0] = 2.0 ** exponent
    p.pool = stands(p.pool8)
    p.scale = 1 / math.sqrt(D) if plane else 1 / (2.0 ** exponent * 100 * math.sqrt(D))
    p.run().check(rows=15)
