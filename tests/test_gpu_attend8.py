"""Attention over a cache in 8 bits against 64 bits, row by row, over the values
that its codes and scales stand for.  The tolerances are those of
cache_model.tolerance where scales are powers of two: a cached value is exact
in the inputs' type.  GPU."""
import numpy as np
import pytest
import torch

import context_lookup_speculative_gb300 as clk
from cache_model import UNIT, masks_of, tolerance
from test_gpu_attend import DT, INF, NAN, Prompt, Tree, f64, ints

pytestmark = pytest.mark.gpu


def eight(x, T, seed, pad=0, odd=False):
    """x's pool in 8 bits: codes of x times a power of two (or, odd, any factor) from block to block; and what they stand for."""
    planes, pages, heads, P, D = x.shape
    g = torch.Generator(device="cuda").manual_seed(seed)
    raw = torch.empty((planes, pages, heads, P, D + pad), dtype=torch.float8_e4m3fn, device="cuda")
    data = raw[..., :D]
    data.copy_((x.float() * 100).clamp(-448, 448).to(torch.float8_e4m3fn))
    scale = torch.exp2(torch.randint(-8, -4, (planes, pages, heads, P // T), generator=g, device="cuda").float())
    if odd:
        scale = scale * (1 + torch.rand(scale.shape, generator=g, device="cuda"))
    stands = (data.double().unflatten(3, (P // T, T)) * scale[..., None, None].double()).flatten(3, 4)
    return clk.ScaledPool(data, scale), stands if odd else stands.to(x.dtype)


class Tree8(Tree):
    def __init__(self, seed, *a, T=16, odd=False, pad8=0, **kw):
        super().__init__(seed, *a, **kw)
        self.pool8, self.pool = eight(self.pool, T, seed, pad8, odd)

    def run(self):
        clk.tree_attend(self.cache, ints(self.slots.tolist()), self.pool8, self.layer, self.q, self.k, self.v, ints(self.nodes),
                        self.dmask, self.scale, self.out, self.scratch, ctx=None if self.ctx is self.lens else ints(self.ctx))
        return self


class Prompt8(Prompt):
    def __init__(self, seed, *a, T=16, odd=False, pad8=0, **kw):
        super().__init__(seed, *a, **kw)
        self.pool8, self.pool = eight(self.pool, T, seed, pad8, odd)
        self.kw["pool"] = self.pool8


@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("D", [64, 128, 16, 48, 80, 96, 112, 8, 256, 33, 1])
def test_types_and_dims(kind, D):
    Tree8(D, 3, 5, [70, 0, 129], 2, 2, D, 16, kind, nodes=[5, 3, 1]).run().check()
    Prompt8(D, [70, 1, 0, 33], 2, 2, D, kind, ctx=[0, 30, 20, 140]).run().check(rows=12)


@pytest.mark.parametrize("P,T", [(16, 16), (32, 16), (32, 32), (64, 16), (64, 32), (64, 64), (128, 16), (128, 32), (128, 64), (128, 128)])
@pytest.mark.parametrize("n", [1, 15, 16, 17, 63, 64, 65, 127, 128, 129, 255, 257, 385, 1000])
def test_context_lengths_pages_and_blocks(P, T, n):
    for kind, D in (("bf16", 128), ("f16", 64)):
        Tree8(n + P, 2, 4, [n, max(0, n - 1)], 4, 1, D, P, kind, nodes=[4, 2], T=T).run().check()


@pytest.mark.parametrize("G", [1, 2, 3, 4, 5, 6, 8, 16, 48, 128, 130])
def test_head_groups(G):
    Tree8(G, 2, 3, [200, 37], G, 2 if G < 12 else 1, 64, 32, "bf16", nodes=[3, 2]).run().check()
    Prompt8(G, [40, 50], G, 2 if G < 8 else 1, 128, "bf16", ctx=[140, 30]).run().check(rows=8)


@pytest.mark.parametrize("N", [1, 2, 15, 16, 17, 32, 33, 63, 64])
@pytest.mark.parametrize("G,D", [(1, 64), (4, 128), (6, 64)])
def test_tree_sizes(N, G, D):
    Tree8(N * G, 3, N, [150, 300, 3], G, 1, D, 64, "f16", nodes=[N, max(1, N // 2), 0]).run().check()


@pytest.mark.parametrize("B", [1, 7, 33, 200])
def test_ragged_batches(B):
    rng = np.random.default_rng(B)
    for D, kind in ((64, "bf16"), (128, "f16")):
        t = Tree8(B, B, 3, rng.integers(0, 700, size=B).tolist(), 2, 2, D, 16, kind).run()
        t.check(only=range(0, B, max(1, B // 12)))


def test_many_requests():
    B = 1500
    rng = np.random.default_rng(0)
    t = Tree8(11, B, 2, rng.integers(0, 90, size=B).tolist(), 2, 1, 64, 16, "bf16").run()
    t.check(only=rng.permutation(B)[:40].tolist() + [0, B - 1])


@pytest.mark.parametrize("D,kind", [(128, "bf16"), (64, "f16"), (64, "bf16"), (128, "f16")])
def test_a_long_context_is_split_and_joined(D, kind):
    Tree8(D, 1, 16, [20011], 4, 1, D, 64, kind, nodes=[16]).run().check()
    Tree8(D, 2, 1, [9000, 1], 8, 2, D, 128, kind, nodes=[1, 1], T=128).run().check()


@pytest.mark.parametrize("kind,D", [("bf16", 128), ("f16", 64), ("f16", 128), ("bf16", 48), ("f32", 40)])
def test_scales_of_any_size(kind, D, monkeypatch):
    """Scales that are no powers of two: a cached element may be rounded to the type, by half a step u relative.  A
    score then is off by at most u a, a the largest sum of |q k| scale over a row's keys, a weight by exp(2 u a) - 1,
    and a value by u.  For normal q (times 1, the mean of |x| is 0.8) and k of size one a is about 0.64 sqrt(D), and
    its largest over these rows below 1.5 times that."""
    import test_gpu_attend

    u = UNIT[kind]
    more = np.expm1(2 * u * 1.5 * 0.64 * np.sqrt(D)) + u

    def looser(kind, ref, size, keys, vmax):
        return tolerance(kind, ref, size, keys, vmax) + more * size

    monkeypatch.setattr(test_gpu_attend, "tolerance", looser)
    Tree8(1, 3, 6, [300, 20, 129], 3, 2, D, 64, kind, nodes=[6, 6, 6], T=32, odd=True).run().check()
    Prompt8(2, [40, 200], 3, 2, D, kind, ctx=[300, 20], P=64, T=64, odd=True).run().check(rows=15)


def test_scales_far_from_one():
    """Blocks that hardly count beside others, and blocks of zeros with the least scale."""
    for kind in ("bf16", "f16"):
        t = Tree8(3, 2, 4, [500, 130], 2, 1, 64, 32, kind, nodes=[4, 4])
        low = 2.0 ** -13 if kind == "f16" else 2.0 ** -60
        t.pool8.scale[:, ::2] = low
        t.pool8.scale[:, 1::3] = 2.0 ** -120
        data = t.pool8.data.view(torch.uint8)
        data[:, 1::3] = 0
        s = t.pool8.scale[..., None].expand(-1, -1, -1, -1, 16).flatten(3)[..., None]
        t.pool = (t.pool8.data.float() * s).to(DT[kind])
        t.run().check()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lo,hi,odd", [(-100, 60, False), (-100, -100, False), (40, 60, False), (-60, 30, False), (-40, 40, True)])
def test_v_scales_far_apart(lo, hi, odd, D, monkeypatch):
    """V's scales from 2^lo to 2^hi within a request (odd: no powers of two, some negative).  A weight times its scale
    is rounded to float16, by half a step of 2^-24 at least where the largest is 2^5 or more: over all keys at most
    keys * 2^-30 * 448 times the largest scale."""
    import test_gpu_attend

    t = Tree8(abs(D + hi), 2, 5, [700, 260], 3, 2, D, 32, "bf16", nodes=[5, 2], T=16)
    g = torch.Generator(device="cuda").manual_seed(hi)
    v = t.pool8.scale[1]
    v.copy_(torch.exp2(torch.randint(lo, hi + 1, v.shape, generator=g, device="cuda").float()))
    if odd:
        v.mul_(torch.rand(v.shape, generator=g, device="cuda") * 2.5 - 1)
    t.pool = (t.pool8.data.double().unflatten(3, (2, 16)) * t.pool8.scale[..., None, None].double()).flatten(3, 4)
    more = 2.0 ** -30 * 448 * float(v.abs().max())
    monkeypatch.setattr(test_gpu_attend, "tolerance", lambda kind, ref, size, keys, vmax: tolerance(kind, ref, size, keys, vmax) + keys * more)
    t.k.mul_(4)
    t.run().check()


@pytest.mark.parametrize("first,then", [(-100, 60), (60, -100), (-100, 90), (90, -60)])
@pytest.mark.parametrize("D,n", [(64, 700), (128, 700), (64, 5000), (128, 5000)])
def test_v_scales_that_change_along_the_context(first, then, D, n, monkeypatch):
    """The first half of a context's V has scales of 2^first, the other of 2^then: tiles, streams and parts of one row with
    references far apart, whose sums of weights count alike.  Tolerance as for scales far apart."""
    import test_gpu_attend

    t = Tree8(D + n, 2, 3, [n, 130], 4, 1, D, 64, "bf16", nodes=[3, 1], T=64)
    for s, length in enumerate([n, 130]):
        slot = int(t.slots[s])
        pages = t.cache.table[slot, :-(-length // 64)].long()
        half = len(pages) // 2
        t.pool8.scale[1][pages[:half]] = 2.0 ** first
        t.pool8.scale[1][pages[half:]] = 2.0 ** then
    t.pool = (t.pool8.data.double() * t.pool8.scale[..., None].double())
    more = 2.0 ** -30 * 448 * 2.0 ** max(first, then)
    monkeypatch.setattr(test_gpu_attend, "tolerance", lambda kind, ref, size, keys, vmax: tolerance(kind, ref, size, keys, vmax) + keys * more)
    t.run().check()


def test_large_scores():
    for kind, D in (("bf16", 64), ("f16", 128)):
        t = Tree8(5, 2, 4, [700, 300], 2, 1, D, 16, kind, nodes=[4, 4], amp=8.0)
        t.pool8.scale[0].mul_(torch.exp2(torch.arange(t.pool.shape[1], device="cuda") % 3 - 1.0).view(-1, 1, 1))
        s = t.pool8.scale[..., None].expand(-1, -1, -1, -1, 16).flatten(3)[..., None]
        t.pool = (t.pool8.data.float() * s).to(DT[kind])
        t.run().check()
        Prompt8(7, [300], 2, 1, D, kind, ctx=[200], amp=10.0).run().check(rows=60)


@pytest.mark.parametrize("scale", [0.0, -0.1, 1.0])
def test_softmax_scales(scale):
    Tree8(7, 2, 4, [130, 20], 2, 1, 64, 16, "bf16", nodes=[4, 4], scale=scale).run().check()


def spoil8(pool, cache, held, codes, scale):
    """Rows that no slot's token holds become `codes`, scales of blocks without such rows `scale`."""
    P, T = cache.page_tokens, pool.data.shape[3] // pool.scale.shape[3]
    keep = torch.zeros((pool.data.shape[1], P), dtype=torch.bool, device="cuda")
    for s, n in enumerate(held):
        for i in range(-(-n // P)):
            keep[cache.table[s, i].long(), :min(P, n - i * P)] = True
    data = pool.data.view(torch.uint8)
    data.copy_(torch.where(keep[None, :, None, :, None], data, torch.tensor(codes, dtype=torch.uint8, device="cuda")))
    used = keep.unflatten(1, (P // T, T)).any(2)
    pool.scale.copy_(torch.where(used[None, :, None], pool.scale, torch.tensor(scale, device="cuda")))


@pytest.mark.parametrize("kind,D", [("bf16", 128), ("f16", 64), ("bf16", 64), ("f16", 128), ("f32", 40)])
@pytest.mark.parametrize("codes,scale", [(0x7f, NAN), (0xff, INF), (0x7e, 3e38), (0x7f, 1.0)])
def test_what_is_not_visible_is_not_counted(kind, D, codes, scale):
    """Rows past ctx, free pages, nodes past the count or off a row's mask hold NaN, infinities and the largest values."""
    N = 12
    base = [masks_of([-1] + list(range(N - 1)), N, N)] * 3
    mask = [[w & ~(1 << 5) & (~0 if n >= 9 else ~(1 << 7)) & (2 ** 64 - 1) for n, w in enumerate(row)] for row in base]
    t = Tree8(9, 3, N, [37, 130, 0], 3, 2, D, 32, kind, nodes=[N, 9, 7], mask=mask, lens=[80, 131, 20])
    held = [min(c, n) for c, n in zip([t.ctx[list(t.slots).index(s)] for s in range(3)], t.by_slot)]
    spoil8(t.pool8, t.cache, held, codes, scale)
    for b in range(3):
        for x in (t.k, t.v, t.q):
            x[b, t.nodes[b]:] = NAN
    t.k[:, 5] = NAN
    t.v[:, 5] = INF
    t.run().check()
    p = Prompt8(5, [33, 130, 7], 2, 1, D, kind, ctx=[20, 0, 100], lead=3, tail=9)
    spoil8(p.pool8, p.cache, p.by_slot, codes, scale)
    for x in (p.q, p.k, p.v):
        x[:3] = NAN
        x[p.off[-1]:] = NAN
    p.run().check()


@pytest.mark.parametrize("P", [16, 32, 64, 128])
def test_prompts_behind_cached_prefixes(P):
    for kind, D in (("bf16", 128), ("f16", 64)):
        Prompt8(P, [40, 1, 200, 0, 130, 64], 3, 2, D, kind, ctx=[0, 77, 130, 50, 1, 3 * P], P=P, T=P).run().check(rows=15)


def test_long_prompts():
    Prompt8(1, [1500, 37, 2300], 6, 2, 64, "f16", ctx=[100, 5000, 0], P=64, T=32).run().check(rows=25)
    Prompt8(2, [2011], 4, 1, 128, "bf16", ctx=[4099], P=64).run().check(rows=40)
    Prompt8(3, [3], 4, 1, 128, "bf16", ctx=[30003], P=64).run().check()


@pytest.mark.parametrize("D,kind", [(128, "bf16"), (64, "f16"), (40, "f32")])
def test_an_unaligned_pool(D, kind):
    Tree8(14, 2, 3, [50, 200], 2, 1, D, 16, kind, nodes=[3, 3], pad8=3).run().check()
    Prompt8(14, [30, 20], 2, 1, D, kind, ctx=[50, 20], pad8=1).run().check(rows=10)


@pytest.mark.parametrize("layer", [0, 2])
def test_layers_and_contexts_shorter_than_the_slot(layer):
    Tree8(12, 2, 4, [100, 45], 2, 3, 64, 16, "bf16", nodes=[4, 3], layers=3, layer=layer).run().check()
    Tree8(13, 3, 4, [10, 0, 99], 2, 1, 128, 32, "bf16", nodes=[4, 4, 4], lens=[90, 33, 99]).run().check()


def test_same_results_every_time():
    for kind, D in (("bf16", 128), ("f16", 64)):
        t = Tree8(16, 5, 6, [3000, 20, 500, 0, 1111], 4, 2, D, 64, kind).run()
        p = Prompt8(17, [300, 20, 1500], 4, 2, D, kind, ctx=[3000, 0, 129], P=64).run()
        torch.cuda.synchronize()
        first = t.out.clone(), p.out.clone()
        for _ in range(5):
            t.out.fill_(NAN)
            t.run()
            p.run()
            torch.cuda.synchronize()
            assert torch.equal(t.out, first[0]) and torch.equal(p.out, first[1])


def test_a_seen_nan_stays_in_its_rows():
    """A cached NaN reaches those rows only that see it; NaN beside it in new tokens too."""
    chain = [masks_of([-1, 0, 1, 2], 4, 4)] * 2
    for kind, D in (("bf16", 128), ("f16", 64)):
        t = Tree8(10, 2, 4, [70, 70], 2, 1, D, 16, kind, nodes=[4, 4], mask=chain)
        t.v[0, 2, 0, 3] = INF
        t.k[1, 3, 0, 0] = NAN
        t.run()
        torch.cuda.synchronize()
        out = t.out.float()
        assert torch.isfinite(out[0, :2]).all() and torch.isfinite(out[1, :3]).all()
        assert not torch.isfinite(out[0, 2:, :, 3]).any() and torch.isnan(out[1, 3]).all()
        t.out[0, 2:], t.out[1, 3] = 0, 0
        t.nodes = [2, 3]
        t.check()


def test_bad_requests_are_latched_and_give_zero():
    t = Tree8(17, 4, 3, [40, 40, 40, 40], 2, 1, 64, 16, "bf16", nodes=[3, 4, 3, -1])
    t.ctx = [40, 40, 41, 40]
    t.run()
    torch.cuda.synchronize()
    assert t.cache.status()[0] == clk.EINVAL
    assert (t.out[1:] == 0).all()
    t.cache.status_clear()
    t.check(only=[0])


def test_captured_and_on_another_stream():
    for D, kind in ((128, "bf16"), (64, "f16")):
        t = Tree8(18, 3, 4, [300, 20, 1500], 2, 2, D, 64, kind, nodes=[4, 4, 4])
        slots, nodes = ints(t.slots.tolist()), ints(t.nodes)

        def call():
            clk.tree_attend(t.cache, slots, t.pool8, 0, t.q, t.k, t.v, nodes, t.dmask, t.scale, t.out, t.scratch)

        torch.cuda.synchronize()
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            call()
        s.synchronize()
        first = t.out.clone()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call()
        t.out.fill_(NAN)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(t.out, first)


def test_an_append_then_an_attention():
    """Rows rotated and appended in 8 bits, then read by the next tokens: the calls together."""
    B, Hq, Hkv, D, P, dt = 2, 4, 2, 64, 32, torch.bfloat16
    h = clk.Cache(B, 8, 16, P)
    pool = clk.ScaledPool.empty(1, 16, Hkv, P, D, block=16)
    rot = clk.Rotary.of(10000.0 ** (-torch.arange(32) / 32.0), 256)
    slots, lens = ints([1, 0]), [70, 33]
    g = torch.Generator(device="cuda").manual_seed(3)
    qkv = torch.empty((sum(lens), Hq + 2 * Hkv, D), dtype=dt, device="cuda").normal_(generator=g)
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    off = ints([0, 70, 103], torch.int64)
    clk.cache_grow(h, slots, ints(lens))
    clk.cache_append_rotary(h, slots, pool, k[None], v[None], ints(lens), rotary=rot, offsets=off, q=q, q_out=q, k_out=k[None])
    scratch = clk.attend_scratch(Hq, Hkv, D)
    new = torch.empty((B, 3, Hq + 2 * Hkv, D), dtype=dt, device="cuda").normal_(generator=g)
    nq, nk, nv = new[:, :, :Hq], new[:, :, Hq:Hq + Hkv], new[:, :, Hq + Hkv:]
    mask = ints([masks_of([-1, 0, 0], 3, 3)] * B, torch.int64)
    nodes = ints([3, 3])
    raw = nk.clone()
    clk.tree_rotate(h, slots, nq, nk, nodes, mask, rot, nq, nk)
    out = torch.zeros((B, 3, Hq, D), dtype=dt, device="cuda")
    clk.tree_attend(h, slots, pool, 0, nq, nk, nv, nodes, mask, D ** -0.5, out, scratch)
    # the accepted nodes' keys go in as they were rotated for the attention: the same as rotated on the way
    path = ints([[0, 2, -1], [0, 1, -1]])
    clk.cache_grow(h, slots, ints([2, 2]))
    clk.cache_append(h, slots, pool, nk[None].contiguous(), nv[None].contiguous(), ints([2, 2]), path=path)
    torch.cuda.synchronize()
    first = pool.data.float().clone(), pool.scale.clone()
    rounded = raw.clone()
    clk.cache_append_rotary(h, slots, pool, rounded[None], nv[None].contiguous(), ints([2, 2]), rotary=rot, path=path)
    torch.cuda.synchronize()
    assert h.status()[0] == 0 and torch.equal(first[1], pool.scale)
    # rounded once instead of twice: at most one step of 8 bits apart
    assert ((first[0] - pool.data.float()).abs() <= first[0].abs() * 2.0 ** -3 + 2.0 ** -9).all()
    # against 64 bits over what the cache held
    table = h.table.cpu()
    values = (pool.data.float().unflatten(3, (2, 16)) * pool.scale[..., None, None]).flatten(3, 4)
    for b, (s, n) in enumerate(zip([1, 0], lens)):
        pages = table[s, :-(-n // P)].long().cuda()
        for hh in range(Hkv):
            kc, vc = (values[x, pages, hh].reshape(-1, D)[:n].double() for x in (0, 1))
            for t, see in enumerate(([0], [0, 1], [0, 2])):
                for gq in (2 * hh, 2 * hh + 1):
                    e = torch.cat([kc, nk[b, see, hh].double()]) @ nq[b, t, gq].double() * D ** -0.5
                    vals = torch.cat([vc, nv[b, see, hh].double()])
                    want, size = torch.softmax(e, 0) @ vals, torch.softmax(e, 0) @ vals.abs()
                    # bf16 weights and result: half a step of 2^-8 each; float32 scores and sums below 2^-14
                    tol = 2.0 ** -8 * want.abs() + (2.0 ** -8 + 2.0 ** -14) * size
                    assert ((out[b, t, gq].double() - want).abs() <= tol).all()


def test_results_are_those_of_the_same_values_in_16_bits():
    """Whether a row's error hides a wrong block: the same call over the 16-bit pool of the values differs by roundings only."""
    t = Tree8(20, 2, 8, [1000, 333], 4, 2, 128, 64, "bf16", nodes=[8, 8]).run()
    first = f64(t.out)
    clk.tree_attend(t.cache, ints(t.slots.tolist()), t.pool.contiguous(), 0, t.q, t.k, t.v, ints(t.nodes), t.dmask, t.scale, t.out, t.scratch)
    second = f64(t.out)
    assert np.abs(first - second).max() <= 2.0 ** -6 * np.abs(second).max()
