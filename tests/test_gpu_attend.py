"""Attention over the paged cache against 64 bits, row by row: head groups,
types, lengths, pages, masks, strides, packing, and what may not be read.
The tolerances are those of cache_model.tolerance.  GPU."""
import math

import numpy as np
import pytest
import torch

import context_lookup_speculative_gb300 as clk
from cache_model import attend_row, masks_of, random_tree, tolerance

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
NAN, INF = float("nan"), float("inf")


def ints(v, dtype=torch.int32):
    return torch.tensor(v, dtype=dtype, device="cuda")


def f64(x):
    return x.detach().double().cpu().numpy()


def make_pool(rng_seed, layers, pages, Hkv, P, D, kind, order="pnht"):
    g = torch.Generator(device="cuda").manual_seed(rng_seed)
    sizes = {"p": 2 * layers, "n": pages, "h": Hkv, "t": P}
    raw = torch.empty([sizes[c] for c in order] + [D], dtype=DT[kind], device="cuda").normal_(generator=g)
    return raw.permute([order.index(c) for c in "pnht"] + [4])


def fill(cache, lens, rng):
    """Grows the slots in shuffled rounds; returns nothing: the table is read back."""
    left = list(lens)
    for part in (3, 2, 1):
        order = rng.permutation(len(lens))
        give = [left[b] // part for b in range(len(lens))]
        left = [x - y for x, y in zip(left, give)]
        clk.cache_grow(cache, ints(order.tolist()), ints([give[b] for b in order]))


def cached(pool, plane, table, n, h, P):
    pages = table[:(n + P - 1) // P]
    return f64(pool[plane][pages.long(), h]).reshape(-1, pool.shape[-1])[:n]


def spoil(pool, cache, lens, fillers):
    """Everything in the pool that no slot's token holds becomes one of the fillers."""
    P, D = cache.page_tokens, pool.shape[-1]
    keep = torch.zeros((pool.shape[1], P), dtype=torch.bool, device="cuda")
    table = cache.table
    for s, n in enumerate(lens):
        for i in range(-(-n // P)):
            keep[table[s, i].long(), :min(P, n - i * P)] = True
    junk = torch.tensor(fillers, device="cuda", dtype=pool.dtype)
    noise = junk[torch.arange(pool.shape[1] * P * D, device="cuda") % len(fillers)].view(pool.shape[1], 1, P, D)
    pool.copy_(torch.where(keep[None, :, None, :, None], pool, noise))


def compare(got, want, size, kind, keys, vmax, what):
    assert np.isfinite(got).all(), what
    bad = np.abs(got - want) > tolerance(kind, want, size, keys, vmax)
    assert not bad.any(), (what, np.abs(got - want).max(), np.argwhere(bad)[:3].tolist())


class Tree:
    def __init__(self, seed, B, N, ctx, G, Hkv, D, P, kind, nodes=None, layers=1, layer=0, order="pnht", scale=None, lens=None,
                 pad=0, mask=None, amp=1.0):
        rng = self.rng = np.random.default_rng(seed)
        self.B, self.N, self.G, self.Hkv, self.D, self.P, self.kind, self.layer = B, N, G, Hkv, D, P, kind, layer
        self.ctx = list(ctx)
        self.lens = list(lens) if lens is not None else self.ctx
        Hq = G * Hkv
        pages = sum(-(-n // P) for n in self.lens) + 3
        self.slots = rng.permutation(B)
        by_slot = [0] * B
        for b in range(B):
            by_slot[self.slots[b]] = self.lens[b]
        self.cache = clk.Cache(B, max(1, max(-(-n // P) for n in self.lens)), pages, P)
        fill(self.cache, by_slot, rng)
        self.by_slot = by_slot
        self.pool = make_pool(seed, layers, pages, Hkv, P, D, kind, order)
        qkv = torch.empty((B, N, Hq + 2 * Hkv + pad, D), dtype=DT[kind], device="cuda").normal_(
            generator=torch.Generator(device="cuda").manual_seed(seed + 1))
        self.q, self.k, self.v = qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hkv], qkv[:, :, Hq + Hkv:Hq + 2 * Hkv]
        self.q.mul_(amp)
        self.nodes = nodes if nodes is not None else rng.integers(0, N + 1, size=B).tolist()
        if mask is None:
            mask = [masks_of(random_tree(rng, N), N, N) for _ in range(B)]
        self.mask = mask
        words = [[w - (1 << 64) if w >> 63 else w for w in row] for row in mask]
        self.dmask = torch.tensor(words, dtype=torch.int64, device="cuda")
        self.scale = 1 / math.sqrt(D) if scale is None else scale
        self.out = torch.full((B, N, Hq, D), NAN, dtype=DT[kind], device="cuda")
        self.scratch = clk.attend_scratch(Hq, Hkv, D)

    def run(self):
        clk.tree_attend(self.cache, ints(self.slots.tolist()), self.pool, self.layer, self.q, self.k, self.v, ints(self.nodes),
                        self.dmask, self.scale, self.out, self.scratch, ctx=None if self.ctx is self.lens else ints(self.ctx))
        return self

    def check(self, only=None):
        torch.cuda.synchronize()
        assert self.cache.status()[0] == 0
        out, q, k, v = f64(self.out), f64(self.q), f64(self.k), f64(self.v)
        for b in range(self.B) if only is None else only:
            n = self.nodes[b]
            assert (out[b, n:] == 0).all(), b
            for h in range(self.Hkv):
                tab = self.cache.table[int(self.slots[b])]
                kc, vc = (cached(self.pool, 2 * self.layer + x, tab, self.ctx[b], h, self.P) for x in (0, 1))
                for t in range(n):
                    see = [m for m in range(n) if self.mask[b][t] >> m & 1]
                    keys = np.concatenate([kc, k[b][see, h]])
                    vals = np.concatenate([vc, v[b][see, h]])
                    vmax = np.abs(vals).max() if len(vals) else 0.0
                    for g in range(self.G):
                        want, size = attend_row(q[b, t, h * self.G + g], keys, vals, self.scale)
                        compare(out[b, t, h * self.G + g], want, size, self.kind, len(keys), vmax, (b, t, h, g))
        return self


# -- trees --------------------------------------------------------------
@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("D", [64, 128, 80, 8, 96, 256, 33, 1])
def test_types_and_dims(kind, D):
    Tree(D, 3, 5, [70, 0, 129], 2, 2, D, 16, kind, nodes=[5, 3, 1]).run().check()


@pytest.mark.parametrize("P", [16, 32, 64, 128])
@pytest.mark.parametrize("n", [0, 1, 15, 16, 17, 63, 127, 128, 129, 255, 256, 257, 1000])
def test_context_lengths_and_pages(P, n):
    for kind, D in (("bf16", 128), ("f16", 64)):
        Tree(n + P, 2, 4, [n, max(0, n - 1)], 4, 1, D, P, kind, nodes=[4, 2]).run().check()


@pytest.mark.parametrize("G", [1, 2, 3, 4, 5, 6, 7, 8, 12, 16, 48, 128, 130])
def test_head_groups(G):
    Tree(G, 2, 3, [200, 37], G, 2 if G < 12 else 1, 64, 32, "bf16", nodes=[3, 2]).run().check()


@pytest.mark.parametrize("N", [1, 2, 8, 15, 16, 17, 31, 32, 33, 48, 63, 64])
@pytest.mark.parametrize("G", [1, 4, 6])
def test_tree_sizes(N, G):
    Tree(N * G, 3, N, [150, 300, 3], G, 1, 64, 64, "f16", nodes=[N, max(1, N // 2), 0]).run().check()


@pytest.mark.parametrize("B", [1, 7, 33, 200])
def test_ragged_batches(B):
    rng = np.random.default_rng(B)
    t = Tree(B, B, 3, rng.integers(0, 700, size=B).tolist(), 2, 2, 64, 16, "bf16").run()
    t.check(only=range(0, B, max(1, B // 12)))


def test_many_requests():
    """More requests than a CTA has threads; every output against the same call in parts."""
    B = 1500
    rng = np.random.default_rng(0)
    t = Tree(11, B, 2, rng.integers(0, 90, size=B).tolist(), 2, 1, 64, 16, "bf16").run()
    t.check(only=rng.permutation(B)[:40].tolist() + [0, B - 1])


@pytest.mark.parametrize("D,kind", [(128, "bf16"), (64, "f16")])
def test_a_long_context_is_split_and_joined(D, kind):
    Tree(D, 1, 16, [20011], 4, 1, D, 64, kind, nodes=[16]).run().check()
    Tree(D, 2, 1, [9000, 1], 8, 2, D, 128, kind, nodes=[1, 1]).run().check()


def test_large_scores():
    """Softmaxes that one key takes almost alone, and a maximum that keeps rising."""
    t = Tree(5, 2, 4, [700, 300], 2, 1, 64, 16, "bf16", nodes=[4, 4], amp=8.0)
    ramp = torch.linspace(0.01, 3.0, t.pool.shape[1], device="cuda").view(-1, 1, 1, 1)
    t.pool[0].mul_(ramp.to(t.pool.dtype))
    t.run().check()


def test_scores_far_below_zero_and_above():
    for sign in (-1.0, 1.0):
        t = Tree(6, 1, 2, [400], 2, 1, 64, 16, "f16", nodes=[2])
        t.q.fill_(1.0)
        t.pool[0].mul_(0.1).add_(sign * 4.0)
        t.k.mul_(0.1).add_(sign * 4.0)
        t.run().check()


@pytest.mark.parametrize("scale", [0.0, -0.1, 1.0])
def test_scales(scale):
    Tree(7, 2, 4, [130, 20], 2, 1, 64, 16, "bf16", nodes=[4, 4], scale=scale).run().check()


def test_masks_of_any_form():
    """Rows that see nothing, everything, only later nodes, only others; bits past the node count."""
    N = 64
    full = (1 << 64) - 1
    mask = [[0] * N, [full] * N, [full ^ (1 << n) for n in range(N)], [full << n & full for n in range(N)], [0] * N, [full] * N]
    t = Tree(8, 6, N, [0, 0, 0, 0, 50, 0], 2, 1, 64, 16, "bf16", nodes=[N, N, N, N, N, 40], mask=mask).run()
    t.check()
    assert (t.out[0] == 0).all()


@pytest.mark.parametrize("kind,D", [("bf16", 128), ("f16", 64), ("f32", 40)])
def test_what_is_not_visible_is_not_counted(kind, D):
    """Rows past ctx, free pages, nodes past the count or off a row's mask hold infinities, NaN and the type's extremes."""
    top = torch.finfo(DT[kind]).max
    N = 12
    # node 5 is seen by nobody, not even itself; node 7 by the nodes from 9 on
    base = [masks_of([-1] + list(range(N - 1)), N, N)] * 3
    mask = [[w & ~(1 << 5) & (~0 if n >= 9 else ~(1 << 7)) & (2 ** 64 - 1) for n, w in enumerate(row)] for row in base]
    for fillers in ([NAN], [INF, -INF], [top, -top], [NAN, INF, -INF, top, 0.0]):
        t = Tree(9, 3, N, [37, 130, 0], 3, 2, D, 32, kind, nodes=[N, 9, 7], mask=mask, lens=[80, 131, 20])
        spoil(t.pool, t.cache, [min(c, n) for c, n in zip([t.ctx[list(t.slots).index(s)] for s in range(3)], t.by_slot)], fillers)
        f = fillers[0]
        for b in range(3):
            t.k[b, t.nodes[b]:] = f
            t.v[b, t.nodes[b]:] = f
            t.q[b, t.nodes[b]:] = f
        t.k[:, 5] = f
        t.v[:, 5] = f
        t.run().check()


def test_infinities_and_nan_that_are_seen_stay_in_their_rows():
    N = 4
    chain = [masks_of([-1, 0, 1, 2], N, N)] * 2
    t = Tree(10, 2, N, [70, 70], 2, 1, 64, 16, "bf16", nodes=[N, N], mask=chain)
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


@pytest.mark.parametrize("order", ["pnht", "pnth", "npth", "hnpt"])
@pytest.mark.parametrize("layer", [0, 2])
def test_pool_orders_and_layers(order, layer):
    Tree(12, 2, 4, [100, 45], 2, 3, 64, 16, "bf16", nodes=[4, 3], layers=3, layer=layer, order=order).run().check()


def test_context_shorter_than_the_slot():
    Tree(13, 3, 4, [10, 0, 99], 2, 1, 128, 32, "bf16", nodes=[4, 4, 4], lens=[90, 33, 99]).run().check()


def test_rows_that_are_not_aligned_to_vectors():
    """Heads of 20 elements (40 bytes), and a query tensor that starts at an odd element."""
    Tree(14, 2, 3, [50, 20], 2, 1, 20, 16, "bf16", nodes=[3, 3]).run().check()
    t = Tree(15, 2, 3, [50, 20], 2, 1, 64, 16, "f16", nodes=[3, 3])
    for name in ("q", "k", "v"):
        x = getattr(t, name)
        wide = torch.zeros(x.shape[:-1] + (x.shape[-1] + 3,), dtype=x.dtype, device="cuda")
        wide[..., 1:-2] = x
        setattr(t, name, wide[..., 1:-2])
    t.run().check()


def test_same_results_every_time_and_for_any_batch():
    """A request's rows do not depend on timing; and the call can be repeated on its scratch."""
    t = Tree(16, 5, 6, [3000, 20, 500, 0, 1111], 4, 2, 128, 64, "bf16").run()
    torch.cuda.synchronize()
    first = t.out.clone()
    for _ in range(5):
        t.out.fill_(NAN)
        t.run()
        torch.cuda.synchronize()
        assert torch.equal(t.out, first)


def test_bad_requests_are_latched_and_give_zero():
    t = Tree(17, 4, 3, [40, 40, 40, 40], 2, 1, 64, 16, "bf16", nodes=[3, 4, 3, -1])
    t.ctx = [40, 40, 41, 40]
    t.run()
    torch.cuda.synchronize()
    assert t.cache.status()[0] == clk.EINVAL
    assert (t.out[1:] == 0).all()
    t.cache.status_clear()
    t.check(only=[0])
    good = t.slots.copy()
    t.slots[0], t.ctx, t.nodes = 4, [40] * 4, [3] * 4
    t.out.fill_(NAN)
    t.run()
    torch.cuda.synchronize()
    assert t.cache.status() == (clk.EINVAL, 0)
    assert (t.out[0] == 0).all()
    t.cache.status_clear()
    t.slots[0] = good[0]
    t.check(only=[1, 2, 3])


# -- prompts ------------------------------------------------------------
class Prompt:
    def __init__(self, seed, lens, G, Hkv, D, kind, ctx=None, P=16, lead=0, tail=0, amp=1.0):
        rng = np.random.default_rng(seed)
        self.lens, self.G, self.Hkv, self.D, self.kind, self.P, self.ctx = list(lens), G, Hkv, D, kind, P, ctx
        B, Hq = len(lens), G * Hkv
        self.off = (np.cumsum([0] + self.lens) + lead).tolist()
        T = self.off[-1] + tail
        qkv = torch.empty((T, Hq + 2 * Hkv, D), dtype=DT[kind], device="cuda").normal_(
            generator=torch.Generator(device="cuda").manual_seed(seed))
        self.q, self.k, self.v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        self.q.mul_(amp)
        self.out = torch.full((T, Hq, D), 5.0, dtype=DT[kind], device="cuda")
        self.scale = 1 / math.sqrt(D)
        self.scratch = clk.attend_scratch(Hq, Hkv, D)
        self.kw = {}
        if ctx is not None:
            pages = sum(-(-n // P) for n in ctx) + 2
            self.slots = rng.permutation(B)
            by_slot = [0] * B
            for b in range(B):
                by_slot[self.slots[b]] = ctx[b]
            self.by_slot = by_slot
            self.cache = clk.Cache(B, max(1, max(-(-n // P) for n in ctx)), pages, P)
            fill(self.cache, by_slot, rng)
            self.pool = make_pool(seed, 1, pages, Hkv, P, D, kind)
            self.kw = dict(cache=self.cache, slots=ints(self.slots.tolist()), pool=self.pool, ctx=ints(ctx))

    def run(self):
        clk.prompt_attend(self.q, self.k, self.v, ints(self.off, torch.int64), self.scale, self.out, self.scratch, **self.kw)
        return self

    def check(self, rows=None):
        """rows: how many rows of a request are looked at (None: all)."""
        torch.cuda.synchronize()
        if self.kw:
            assert self.cache.status()[0] == 0
        out, q, k, v = f64(self.out), f64(self.q), f64(self.k), f64(self.v)
        inside = np.zeros(len(out), dtype=bool)
        for b, n in enumerate(self.lens):
            lo = self.off[b]
            inside[lo:lo + n] = True
            c = self.ctx[b] if self.ctx is not None else 0
            pick = range(n) if rows is None or n <= rows else sorted({0, n - 1, n // 2, *np.random.default_rng(b).integers(0, n, rows)})
            for h in range(self.Hkv):
                kc = vc = np.zeros((0, self.D))
                if c:
                    tab = self.cache.table[int(self.slots[b])]
                    kc, vc = (cached(self.pool, x, tab, c, h, self.P) for x in (0, 1))
                keys, vals = np.concatenate([kc, k[lo:lo + n, h]]), np.concatenate([vc, v[lo:lo + n, h]])
                for t in pick:
                    for g in range(self.G):
                        kk, vv = keys[:c + t + 1], vals[:c + t + 1]
                        want, size = attend_row(q[lo + t, h * self.G + g], kk, vv, self.scale)
                        compare(out[lo + t, h * self.G + g], want, size, self.kind, len(kk), np.abs(vv).max(), (b, t, h, g))
        assert (out[~inside] == 5.0).all()
        return self


@pytest.mark.parametrize("kind,D", [("bf16", 128), ("f16", 64), ("bf16", 64), ("f16", 128), ("f32", 64), ("bf16", 80), ("f16", 256),
                                    ("bf16", 24)])
def test_prompt_types_and_dims(kind, D):
    Prompt(D, [70, 1, 0, 133, 20], 2, 2, D, kind).run().check(rows=20)


@pytest.mark.parametrize("n", [1, 2, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 300, 513])
@pytest.mark.parametrize("G", [1, 4])
def test_prompt_lengths(n, G):
    Prompt(n, [n], G, 1, 64, "bf16").run().check(rows=40)


@pytest.mark.parametrize("G", [1, 2, 3, 4, 5, 6, 7, 8, 16, 40, 128, 129])
def test_prompt_head_groups(G):
    Prompt(G, [90, 150], G, 2 if G < 8 else 1, 128, "bf16").run().check(rows=10)


@pytest.mark.parametrize("P", [16, 32, 64, 128])
def test_prompts_behind_cached_prefixes(P):
    for kind, D in (("bf16", 128), ("f16", 64)):
        Prompt(P, [40, 1, 200, 0, 130, 64], 3, 2, D, kind, ctx=[0, 77, 130, 50, 1, 3 * P], P=P).run().check(rows=15)


def test_a_long_prompt():
    Prompt(1, [6011], 4, 1, 128, "bf16").run().check(rows=60)
    Prompt(2, [1500, 37, 2300], 6, 2, 64, "f16", ctx=[100, 5000, 0], P=64).run().check(rows=25)


def test_few_rows_behind_a_long_prefix():
    Prompt(3, [3], 4, 1, 128, "bf16", ctx=[30003], P=64).run().check()


def test_many_short_prompts():
    rng = np.random.default_rng(4)
    Prompt(4, rng.integers(0, 9, size=700).tolist(), 2, 1, 64, "bf16").run().check(rows=3)


def test_prompt_rows_outside_are_neither_read_nor_written():
    """Rows before the first, after the last and of other requests hold NaN; free and stale page rows too."""
    for fillers in ([NAN], [INF, -INF, 3e38]):
        p = Prompt(5, [33, 130, 7], 2, 1, 64, "bf16", ctx=[20, 0, 100], lead=3, tail=9)
        spoil(p.pool, p.cache, p.by_slot, fillers)
        for x in (p.q, p.k, p.v):
            x[:3] = NAN
            x[p.off[-1]:] = NAN
        p.run().check()


def test_a_later_token_reaches_no_earlier_row():
    p = Prompt(6, [200], 2, 1, 128, "bf16")
    p.k[150:], p.v[150:] = NAN, INF
    p.run()
    torch.cuda.synchronize()
    assert not torch.isfinite(p.out[150:].float()).any()
    p.lens, p.out[150:] = [150], 5.0
    p.check()
    p = Prompt(6, [200], 2, 1, 64, "f16")
    p.v[131, 0, 5] = NAN
    p.run()
    torch.cuda.synchronize()
    assert torch.isnan(p.out[131:, :, 5]).all()
    p.lens, p.out[131:] = [131], 5.0
    p.check()


def test_prompt_large_scores():
    Prompt(7, [300], 2, 1, 64, "bf16", amp=10.0).run().check(rows=60)


def test_bad_offsets_and_contexts():
    p = Prompt(8, [20, 30, 10], 2, 1, 64, "bf16", ctx=[5, 6, 7])
    p.kw["ctx"] = ints([5, 7, -1])
    p.run()
    torch.cuda.synchronize()
    assert p.cache.status()[0] == clk.EINVAL
    p.cache.status_clear()
    assert (p.out[20:] == 5.0).all()
    p.lens = [20, 0, 0]
    p.check()
    p = Prompt(9, [20, 30], 2, 1, 64, "bf16")
    good = list(p.off)
    for off in ([0, 20, 51], [-1, 20, 50], [0, 20, 19]):
        p.off = off
        p.run()
    torch.cuda.synchronize()
    p.off = good
    p.check()


def test_attention_on_another_stream_and_in_a_graph():
    t = Tree(18, 2, 4, [300, 50], 2, 1, 128, 16, "bf16", nodes=[4, 4])
    p = Prompt(10, [100, 50], 2, 1, 128, "bf16")
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        t.run()
        p.run()
    s.synchronize()
    t.check()
    p.check(rows=10)
    slots, nodes, off = ints(t.slots.tolist()), ints(t.nodes), ints(p.off, torch.int64)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        clk.tree_attend(t.cache, slots, t.pool, 0, t.q, t.k, t.v, nodes, t.dmask, t.scale, t.out, t.scratch)
        clk.prompt_attend(p.q, p.k, p.v, off, p.scale, p.out, p.scratch)
    t.q.mul_(-0.5)
    p.q.mul_(-0.5)
    t.out.zero_()
    p.out.fill_(5.0)
    g.replay()
    t.check()
    p.check(rows=10)


def test_refusals():
    t = Tree(19, 2, 3, [20, 20], 2, 1, 64, 16, "bf16", nodes=[3, 3])
    ok = dict(h=t.cache, slots=ints([0, 1]), pool=t.pool, layer=0, q=t.q, k=t.k, v=t.v, nodes=ints([3, 3]), mask=t.dmask, scale=0.1,
              out=t.out, scratch=t.scratch)
    clk.tree_attend(**ok)
    for bad in (dict(q=t.q.float()), dict(out=t.out[:, :2]), dict(k=t.k[:, :2]), dict(mask=t.dmask.int()), dict(nodes=ints([3])),
                dict(slots=ints([0, 1, 1])), dict(pool=t.pool[:, :2]), dict(pool=t.pool[:, :, :, :8]), dict(q=t.q[0])):
        with pytest.raises(ValueError):
            clk.tree_attend(**{**ok, **bad})
    for bad in (dict(layer=1), dict(layer=-1), dict(scale=NAN), dict(pool=t.pool.float())):
        with pytest.raises(clk.ClkError):
            clk.tree_attend(**{**ok, **bad})
    with pytest.raises(ValueError):
        clk.prompt_attend(t.q[0], t.k[0], t.v[0], ints([0, 3], torch.int64), 0.1, t.out[0], t.scratch, ctx=ints([1]))
    clk.prompt_attend(t.q[0], t.k[0], t.v[0], ints([0, 3], torch.int64), 0.1, t.out[0], t.scratch)


@pytest.mark.parametrize("scale", [1e-38, 1e-25, 1e-3, 20.0])
def test_scales_at_the_ends_of_the_range(scale):
    Tree(20, 2, 4, [130, 20], 2, 1, 64, 16, "bf16", nodes=[4, 4], scale=scale).run().check()


def test_a_pool_of_more_than_two_to_the_32_elements():
    """Pages whose elements lie past 32 bits, read by both kernels."""
    pages, P, Hkv, D = 8700, 128, 16, 128
    cache = clk.Cache(3, pages, pages, P)
    pool = torch.empty((2, pages, Hkv, P, D), dtype=torch.bfloat16, device="cuda")
    assert pool.numel() > 1 << 32
    n = 300
    clk.cache_grow(cache, ints([0]), ints([(pages - 4) * P]))
    clk.cache_grow(cache, ints([2]), ints([n]))
    torch.cuda.synchronize()
    assert cache.table[2, 0].item() == pages - 4
    pool[:, pages - 4:].normal_()
    g = torch.Generator(device="cuda").manual_seed(3)
    qkv = torch.empty((1, 2, 3 * Hkv, D), dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    q, k, v = qkv.split(Hkv, 2)
    mask = torch.tensor([[1, 3]], dtype=torch.int64, device="cuda")
    for scale in (0.09, -0.09):  # a negative scale goes through the general kernel
        out = torch.zeros((1, 2, Hkv, D), dtype=torch.bfloat16, device="cuda")
        clk.tree_attend(cache, ints([2]), pool, 0, q, k, v, ints([2]), mask, scale, out, clk.attend_scratch(Hkv, Hkv, D))
        for h in (0, Hkv - 1):
            kc, vc = (cached(pool, x, cache.table[2], n, h, P) for x in (0, 1))
            for t in range(2):
                keys, vals = np.concatenate([kc, f64(k)[0, :t + 1, h]]), np.concatenate([vc, f64(v)[0, :t + 1, h]])
                want, size = attend_row(f64(q)[0, t, h], keys, vals, scale)
                compare(f64(out)[0, t, h], want, size, "bf16", len(keys), np.abs(vals).max(), (scale, h, t))


def test_broadcast_inputs():
    """Strides of 0: one K/V row shared by the heads, one query shared by the requests."""
    t = Tree(21, 3, 4, [40, 0, 130], 2, 2, 64, 16, "bf16", nodes=[4, 2, 3])
    t.k, t.v = (x[:, :, :1].expand(-1, -1, 2, -1) for x in (t.k, t.v))
    t.q = t.q[:1].expand(3, -1, -1, -1)
    t.run().check()
    p = Prompt(22, [70, 9], 2, 2, 128, "f16")
    p.k, p.v = (x[:, :1].expand(-1, 2, -1) for x in (p.k, p.v))
    p.run().check(rows=10)


def test_keys_and_values_of_different_strides():
    t = Tree(23, 2, 5, [60, 33], 3, 2, 64, 16, "bf16", nodes=[5, 4])
    t.v = t.v.permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3)
    t.q = t.q.contiguous()
    t.run().check()


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("step", [2.0, 9.0, 60.0])
def test_maxima_that_rise_tile_after_tile(kind, step):
    """Every 128 keys the scores rise by `step` (log2 units), slowly and in jumps, in some rows only."""
    D, n = 64, 1300
    t = Tree(24, 2, 4, [n, n - 37], 2, 1, D, 128, kind, nodes=[4, 4], scale=math.log(2.0) / 8)
    for s in range(2):
        for i in range(-(-n // 128)):
            # element 0 of the keys carries the level: scores = 8 * level * q0 / 8 log2 units
            page = t.cache.table[s, i].long()
            if page >= 0:
                t.pool[0, page, 0] *= 0.1
                t.pool[0, page, 0, :, 0] = step * i
    t.q.mul_(0.1)
    t.q[..., 0] = 1.0
    t.q[:, 1, 0, 0] = -1.0  # a row whose scores fall
    t.q[:, 2, 1, 0] = 0.0   # and one where they stay
    t.k.mul_(0.1)
    t.run().check()


# -- the general kernel's shares: rows a warp, warps a tile, CTAs a row ---
@pytest.mark.parametrize("kind,D", [("f32", 40), ("f32", 128), ("bf16", 250)])
@pytest.mark.parametrize("B,N,G", [(1, 1, 1), (1, 1, 5), (1, 2, 2), (1, 4, 3), (1, 9, 3), (1, 16, 2), (1, 64, 1), (3, 5, 33), (1, 1, 70),
                                   (40, 3, 4)])
def test_shares_of_the_general_kernel_for_trees(B, N, G, kind, D):
    ctx = [(700, 0, 64, 1, 513, 129)[b % 6] for b in range(B)]
    nodes = [N if b % 3 == 0 else max(0, N - b % 4) for b in range(B)]
    Tree(B + N + G, B, N, ctx, G, 1, D, 32, kind, nodes=nodes).run().check()


@pytest.mark.parametrize("lens", [[1], [8], [300], [5] * 30, [33, 0, 420, 1]])
@pytest.mark.parametrize("G", [1, 3, 40])
@pytest.mark.parametrize("kind,D", [("f32", 40), ("f16", 200)])
def test_shares_of_the_general_kernel_for_prompts(lens, G, kind, D):
    Prompt(len(lens) + G, lens, G, 1, D, kind, ctx=[(130, 0, 64)[b % 3] for b in range(len(lens))]).run().check(rows=12)


@pytest.mark.parametrize("D", [40, 160])
def test_hidden_values_in_the_general_kernel(D):
    """A new token that only some rows see holds NaN: the others' results are what they are without it."""
    mask = [[1, 3, 5, 9, 17, 1, 1, 1]]  # token 3 is seen by itself alone
    nodes = [8]
    a = Tree(3, 1, 8, [200], 2, 1, D, 16, "f32", nodes=nodes, mask=mask)
    a.run().check()
    want = a.out.clone()
    a.v[0, 3] = NAN
    a.k[0, 4] = INF
    a.run()
    keep = [t for t in range(8) if t not in (3, 4)]
    assert torch.equal(a.out[0, keep], want[0, keep])
    assert a.out[0, 3].isnan().all()


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("D", [8, 16, 24, 32, 48, 56, 72, 104])
def test_rows_that_do_not_fill_a_tile(kind, D):
    """Tensor-core tiles of 64 or 128 columns, of which D are there."""
    Tree(D, 3, 5, [300, 0, 129], 3, 2, D, 32, kind, nodes=[5, 3, 1]).run().check()
    Prompt(D, [140, 1, 260], 3, 2, D, kind, ctx=[40, 200, 0]).run().check(rows=15)
