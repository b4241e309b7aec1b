"""Position rotation of drafted trees and of appended rows, bit for bit against
a float32 model: types, row lengths, pairings, layouts, batches, and what may
not be read or written.  GPU."""
import numpy as np
import pytest
import torch

import context_lookup_speculative_gb300 as clk
from cache_model import masks_of, random_tree
from rotary_model import angles, same, turned
from test_gpu_attend import DT, NAN, fill, ints

pytestmark = pytest.mark.gpu


def words(rows):
    return ints([[w - (1 << 64) if w >> 63 else w for w in row] for row in rows], torch.int64)


def normal(shape, kind, seed):
    return torch.empty(shape, dtype=DT[kind], device="cuda").normal_(generator=torch.Generator(device="cuda").manual_seed(seed))


class Slots:
    """A cache whose slots hold `lens` rows."""

    def __init__(self, lens, P, rng, more=3):
        self.lens, self.P = list(lens), P
        pages = sum(-(-n // P) for n in lens) + more
        self.h = clk.Cache(len(lens), max(1, max(-(-n // P) for n in lens)), pages, P)
        fill(self.h, lens, rng)
        self.table = self.h.table.cpu()

    def place(self, slot, pos):
        return int(self.table[slot, pos // self.P]), pos % self.P


# -- trees --------------------------------------------------------------
def tree_case(seed, B, N, Hq, Hkv, D, pairs, kind, neighbours=False, ctx=None, nodes=None, mask=None, layout="sliced", positions=None,
              status=0):
    rng = np.random.default_rng(seed)
    lens = rng.integers(0, 300, size=B).tolist()
    c = Slots(lens, 16, rng)
    slots = rng.permutation(B).tolist()
    at = [lens[s] for s in slots] if ctx is None else ctx
    nodes = rng.integers(0, N + 1, size=B).tolist() if nodes is None else nodes
    mask = [masks_of(random_tree(rng, N), N, N) for _ in range(B)] if mask is None else mask
    positions = positions or max(at + [0]) + N
    table = angles(positions, pairs)
    wide = normal((B, N, Hq + 2 * Hkv, D), kind, seed)
    q, k = wide[:, :, :Hq], wide[:, :, Hq:Hq + Hkv]
    if layout == "odd":  # rows that start at odd elements
        pad = torch.zeros((B, N, Hq + 2 * Hkv, D + 3), dtype=DT[kind], device="cuda")
        pad[..., 1:-2] = wide
        q, k = pad[:, :, :Hq, 1:-2], pad[:, :, Hq:Hq + Hkv, 1:-2]
    elif layout == "heads first":
        q, k = (x.permute(2, 0, 1, 3).contiguous().permute(1, 2, 0, 3) for x in (q, k))
    q0, k0 = q.cpu().clone(), k.cpu().clone()
    qo, ko = (q, k) if layout == "in place" else (torch.full(q.shape, 3.0, dtype=q.dtype, device="cuda"), torch.full(k.shape, 3.0, dtype=k.dtype, device="cuda"))
    want = [x.cpu().clone() for x in (qo, ko)]
    clk.tree_rotate(c.h, ints(slots), q, k, ints(nodes), words(mask), clk.Rotary(table.cuda(), neighbours), qo, ko,
                    ctx=None if ctx is None else ints(ctx))
    torch.cuda.synchronize()
    for b in range(B):
        n = nodes[b]
        if not 0 <= n <= N or not 0 <= at[b] <= lens[slots[b]]:
            continue
        pos = [at[b] + max(0, bin(w & ((1 << n) - 1)).count("1") - 1) for w in mask[b][:n]]
        keep = [i for i, p in enumerate(pos) if p < positions]
        for x, y in ((q0, want[0]), (k0, want[1])):
            if keep:
                y[b, keep] = turned(x[b, keep], [pos[i] for i in keep], table, neighbours).to(DT[kind])
    assert c.h.status()[0] == status
    assert same(qo, want[0]) and same(ko, want[1])


@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("neighbours", [False, True])
@pytest.mark.parametrize("D,pairs", [(128, 64), (64, 32), (128, 16), (16, 8), (96, 48), (80, 40), (112, 24), (256, 128), (64, 20), (33, 7), (2, 1)])
def test_trees_types_and_rows(kind, neighbours, D, pairs):
    tree_case(D + pairs, 4, 9, 6, 2, D, pairs, kind, neighbours)


@pytest.mark.parametrize("N", [1, 2, 15, 16, 17, 33, 63, 64])
def test_tree_sizes(N):
    tree_case(N, 5, N, 4, 1, 64, 32, "bf16")


@pytest.mark.parametrize("layout", ["in place", "odd", "heads first"])
@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_tree_layouts(layout, kind):
    tree_case(3, 4, 18, 8, 2, 128, 64, kind, layout=layout)


@pytest.mark.parametrize("B", [1, 255, 256, 257, 900])
def test_tree_batches(B):
    tree_case(B, B, 3, 2, 1, 64, 32, "bf16")


def test_many_heads_and_trees():
    tree_case(5, 40, 64, 48, 8, 128, 64, "f16")


def test_masks_of_any_form_and_contexts():
    full = (1 << 64) - 1
    N = 64
    mask = [[0] * N, [full] * N, [full << n & full for n in range(N)], [1 << n for n in range(N)]]
    tree_case(6, 4, N, 2, 1, 64, 32, "bf16", mask=mask, nodes=[N, N, 40, 0])
    tree_case(6, 4, N, 2, 1, 64, 32, "bf16", mask=mask, nodes=[N, N, 40, 0], ctx=[0, 0, 0, 0])


def test_bad_trees_are_left_out():
    tree_case(7, 4, 4, 2, 1, 64, 32, "bf16", nodes=[4, 5, -1, 4], ctx=[0, 0, 0, 100000], positions=50, status=clk.EINVAL)
    tree_case(7, 3, 4, 2, 1, 64, 32, "bf16", nodes=[4, 4, 4], ctx=[0, 0, 0], positions=2, status=clk.EINVAL)


# -- appended rows --------------------------------------------------------
def append_case(seed, counts, lens, Hq, Hkv, D, pairs, kind, form="packed", layers=1, layer=0, P=16, neighbours=False, sides=True,
                in_place=False, order="pnht", rows=None, spare=0):
    """Rows behind `lens` rows of each slot; form: packed, dense, or path (accepted nodes)."""
    rng = np.random.default_rng(seed)
    B = len(counts)
    slots = rng.permutation(B).tolist()
    by_slot = [0] * B
    for b, s in enumerate(slots):
        by_slot[s] = lens[b] + counts[b]
    c = Slots(by_slot, P, rng)
    sizes = {"p": 2 * (layer + layers), "n": c.h.num_pages, "h": Hkv, "t": P}
    pool = normal([sizes[x] for x in order] + [D], kind, seed).permute([order.index(x) for x in "pnht"] + [4])
    table = angles(max(by_slot) + 1, pairs) if pairs else None
    N = max(counts + [1]) + spare
    lead = (sum(counts) + spare,) if form == "packed" else (B, N)
    wide = normal((layers,) + lead + (Hq + 2 * Hkv, D), kind, seed + 1)
    q, k, v = wide[0][..., :Hq, :], wide[..., Hq:Hq + Hkv, :], wide[..., Hq + Hkv:, :]
    q0, k0 = q.cpu().clone(), k.cpu().clone()
    kw = {}
    if form == "packed":
        off = np.cumsum([0] + counts).tolist()
        kw["offsets"] = ints(off, torch.int64)
    if form == "path":
        path = [rng.integers(0, N, size=N).tolist() for _ in range(B)]
        kw["path"] = ints(path)
    if pairs:
        kw["rotary"] = clk.Rotary(table.cuda(), neighbours)
    want_q = want_k = None
    if sides and pairs and layers == 1 and form != "path":
        qo, ko = (q, k) if in_place else (torch.full_like(q, 3.0), torch.full_like(k, 3.0))
        want_q, want_k = qo.cpu().clone(), ko.cpu().clone()
        kw.update(q=q, q_out=qo, k_out=ko)
    want = pool.cpu().clone()
    v0 = v.cpu().clone()
    clk.cache_append_rotary(c.h, ints(slots), pool, k, v, ints(counts), layer=layer, **kw)
    torch.cuda.synchronize()
    for b in range(B):
        n, p0 = counts[b], lens[b]
        if n == 0:
            continue
        at = list(range(off[b], off[b] + n)) if form == "packed" else (path[b][:n] if form == "path" else list(range(n)))
        pos = list(range(p0, p0 + n))
        for l in range(layers):
            rk, rv = (x[l][at] if form == "packed" else x[l, b, at] for x in (k0, v0))
            rk = turned(rk, pos, table, neighbours).to(DT[kind]) if pairs else rk
            for i, p in enumerate(pos):
                page, line = c.place(slots[b], p)
                want[2 * (layer + l), page, :, line], want[2 * (layer + l) + 1, page, :, line] = rk[i], rv[i]
            if want_k is not None:
                rq = turned(q0[at] if form == "packed" else q0[b, at], pos, table, neighbours).to(DT[kind])
                if form == "packed":
                    want_k[0, at], want_q[at] = rk, rq
                else:
                    want_k[0, b, at], want_q[b, at] = rk, rq
    assert c.h.status()[0] == 0
    assert same(pool, want)
    if want_k is not None:
        assert same(ko, want_k) and same(qo, want_q)


@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("form", ["packed", "dense", "path"])
@pytest.mark.parametrize("D,pairs", [(128, 64), (64, 32), (64, 8), (96, 24), (256, 128), (33, 7)])
def test_appended_rows(kind, form, D, pairs):
    append_case(D + pairs, [5, 0, 17, 40, 1], [3, 20, 15, 0, 31], 4, 2, D, pairs, kind, form, neighbours=D == 64)


@pytest.mark.parametrize("P", [16, 32, 64, 128])
@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 33, 129])
def test_appended_lengths_and_pages(P, n):
    append_case(n, [n, 1, max(1, n - 1)], [P - 1, P, 0], 2, 1, 64, 32, "bf16", P=P)


@pytest.mark.parametrize("order", ["pnht", "pnth", "npth", "hnpt"])
def test_pool_orders_layers_and_in_place(order):
    append_case(1, [5, 30], [10, 3], 0, 3, 64, 32, "bf16", "dense", layers=3, layer=1, order=order, spare=2)
    append_case(2, [5, 30], [10, 3], 4, 3, 64, 32, "f16", "packed", layer=1, order=order, in_place=True, spare=5)


def test_without_a_rotation_it_appends():
    append_case(3, [5, 30, 1], [10, 3, 100], 0, 2, 128, 0, "bf16", "packed", layers=2)
    append_case(4, [5, 30, 1], [10, 3, 100], 0, 2, 40, 0, "f32", "path", layers=2)


@pytest.mark.parametrize("B", [1, 256, 300, 700])
def test_append_batches(B):
    rng = np.random.default_rng(B)
    append_case(B, rng.integers(0, 20, size=B).tolist(), rng.integers(0, 40, size=B).tolist(), 2, 1, 64, 32, "bf16")


def test_a_long_prompt_of_many_heads():
    append_case(9, [3001, 77], [100, 4000], 32, 8, 128, 64, "bf16", P=64)


def test_requests_that_are_left_out():
    """Bad slots, counts, paths, offsets and positions past the table; the others are written."""
    rng = np.random.default_rng(0)
    c = Slots([40, 40, 40, 40, 40], 16, rng)
    table = angles(45, 32)
    rot = clk.Rotary(table.cuda())
    pool = normal((2, c.h.num_pages, 1, 16, 64), "bf16", 1)
    k, v = normal((1, 4, 3, 1, 64), "bf16", 2), normal((1, 4, 3, 1, 64), "bf16", 3)

    def check(slots, counts, good, **kw):
        want = pool.cpu().clone()
        clk.cache_append_rotary(c.h, ints(slots), pool, k.flatten(1, 2) if "offsets" in kw else k, v.flatten(1, 2) if "offsets" in kw else v,
                                ints(counts), rotary=rot, **kw)
        torch.cuda.synchronize()
        off = kw["offsets"].tolist() if "offsets" in kw else [0, 3, 6, 9, 12]
        for b in good:
            n = counts[b]
            pos = list(range(40 - n, 40))
            r = list(range(off[b], off[b] + n))
            rk = turned(k.cpu().flatten(1, 2)[0, r], pos, table, False).to(torch.bfloat16)
            for i, p in enumerate(pos):
                page, line = c.place(slots[b], p)
                want[0, page, :, line], want[1, page, :, line] = rk[i], v.cpu().flatten(1, 2)[0, r[i]]
        assert same(pool, want)
        assert c.h.status()[0] == clk.EINVAL
        c.h.status_clear()

    check([0, 7, -1, 3], [3, 3, 3, 2], [0, 3])
    check([0, 1, 2, 3], [4, -1, 3, 3], [2, 3])
    check([0, 1, 2, 3], [2, 3, 3, 3], [0, 3], offsets=ints([0, 3, 20, 6, 12], torch.int64))
    check([0, 1, 2, 3], [2, 3, 3, 3], [1, 3], offsets=ints([3, 0, 6, 4, 12], torch.int64))
    # a page that is not there, by a table entry out of range
    path = [[0, 1, 2], [0, 5, 1], [0, 1, -1], [2, 1, 0]]
    before = pool.cpu().clone()
    clk.cache_append_rotary(c.h, ints([0, 1, 2, 3]), pool, k, v, ints([1, 1, 1, 1]), rotary=rot, path=ints([[9, 0, 0], [-1, 0, 0], [3, 0, 0], [1 << 30, 0, 0]]))
    torch.cuda.synchronize()
    assert c.h.status()[0] == clk.EINVAL and same(pool, before) and path
    c.h.status_clear()
    # positions up to the table's end are taken, past it the request is left out
    short = clk.Rotary(table[:39].contiguous().cuda())
    clk.cache_append_rotary(c.h, ints([0, 1, 2, 3]), pool, k, v, ints([1, 1, 1, 1]), rotary=short)
    torch.cuda.synchronize()
    assert c.h.status()[0] == clk.EINVAL and same(pool, before)
    c.h.status_clear()
    clk.cache_append_rotary(c.h, ints([0, 1, 2, 3]), pool, k, v, ints([1, 1, 1, 1]), rotary=clk.Rotary(table[:40].contiguous().cuda()))
    torch.cuda.synchronize()
    assert c.h.status()[0] == 0 and not same(pool, before)


def test_rows_that_others_hold_are_not_written():
    rng = np.random.default_rng(0)
    h = clk.Cache(2, 4, 8, 16)
    clk.cache_grow(h, ints([0]), ints([20]))
    pool = normal((2, 8, 1, 16, 64), "bf16", 1)
    clk.cache_fork(h, ints([0]), ints([1]), pool)
    k = normal((1, 1, 20, 1, 64), "bf16", 2)
    before = pool.cpu().clone()
    clk.cache_append_rotary(h, ints([1]), pool, k, k.clone(), ints([5]), rotary=clk.Rotary(angles(64, 32).cuda()))
    torch.cuda.synchronize()
    assert h.status()[0] == clk.EINVAL and same(pool, before) and rng is not None


def test_tables_of_the_framework():
    freq = 10000.0 ** (-torch.arange(32, dtype=torch.float64) / 32)
    r = clk.Rotary.of(freq, 1000, factor=1.25)
    a = torch.arange(1000, dtype=torch.float64)[:, None] * freq
    want = torch.stack([a.cos(), a.sin()], 1) * 1.25
    # float32 of a value below 2: half a step of 2^-23
    assert r.table.shape == (1000, 2, 32) and (r.table.cpu().double() - want).abs().max() <= 2.0 ** -24 + 2.0 ** -40


def test_captured_and_on_another_stream():
    rng = np.random.default_rng(0)
    c = Slots([50, 9], 16, rng)
    table = angles(64, 32)
    rot = clk.Rotary(table.cuda())
    q, k, v = normal((2, 4, 4, 64), "bf16", 1), normal((2, 4, 2, 64), "bf16", 2), normal((2, 4, 2, 64), "bf16", 3)
    qo, ko = torch.zeros_like(q), torch.zeros_like(k)
    pool = normal((2, c.h.num_pages, 2, 16, 64), "bf16", 4)
    nodes, mask, slots, count = ints([4, 4]), words([masks_of([-1, 0, 1, 2], 4, 4)] * 2), ints([0, 1]), ints([4, 4])

    def both():
        clk.tree_rotate(c.h, slots, q, k, nodes, mask, rot, qo, ko)
        clk.cache_append_rotary(c.h, slots, pool, k[None], v[None], count, rotary=rot)

    def results():
        return qo.clone(), ko.clone(), pool.clone()

    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        both()
    s.synchronize()
    first = results()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        both()
    k.mul_(2.0)
    qo.fill_(NAN)
    g.replay()
    torch.cuda.synchronize()
    got = results()
    assert torch.equal(got[0], first[0]) and torch.equal(got[1], first[1] * 2)
    want = first[2].clone()
    for slot, n in ((0, 50), (1, 9)):
        for p in range(n - 4, n):
            page, line = c.place(slot, p)
            want[0, page, :, line] *= 2
    assert torch.equal(got[2], want)
