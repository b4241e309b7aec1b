"""A cache in 8 bits: rows that come in, blocks whose scale grows, forks and
compaction, bit for bit against a model.  GPU."""
import numpy as np
import pytest
import torch

import context_lookup_speculative_gb300 as clk
from rotary_model import Eight, angles, same, turned
from test_gpu_attend import DT, INF, NAN, ints
from test_gpu_rotary import Slots, normal

pytestmark = pytest.mark.gpu


def pool8(planes, pages, heads, P, D, T, seed, order="pnht", pad=0):
    """A pool of random codes (NaN among them) and random scales, in a given order of its axes."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    sizes = {"p": planes, "n": pages, "h": heads, "t": P}
    raw = torch.randint(0, 256, [sizes[x] for x in order] + [D + pad], generator=g, device="cuda", dtype=torch.uint8)
    data = raw.view(torch.float8_e4m3fn).permute([order.index(x) for x in "pnht"] + [4])[..., :D]
    scale = torch.exp2(torch.randint(-12, 6, (P // T, planes, pages, heads), generator=g, device="cuda").float()).permute(1, 2, 3, 0)
    return clk.ScaledPool(data, scale)


class Case:
    def __init__(self, seed, B, Hkv, D, T, kind, P=None, layers=1, layer=0, pages=40, pairs=0, neighbours=False, order="pnht", pad=0):
        self.rng = np.random.default_rng(seed)
        self.P = P or max(T, 32)
        self.h = clk.Cache(B, pages, B * pages, self.P)
        self.kind, self.Hkv, self.D, self.layers, self.layer, self.B = kind, Hkv, D, layers, layer, B
        self.pool = pool8(2 * (layer + layers), B * pages, Hkv, self.P, D, T, seed, order, pad)
        self.model = Eight(self.pool.data, self.pool.scale)
        self.table = angles(pages * self.P, pairs) if pairs else None
        self.neighbours = neighbours
        self.rot = clk.Rotary(self.table.cuda(), neighbours) if pairs else None
        self.seed = seed * 1000

    def rows(self, n, size=1.0):
        self.seed += 1
        return normal((self.layers, n, self.Hkv, self.D), self.kind, self.seed) * size

    def add(self, slots, counts, form="packed", size=1.0, k=None, v=None, sides=False):
        clk.cache_grow(self.h, ints(slots), ints(counts))
        self.write(slots, counts, form, size, k, v, sides)

    def write(self, slots, counts, form="packed", size=1.0, k=None, v=None, sides=False):
        B = len(slots)
        kw = {}
        if form == "packed":
            off = np.cumsum([0] + counts).tolist()
            at = [list(range(off[b], off[b + 1])) for b in range(B)]
            n = off[-1]
            kw["offsets"] = ints(off, torch.int64)
        else:
            N = max(counts + [1])
            n = B * N
            at = [[b * N + i for i in range(counts[b])] for b in range(B)]
            if form == "path":
                path = [self.rng.integers(0, N, size=N).tolist() for _ in range(B)]
                kw["path"] = ints(path)
                at = [[b * N + path[b][i] for i in range(counts[b])] for b in range(B)]
        k = self.rows(n, size) if k is None else k
        v = self.rows(n, size) if v is None else v
        shape = k.shape if form == "packed" else (self.layers, B, -1, self.Hkv, self.D)
        if sides:
            q = normal(shape[1:-2] + (3, self.D), self.kind, self.seed + 7) if form == "packed" else normal((B, N, 3, self.D), self.kind, self.seed + 7)
            qo, ko = torch.zeros_like(q), torch.zeros_like(k.reshape(shape))
            kw.update(q=q, q_out=qo, k_out=ko)
        clk.cache_append_rotary(self.h, ints(slots), self.pool, k.reshape(shape), v.reshape(shape), ints(counts), rotary=self.rot, layer=self.layer, **kw)
        torch.cuda.synchronize()
        table, length = self.h.table.cpu(), self.h.length.cpu()
        k, v = k.cpu(), v.cpu()
        for b, s in enumerate(slots):
            p0, n = int(length[s]) - counts[b], counts[b]
            if n == 0:
                continue
            for l in range(self.layers):
                rk = turned(k[l][at[b]], range(p0, p0 + n), self.table, self.neighbours) if self.rot else k[l][at[b]].float()
                for x, y in ((0, rk), (1, v[l][at[b]].float())):
                    self.model.append(2 * (self.layer + l) + x, table[s].tolist(), p0, y)
                if sides:
                    rq = turned(q.cpu().flatten(0, -3)[at[b]], range(p0, p0 + n), self.table, self.neighbours).to(DT[self.kind])
                    assert same(qo.flatten(0, -3).cpu()[at[b]], rq) and same(ko[0].flatten(0, -3).cpu()[at[b]], rk.to(DT[self.kind]))

    def check(self, status=0):
        assert self.h.status()[0] == status
        assert same(self.pool.scale, self.model.scale)
        assert same(self.pool.data, self.model.codes)


@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("T", [16, 32, 64, 128])
@pytest.mark.parametrize("D,pairs", [(128, 64), (64, 32), (64, 0), (96, 24), (80, 40), (16, 8), (256, 128), (33, 7)])
def test_rows_in_8_bits(kind, T, D, pairs):
    c = Case(D + T, 3, 2, D, T, kind, pairs=pairs, neighbours=D == 96, pages=10 if T > 32 else 20)
    c.add([2, 0, 1], [T + 3, 1, 2 * T])
    c.add([1, 2, 0], [5, T // 2, 7], "dense", size=3.0)
    c.add([0, 1, 2], [9, 3, 1], "path", size=0.1)
    c.check()


@pytest.mark.parametrize("T,P", [(16, 16), (16, 64), (16, 128), (32, 128), (64, 64), (128, 128)])
def test_single_tokens_that_grow_their_blocks(T, P):
    """Each token larger than those before, then smaller; scales grow and earlier rows are rounded again."""
    c = Case(T + P, 2, 2, 64, T, "bf16", P=P, pairs=32, pages=4)
    for i in range(40):
        c.add([0, 1], [1, i % 3], size=0.01 * 1.5 ** (i if i < 25 else 50 - i))
    c.check()


@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 31, 33, 127, 129, 500])
def test_lengths(n):
    c = Case(n, 2, 1, 128, 32, "f16", P=64, pairs=64)
    c.add([0, 1], [n, max(1, n // 2)])
    c.add([0, 1], [3, n])
    c.check()


@pytest.mark.parametrize("order", ["pnht", "pnth", "npth", "hnpt"])
def test_pool_orders_layers_and_odd_rows(order):
    c = Case(1, 2, 3, 64, 16, "bf16", layers=3, layer=1, pairs=32, order=order)
    c.add([0, 1], [20, 37])
    c.add([0, 1], [5, 1], "path", size=4.0)
    c.check()
    c = Case(2, 2, 3, 64, 16, "bf16", layers=2, pairs=32, order=order, pad=5)
    c.add([0, 1], [20, 37])
    c.add([0, 1], [5, 1], "dense", size=4.0)
    c.check()


def test_queries_and_keys_beside_the_pages():
    for form in ("packed", "dense"):
        for kind, D in (("bf16", 128), ("f32", 40)):
            c = Case(3, 3, 2, D, 16, kind, pairs=D // 2)
            c.add([0, 2], [5, 40], form, sides=True)
            c.add([2, 1], [1, 1], form, sides=True)
            c.check()


@pytest.mark.parametrize("kind,D", [("bf16", 64), ("f32", 24)])
def test_extreme_values(kind, D):
    """Zeros, infinities, NaN, the type's ends, values on and next to the border of a scale."""
    top = torch.finfo(DT[kind]).max
    tiny = torch.finfo(DT[kind]).tiny
    for seed, fill in enumerate([[0.0], [-0.0], [INF, 1.0], [-INF], [NAN], [NAN, INF, 2.0], [top, -top], [tiny, -tiny, 0.0], [448.0, 1.0],
                                 [449.0, 1.0], [450.0, -1.0], [-448.0 * 2 ** -20, 0.0], [1e-30, 1e30], [2.0 ** -133]]):
        c = Case(seed, 1, 1, D, 16, kind)
        x = torch.tensor(fill, device="cuda").to(DT[kind])
        c.add([0], [7], k=x[torch.arange(7 * D, device="cuda") % len(fill)].view(1, 7, 1, D))
        c.add([0], [4], size=0.25)
        c.add([0], [8], v=x[torch.arange(8 * D, device="cuda") % len(fill)].view(1, 8, 1, D))
        c.check()


def test_scales_that_came_from_elsewhere():
    """A block's scale may be any positive number, and one that is none does not count."""
    for had in (0.3, 1e-3, 77.7, 0.0, -1.0, NAN, INF, 1e-40, 3e38):
        for kind, D in (("bf16", 64), ("f32", 24)):
            c = Case(4, 1, 2, D, 16, kind, pairs=8)
            c.add([0], [5])
            c.pool.scale.fill_(had)
            c.model.scale.fill_(had)
            c.add([0], [6])
            c.check()


def test_repeated_and_layer_by_layer():
    c = Case(5, 2, 2, 64, 16, "bf16", layers=1)
    c.add([0, 1], [19, 5])
    k, v = c.rows(9), c.rows(9)
    clk.cache_grow(c.h, ints([0, 1]), ints([4, 5]))
    for _ in range(3):
        c.write([0, 1], [4, 5], k=k, v=v)
    c.check()


def test_many_requests():
    B = 700
    c = Case(6, B, 1, 64, 16, "bf16", P=16, pages=4, pairs=32)
    order = c.rng.permutation(B).tolist()
    c.add(order, c.rng.integers(0, 33, size=B).tolist())
    c.add(order[::-1], c.rng.integers(0, 4, size=B).tolist(), "dense", size=2.0)
    c.check()


def test_a_long_prompt_in_large_blocks():
    c = Case(7, 2, 4, 128, 128, "bf16", P=128, pages=20, pairs=64)
    c.add([0, 1], [1501, 700], sides=True)
    c.check()


def test_bad_requests_are_left_out():
    c = Case(8, 4, 1, 64, 16, "bf16", pairs=32)
    c.add([0, 1, 2, 3], [20, 20, 20, 20])
    k = c.rows(12)
    clk.cache_append_rotary(c.h, ints([0, 9, 2, 3]), c.pool, k, k.clone(), ints([3, 3, 30, -1]), rotary=c.rot, offsets=ints([3, 0, 6, 9, 12], torch.int64))
    torch.cuda.synchronize()
    c.check(status=clk.EINVAL)


def same_rows(c, a, b, n):
    """Slots a and b stand for the same rows."""
    table, P, T = c.h.table.cpu(), c.P, c.model.T
    data, scale = c.pool.data.float().cpu(), c.pool.scale.cpu()
    for p in range(n):
        x, y = int(table[a, p // P]), int(table[b, p // P])
        assert same(data[:, x, :, p % P], data[:, y, :, p % P]) and same(scale[:, x, :, p % P // T], scale[:, y, :, p % P // T])


@pytest.mark.parametrize("order,pad", [("pnht", 0), ("npth", 0), ("pnht", 3)])
def test_forks_take_their_scales_along(order, pad):
    c = Case(9, 4, 2, 64, 16, "bf16", P=64, layers=2, pages=6, order=order, pad=pad)
    c.add([0, 1], [150, 64])
    clk.cache_fork(c.h, ints([0, 1]), ints([2, 3]), c.pool)
    torch.cuda.synchronize()
    assert c.h.length.tolist() == [150, 64, 150, 64]
    same_rows(c, 0, 2, 150)
    same_rows(c, 1, 3, 64)
    first = int(c.h.table[0, 2]), int(c.h.table[2, 2])
    assert first[0] != first[1]
    # each goes on by itself
    c.model = Eight(c.pool.data, c.pool.scale)
    c.add([2, 0], [3, 3], size=9.0)
    c.check()
    for bad in ([0], [2]):
        clk.cache_fork(c.h, ints(bad), ints([3]), c.pool)
    torch.cuda.synchronize()
    c.check(status=clk.EINVAL)


@pytest.mark.parametrize("pages", [6, 200])
def test_compaction_moves_scales(pages):
    """Small tables (one launch fewer) and larger ones."""
    c = Case(10, 16, 2, 64, 16, "bf16", P=32, layers=2, pages=pages)
    lens = c.rng.integers(1, 150, size=16).tolist()
    c.add(list(range(16)), lens)

    def held():
        torch.cuda.synchronize()
        table, P, T = c.h.table.cpu(), c.P, c.model.T
        data, scale = c.pool.data.float().cpu(), c.pool.scale.cpu()
        return [[(data[:, int(table[s, p // P]), :, p % P].clone(), scale[:, int(table[s, p // P]), :, p % P // T].clone()) for p in range(lens[s])]
                for s in range(1, 16, 2)]

    before = held()
    clk.cache_free(c.h, ints(list(range(0, 16, 2))))
    moved = ints([0])
    clk.cache_compact(c.h, c.pool, moved)
    after = held()
    assert int(moved) > 0 and c.h.status()[0] == 0
    assert all(same(a, x) and same(b, y) for r, t in zip(before, after) for (a, b), (x, y) in zip(r, t))


def test_pools_and_arguments_that_do_not_fit():
    h = clk.Cache(2, 4, 8, 32)
    p = clk.ScaledPool.empty(1, 8, 2, 32, 64, block=16)
    assert p.data.shape == (2, 8, 2, 32, 64) and p.scale.shape == (2, 8, 2, 2)
    data, scale = p.data, p.scale
    for d, s in ((data.float(), scale), (data, scale.half()), (data[0], scale), (data, scale[:, :7]), (data, scale[..., :0]), (data, scale[:1]),
                 (data, torch.ones((2, 8, 2, 4), device="cuda")), (data.cpu(), scale), (data, scale.cpu()),
                 (data.transpose(3, 4), scale)):
        with pytest.raises(ValueError):
            clk.ScaledPool(d, s)
    k = normal((1, 2, 3, 2, 64), "bf16", 1)
    n = ints([3, 3])
    rot = clk.Rotary(angles(64, 32).cuda())
    with pytest.raises(ValueError):
        clk.cache_append_rotary(clk.Cache(2, 4, 9, 32), ints([0, 1]), p, k, k, n)
    with pytest.raises(ValueError):
        clk.cache_append_rotary(h, ints([0, 1]), p, k[..., :32], k[..., :32], n)
    with pytest.raises(ValueError):
        clk.cache_append_rotary(h, ints([0, 1]), data, k, k, n)
    with pytest.raises(ValueError):
        clk.cache_append_rotary(h, ints([0, 1]), p, k, k, n, rotary=rot, q=k[0])
    with pytest.raises(ValueError):
        clk.cache_append_rotary(h, ints([0, 1]), p, k, k, n, k_out=k)
    with pytest.raises(ValueError):
        clk.cache_append_rotary(h, ints([0, 1]), p, k, k, n, rotary=rot, k_out=k, path=ints([[0, 1, 2]] * 2))
    with pytest.raises(clk.ClkError):
        clk.cache_append_rotary(h, ints([0, 1]), p, k, k, n, rotary=clk.Rotary(angles(64, 33).cuda()))
    for bad in (angles(4, 2), angles(4, 2).cuda().half(), angles(4, 2).cuda()[:, :1], angles(4, 4).cuda()[..., :2]):
        with pytest.raises(ValueError):
            clk.Rotary(bad)
