"""The paged cache's calls against a plain model of it: page numbers, lengths
and holder counts exactly, and every row that a slot holds bit for bit.  GPU."""
import numpy as np
import pytest
import torch

import context_lookup_speculative_gb300 as clk
from cache_model import CacheModel

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def ints(v, dtype=torch.int32):
    return torch.tensor(v, dtype=dtype, device="cuda")


class Both:
    """The cache and the model, driven together.  Rows carry marks: the row
    of mark m holds m + plane, spread over heads and elements."""

    def __init__(self, slots, max_pages, pages, P, layers=1, heads=2, dim=8, kind="bf16", order="phtd"):
        self.h = clk.Cache(slots, max_pages, pages, P)
        self.m = CacheModel(slots, max_pages, pages, P)
        self.P, self.layers, self.heads, self.dim, self.dt = P, layers, heads, dim, DT[kind]
        sizes = {"p": 2 * layers, "n": pages + 3, "h": heads, "t": P}
        names = {"phtd": "pnht", "pthd": "pnth", "npth": "npth", "hnpt": "hnpt"}[order]
        raw = torch.full([sizes[c] for c in names] + [dim], -7.0, dtype=self.dt, device="cuda")
        self.pool = raw.permute([names.index(c) for c in "pnht"] + [4])
        self.mark = 0

    def value(self, marks, plane):
        """[rows, heads, dim] of small whole numbers that every type holds exactly."""
        m = np.asarray(marks, dtype=np.int64).reshape(-1, 1, 1)
        h = np.arange(self.heads).reshape(1, -1, 1)
        d = np.arange(self.dim).reshape(1, 1, -1)
        return ((m * 7 + plane * 31 + h * 13 + d * 3) % 251).astype(np.float32)

    def grow(self, slots, counts):
        clk.cache_grow(self.h, ints(slots), ints(counts))
        return self.m.grow(slots, counts)

    def append(self, slots, counts, path=None, packed=False):
        B = len(slots)
        N = max([1] + list(counts)) + 2
        if path is not None:
            N = max(N, max(max(p + [0]) for p in path) + 1)
        if packed:
            off = np.concatenate([[0], np.cumsum([c + i % 2 for i, c in enumerate(counts)])])
            rows = int(off[-1])
        else:
            off, rows = np.arange(B + 1) * N, B * N
        marks = np.arange(self.mark, self.mark + rows)
        self.mark += rows
        k = np.stack([self.value(marks, 2 * l) for l in range(self.layers)])
        v = np.stack([self.value(marks, 2 * l + 1) for l in range(self.layers)])
        shape = (self.layers, rows) if packed else (self.layers, B, N)
        # sources lie inside a wider tensor, as slices of a projection's output do
        wide = torch.zeros(shape + (2 * self.heads, self.dim), dtype=self.dt, device="cuda")
        wide[..., :self.heads, :] = torch.from_numpy(k).to("cuda", self.dt).view(*shape, self.heads, self.dim)
        wide[..., self.heads:, :] = torch.from_numpy(v).to("cuda", self.dt).view(*shape, self.heads, self.dim)
        p = None
        if path is not None:
            p = ints([q + [-1] * (N - len(q)) for q in path])
        clk.cache_append(self.h, ints(slots), self.pool, wide[..., :self.heads, :], wide[..., self.heads:, :], ints(counts),
                         path=p, offsets=ints(off, torch.int64) if packed else None)
        self.m.append(slots, [[int(off[b]) + marks[0] + (path[b][i] if path else i) for i in range(c)]
                              for b, c in enumerate(counts)])

    def check(self, status=0):
        torch.cuda.synchronize()
        assert self.h.status()[0] == status
        assert self.h.length.tolist() == self.m.len
        assert self.h.refs.tolist() == self.m.refs
        want = [t + [-1] * (self.h.max_pages - len(t)) for t in self.m.table]
        assert self.h.table.tolist() == want
        pool = self.pool.float().cpu().numpy()
        keys = list(self.m.rows)
        if keys:
            pages, rows = np.array(keys).T
            marks = np.array([self.m.rows[k] for k in keys])
            for plane in range(2 * self.layers):
                assert np.array_equal(pool[plane][pages, :, rows], self.value(marks, plane))
        untouched = np.ones(pool.shape[1:2] + (self.P,), dtype=bool)
        for p, r in keys:
            untouched[p, r] = False
        assert (pool.transpose(1, 3, 0, 2, 4)[untouched] == -7.0).all()


@pytest.mark.parametrize("P", [16, 32, 64, 128])
@pytest.mark.parametrize("kind,dim,order", [("bf16", 8, "phtd"), ("f16", 5, "pthd"), ("f32", 1, "npth"), ("bf16", 200, "hnpt"),
                                            ("f16", 6, "phtd"), ("f32", 256, "pthd"), ("bf16", 36, "npth")])
def test_life_of_a_cache(P, kind, dim, order):
    """Prompts, a step's accepted rows, forks, freeing and compaction."""
    rng = np.random.default_rng(P + dim)
    c = Both(12, 9, 70, P, layers=2, heads=3, dim=dim, kind=kind, order=order)
    slots, counts = [4, 0, 9, 2], [3 * P + 5, P, 1, 0]
    assert c.grow(slots, counts) == []
    c.append(slots, counts, packed=True)
    c.check()
    assert c.grow([2, 4, 0], [2 * P + 1, P, P - 1]) == []
    c.append([2, 4, 0], [2 * P + 1, P, P - 1])
    c.check()
    assert c.m.fork([4, 4, 0, 9], [1, 3, 5, 6]) == []
    clk.cache_fork(c.h, ints([4, 4, 0, 9]), ints([1, 3, 5, 6]), c.pool)
    c.check()
    path = [[0, 2, 3], [0], [0, 1, 4, 7], [0, 5]]
    counts = [len(p) for p in path]
    assert c.grow([1, 3, 4, 9], counts) == []
    c.append([1, 3, 4, 9], counts, path=path)
    c.check()
    for gone in ([4, 0], [6, 3]):
        c.m.free(gone)
        clk.cache_free(c.h, ints(gone))
        c.check()
    moved = ints([-1])
    clk.cache_compact(c.h, c.pool, moved)
    assert moved.tolist() == [c.m.compact()]
    c.check()
    more = rng.integers(0, P, size=3).tolist()
    assert c.grow([1, 0, 2], more) == []
    c.append([1, 0, 2], more)
    c.check()


@pytest.mark.parametrize("seed", range(4))
def test_random_calls(seed):
    rng = np.random.default_rng(seed)
    c = Both(40, 6, 150, 16, heads=1, dim=8)
    failures = 0
    for _ in range(25):
        used = [s for s in range(40) if c.m.len[s]]
        empty = [s for s in range(40) if not c.m.len[s]]
        what = rng.integers(0, 5)
        if what <= 1:
            slots = rng.permutation(40)[:rng.integers(1, 20)].tolist()
            counts = rng.integers(0, 40, size=len(slots)).tolist()
            bad = c.grow(slots, counts)
            failures += len(bad)
            good = [b for b in range(len(slots)) if b not in bad]
            if good:
                c.append([slots[b] for b in good], [counts[b] for b in good], packed=bool(what))
        elif what == 2 and used and empty:
            n = int(rng.integers(1, len(empty) + 1))
            src = rng.choice(used, size=n).tolist()
            failures += len(c.m.fork(src, empty[:n]))
            clk.cache_fork(c.h, ints(src), ints(empty[:n]), c.pool)
        elif what == 3 and used:
            gone = rng.permutation(used)[:rng.integers(1, len(used) + 1)].tolist()
            c.m.free(gone)
            clk.cache_free(c.h, ints(gone))
        else:
            c.m.compact()
            clk.cache_compact(c.h, c.pool)
        st = c.h.status()[0]
        assert st in (0, clk.ECAPACITY)
        c.h.status_clear()
        c.check()


def test_lack_of_pages_leaves_the_request_as_it_was():
    c = Both(6, 4, 7, 16, heads=1)
    assert c.grow([0, 1], [33, 17]) == []  # 3 + 2 pages
    c.append([0, 1], [33, 17])
    # 2 free pages: the second of these does not fit, nor does the fourth after it; the third needs none
    assert c.grow([2, 3, 0, 4], [16, 32, 5, 16]) == [1, 3]
    c.check(status=clk.ECAPACITY)
    assert c.h.status()[1] in (3, 4)
    c.h.status_clear()
    assert c.grow([5], [65]) == [0]  # more than the table holds
    c.check(status=clk.ECAPACITY)
    c.h.status_clear()
    assert c.m.fork([0, 1], [3, 4]) == [1]
    clk.cache_fork(c.h, ints([0, 1]), ints([3, 4]), c.pool)
    c.check(status=clk.ECAPACITY)
    assert c.h.status()[1] == 4


def test_large_batches_and_many_pages():
    """More requests than a planning CTA has threads, more pages than one scan step sees."""
    c = clk.Cache(3000, 90, 200000, 16)
    rng = np.random.default_rng(5)
    slots = rng.permutation(3000)
    counts = rng.integers(0, 1400, size=3000)
    clk.cache_grow(c, ints(slots), ints(counts))
    pages = (counts + 15) // 16
    first = np.cumsum(pages) - pages
    ok = (first + pages <= 200000) | (pages == 0)
    torch.cuda.synchronize()
    assert (c.status()[0] == clk.ECAPACITY) == (not ok.all())
    table, length = c.table.cpu().numpy(), c.length.cpu().numpy()
    for b in range(3000):
        n = pages[b] if ok[b] else 0
        assert length[slots[b]] == (counts[b] if ok[b] else 0)
        assert table[slots[b], :n].tolist() == list(range(first[b], first[b] + n)) and (table[slots[b], n:] == -1).all()


@pytest.mark.parametrize("call", ["grow", "append", "fork", "free"])
def test_bad_slots_and_counts_are_latched_and_skipped(call):
    c = Both(4, 4, 16, 16, heads=1)
    c.grow([0], [20])
    c.append([0], [20])
    k = torch.zeros((1, 2, 8, 1, 8), dtype=c.dt, device="cuda")
    for bad in (-1, 4):
        if call == "grow":
            clk.cache_grow(c.h, ints([bad, 1]), ints([3, 3]))
            c.m.grow([1], [3])
        elif call == "append":
            clk.cache_append(c.h, ints([bad, 2]), c.pool, k, k, ints([1, 0]))
        elif call == "fork":
            clk.cache_fork(c.h, ints([bad]), ints([3]), c.pool)
            c.check(status=clk.EINVAL)
            clk.cache_fork(c.h, ints([0]), ints([bad]), c.pool)
        else:
            clk.cache_free(c.h, ints([bad, 3]))
        c.check(status=clk.EINVAL)
        assert c.h.status()[1] == 0  # the batch position
        c.h.status_clear()
    if call == "grow":
        clk.cache_grow(c.h, ints([2]), ints([-1]))
    elif call == "append":
        for n, path in ((21, None), (9, None), (-1, None), (2, [0, 8]), (2, [-1, 0])):
            # more than held, more than given, negative, a path out of range
            c.h.status_clear()
            kk = torch.full((1, 1, 8, 1, 8), -7.0, dtype=c.dt, device="cuda")
            p = None if path is None else ints([path + [0] * 6])
            if path is not None:
                # the rows that can be written are
                c.m.rows = {q: m for q, m in c.m.rows.items() if q[1] not in (2, 3) or q[0] != c.m.table[0][1]}
            clk.cache_append(c.h, ints([0]), c.pool, kk, kk, ints([n]), path=p)
            assert c.h.status() == (clk.EINVAL, 0)
        c.pool[:, c.m.table[0][1], :, 2:4] = -7.0
        c.check(status=clk.EINVAL)
        c.h.status_clear()
        for off in ([0, 9], [-1, 3], [3, 2]):
            clk.cache_append(c.h, ints([0]), c.pool, kk[:, 0], kk[:, 0], ints([3]), offsets=ints(off, torch.int64))
            assert c.h.status() == (clk.EINVAL, 0)
            c.h.status_clear()
        return
    elif call == "fork":
        clk.cache_fork(c.h, ints([0]), ints([0]), c.pool)
    else:
        return
    c.check(status=clk.EINVAL)


def test_a_slot_listed_twice_is_freed_once():
    c = Both(4, 4, 16, 16, heads=1)
    c.grow([0, 1], [40, 20])
    clk.cache_free(c.h, ints([1, 1, 0]))
    c.m.free([1, 0])
    c.check()


def test_a_pool_of_more_than_two_to_the_32_elements():
    """Offsets past 32 bits: the last pages of a pool of 4.5 billion elements."""
    pages, P, heads, dim = 8600, 128, 16, 128
    h = clk.Cache(3, pages, pages, P)
    pool = torch.empty((2, pages, heads, P, dim), dtype=torch.bfloat16, device="cuda")
    assert pool.numel() > 1 << 32
    n = (pages - 2) * P - 3
    clk.cache_grow(h, ints([0]), ints([n]))
    clk.cache_grow(h, ints([0]), ints([7]))
    k = torch.randn((1, 1, 7, heads, dim), device="cuda").to(torch.bfloat16)
    v = torch.randn((1, 1, 7, heads, dim), device="cuda").to(torch.bfloat16)
    clk.cache_append(h, ints([0]), pool, k, v, ints([7]))
    clk.cache_fork(h, ints([0]), ints([2]), pool)
    torch.cuda.synchronize()
    assert h.status()[0] == 0
    last = pages - 2
    assert h.table[0, last].item() == last and h.table[2, last].item() == last + 1
    for plane, x in ((0, k), (1, v)):
        got = torch.cat([pool[plane, last - 1, :, P - 3:], pool[plane, last, :, :4]], 1)
        assert torch.equal(got, x[0, 0].transpose(0, 1))
        assert torch.equal(pool[plane, last + 1, :, :4], x[0, 0, 3:].transpose(0, 1))
    clk.cache_free(h, ints([0]))
    moved = ints([-1])
    clk.cache_compact(h, pool, moved)
    assert moved.item() == 1
    assert torch.equal(pool[1, last, :, :4], v[0, 0, 3:].transpose(0, 1))
    assert torch.equal(pool[0, last - 1, :, P - 3:], k[0, 0, :3].transpose(0, 1))


def test_in_a_graph_and_on_another_stream():
    c = Both(8, 4, 40, 16, layers=1, heads=2, dim=8)
    c.grow([0, 1], [30, 7])
    c.append([0, 1], [30, 7])
    s = torch.cuda.Stream()
    src, dst = ints([0, 1]), ints([2, 3])
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        clk.cache_fork(c.h, src, dst, c.pool)
    s.synchronize()
    c.m.fork([0, 1], [2, 3])
    c.check()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        clk.cache_free(c.h, dst)
        clk.cache_fork(c.h, src, dst, c.pool)
        clk.cache_compact(c.h, c.pool)
    for _ in range(2):
        g.replay()
        c.m.free([2, 3])
        c.m.fork([0, 1], [2, 3])
        c.m.compact()
        c.check()


@pytest.mark.parametrize("max_slots,max_pages", [(12, 9), (12, 170), (12, 171), (2000, 9)])
def test_compaction_of_small_and_large_tables(max_slots, max_pages):
    """One CTA rewrites small tables, one per slot large ones (the limit lies between 170 and 171)."""
    c = Both(max_slots, max_pages, 70, 16, layers=1, heads=2, dim=8)
    slots, counts = [4, 0, 9, 2], [3 * 16 + 5, 16, 33, 90]
    assert c.grow(slots, counts) == []
    c.append(slots, counts, packed=True)
    assert c.m.fork([4, 2, 2], [1, 3, 11]) == []
    clk.cache_fork(c.h, ints([4, 2, 2]), ints([1, 3, 11]), c.pool)
    for gone in ([0, 4], [2], [1, 9]):
        c.m.free(gone)
        clk.cache_free(c.h, ints(gone))
        moved = ints([-1])
        clk.cache_compact(c.h, c.pool, moved)
        assert moved.tolist() == [c.m.compact()]
        c.check()


@pytest.mark.parametrize("layers,dim", [(1, 8), (2, 8), (4, 16), (2, 200)])
def test_groups_of_rows_of_every_size(layers, dim):
    """8, 16 or 32 rows a CTA, by their size and number: packed rows, paths, and tails of forks, ragged at every end."""
    rng = np.random.default_rng(layers + dim)
    c = Both(140, 5, 400, 16, layers=layers, heads=1, dim=dim)
    slots = rng.permutation(70).tolist()
    counts = [int(x) for x in rng.integers(0, 60, size=70)]
    assert c.grow(slots, counts) == []
    c.append(slots, counts, packed=True)
    c.check()
    dst = [70 + b for b in range(70)]
    bad = c.m.fork(slots, dst)
    assert bad == []
    clk.cache_fork(c.h, ints(slots), ints(dst), c.pool)
    c.check()
    path = [sorted(rng.choice(13, size=1 + b % 5, replace=False).tolist()) for b in range(70)]
    counts = [len(p) for p in path]
    assert c.grow(dst, counts) == []
    c.append(dst, counts, path=path)
    c.check()
