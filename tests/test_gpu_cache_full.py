"""What cache_append may write: only rows that a grow made room for, and never
rows that another slot holds too.  An exhausted pool is the ordinary way to a
grow that fails, and no call synchronises, so that the append with the same
counts follows it unseen.  GPU."""
import math

import pytest
import torch

import context_lookup_speculative_gb300 as clk
from test_gpu_cache import Both, ints

pytestmark = pytest.mark.gpu


def append_to(c, slots, counts, good, **kw):
    """Appends for all slots, where the rows of batch positions `good` alone are to be written."""
    whole = c.m.append

    def some(at, marks):
        whole([at[b] for b in good], [marks[b] for b in good])

    c.m.append = some
    c.append(slots, counts, **kw)
    c.m.append = whole


@pytest.mark.parametrize("packed", [False, True])
def test_append_after_a_grow_that_failed(packed):
    """Slots 0 and 1 share two full pages, slot 2 ends inside its second page, slot 3 has room: 5 pages, all taken."""
    c = Both(6, 4, 5, 16, layers=2, heads=2)
    assert c.grow([0, 2, 3], [32, 20, 5]) == []
    c.append([0, 2, 3], [32, 20, 5])
    assert c.m.fork([0], [1]) == []
    clk.cache_fork(c.h, ints([0]), ints([1]), c.pool)
    c.check()
    slots, counts = [0, 1, 2, 3], [3, 2, 13, 4]
    assert c.grow(slots, counts) == [0, 1, 2]
    append_to(c, slots, counts, good=[3], packed=packed)
    c.check(status=clk.ECAPACITY)
    # again, after the host has seen the failure and cleared it
    c.h.status_clear()
    append_to(c, slots, counts, good=[3], packed=packed)
    c.check(status=clk.EINVAL)
    c.h.status_clear()
    # with pages to be had the same slots go on
    c.m.free([2])
    clk.cache_free(c.h, ints([2]))
    assert c.grow([0, 1], [3, 2]) == []
    c.append([0, 1], [3, 2], packed=packed)
    c.check()


def test_append_by_path_after_a_grow_that_failed():
    c = Both(4, 4, 4, 16)
    assert c.grow([0, 1], [32, 30]) == []
    c.append([0, 1], [32, 30])
    path = [[0, 3], [0, 2]]
    assert c.grow([0, 1], [2, 2]) == [0]
    append_to(c, [0, 1], [2, 2], good=[1], path=path)
    c.check(status=clk.ECAPACITY)


def test_append_after_a_count_that_grow_refused():
    c = Both(4, 3, 12, 16)
    assert c.grow([0, 1], [20, 20]) == []
    c.append([0, 1], [20, 20])
    assert c.grow([0, 1], [-1, 29]) == [0, 1]
    c.check(status=clk.EINVAL) if c.h.status()[0] == clk.EINVAL else c.check(status=clk.ECAPACITY)
    append_to(c, [0, 1], [1, 20], good=[])
    c.h.status_clear()
    c.append([0, 1], [0, 0])  # nothing to write is never wrong
    c.check()


def test_rows_that_two_slots_hold_are_not_written():
    c = Both(6, 4, 12, 16)
    assert c.grow([0, 2], [32, 20]) == []
    c.append([0, 2], [32, 20])
    assert c.m.fork([0, 2], [1, 3]) == []
    clk.cache_fork(c.h, ints([0, 2]), ints([1, 3]), c.pool)
    for slot in (0, 1):  # both pages are shared
        append_to(c, [slot], [1], good=[])
        c.check(status=clk.EINVAL)
        c.h.status_clear()
    for slot in (2, 3):  # the first page is shared, the last four rows are the slot's own
        append_to(c, [slot], [5], good=[])
        c.check(status=clk.EINVAL)
        c.h.status_clear()
        c.append([slot], [4])
        c.check()
    assert c.grow([0, 1], [3, 2]) == []
    append_to(c, [0, 1], [4, 2], good=[1])
    c.check(status=clk.EINVAL)
    c.h.status_clear()
    c.append([0], [3])
    c.check()


def test_rows_of_several_grows_and_rows_written_again():
    """Room taken in rounds is filled by one append, and an append may be repeated."""
    c = Both(4, 5, 20, 16, layers=2)
    for n in (3, 20, 9):
        assert c.grow([1, 2], [n, 2 * n]) == []
    c.append([1, 2], [32, 64])
    c.append([1, 2], [32, 60])
    c.check()
    c.m.free([2])
    clk.cache_free(c.h, ints([2]))
    assert c.grow([2], [7]) == []
    c.append([2], [7])
    c.check()
    c.h.reset()
    c.m.free([1, 2])
    assert c.grow([1, 2], [16, 3]) == []
    c.append([1, 2], [16, 3])
    c.m.rows = {at: m for at, m in c.m.rows.items() if at in {(c.m.table[s][i // 16], i % 16) for s in (1, 2) for i in range(c.m.len[s])}}
    torch.cuda.synchronize()
    pool, keys = c.pool.float().cpu().numpy(), list(c.m.rows)
    for page, row in keys:
        assert (pool[0][page, :, row] == c.value([c.m.rows[page, row]], 0)[0]).all()


def test_a_full_pool_leaves_the_other_requests_attention_as_it_was():
    P, D, Hkv, G = 16, 64, 1, 2
    h = clk.Cache(4, 4, 2, P)
    g = torch.Generator(device="cuda").manual_seed(1)
    pool = torch.empty((2, 2, Hkv, P, D), dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    clk.cache_grow(h, ints([0]), ints([32]))
    clk.cache_fork(h, ints([0]), ints([1]), pool)
    qkv = torch.empty((1, 4, G * Hkv + 2 * Hkv, D), dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    q, k, v = qkv[:, :, :G * Hkv], qkv[:, :, G * Hkv:-Hkv], qkv[:, :, -Hkv:]
    mask = torch.tensor([[1, 3, 7, 15]], dtype=torch.int64, device="cuda")
    scratch = clk.attend_scratch(G * Hkv, Hkv, D)

    def attend(slot):
        out = torch.zeros((1, 4, G * Hkv, D), dtype=torch.bfloat16, device="cuda")
        clk.tree_attend(h, ints([slot]), pool, 0, q, k, v, ints([4]), mask, 1 / math.sqrt(D), out, scratch)
        torch.cuda.synchronize()
        return out

    before = attend(1)
    clk.cache_grow(h, ints([0]), ints([3]))  # no page left
    clk.cache_append(h, ints([0]), pool, k[None], v[None], ints([3]))
    assert torch.equal(attend(1), before)
    assert torch.equal(attend(0), before)
    assert h.status() == (clk.ECAPACITY, 0)
