"""The cache, tree and attention calls refuse bad arguments before anything is
launched.  CPU only: pointers are made up, and no call here reaches a GPU."""
import ctypes
import os

import pytest

P = 0x10000  # an aligned, made-up device pointer


@pytest.fixture(scope="module")
def clk():
    import context_lookup_speculative_gb300 as clk_mod
    if not os.path.exists(clk_mod.LIB_PATH):
        from context_lookup_speculative_gb300 import build
        build.build()
    return clk_mod


@pytest.fixture()
def cache(clk):
    L = clk.lib()
    n = ctypes.c_size_t()
    assert L.clk_cache_workspace_bytes(4, 8, 32, ctypes.byref(n)) == 0
    h = ctypes.c_void_p()
    assert L.clk_cache_create(ctypes.byref(h), 4, 8, 32, 16, 1 << 20, n.value) == 0
    yield h
    L.clk_cache_destroy(h)


def pool_of(clk, **kw):
    d = dict(d_base=P, dtype=clk.BF16, planes=4, heads=2, dim=64, plane_stride=32 * 2 * 16 * 64, page_stride=2 * 16 * 64,
             head_stride=16 * 64, tok_stride=64)
    d.update(kw)
    return clk.PoolDesc(**d)


BAD_POOLS = [dict(d_base=None), dict(d_base=P + 1), dict(dtype=3), dict(planes=3), dict(planes=0), dict(heads=0), dict(dim=0),
             dict(dim=257), dict(page_stride=-1), dict(plane_stride=-1), dict(head_stride=-1), dict(tok_stride=-1)]


def attn_of(clk, **kw):
    d = dict(dtype=clk.BF16, q_heads=4, kv_heads=2, dim=64, scale=0.1, d_q=P, d_k=P, d_v=P, d_out=P, q_req=1024, q_row=256,
             q_head=64, k_req=512, k_row=128, k_head=64, v_req=512, v_row=128, v_head=64)
    d.update(kw)
    return clk.AttnDesc(**d)


BAD_ATTN = [dict(dtype=5), dict(q_heads=3), dict(q_heads=1), dict(kv_heads=0), dict(dim=0), dict(dim=257), dict(dim=128),
            dict(scale=float("nan")), dict(scale=float("inf")), dict(d_q=P + 1), dict(d_out=P + 1), dict(q_row=-1), dict(v_head=-1),
            dict(d_k=None), dict(d_out=None)]


def test_cache_sizes_and_creation(clk):
    L = clk.lib()
    n = ctypes.c_size_t()
    for bad in ((0, 1, 1), (1, 0, 1), (1, 1, 0), (1 << 16, 1 << 15, 1), (-1, 1, 1)):
        assert L.clk_cache_workspace_bytes(*bad, ctypes.byref(n)) == clk.EINVAL
    assert L.clk_cache_workspace_bytes(4, 8, 32, None) == clk.EINVAL
    assert L.clk_cache_workspace_bytes(64, 500, 30000, ctypes.byref(n)) == 0
    assert 4 * (64 * 500 + 4 * 30000) < n.value < 4 * (64 * 500 + 4 * 30000) * 1.1 + 8192
    h = ctypes.c_void_p()
    args = (4, 8, 32, 16, 1 << 20, 1 << 20)
    for i, bad in ((0, 0), (3, 8), (3, 48), (3, 256), (4, None), (4, (1 << 20) + 128), (5, 100)):
        a = list(args)
        a[i] = bad
        assert L.clk_cache_create(ctypes.byref(h), *a) == clk.EINVAL, (i, bad)
        assert not h.value
    assert L.clk_cache_create(None, *args) == clk.EINVAL
    assert L.clk_cache_create(ctypes.byref(h), 1, 1 << 27, 32, 16, 1 << 20, 1 << 40) == clk.EINVAL  # 2^31 tokens a slot
    L.clk_cache_destroy(None)


def test_cache_calls(clk, cache):
    L = clk.lib()
    pool = pool_of(clk)
    p = ctypes.byref(pool)
    for call in (lambda h: L.clk_cache_reset(h, None), lambda h: L.clk_cache_grow(h, P, 1, P, None), lambda h: L.clk_cache_free(h, P, 1, None),
                 lambda h: L.clk_cache_fork(h, P, P, 1, p, None), lambda h: L.clk_cache_compact(h, p, None, None),
                 lambda h: L.clk_cache_append(h, P, 1, p, 0, 1, P, P, 0, 0, 0, 1, None, None, P, None),
                 lambda h: L.clk_cache_buffers(h, None, None, None), lambda h: L.clk_cache_status_clear(h, None)):
        assert call(None) == clk.ESTATE
    for B in (-1, 5):
        assert L.clk_cache_grow(cache, P, B, P, None) == clk.EINVAL
        assert L.clk_cache_free(cache, P, B, None) == clk.EINVAL
        assert L.clk_cache_fork(cache, P, P, B, p, None) == clk.EINVAL
    assert L.clk_cache_grow(cache, P, 0, P, None) == L.clk_cache_free(cache, P, 0, None) == L.clk_cache_fork(cache, P, P, 0, p, None) == 0
    assert L.clk_cache_grow(cache, None, 1, P, None) == L.clk_cache_grow(cache, P, 1, P + 2, None) == clk.EINVAL
    assert L.clk_cache_fork(cache, P, None, 1, p, None) == L.clk_cache_free(cache, P + 1, 1, None) == clk.EINVAL
    assert L.clk_cache_status(cache, None, None, None) == clk.EINVAL
    assert L.clk_cache_compact(cache, p, P + 1, None) == clk.EINVAL
    for bad in BAD_POOLS:
        q = ctypes.byref(pool_of(clk, **bad))
        assert L.clk_cache_fork(cache, P, P, 1, q, None) == clk.EINVAL, bad
        assert L.clk_cache_compact(cache, q, None, None) == clk.EINVAL, bad
        assert L.clk_cache_append(cache, P, 1, q, 0, 1, P, P, 0, 0, 0, 1, None, None, P, None) == clk.EINVAL, bad
    good = dict(slots=P, B=1, pool=p, layer0=0, layers=2, k=P, v=P, ls=0, rs=0, hs=0, N=4, off=None, path=None, count=P)
    for bad in (dict(slots=None), dict(layer0=1), dict(layers=3), dict(layer0=-1), dict(layers=-1), dict(k=None), dict(v=P + 1), dict(ls=-1),
                dict(rs=-1), dict(hs=-1), dict(N=-1), dict(count=None), dict(off=P, path=P), dict(off=P + 4), dict(path=P + 2),
                dict(N=1 << 60)):
        a = {**good, **bad}
        assert L.clk_cache_append(cache, *a.values(), None) == clk.EINVAL, bad
    for nothing in (dict(B=0), dict(N=0), dict(layers=0)):
        assert L.clk_cache_append(cache, *{**good, **nothing}.values(), None) == 0
    at = [ctypes.c_void_p() for _ in range(3)]
    assert L.clk_cache_buffers(cache, *(ctypes.byref(x) for x in at)) == 0
    assert all(x.value % 256 == 0 and x.value >= 1 << 20 for x in at) and len({x.value for x in at}) == 3


def test_tree_calls(clk):
    L = clk.lib()
    for B, N in ((-1, 4), (clk.MAX_BATCH + 1, 4), (1, 0), (1, clk.TREE_MAX + 1)):
        assert L.clk_tree_masks(B, N, P, P, P, None) == clk.EINVAL
        assert L.clk_tree_accept(B, N, P, P, P, P, P, P, P, P, None) == clk.EINVAL
    assert L.clk_tree_masks(0, 4, None, None, None, None) == 0
    assert L.clk_tree_accept(0, 4, *[None] * 8, None) == 0
    for i in range(3):
        for bad in (None, P + 1):
            a = [P] * 3
            a[i] = bad
            assert L.clk_tree_masks(1, 4, *a, None) == clk.EINVAL
    assert L.clk_tree_masks(1, 4, P, P, P + 4, None) == clk.EINVAL  # masks are 64-bit words
    for i in range(8):
        a = [P] * 8
        a[i] = None
        assert L.clk_tree_accept(1, 4, *a, None) == clk.EINVAL


def test_attention_calls(clk, cache):
    L = clk.lib()
    n = ctypes.c_size_t()
    for bad in ((4, 3, 64), (2, 4, 64), (4, 0, 64), (4, 2, 0), (4, 2, 257)):
        assert L.clk_attend_scratch_bytes(*bad, ctypes.byref(n)) == clk.EINVAL
    assert L.clk_attend_scratch_bytes(4, 2, 64, None) == clk.EINVAL
    assert L.clk_attend_scratch_bytes(4, 2, 200, ctypes.byref(n)) == 0 and n.value == 16
    pool, attn = pool_of(clk), attn_of(clk)
    good = dict(h=cache, slots=P, B=1, pool=ctypes.byref(pool), layer=0, a=ctypes.byref(attn), N=4, nodes=P, mask=P, ctx=None,
                scratch=P, bytes=1 << 30)

    def tree(**kw):
        return L.clk_tree_attend(*{**good, **kw}.values(), None)

    assert tree(h=None) == clk.ESTATE
    for bad in (dict(slots=None), dict(B=5), dict(B=-1), dict(layer=2), dict(layer=-1), dict(a=None), dict(N=0), dict(N=65),
                dict(nodes=None), dict(mask=None), dict(mask=P + 4), dict(ctx=P + 2), dict(pool=None)):
        assert tree(**bad) == clk.EINVAL, bad
    for bad in BAD_POOLS + [dict(dtype=clk.F16), dict(heads=1), dict(dim=32)]:
        assert tree(pool=ctypes.byref(pool_of(clk, **bad))) == clk.EINVAL, bad
    for bad in BAD_ATTN:
        assert tree(a=ctypes.byref(attn_of(clk, **bad))) == clk.EINVAL, bad
    assert tree(B=0) == 0
    good = dict(a=ctypes.byref(attn), off=P, B=1, T=10, h=None, slots=None, pool=None, layer=0, ctx=None, scratch=P, bytes=1 << 30)

    def prompt(**kw):
        return L.clk_prompt_attend(*{**good, **kw}.values(), None)

    for bad in (dict(a=None), dict(off=None), dict(off=P + 4), dict(B=-1), dict(B=clk.MAX_BATCH + 1), dict(T=-1), dict(T=(1 << 30) + 1),
                dict(ctx=P), dict(h=cache, pool=None), dict(h=cache, pool=ctypes.byref(pool), slots=None),
                dict(h=cache, pool=ctypes.byref(pool), slots=P, layer=2), dict(h=cache, pool=ctypes.byref(pool), slots=P, ctx=P + 1)):
        assert prompt(**bad) == clk.EINVAL, bad
    for bad in BAD_ATTN:
        if "dim" in bad and bad["dim"] == 128:
            continue  # no pool to disagree with
        assert prompt(a=ctypes.byref(attn_of(clk, **bad))) == clk.EINVAL, bad
    assert prompt(B=0) == 0 and prompt(T=0) == 0
