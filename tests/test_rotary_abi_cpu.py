"""The rotation calls and those over a cache in 8 bits refuse bad arguments
before anything is launched.  CPU only: pointers are made up, and no call here
reaches a GPU."""
import ctypes

import pytest

from test_operators_abi_cpu import BAD_ATTN, BAD_POOLS, P, attn_of, cache, clk, pool_of  # noqa: F401


def pool8_of(clk, **kw):
    return pool_of(clk, **{"dtype": clk.E4M3, **kw})


def scales_of(clk, **kw):
    return clk.ScalesDesc(**{**dict(d_base=P, tokens=16, plane_stride=64, page_stride=2, head_stride=1, block_stride=1), **kw})


def rotary_of(clk, **kw):
    return clk.RotaryDesc(**{**dict(d_table=P, positions=100, pairs=32, neighbours=0), **kw})


def turn_of(clk, **kw):
    d = dict(dtype=clk.BF16, q_heads=4, kv_heads=2, dim=64, d_q=P, d_k=P, d_q_out=P, d_k_out=P)
    d.update({n: 64 for n, _ in clk.TurnDesc._fields_[8:]})
    return clk.TurnDesc(**{**d, **kw})


BAD_SCALES = [dict(d_base=None), dict(d_base=P + 2), dict(tokens=0), dict(tokens=8), dict(tokens=32), dict(tokens=24), dict(tokens=-16),
              dict(plane_stride=-1), dict(page_stride=-1), dict(head_stride=-1), dict(block_stride=-1)]
BAD_ROTARY = [dict(d_table=None), dict(d_table=P + 2), dict(positions=0), dict(positions=-1), dict(positions=1 << 40), dict(pairs=0),
              dict(pairs=-1), dict(pairs=33), dict(neighbours=2), dict(neighbours=-1)]
# of a pool with scales; the other types go without
BAD_POOLS8 = [b for b in BAD_POOLS if "dtype" not in b and b != dict(d_base=P + 1)] + [dict(dtype=t) for t in (0, 1, 2, 4, -1)]
ref = ctypes.byref


def test_forks_and_compaction_with_scales(clk, cache):  # noqa: F811
    L = clk.lib()
    pool, scales = pool8_of(clk), scales_of(clk)
    assert L.clk_cache_fork_scaled(None, P, P, 1, ref(pool), ref(scales), None) == clk.ESTATE
    assert L.clk_cache_compact_scaled(None, ref(pool), ref(scales), None, None) == clk.ESTATE
    assert L.clk_cache_fork_scaled(cache, P, P, 0, ref(pool), ref(scales), None) == 0
    for p, s in [(pool8_of(clk, **b), scales) for b in BAD_POOLS8] + [(pool, scales_of(clk, **b)) for b in BAD_SCALES]:
        assert L.clk_cache_fork_scaled(cache, P, P, 1, ref(p), ref(s), None) == clk.EINVAL
        assert L.clk_cache_compact_scaled(cache, ref(p), ref(s), None, None) == clk.EINVAL
    for a in ((None, ref(scales)), (ref(pool), None)):
        assert L.clk_cache_fork_scaled(cache, P, P, 1, *a, None) == clk.EINVAL
        assert L.clk_cache_compact_scaled(cache, *a, None, None) == clk.EINVAL
    assert L.clk_cache_fork_scaled(cache, None, P, 1, ref(pool), ref(scales), None) == clk.EINVAL
    assert L.clk_cache_fork_scaled(cache, P, P, 5, ref(pool), ref(scales), None) == clk.EINVAL
    assert L.clk_cache_compact_scaled(cache, ref(pool), ref(scales), P + 2, None) == clk.EINVAL


def test_pools_of_8_bits_need_their_scales(clk, cache):  # noqa: F811
    L = clk.lib()
    pool = pool8_of(clk)
    assert L.clk_cache_fork(cache, P, P, 1, ref(pool), None) == clk.EINVAL
    assert L.clk_cache_compact(cache, ref(pool), None, None) == clk.EINVAL
    assert L.clk_cache_append(cache, P, 1, ref(pool), 0, 1, P, P, 0, 0, 0, 1, None, None, P, None) == clk.EINVAL
    a = attn_of(clk)
    assert L.clk_tree_attend(cache, P, 1, ref(pool), 0, ref(a), 4, P, P, None, P, 1 << 30, None) == clk.EINVAL
    assert L.clk_prompt_attend(ref(a), P, 1, 4, cache, P, ref(pool), 0, P, P, 1 << 30, None) == clk.EINVAL


def test_tree_rotate(clk, cache):  # noqa: F811
    L = clk.lib()
    t, r = turn_of(clk), rotary_of(clk)
    good = dict(slots=P, B=1, turn=ref(t), N=4, nodes=P, mask=P, ctx=None, rotary=ref(r))

    def call(h=cache, **kw):
        return L.clk_tree_rotate(h, *{**good, **kw}.values(), None)

    assert call(h=None) == clk.ESTATE
    assert call(B=0) == 0
    for bad in (dict(B=-1), dict(B=5), dict(N=0), dict(N=clk.TREE_MAX + 1), dict(turn=None), dict(rotary=None), dict(slots=None), dict(slots=P + 1),
                dict(nodes=None), dict(nodes=P + 2), dict(mask=None), dict(mask=P + 4), dict(ctx=P + 1)):
        assert call(**bad) == clk.EINVAL, bad
    for bad in BAD_ROTARY:
        assert call(rotary=ref(rotary_of(clk, **bad))) == clk.EINVAL, bad
    for bad in [dict(dtype=clk.E4M3), dict(dtype=5), dict(dtype=-1), dict(q_heads=0), dict(kv_heads=0), dict(q_heads=65536), dict(dim=0), dict(dim=257)] + \
            [{n: x} for n in ("d_q", "d_k", "d_q_out", "d_k_out") for x in (None, P + 1)] + [{n: -1} for n, _ in clk.TurnDesc._fields_[8:]]:
        assert call(turn=ref(turn_of(clk, **bad))) == clk.EINVAL, bad


@pytest.mark.parametrize("eight", [False, True])
def test_append_rotary(clk, cache, eight):  # noqa: F811
    L = clk.lib()
    pool, scales, r, t = (pool8_of if eight else pool_of)(clk), scales_of(clk), rotary_of(clk), turn_of(clk)
    good = dict(slots=P, B=1, pool=ref(pool), scales=ref(scales) if eight else None, layer0=0, layers=1, dtype=clk.BF16, k=P, v=P, ls=0, rs=0,
                hs=0, N=4, off=None, path=None, count=P, rotary=ref(r), turn=ref(t))

    def call(h=cache, **kw):
        return L.clk_cache_append_rotary(h, *{**good, **kw}.values(), None)

    assert call(h=None) == clk.ESTATE
    for nothing in (dict(B=0), dict(N=0), dict(layers=0)):
        assert call(**nothing) == 0
    for bad in (dict(B=-1), dict(B=5), dict(slots=None), dict(layer0=2), dict(layers=3), dict(layer0=-1), dict(layers=-1), dict(k=None), dict(v=P + 1),
                dict(ls=-1), dict(rs=-1), dict(hs=-1), dict(N=-1), dict(N=1 << 60), dict(count=None), dict(count=P + 2), dict(off=P, path=P, turn=None),
                dict(off=P + 4), dict(path=P + 2, turn=None), dict(path=P), dict(layers=2), dict(rotary=None), dict(dtype=clk.E4M3), dict(dtype=7),
                dict(pool=None)):
        assert call(**bad) == clk.EINVAL, bad
    # rows of another type than a pool without scales, and scales that do not go with the pool
    assert call(pool=ref(pool_of(clk) if eight else pool8_of(clk))) == clk.EINVAL
    assert call(scales=None if eight else ref(scales)) == clk.EINVAL
    if not eight:
        assert call(dtype=clk.F16, turn=None) == clk.EINVAL
    for bad in BAD_ROTARY:
        assert call(rotary=ref(rotary_of(clk, **bad))) == clk.EINVAL, bad
    for bad in BAD_POOLS8 if eight else BAD_POOLS:
        assert call(pool=ref((pool8_of if eight else pool_of)(clk, **bad))) == clk.EINVAL, bad
    if eight:
        for bad in BAD_SCALES:
            assert call(scales=ref(scales_of(clk, **bad))) == clk.EINVAL, bad
    for bad in (dict(dtype=clk.F16), dict(dim=32), dict(kv_heads=1), dict(q_heads=0), dict(d_q=None), dict(d_q_out=None), dict(d_q=P + 1),
                dict(d_q_out=P + 1), dict(d_k_out=P + 1), dict(q_row=-1), dict(q_head=-1), dict(qo_row=-1), dict(qo_head=-1), dict(ko_row=-1),
                dict(ko_head=-1)):
        assert call(turn=ref(turn_of(clk, **bad))) == clk.EINVAL, bad


def test_attention_over_8_bits(clk, cache):  # noqa: F811
    L = clk.lib()
    pool, scales, a = pool8_of(clk), scales_of(clk), attn_of(clk)
    tree = dict(slots=P, B=1, pool=ref(pool), scales=ref(scales), layer=0, a=ref(a), N=4, nodes=P, mask=P, ctx=None, scratch=P, bytes=1 << 30)
    prompt = dict(a=ref(a), off=P, B=1, T=4, h=cache, slots=P, pool=ref(pool), scales=ref(scales), layer=0, ctx=P, scratch=P, bytes=1 << 30)

    def trees(h=cache, **kw):
        return L.clk_tree_attend_scaled(h, *{**tree, **kw}.values(), None)

    def prompts(**kw):
        return L.clk_prompt_attend_scaled(*{**prompt, **kw}.values(), None)

    assert trees(h=None) == prompts(h=None) == clk.ESTATE
    assert trees(B=0) == prompts(B=0) == prompts(T=0) == 0
    for bad in (dict(scales=None), dict(pool=None), dict(a=None), dict(B=-1), dict(layer=2), dict(layer=-1), dict(slots=None), dict(ctx=P + 2)):
        assert trees(**bad) == clk.EINVAL, bad
        assert prompts(**bad) == clk.EINVAL, bad
    for bad in (dict(N=0), dict(N=65), dict(nodes=None), dict(mask=P + 4)):
        assert trees(**bad) == clk.EINVAL, bad
    for bad in (dict(T=-1), dict(T=(1 << 30) + 1), dict(off=None), dict(off=P + 4)):
        assert prompts(**bad) == clk.EINVAL, bad
    for p, s in [(pool8_of(clk, **b), scales) for b in BAD_POOLS8] + [(pool, scales_of(clk, **b)) for b in BAD_SCALES]:
        assert trees(pool=ref(p), scales=ref(s)) == prompts(pool=ref(p), scales=ref(s)) == clk.EINVAL
    for bad in BAD_ATTN:
        b = ref(attn_of(clk, **bad))
        assert trees(a=b) == prompts(a=b) == clk.EINVAL, bad
