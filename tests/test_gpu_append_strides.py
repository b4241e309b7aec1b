"""cache_append and the pool's layout: a stride of an axis of one element means
nothing and refuses nothing.  GPU."""
import pytest
import torch

import context_lookup_speculative_gb300 as clk
from test_gpu_cache import ints

pytestmark = pytest.mark.gpu


def filled(P, heads, dim, lens):
    h = clk.Cache(len(lens), 4, 4 * len(lens), P)
    pool = torch.zeros((4, 4 * len(lens), heads, P, dim), dtype=torch.bfloat16, device="cuda")
    clk.cache_grow(h, ints(range(len(lens))), ints(lens))
    return h, pool


def rows_of(h, pool, plane, slot, first, n):
    at = torch.arange(first, first + n, device="cuda")
    return pool[plane, h.table[slot, at // h.page_tokens].long(), :, at % h.page_tokens]


@pytest.mark.parametrize("heads", [1, 3])
@pytest.mark.parametrize("layers", [1, 2])
@pytest.mark.parametrize("B", [1, 3])
def test_one_token_a_request_from_a_projection(B, layers, heads):
    """Decoding by single tokens: K and V are slices of one projection, with a token axis put in."""
    P, dim = 16, 8
    h, pool = filled(P, heads, dim, [20 + b for b in range(B)])
    qkv = torch.randn((layers, B, 5 + 2 * heads, dim), device="cuda").to(torch.bfloat16)
    k, v = (qkv[:, :, x:x + heads].unsqueeze(2) for x in (5, 5 + heads))
    clk.cache_append(h, ints(range(B)), pool, k, v, ints([1] * B))
    assert h.status()[0] == 0
    for layer in range(layers):
        for b in range(B):
            for x, src in ((0, k), (1, v)):
                assert torch.equal(rows_of(h, pool, 2 * layer + x, b, 19 + b, 1)[0], src[layer, b, 0])


@pytest.mark.parametrize("N", [1, 3])
def test_strides_of_axes_of_one_element(N):
    """K and V whose strides differ on axes of one element only (layers, requests, heads, and tokens where N = 1)."""
    P, dim = 16, 8
    h, pool = filled(P, 1, dim, [20])
    k, v = (torch.randn((1, 1, N, 1, dim), device="cuda").to(torch.bfloat16) for _ in range(2))
    odd = [7, 1001, dim if N > 1 else 333, 13, 1]
    k = k.as_strided(k.shape, odd)
    clk.cache_append(h, ints([0]), pool, k, v, ints([N]))
    assert h.status()[0] == 0
    for x, src in ((0, k), (1, v)):
        assert torch.equal(rows_of(h, pool, x, 0, 20 - N, N)[:, 0], src[0, 0, :, 0])
    clk.cache_append(h, ints([0]), pool, v[:, 0], k[:, 0], ints([N]), offsets=ints([0, N], torch.int64))
    assert h.status()[0] == 0
    for x, src in ((0, v), (1, k)):
        assert torch.equal(rows_of(h, pool, x, 0, 20 - N, N)[:, 0], src[0, 0, :, 0])


def test_layouts_that_differ_are_still_refused():
    h, pool = filled(16, 2, 8, [20, 20])
    k = torch.zeros((1, 2, 3, 2, 8), dtype=torch.bfloat16, device="cuda")
    apart = torch.zeros((1, 2, 4, 2, 8), dtype=torch.bfloat16, device="cuda")[:, :, :3]
    for kk, vv in ((k, k.transpose(2, 3).contiguous().transpose(2, 3)), (apart, apart)):
        with pytest.raises(ValueError):
            clk.cache_append(h, ints([0, 1]), pool, kk, vv, ints([3, 3]))


def test_a_pool_of_rows_of_one_element():
    """Its last axis has one element, so that its stride is whatever it came with."""
    P = 16
    h = clk.Cache(2, 4, 8, P)
    wide = torch.zeros((2, 8, 1, P, 1), dtype=torch.float32, device="cuda")
    pool = wide.as_strided(wide.shape, wide.stride()[:4] + (5,))
    clk.cache_grow(h, ints([1]), ints([20]))
    k = torch.randn((1, 1, 20, 1, 1), device="cuda")
    clk.cache_append(h, ints([1]), pool, k, -k, ints([20]))
    assert h.status()[0] == 0
    assert torch.equal(rows_of(h, wide, 0, 1, 0, 20), k[0, 0]) and torch.equal(rows_of(h, wide, 1, 1, 0, 20), -k[0, 0])
