"""The appending call counts a block's heads of all layers, K and V, and of q in 32 bits: more are refused.  CPU only."""
import ctypes

import pytest

from test_operators_abi_cpu import P, cache, clk, pool_of  # noqa: F401
from test_rotary_abi_cpu import pool8_of, scales_of

ref = ctypes.byref


@pytest.mark.parametrize("eight", [False, True])
@pytest.mark.parametrize("layers,heads", [(32767, 65535), (32767, 16385), (16384, 32769)])
def test_too_many_heads_and_layers(clk, cache, eight, layers, heads):  # noqa: F811
    pool = (pool8_of if eight else pool_of)(clk, planes=2 * layers, heads=heads, dim=1)
    scales = scales_of(clk)
    got = clk.lib().clk_cache_append_rotary(cache, P, 1, ref(pool), ref(scales) if eight else None, 0, layers, clk.BF16, P, P, 0, 0, 0, 4,
                                            None, None, P, None, None, None)
    assert got == clk.EINVAL
