"""clk_attend_status refuses bad arguments before it touches a GPU.  CPU only."""
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


def test_refusals(clk):
    L = clk.lib()
    st = ctypes.c_int32(7)
    for scratch, out in ((None, ctypes.byref(st)), (P + 8, ctypes.byref(st)), (P, None)):
        assert L.clk_attend_status(scratch, out, None) == clk.EINVAL
    assert st.value == 7
    n = ctypes.c_size_t()
    # the status has its place in the smallest scratch too
    assert L.clk_attend_scratch_bytes(4, 2, 200, ctypes.byref(n)) == 0 and n.value >= 16
