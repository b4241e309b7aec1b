"""The same over a cache in 8 bits: a wait between CTAs that runs out is reported, and the next call is whole.  GPU."""
import pytest
import torch

import context_lookup_speculative_gb300 as clk
from test_gpu_attend8 import Prompt8, Tree8
from test_gpu_attend_status import disagree

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind,D", [("bf16", 128), ("f16", 64)])
def test_waits_that_run_out(kind, D):
    for c in (Tree8(2, 1, 16, [20000], 4, 2, D, 64, kind, nodes=[16]), Prompt8(3, [500], 4, 2, D, kind, ctx=[9000], P=64)):
        c.run()
        assert clk.attend_status(c.scratch) == 0 and c.cache.status()[0] == 0
        disagree(c.scratch)
        c.run()
        torch.cuda.synchronize()
        assert c.cache.status() == (clk.ECUDA, -1) and clk.attend_status(c.scratch) == clk.ECUDA
        c.cache.status_clear()
        c.scratch.zero_()
        c.out.fill_(5.0)
        c.run().check(*(() if isinstance(c, Tree8) else (20,)))
        assert clk.attend_status(c.scratch) == 0
