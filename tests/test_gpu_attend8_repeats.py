"""Attention over a cache in 8 bits, called many times in a row: CTAs without work and warps without a role beside busy
ones, calls of one and of many items.  Every call ends, and all give the first one's results.  GPU."""
import pytest
import torch

from test_gpu_attend import NAN
from test_gpu_attend8 import Prompt8, Tree8

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("ctx,times", [([1], 1500), ([130, 5, 0], 1000), ([3000, 700], 500), ([400] * 48, 300)])
def test_repeated_calls(ctx, times, D, kind):
    t = Tree8(D, len(ctx), 4, ctx, 2, 2, D, 16, kind, nodes=[4] * len(ctx)).run()
    p = Prompt8(D, [20] * len(ctx), 2, 2, D, kind, ctx=ctx).run()
    torch.cuda.synchronize()
    for c in (t, p):
        first = c.out.clone()
        c.out.fill_(NAN)
        for _ in range(times):
            c.run()
        torch.cuda.synchronize()
        assert torch.equal(c.out, first) and c.cache.status()[0] == 0
