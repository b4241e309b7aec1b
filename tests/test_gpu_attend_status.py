"""A wait between an attention's CTAs that runs out ends the call, and is
reported: in the cache where there is one, and in the scratch, which is all
that a prompt without a cache has.  The waits are made to run out by flags
that do not agree (they count a scratch's calls, after its 128 bytes of
status): some CTAs' neighbours then look like last call's.  Each gives up after
about two seconds.  GPU."""
import pytest
import torch

import context_lookup_speculative_gb300 as clk
from test_gpu_attend import Prompt, Tree

pytestmark = pytest.mark.gpu


def disagree(scratch):
    ctas = torch.cuda.get_device_properties(0).multi_processor_count
    g = torch.Generator(device="cuda").manual_seed(0)
    flags = scratch[128:128 + 4 * ctas].view(torch.int32)
    flags.copy_(-torch.randint(0, 2, (ctas,), generator=g, device="cuda", dtype=torch.int32))


def test_a_prompt_without_a_cache():
    p = Prompt(1, [5000], 4, 2, 128, "bf16")
    p.run()
    assert clk.attend_status(p.scratch) == 0
    disagree(p.scratch)
    p.run()
    assert clk.attend_status(p.scratch) == clk.ECUDA
    assert clk.attend_status(p.scratch) == clk.ECUDA  # stays until the scratch is zeroed
    p.scratch.zero_()
    p.out.fill_(5.0)
    p.run().check(rows=20)
    assert clk.attend_status(p.scratch) == 0


def test_a_tree_over_a_cache():
    t = Tree(2, 1, 16, [12000], 4, 2, 64, 64, "f16", nodes=[16])
    disagree(t.scratch)
    t.run()
    torch.cuda.synchronize()
    assert t.cache.status() == (clk.ECUDA, -1) and clk.attend_status(t.scratch) == clk.ECUDA
    t.cache.status_clear()
    t.scratch.zero_()
    t.run().check()
    assert clk.attend_status(t.scratch) == 0


def test_refusals():
    with pytest.raises(ValueError):
        clk.attend_status(torch.zeros(128, dtype=torch.uint8))
    with pytest.raises(ValueError):
        clk.attend_status(torch.zeros(32, dtype=torch.int32, device="cuda"))
    assert clk.attend_status(clk.attend_scratch(4, 2, 200)) == 0
