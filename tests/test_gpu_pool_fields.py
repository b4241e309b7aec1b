"""The tensors of a pool in 8 bits and of a rotation, whose addresses the calls have, cannot be replaced.  GPU."""
import pytest
import torch

import context_lookup_speculative_gb300 as clk

pytestmark = pytest.mark.gpu


def test_fields_are_not_replaced():
    pool = clk.ScaledPool.empty(1, 2, 1, 16, 16)
    rot = clk.Rotary.of(torch.ones(4), 10)
    for x, name, other in ((pool, "scale", pool.scale.clone()), (pool, "data", pool.data.clone()), (rot, "table", rot.table.clone()),
                           (rot, "neighbours", True)):
        with pytest.raises(AttributeError):
            setattr(x, name, other)
    pool.scale.fill_(2.0)
    assert bool((pool.scale == 2).all()) and rot.neighbours is False
