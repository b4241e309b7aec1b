"""Rotation from several host threads at once, each with a cache, a stream and a batch size of its own, large enough that the
counts of its requests' blocks need more shared memory than a kernel has by default.  GPU."""
import threading

import pytest
import torch

import context_lookup_speculative_gb300 as clk
from rotary_model import angles
from test_gpu_attend import ints

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [64, 24])
def test_large_batches_from_several_threads(D):
    rot = clk.Rotary(angles(40, D // 2).cuda())
    wrong = []

    def work(B):
        try:
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                h = clk.Cache(B, 1, B, 16)
                slots = torch.arange(B, dtype=torch.int32, device="cuda")
                clk.cache_grow(h, slots, slots % 8)
                q, k = torch.ones((B, 1, 1, D), device="cuda").half(), torch.ones((B, 1, 1, D), device="cuda").half()
                qo, ko = torch.zeros_like(q), torch.zeros_like(k)
                nodes, mask = torch.ones_like(slots), ints([[1]] * B, torch.int64)
                for _ in range(1500):
                    clk.tree_rotate(h, slots, q, k, nodes, mask, rot, qo, ko)
                s.synchronize()
                # at position p the first pair of ones becomes (cos - sin, ..)
                want = (rot.table[:8, 0] - rot.table[:8, 1]).half()[(slots % 8).long()]
                if not (torch.equal(qo[:, 0, 0, :D // 2], want) and torch.equal(ko, qo)):
                    wrong.append((B, "values"))
                if h.status()[0] != 0:
                    wrong.append((B, h.status()))
        except Exception as e:  # noqa: BLE001 (what the thread met is the test's result)
            wrong.append((B, repr(e)))

    threads = [threading.Thread(target=work, args=(B,)) for B in (8192, 4200, 5000, 8000)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong
