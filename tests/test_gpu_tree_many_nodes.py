"""Greedy verification of trees of any size with the framework's own argmax:
verify_greedy takes blocks of 16 rows, so a tree of N nodes, padded to a
multiple of 16, is N / 16 blocks of it.  GPU."""
import numpy as np
import pytest
import torch

import context_lookup_speculative_gb300 as clk
from cache_model import accept_of, random_tree
from test_gpu_cache import ints

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("N", [16, 32, 48, 64])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_trees_through_verify_greedy(N, dtype):
    B, V = 5, 1000
    rng = np.random.default_rng(N)
    nodes = [N, N - 5, 1, 0, N // 2 + 1]
    parent = [random_tree(rng, N) for _ in range(B)]
    logits = torch.randn((B, N, V), generator=torch.Generator(device="cuda").manual_seed(N), device="cuda").to(dtype)
    top = logits.float().max(-1, keepdim=True).values
    lowest = torch.where(logits.float() == top, torch.arange(V, device="cuda"), V).min(-1).values  # of equal maxima
    want = lowest.cpu().numpy()
    tok = [[-1] + [int(want[b][parent[b][n]]) if rng.random() < 0.8 else 7 for n in range(1, N)] for b in range(B)]
    blocks = N // 16 * B
    d = {n: torch.zeros(s, dtype=torch.int32, device="cuda") for n, s in
         dict(argmax=(blocks, 16), accept=(blocks,), emitted=(blocks,), out=(blocks, 16)).items()}
    clk.verify_greedy(logits.view(blocks, 16, V), ints(tok).view(blocks, 16), torch.full((blocks,), 16, dtype=torch.int32, device="cuda"),
                      d["argmax"], d["accept"], d["emitted"], d["out"], clk.verify_scratch(blocks))
    argmax = d["argmax"].view(B, N)
    assert np.array_equal(argmax.cpu().numpy(), want)
    accept, path, emitted, out = (torch.zeros(s, dtype=torch.int32, device="cuda") for s in ((B,), (B, N), (B,), (B, N)))
    clk.tree_accept(ints(tok), ints(parent), ints(nodes), argmax, accept, path, emitted, out)
    for b in range(B):
        p = accept_of(tok[b], parent[b], nodes[b], want[b])
        assert path[b].tolist() == p + [-1] * (N - len(p))
        assert emitted[b].item() == len(p) and out[b, :len(p)].tolist() == [int(want[b][n]) for n in p]
