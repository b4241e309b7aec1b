"""Ancestor masks and greedy verification of trees against a walk in plain Python.  GPU."""
import numpy as np
import pytest
import torch

import context_lookup_speculative_gb300 as clk
from cache_model import accept_of, masks_of, random_tree

pytestmark = pytest.mark.gpu


def run(tok, parent, nodes, argmax):
    B, N = tok.shape
    dev = [torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).cuda() for x in (tok, parent, nodes, argmax)]
    mask = torch.full((B, N), 77, dtype=torch.int64, device="cuda")
    out = [torch.full(s, 77, dtype=torch.int32, device="cuda") for s in ((B,), (B, N), (B,), (B, N))]
    clk.tree_masks(dev[1], dev[2], mask)
    clk.tree_accept(*dev, *out)
    torch.cuda.synchronize()
    return mask.cpu().numpy(), [o.cpu().numpy() for o in out]


def check(tok, parent, nodes, argmax):
    mask, (accept, path, emitted, out_tok) = run(tok, parent, nodes, argmax)
    B, N = tok.shape
    for b in range(B):
        n = nodes[b] if 0 <= nodes[b] <= N else 0
        assert [int(x) & (2 ** 64 - 1) for x in mask[b]] == masks_of(parent[b], n, N), b
        want = accept_of(tok[b], parent[b], n, argmax[b])
        assert path[b].tolist() == want + [-1] * (N - len(want)), b
        assert out_tok[b].tolist() == [argmax[b][p] for p in want] + [clk.SENT] * (N - len(want)), b
        assert accept[b] == max(0, len(want) - 1) and emitted[b] == len(want), b


@pytest.mark.parametrize("N", [1, 2, 7, 16, 31, 32, 33, 63, 64])
def test_trees(N):
    rng = np.random.default_rng(N)
    B = 60
    parent = np.array([random_tree(rng, N, wide=1 + b % 6) for b in range(B)])
    # few tokens, so that answers agree often and siblings share tokens
    tok, argmax = rng.integers(0, 2, size=(B, N)), rng.integers(0, 2, size=(B, N))
    tok[::3] = np.where(rng.random((20, N)) < 0.95, np.take_along_axis(argmax[::3], np.maximum(parent[::3], 0), 1), tok[::3])
    check(tok, parent, rng.integers(0, N + 1, size=B), argmax)


def test_bad_parents_counts_and_sentinels():
    N = 5
    parent = np.array([[-1, 0, 1, 2, 3], [9, 0, 2, 5, -3], [0, 1, 0, 2, 3], [-1, 0, 1, 2, 3], [-1, 0, 1, 2, 3], [-1, 0, 1, 2, 3]])
    tok = np.full((6, N), 4)
    argmax = np.full((6, N), 4)
    tok[3, 2] = argmax[3, 1] = clk.SENT  # a sentinel never matches, not even a sentinel
    check(tok, parent, np.array([5, 5, 5, 5, -1, 6]), argmax)


def test_a_chain_is_the_greedy_verification_of_a_block():
    """accept, emitted and out_tok of a chain are verify_greedy's."""
    rng = np.random.default_rng(3)
    B, V = 20, 1000
    x = torch.from_numpy(rng.integers(-30, 30, size=(B, 16, V)).astype(np.float32)).cuda()
    g = x.argmax(dim=2).to(torch.int32)
    L = torch.from_numpy(rng.integers(1, 17, size=B).astype(np.int32)).cuda()
    blk = torch.cat([torch.zeros((B, 1), dtype=torch.int32, device="cuda"), g[:, :15]], 1)
    blk[torch.from_numpy(rng.random((B, 16)) < 0.1).cuda()] = 5
    i32 = dict(dtype=torch.int32, device="cuda")
    arg, acc, em, out = torch.zeros((B, 16), **i32), torch.zeros(B, **i32), torch.zeros(B, **i32), torch.zeros((B, 16), **i32)
    clk.verify_greedy(x, blk, L, arg, acc, em, out, clk.verify_scratch(B))
    parent = torch.arange(-1, 15, **i32).repeat(B, 1)
    acc2, path, em2, out2 = torch.zeros_like(acc), torch.zeros_like(out), torch.zeros_like(em), torch.zeros_like(out)
    clk.tree_accept(blk, parent, L, arg, acc2, path, em2, out2)
    assert torch.equal(acc, acc2) and torch.equal(em, em2) and torch.equal(out, out2)
    assert len(set(acc.tolist())) > 3
