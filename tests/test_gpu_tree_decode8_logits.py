"""Decoding over a cache in 8 bits with the rotating calls against the same with keys and queries rotated by plain
operations at positions of their own counting: in float32 both round alike, so that logits, tokens, codes and scales are
equal bit for bit.  GPU."""
import os
import sys

import pytest
import torch

import context_lookup_speculative_gb300 as clk

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
MOST = 320  # tokens of a request


def decode(rotating, tree, steps=10):
    """Tokens, every forward pass's logits, and the pool, of three requests about one document."""
    import tree_decode

    t = tree_decode.Target(dtype=torch.float32)
    if not rotating:
        table = clk.Rotary.of(t.freq, MOST).table

        def rotate(x, pos):
            c, s = (table[pos.long()][..., i, :].unsqueeze(-2) for i in (0, 1))
            u, v = x.chunk(2, -1)
            return torch.cat([u * c - v * s, v * c + u * s], -1)

        t.rotate = rotate
    logits = []
    forward = t.forward

    def recorded(*a, **kw):
        logits.append(forward(*a, **kw))
        return logits[-1]

    t.forward = recorded
    d = tree_decode.Decoder(t, 4, MOST, cache8=True)
    if not rotating:
        d.rotary = None
    g = torch.Generator().manual_seed(1)
    doc = torch.randint(0, t.vocab, (150,), generator=g, dtype=torch.int32)
    asked = [torch.randint(0, t.vocab, (8 + 5 * r,), generator=g, dtype=torch.int32) for r in range(3)]
    i32 = dict(dtype=torch.int32, device="cuda")
    base, slots = torch.tensor([3], **i32), torch.arange(3, **i32)
    d.ingest(base, [doc], torch.zeros(1, **i32))
    clk.cache_fork(d.cache, base.repeat(3), slots, d.pool)
    last = d.ingest(slots, asked, torch.full((3,), 150, **i32))
    d.start(slots, [torch.cat([doc, q]) for q in asked], last)
    tokens = []
    for _ in range(steps):
        d.step(tree)
        tokens.append((d.emitted.tolist(), [row[:n] for n, row in zip(d.emitted.tolist(), d.out_tok.tolist())]))
    torch.cuda.synchronize()
    assert d.cache.status()[0] == d.lookup.status()[0] == 0
    return tokens, logits, d


@pytest.mark.parametrize("tree", [True, False])
def test_the_rotating_calls_and_plain_rotation_agree(tree):
    tokens, logits, d = decode(True, tree)
    want, plain, e = decode(False, tree)
    assert tokens == want and len(logits) == len(plain)
    assert all(torch.equal(a, b) for a, b in zip(logits, plain))
    assert torch.equal(d.cache.length, e.cache.length) and torch.equal(d.cache.table, e.cache.table)
    assert torch.equal(d.pool.data.view(torch.uint8), e.pool.data.view(torch.uint8)) and torch.equal(d.pool.scale, e.pool.scale)
    # something was appended in every layer
    assert all(bool((d.pool.scale[p] != 1).any()) and bool((d.pool.data[p].float() != 0).any()) for p in range(d.pool.data.shape[0]))
