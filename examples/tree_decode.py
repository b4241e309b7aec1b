"""Decoding with drafted trees over a paged cache: the framework's calls together.

A small attention-only target with random weights continues several questions
about one document.  The document goes through the target once; its pages are
shared by all requests (fork), and each question's tokens are a prompt behind
that cached prefix.  Then every step

    lookup_propose   draft from the request's own history
    (bigrams)        seven cheap proposals, a stand-in for a draft model
    tree_masks       both drafts as branches of one tree below the last token
    tree_attend      the target's attention, layer by layer
    verify_greedy    the target's answer at every node
    tree_accept      the accepted path
    cache_grow, cache_append   the accepted nodes' K and V into the pages
    lookup_append    their tokens into the history

At the end half of the requests are freed and the pool is compacted.

    python examples/tree_decode.py [--requests 4] [--document 600] [--tokens 64] [--no-tree]
"""
from __future__ import annotations

import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import context_lookup_speculative_gb300 as clk  # noqa: E402

NODES = 16  # the last token, 8 looked-up tokens, 7 bigram tokens


class Target:
    """Attention layers with residuals over embeddings; rotary positions.  The
    attention is weak beside the token itself, so that text comes to repeat and
    the cheap drafts are right now and then, as in real text."""

    def __init__(self, vocab=512, layers=2, q_heads=8, kv_heads=2, dim=64, dtype=torch.bfloat16, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.layers, self.q_heads, self.kv_heads, self.dim, self.vocab, self.dtype = layers, q_heads, kv_heads, dim, vocab, dtype
        width = q_heads * dim

        def w(*shape):
            return (torch.randn(shape, generator=g, device="cuda") / math.sqrt(shape[0])).to(dtype)

        self.embed = torch.randn((vocab, width), generator=g, device="cuda").to(dtype)
        self.qkv = [w(width, (q_heads + 2 * kv_heads) * dim) for _ in range(layers)]
        self.proj = [0.3 * w(width, width) for _ in range(layers)]
        self.head = w(width, vocab)
        self.freq = 10000.0 ** (-torch.arange(0, dim, 2, device="cuda") / dim)

    def rotate(self, x, pos):
        a = (pos[..., None].float() * self.freq)[..., None, :]
        c, s = a.cos(), a.sin()
        u, v = x.float().chunk(2, -1)
        return torch.cat([u * c - v * s, u * s + v * c], -1).to(self.dtype)

    def forward(self, tok, pos, attend):
        """Logits of tok at pos; attend(layer, q, k, v) is the attention."""
        h = self.embed[tok.long()]
        for i in range(self.layers):
            x = torch.nn.functional.rms_norm(h, h.shape[-1:])
            q, k, v = (x @ self.qkv[i]).unflatten(-1, (-1, self.dim)).split([self.q_heads, self.kv_heads, self.kv_heads], -2)
            o = attend(i, self.rotate(q, pos), self.rotate(k, pos), v)
            h = h + o.flatten(-2) @ self.proj[i]
        return torch.nn.functional.rms_norm(h, h.shape[-1:]).float() @ self.head.float()


class Decoder:
    """The target's cache, the lookup's histories and the buffers of a step."""

    def __init__(self, target, max_slots, max_tokens, page_tokens=16, pages=None):
        self.t = target
        per = -(-max_tokens // page_tokens)
        self.cache = clk.Cache(max_slots, per, pages or max_slots * per, page_tokens)
        self.pool = torch.zeros((2 * target.layers, self.cache.num_pages, target.kv_heads, page_tokens, target.dim),
                                dtype=target.dtype, device="cuda")
        self.lookup = clk.Lookup(max_slots, max_tokens + NODES, target.vocab)
        self.scratch = clk.attend_scratch(target.q_heads, target.kv_heads, target.dim)
        self.scale = 1 / math.sqrt(target.dim)
        single = torch.arange(target.vocab, device="cuda", dtype=torch.int32)
        # a token's successor by itself: the attention of one token is its own v
        logits = target.forward(single, torch.zeros_like(single), lambda i, q, k, v: v.repeat_interleave(target.q_heads // target.kv_heads, -2))
        self.bigram = logits.argmax(-1).to(torch.int32)

    def ingest(self, slots, prompts, ctx):
        """Packed prompts behind the slots' first ctx tokens; returns the tokens that follow."""
        t = self.t
        off = torch.tensor([0] + [len(p) for p in prompts]).cumsum(0)
        where = torch.cat([torch.arange(len(p)) + int(c) for p, c in zip(prompts, ctx.tolist())])
        tok, off, pos = torch.cat(prompts).cuda(), off.cuda(), where.cuda()
        count = (off[1:] - off[:-1]).to(torch.int32)
        clk.cache_grow(self.cache, slots, count)

        def attend(layer, q, k, v):
            out = torch.empty_like(q)
            clk.prompt_attend(q, k, v, off, self.scale, out, self.scratch, cache=self.cache, slots=slots, pool=self.pool,
                              layer=layer, ctx=ctx)
            clk.cache_append(self.cache, slots, self.pool, k[None].contiguous(), v[None].contiguous(), count, layer=layer,
                             offsets=off)
            return out

        return t.forward(tok, pos, attend)[off[1:] - 1].argmax(-1).to(torch.int32)

    def start(self, slots, histories, last):
        """Histories for the lookup: everything that is in the cache, then the token that follows."""
        off = torch.tensor([0] + [len(h) for h in histories]).cumsum(0).cuda()
        clk.lookup_init(self.lookup, slots, torch.cat(histories).to(torch.int32).cuda(), off)
        B = slots.numel()
        i32 = dict(dtype=torch.int32, device="cuda")
        self.slots, self.B = slots, B
        self.tok = torch.zeros((B, NODES), **i32)
        self.tok[:, 0] = last
        clk.lookup_append(self.lookup, slots, self.tok, torch.ones(B, **i32))
        half = NODES // 2
        self.parent = torch.tensor([-1] + [0 if n == half + 1 else n - 1 for n in range(1, NODES)], **i32).repeat(B, 1)
        self.depth = torch.tensor([0] + [n if n <= half else n - half for n in range(1, NODES)], device="cuda")
        self.draft, self.k, self.j = torch.zeros((B, NODES), **i32), torch.zeros(B, **i32), torch.zeros(B, **i32)
        self.mask = torch.zeros((B, NODES), dtype=torch.int64, device="cuda")
        self.argmax, self.path, self.out_tok = (torch.zeros((B, NODES), **i32) for _ in range(3))
        self.accept, self.emitted = torch.zeros(B, **i32), torch.zeros(B, **i32)
        self.vscratch = clk.verify_scratch(B)
        t = self.t
        self.kv = torch.zeros((2, t.layers, B, NODES, t.kv_heads, t.dim), dtype=t.dtype, device="cuda")

    def step(self, tree=True):
        """One step of every request; self.out_tok and self.emitted hold its tokens."""
        t, B, half = self.t, self.B, NODES // 2
        if tree:
            clk.lookup_propose(self.lookup, self.slots, self.draft, self.k, self.j)
            self.tok[:, 1:half + 1] = self.draft[:, :half]
            at = self.tok[:, 0]
            for n in range(half + 1, NODES):
                at = self.bigram[at.long()]
                self.tok[:, n] = at
        nodes = torch.full((B,), NODES if tree else 1, dtype=torch.int32, device="cuda")
        clk.tree_masks(self.parent, nodes, self.mask)
        length = self.cache.length[self.slots.long()]

        def attend(layer, q, k, v):
            out = torch.empty_like(q)
            clk.tree_attend(self.cache, self.slots, self.pool, layer, q, k, v, nodes, self.mask, self.scale, out, self.scratch)
            self.kv[0, layer], self.kv[1, layer] = k, v
            return out

        logits = t.forward(self.tok.clamp(min=0), length[:, None] + self.depth, attend)
        clk.verify_greedy(logits, self.tok, nodes, self.argmax, self.accept, self.emitted, self.out_tok, self.vscratch)
        clk.tree_accept(self.tok, self.parent, nodes, self.argmax, self.accept, self.path, self.emitted, self.out_tok)
        clk.cache_grow(self.cache, self.slots, self.emitted)
        clk.cache_append(self.cache, self.slots, self.pool, self.kv[0], self.kv[1], self.emitted, path=self.path)
        clk.lookup_append(self.lookup, self.slots, self.out_tok, self.emitted)
        self.tok[:, 0] = torch.gather(self.out_tok, 1, (self.emitted[:, None] - 1).long())[:, 0]


def run(requests=4, document=600, tokens=64, tree=True, dtype=torch.bfloat16, seed=0):
    """Decodes; returns each request's tokens, the number of steps and the pool's state."""
    t = Target(dtype=dtype, seed=seed)
    d = Decoder(t, requests + 1, document + 64 + tokens + 2 * NODES)
    g = torch.Generator().manual_seed(seed + 1)
    doc = torch.randint(0, t.vocab, (document,), generator=g, dtype=torch.int32)
    questions = [torch.randint(0, t.vocab, (8 + 5 * r,), generator=g, dtype=torch.int32) for r in range(requests)]
    i32 = dict(dtype=torch.int32, device="cuda")
    base, slots = torch.tensor([requests], **i32), torch.arange(requests, **i32)
    d.ingest(base, [doc], torch.zeros(1, **i32))
    clk.cache_fork(d.cache, base.repeat(requests), slots, d.pool)
    last = d.ingest(slots, questions, torch.full((requests,), document, **i32))
    d.start(slots, [torch.cat([doc, q]) for q in questions], last)
    out = [[int(x)] for x in last.tolist()]
    steps = 0
    while min(map(len, out)) < tokens and steps < tokens:
        d.step(tree)
        steps += 1
        for r, (n, row) in enumerate(zip(d.emitted.tolist(), d.out_tok.tolist())):
            out[r] += row[:n]
    clk.cache_free(d.cache, torch.cat([slots[::2], base]))
    moved = torch.zeros(1, **i32)
    clk.cache_compact(d.cache, d.pool, moved)
    used = int((d.cache.refs > 0).sum())
    status = (d.cache.status()[0], d.lookup.status()[0])
    return dict(tokens=[o[:tokens] for o in out], steps=steps, moved=int(moved), used=used, status=status, decoder=d)


def main():
    p = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    p.add_argument("--requests", type=int, default=4)
    p.add_argument("--document", type=int, default=600)
    p.add_argument("--tokens", type=int, default=64)
    p.add_argument("--no-tree", action="store_true", help="one token a step")
    a = p.parse_args()
    r = run(a.requests, a.document, a.tokens, not a.no_tree)
    made = sum(map(len, r["tokens"]))
    print(f"{made} tokens of {a.requests} requests in {r['steps']} steps ({made / a.requests / r['steps']:.2f} a step); "
          f"{r['moved']} pages moved, {r['used']} in use; status {r['status']}")


if __name__ == "__main__":
    main()
