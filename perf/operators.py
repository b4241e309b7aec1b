"""Cases of the paged-cache and attention operators: what a pass computes, its inputs, its plain form and its floor.

Four operators of a decode loop that verifies drafted tokens:

tree    attention of a step's drafted tokens (a tree, or one token) over a paged cache
prompt  causal attention of packed prompts, each behind a cached prefix of its own (or none)
commit  the end of a step on forked requests: fork, tree masks, accepted path, pages, accepted rows into the pages
life    a batch's cache from its prompts to a compacted pool: pages, rows, freeing half of it, compaction

A cache is a pool [2 * layers, pages, kv heads, page tokens, dim] (planes 2l and
2l + 1 hold layer l's K and V), a page table per slot and a length per slot.
Free pages are handed out lowest number first, in batch order.
"""
import math
import random

import numpy as np
import torch

own = False
SENT = -1
DEV = "cuda"


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # one request, one token: plain decoding in a chat, where the latency of a call is what counts
        dict(name="tree-token-2k", op="tree", B=1, N=1, tree="chain", lo=2048, hi=2048, Hq=32, Hkv=8, D=128, P=64,
             dtype="bf16", lens=1),
        # one request copying out of a 25,000-token document, both drafts of the step as branches of one tree
        dict(name="tree-restate-25k", op="tree", B=1, N=16, tree="branches", lo=25000, hi=25000, Hq=32, Hkv=8, D=128,
             P=64, dtype="bf16", lens=2),
        # the mixed serving batch: 64 requests of 2,000 to 32,000 tokens, blocks of 16 and of 8
        dict(name="tree-mixed-64", op="tree", B=64, N=16, tree="branches", lo=2000, hi=32000, Hq=32, Hkv=8, D=128,
             P=64, dtype="bf16", lens=3),
        # eight very long requests, few heads of keys, chains of 16
        dict(name="tree-long-262k", op="tree", B=8, N=16, tree="chain", lo=262100, hi=262144, Hq=16, Hkv=2, D=128,
             P=128, dtype="f16", lens=4),
        # a wide batch of short requests, an odd number of heads a group, bushy trees, small pages
        dict(name="tree-wide-256", op="tree", B=256, N=13, tree="random", lo=300, hi=4096, Hq=24, Hkv=4, D=64, P=16,
             dtype="f16", lens=5),
        # three short prompts as they arrive in a chat: one token, and odd lengths
        dict(name="prompt-short", op="prompt", B=3, lo=1, hi=130, clo=0, chi=0, Hq=32, Hkv=8, D=128, P=64,
             dtype="bf16", lens=6),
        # chunks of prompts behind cached prefixes (a shared document, or the prompt's earlier chunks)
        dict(name="prompt-chunks-16", op="prompt", B=16, lo=100, hi=2000, clo=0, chi=8192, Hq=24, Hkv=4, D=64, P=32,
             dtype="f16", lens=7),
        # one 25,000-token document, the whole prompt at once
        dict(name="prompt-document-25k", op="prompt", B=1, lo=25000, hi=25000, clo=0, chi=0, Hq=32, Hkv=8, D=128,
             P=64, dtype="bf16", lens=8),
        # the end of one request's step: its latency
        dict(name="commit-1", op="commit", B=1, N=16, tree="branches", lo=2000, hi=2000, Hkv=8, D=128, P=64, layers=2,
             dtype="bf16", lens=9),
        # the end of the mixed batch's step, every request forked into a second continuation
        dict(name="commit-64", op="commit", B=64, N=16, tree="branches", lo=200, hi=2000, Hkv=8, D=128, P=64,
             layers=8, dtype="bf16", lens=10),
        # a few prompts of one layer through the cache's whole life
        dict(name="life-5", op="life", B=5, lo=1, hi=700, Hkv=4, D=64, P=16, layers=1, dtype="f16", lens=11),
        # 64 prompts of 200 to 2,000 tokens, eight layers, half of them freed and the pool compacted
        dict(name="life-64", op="life", B=64, lo=200, hi=2000, Hkv=8, D=128, P=64, layers=8, dtype="bf16", lens=12),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tree", "tree", "prompt", "commit", "life"])
    Hkv = rng.choice([1, 2, 4, 8])
    D, P, dtype, lens = rng.choice([64, 128]), rng.choice([16, 32, 64, 128]), rng.choice(["bf16", "f16"]), rng.randrange(1 << 20)
    if op == "tree":
        B, N, G = _log(rng, 1, 256), _log(rng, 1, 64), rng.choice([1, 3, 4, 5, 6, 8])
        hi = _log(rng, 64, min(262144, 8e9 / (B * Hkv * D * 4), 1.5e10 / (B * Hkv * G * N * 4)))
        return dict(op=op, B=B, N=N, tree=rng.choice(["chain", "branches", "random"]), lo=max(0, hi // 8), hi=hi, Hq=G * Hkv,
                    Hkv=Hkv, D=D, P=P, dtype=dtype, lens=lens)
    if op == "prompt":
        B, G, hi = _log(rng, 1, 16), rng.choice([1, 2, 4, 6, 8]), _log(rng, 16, 8000)
        hi = min(hi, 16000 // B)
        chi = rng.choice([0, _log(rng, 64, 16000 // B)])
        return dict(op=op, B=B, lo=max(1, hi // 8), hi=hi, clo=0, chi=chi, Hq=G * Hkv, Hkv=Hkv, D=D, P=P, dtype=dtype, lens=lens)
    if op == "commit":
        hi = _log(rng, 100, 2000)
        return dict(op=op, B=_log(rng, 1, 64), N=_log(rng, 1, 32), tree=rng.choice(["chain", "branches", "random"]), lo=hi // 8,
                    hi=hi, Hkv=Hkv, D=D, P=P, layers=rng.randint(1, 8), dtype=dtype, lens=lens)
    hi = _log(rng, 64, 2000)
    return dict(op=op, B=_log(rng, 1, 64), lo=hi // 8, hi=hi, Hkv=Hkv, D=D, P=P, layers=rng.randint(1, 8), dtype=dtype, lens=lens)


def _sizes(case):
    """Everything that the case alone fixes, whatever the seed: lengths, trees, node counts, packing offsets."""
    r = random.Random(case["lens"])
    c = dict(case)
    B = case["B"]
    c["len"] = [r.randint(case["lo"], case["hi"]) for _ in range(B)]
    c["ctx"] = [r.randint(case["clo"], case["chi"]) for _ in range(B)] if case["op"] == "prompt" else c["len"]
    c["off"] = [0]
    for n in c["len"]:
        c["off"].append(c["off"][-1] + n)
    if "N" in case:
        N = case["N"]
        # every other block is a long one, as in a batch where half of the requests copy
        c["nodes"] = [N if b % 2 == 0 else max(1, N // 2) for b in range(B)]
        if case["tree"] == "chain":
            par = [list(range(-1, N - 1)) for _ in range(B)]
        elif case["tree"] == "branches":
            half = (N + 1) // 2
            par = [[-1] + [0 if i == half + 1 else i - 1 for i in range(1, N)] for _ in range(B)]
        else:
            par = [[-1] + [max(0, i - 1 - r.randrange(4)) for i in range(1, N)] for _ in range(B)]
        c["parent"] = par
    return c


def _ancestors(par, n):
    """Ancestors of every node, itself among them, as lists."""
    out = []
    for i in range(n):
        out.append((out[par[i]] if i and 0 <= par[i] < i else []) + [i])
    return out


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float16


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _gen(seed, what):
    return torch.Generator(device=DEV).manual_seed(seed * 16 + what)


def _normal(shape, dtype, seed, what):
    return torch.empty(shape, dtype=dtype, device=DEV).normal_(generator=_gen(seed, what))


def _pages(n, P):
    return -(-n // P)


def _mask_bits(c):
    """The ancestor masks as 64-bit words, [B, N]."""
    rows = []
    for par, n in zip(c["parent"], c["nodes"]):
        anc = _ancestors(par, n)
        words = [sum(1 << i for i in a) for a in anc] + [0] * (c["N"] - n)
        rows.append([w - (1 << 64) if w >> 63 else w for w in words])
    return torch.tensor(rows, dtype=torch.int64, device=DEV)


def _cache(c, slots, most, pages):
    """An empty cache: the plain one's arrays, and the framework's own where that is asked for."""
    s = dict(P=c["P"], refs=torch.zeros(pages, dtype=torch.int32, device=DEV), length=torch.zeros(slots, dtype=torch.int32, device=DEV),
             table=torch.full((slots, most), -1, dtype=torch.int32, device=DEV))
    if own:
        import context_lookup_speculative_gb300 as clk

        s["clk"] = clk
        s["cache"] = clk.Cache(max_slots=slots, max_pages=most, num_pages=pages, page_tokens=c["P"])
    return s


def _fill(s, slots, lens, r):
    """Grows the slots to their lengths in shuffled rounds, so that their pages lie in between one another's."""
    left = list(lens)
    for part in (3, 2, 1):
        order = list(range(len(lens)))
        r.shuffle(order)
        give = [left[b] // part for b in range(len(lens))]
        left = [x - y for x, y in zip(left, give)]
        at, count = _ints([slots[b] for b in order]), _ints([give[b] for b in order])
        if own:
            s["clk"].cache_grow(s["cache"], at, count)
        else:
            _grow(s, at, count)


def prepare(case, seed):
    c = _sizes(case)
    op, B, P, D, Hkv, dt = c["op"], c["B"], c["P"], c["D"], c["Hkv"], _dtype(c)
    r = random.Random(seed)
    if op in ("tree", "prompt"):
        need = sum(_pages(n, P) for n in c["ctx"])
        pages = need + need // 8 + 8
        s = _cache(c, B, max(1, max(_pages(n, P) for n in c["ctx"])), pages)
        s["slots"] = _ints(r.sample(range(B), B))
        _fill(s, s["slots"].tolist(), c["ctx"], r)
        s["pool"] = _normal((2, pages, Hkv, P, D), dt, seed, 0)
        Hq = c["Hq"]
        rows = (B, c["N"]) if op == "tree" else (c["off"][-1],)
        # queries, keys and values are slices of one projection's output
        qkv = _normal(rows + (Hq + 2 * Hkv, D), dt, seed, 1)
        qkv[..., :Hq, :] *= 1.5
        s.update(op=op, c=c, q=qkv[..., :Hq, :], k=qkv[..., Hq:Hq + Hkv, :], v=qkv[..., Hq + Hkv:, :], scale=1 / math.sqrt(D),
                 ctx=_ints(c["ctx"]), out=torch.empty(rows + (Hq, D), dtype=dt, device=DEV))
        if op == "tree":
            s.update(nodes=_ints(c["nodes"]), mask=_mask_bits(c))
        else:
            s["off"] = torch.tensor(c["off"], dtype=torch.int64, device=DEV)
        if own:
            s["scratch"] = s["clk"].attend_scratch(Hq, Hkv, D)
        return s
    L = c["layers"]
    if op == "commit":
        N = c["N"]
        pages = sum(_pages(n, P) for n in c["len"]) + B * (2 + _pages(N, P)) + 8
        s = _cache(c, 2 * B, max(_pages(n + N, P) for n in c["len"]), pages)
        s["src"], s["dst"] = _ints(range(B)), _ints(range(B, 2 * B))
        _fill(s, list(range(B)), c["len"], r)
        par = torch.tensor(c["parent"], dtype=torch.int32, device=DEV)
        # what the target answers at every node, and drafts that agree with it at four nodes in five
        argmax = torch.randint(0, 32000, (B, N), generator=_gen(seed, 2), device=DEV, dtype=torch.int32)
        tok = torch.gather(argmax, 1, par.clamp(min=0).long())
        miss = torch.rand((B, N), generator=_gen(seed, 3), device=DEV) < 0.2
        s["k"] = _normal((L, B, N, Hkv, D), dt, seed, 1)
        s["v"] = _normal((L, B, N, Hkv, D), dt, seed, 4)
        s.update(parent=par, argmax=argmax, tok=torch.where(miss, tok + 1, tok), nodes=_ints(c["nodes"]))
        if own:
            i32 = dict(dtype=torch.int32, device=DEV)
            s.update(mask=torch.empty((B, N), dtype=torch.int64, device=DEV), accept=torch.empty(B, **i32), emitted=torch.empty(B, **i32),
                     path=torch.empty((B, N), **i32), out_tok=torch.empty((B, N), **i32))
    else:
        pages = sum(_pages(n, P) for n in c["len"]) + 8
        s = _cache(c, B, max(_pages(n, P) for n in c["len"]) + 1, pages)
        s["slots"], s["freed"] = _ints(range(B)), _ints(range(0, B, 2))
        s["count"], s["off"] = _ints(c["len"]), torch.tensor(c["off"], dtype=torch.int64, device=DEV)
        s["k"] = _normal((L, c["off"][-1], Hkv, D), dt, seed, 1)
        s["v"] = _normal((L, c["off"][-1], Hkv, D), dt, seed, 4)
        if own:
            s["moved"] = torch.empty(1, dtype=torch.int32, device=DEV)
    s["pool"] = _normal((2 * L, pages, Hkv, P, D), dt, seed, 0)
    s.update(op=op, c=c)
    return s


# ---------------------------------------------------------------------------
# Plain forms: the page table
# ---------------------------------------------------------------------------
def _free(s, slots):
    at = slots.long()
    rows = s["table"][at]
    used = rows[rows >= 0].long()
    s["refs"].index_add_(0, used, torch.full_like(used, -1, dtype=torch.int32))
    s["table"][at] = -1
    s["length"][at] = 0


def _take(s, need):
    """The lowest free pages, need[i] of them for each i in turn: (i of each page, its rank for i, the page)."""
    free = torch.nonzero(s["refs"] == 0).flatten()
    first = torch.cumsum(need, 0) - need
    who = torch.repeat_interleave(torch.arange(need.numel(), device=DEV), need)
    page = free[:who.numel()]
    s["refs"][page] = 1
    return who, torch.arange(who.numel(), device=DEV) - first[who], page


def _grow(s, slots, count):
    P, at = s["P"], slots.long()
    old = s["length"][at].long()
    new = old + count.long()
    held = (old + P - 1) // P
    who, rank, page = _take(s, (new + P - 1) // P - held)
    s["table"][at[who], held[who] + rank] = page.int()
    s["length"][at] = new.int()


def _copy_rows(s, src, dst, rows):
    """The first rows[i] rows of page src[i] to page dst[i], in every plane."""
    who = torch.repeat_interleave(torch.arange(rows.numel(), device=DEV), rows)
    row = torch.arange(who.numel(), device=DEV) - (torch.cumsum(rows, 0) - rows)[who]
    s["pool"][:, dst[who], :, row] = s["pool"][:, src[who], :, row]


def _fork(s, src, dst):
    P, a, b = s["P"], src.long(), dst.long()
    n = s["length"][a].long()
    whole, part = n // P, n % P
    col = torch.arange(s["table"].shape[1], device=DEV)
    rows = torch.where(col < whole[:, None], s["table"][a], -1)
    used = rows[rows >= 0].long()
    s["refs"].index_add_(0, used, torch.ones_like(used, dtype=torch.int32))
    s["table"][b], s["length"][b] = rows, n.int()
    who, _, page = _take(s, (part > 0).long())
    old = s["table"][a[who], whole[who]].long()
    s["table"][b[who], whole[who]] = page.int()
    _copy_rows(s, old, page, part[who])


def _append(s, slots, k, v, count, base, path=None):
    """Rows base[b] + (path[b, i], or i) of k and v, i < count[b], to the last count[b] positions of slot b."""
    P, at, count = s["P"], slots.long(), count.long()
    who = torch.repeat_interleave(torch.arange(count.numel(), device=DEV), count)
    i = torch.arange(who.numel(), device=DEV) - (torch.cumsum(count, 0) - count)[who]
    row = base[who] + (i if path is None else path[who, i].long())
    pos = (s["length"][at].long() - count)[who] + i
    page = s["table"][at[who], pos // P].long()
    s["pool"][0::2][:, page, :, pos % P] = k[:, row].transpose(0, 1)
    s["pool"][1::2][:, page, :, pos % P] = v[:, row].transpose(0, 1)


def _compact(s):
    P, live = s["P"], s["refs"] > 0
    at = torch.arange(live.numel(), device=DEV)
    kept = live.sum()
    src = torch.nonzero(live & (at >= kept)).flatten()
    dst = torch.nonzero(~live & (at < kept)).flatten()
    held = s["table"] >= 0
    col = torch.arange(s["table"].shape[1], device=DEV) * P
    rows = torch.zeros_like(at)
    rows[s["table"][held].long()] = (s["length"].long()[:, None] - col).clamp(max=P)[held]
    _copy_rows(s, src, dst, rows[src])
    to = at.int()
    to[src] = dst.int()
    s["table"][held] = to[s["table"][held].long()]
    s["refs"][dst] = s["refs"][src]
    s["refs"][src] = 0
    return torch.full((1,), src.numel(), dtype=torch.int32, device=DEV)


# ---------------------------------------------------------------------------
# Plain forms: trees and attention
# ---------------------------------------------------------------------------
def _closure(parent, nodes):
    """anc[b, n, m]: node m is node n or one of its ancestors."""
    B, N = parent.shape
    at = torch.arange(N, device=DEV)
    valid = at < nodes[:, None]
    edge = (parent >= 0) & (parent < at) & (at > 0) & valid
    step = torch.eye(N, device=DEV) + ((at == parent[:, :, None]) & edge[:, :, None]).float()
    return (torch.matrix_power(step, N) > 0) & valid[:, :, None], edge


def _tree(s):
    parent, nodes, tok, argmax = s["parent"], s["nodes"], s["tok"], s["argmax"]
    N = parent.shape[1]
    at = torch.arange(N, device=DEV)
    anc, edge = _closure(parent, nodes)
    mask = (anc.long() << at).sum(2)
    ok = edge & (tok == torch.gather(argmax, 1, parent.clamp(0, N - 1).long()))
    # of siblings with one token the first is taken
    twin = (parent[:, :, None] == parent[:, None, :]) & (tok[:, :, None] == tok[:, None, :]) & ok[:, None, :] & (at < at[:, None])
    ok = (ok & ~twin.any(2)) | ((at == 0) & (nodes[:, None] > 0))
    hit = ok & ~(anc & ~ok[:, None, :]).any(2)
    emitted = hit.sum(1).int()
    path = torch.sort(torch.where(hit, at, N), 1).values
    out = torch.where(path < N, torch.gather(argmax, 1, path.clamp(max=N - 1)), SENT)
    return dict(mask=mask, accept=emitted - 1, emitted=emitted, path=torch.where(path < N, path, -1).int(), out_tok=out.int())


def _softmax_product(scores, seen, v):
    """softmax over the seen places, times v; a row that sees nothing gives 0."""
    scores.masked_fill_(~seen, -math.inf)
    top = scores.amax(-1, keepdim=True).clamp(min=torch.finfo(torch.float32).min)
    scores.sub_(top).exp_()
    return torch.matmul(scores, v) / scores.sum(-1, keepdim=True).clamp(min=torch.finfo(torch.float32).tiny)


def _gathered(s, plane):
    """The slots' cached rows, padded to whole pages of the longest: [B, kv heads, positions, dim]."""
    rows = s["pool"][plane][s["table"][s["slots"].long()].clamp(min=0).long()]
    return rows.permute(0, 2, 1, 3, 4).flatten(2, 3).float()


def _tree_attend(s):
    q, k, v = s["q"], s["k"], s["v"]
    B, N, Hq, D = q.shape
    Hkv = k.shape[2]
    keys = torch.cat([_gathered(s, 0), k.transpose(1, 2).float()], 2)
    vals = torch.cat([_gathered(s, 1), v.transpose(1, 2).float()], 2)
    rows = q.float().view(B, N, Hkv, Hq // Hkv, D).permute(0, 2, 1, 3, 4).flatten(2, 3)
    scores = torch.matmul(rows, keys.transpose(2, 3)).mul_(s["scale"])
    at = torch.arange(keys.shape[2] - N, device=DEV)
    near = (s["mask"][:, :, None] >> torch.arange(N, device=DEV)) & 1
    valid = torch.arange(N, device=DEV) < s["nodes"][:, None]
    seen = torch.cat([(at < s["ctx"][:, None])[:, None, :].expand(B, N, -1), (near > 0) & valid[:, None, :]], 2) & valid[:, :, None]
    out = _softmax_product(scores, seen.repeat_interleave(Hq // Hkv, 1)[:, None], vals)
    return out.view(B, Hkv, N, Hq // Hkv, D).permute(0, 2, 1, 3, 4).reshape(B, N, Hq, D).to(q.dtype)


def _prompt_attend(s):
    q, k, v, off = s["q"], s["k"], s["v"], s["off"]
    T, Hq, D = q.shape
    B, Hkv, P = off.numel() - 1, k.shape[1], s["P"]
    ctx, at = s["ctx"].long(), torch.arange(B, device=DEV)
    who = torch.repeat_interleave(at, off[1:] - off[:-1])
    pos = torch.arange(T, device=DEV) - off[who] + ctx[who]
    # the cached rows of all requests one after the other, then the new ones
    old = torch.repeat_interleave(at, ctx)
    opos = torch.arange(old.numel(), device=DEV) - (torch.cumsum(ctx, 0) - ctx)[old]
    page = s["table"][s["slots"].long()[old], opos // P].long()
    keys = torch.cat([s["pool"][0][page, :, opos % P], k]).float().transpose(0, 1)
    vals = torch.cat([s["pool"][1][page, :, opos % P], v]).float().transpose(0, 1)
    seen = (who[:, None] == torch.cat([old, who])) & (torch.cat([opos, pos]) <= pos[:, None])
    rows = q.float().view(T, Hkv, Hq // Hkv, D).permute(1, 2, 0, 3)
    out = _softmax_product(torch.matmul(rows, keys[:, None].transpose(2, 3)).mul_(s["scale"]), seen, vals[:, None])
    return out.permute(2, 0, 1, 3).reshape(T, Hq, D).to(q.dtype)


def _whole(s, more):
    return dict(more, pool=s["pool"], table=s["table"], length=s["length"], refs=s["refs"])


def _run_own(s):
    clk, h = s["clk"], s["cache"]
    if s["op"] == "tree":
        clk.tree_attend(h, s["slots"], s["pool"], 0, s["q"], s["k"], s["v"], s["nodes"], s["mask"], s["scale"], s["out"], s["scratch"])
        return s["out"]
    if s["op"] == "prompt":
        clk.prompt_attend(s["q"], s["k"], s["v"], s["off"], s["scale"], s["out"], s["scratch"], cache=h, slots=s["slots"], pool=s["pool"],
                          layer=0, ctx=s["ctx"])
        return s["out"]
    if s["op"] == "commit":
        clk.cache_free(h, s["dst"])
        clk.cache_fork(h, s["src"], s["dst"], s["pool"])
        clk.tree_masks(s["parent"], s["nodes"], s["mask"])
        clk.tree_accept(s["tok"], s["parent"], s["nodes"], s["argmax"], s["accept"], s["path"], s["emitted"], s["out_tok"])
        clk.cache_grow(h, s["dst"], s["emitted"])
        clk.cache_append(h, s["dst"], s["pool"], s["k"], s["v"], s["emitted"], path=s["path"])
        more = {n: s[n] for n in ("mask", "accept", "emitted", "path", "out_tok")}
    else:
        clk.cache_free(h, s["slots"])
        clk.cache_grow(h, s["slots"], s["count"])
        clk.cache_append(h, s["slots"], s["pool"], s["k"], s["v"], s["count"], offsets=s["off"])
        clk.cache_free(h, s["freed"])
        clk.cache_compact(h, s["pool"], s["moved"])
        more = dict(moved=s["moved"])
    return dict(more, pool=s["pool"], table=h.table, length=h.length, refs=h.refs)


def run(s):
    if own:
        return _run_own(s)
    if s["op"] == "tree":
        return _tree_attend(s)
    if s["op"] == "prompt":
        return _prompt_attend(s)
    if s["op"] == "commit":
        _free(s, s["dst"])
        _fork(s, s["src"], s["dst"])
        t = _tree(s)
        _grow(s, s["dst"], t["emitted"])
        B, N = s["tok"].shape
        _append(s, s["dst"], s["k"].flatten(1, 2), s["v"].flatten(1, 2), t["emitted"], torch.arange(B, device=DEV) * N, t["path"])
        return _whole(s, t)
    _free(s, s["slots"])
    _grow(s, s["slots"], s["count"])
    _append(s, s["slots"], s["k"], s["v"], s["count"], s["off"][:-1])
    _free(s, s["freed"])
    return _whole(s, dict(moved=_compact(s)))


# ---------------------------------------------------------------------------
# The definition in 64 bits, request by request
# ---------------------------------------------------------------------------
def exact(case, seed):
    global own
    if case["op"] not in ("tree", "prompt"):
        return None  # rows are moved and whole numbers are computed
    c, was = _sizes(case), own
    own = False
    s = prepare(case, seed)
    own = was
    G, P = c["Hq"] // c["Hkv"], c["P"]
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device=DEV)
    slots = s["slots"].tolist()
    for b in range(c["B"]):
        n, N = c["ctx"][b], c["nodes"][b] if c["op"] == "tree" else c["len"][b]
        pages = s["table"][slots[b], :_pages(n, P)].long()
        new = (b, slice(0, N)) if c["op"] == "tree" else (slice(c["off"][b], c["off"][b] + N),)
        if c["op"] == "tree":
            sees = torch.zeros((N, N), dtype=torch.bool)
            for i, a in enumerate(_ancestors(c["parent"][b], N)):
                sees[i, a] = True
            sees = sees.to(DEV)
        else:
            sees = torch.ones((N, N), dtype=torch.bool, device=DEV).tril()
        for h in range(c["Hkv"]):
            k, v = (torch.cat([s["pool"][x][pages, h].reshape(-1, c["D"])[:n], s["kv"[x]][new][:, h]]).double() for x in (0, 1))
            for g in range(h * G, h * G + G):
                e = (s["q"][new][:, g].double() @ k.T) * s["scale"]
                e[:, n:][~sees] = -math.inf
                out[new + (g,)] = torch.softmax(e, 1) @ v
    return out


# ---------------------------------------------------------------------------
# The floor
# ---------------------------------------------------------------------------
def work(case):
    c = _sizes(case)
    op, B, P, row = c["op"], c["B"], c["P"], c["Hkv"] * c["D"] * 2  # bytes of a token's K (or V)
    if op == "tree":
        pairs = sum(n * m + sum(map(len, _ancestors(p, m))) for n, m, p in zip(c["ctx"], c["nodes"], c["parent"]))
        rows = sum(c["nodes"])
        return dict(bytes=2 * row * (sum(c["ctx"]) + rows) + 2 * c["D"] * c["Hq"] * (rows + B * c["N"]) + 4 * sum(_pages(n, P) for n in c["ctx"]),
                    flops=4 * c["D"] * c["Hq"] * pairs)
    if op == "prompt":
        pairs = sum(n * m + m * (m + 1) // 2 for n, m in zip(c["ctx"], c["len"]))
        return dict(bytes=2 * row * (sum(c["ctx"]) + sum(c["len"])) + 4 * c["D"] * c["Hq"] * sum(c["len"]), flops=4 * c["D"] * c["Hq"] * pairs)
    if op == "commit":
        # the tail pages' rows that a fork copies, and the accepted rows (about 0.8 of the chain survives each node)
        tails = sum(n % P for n in c["len"])
        taken = sum(sum(0.8 ** i for i in range(max(map(len, _ancestors(p, m))))) for p, m in zip(c["parent"], c["nodes"]))
        return dict(bytes=2 * 2 * c["layers"] * row * (tails + taken), flops=0)
    # every row in once, and the rows of live pages that lie beyond the number of live pages
    first, rows = 0, []
    for b, n in enumerate(c["len"]):
        if b % 2:
            rows += [(first + i, min(P, n - i * P)) for i in range(_pages(n, P))]
        first += _pages(n, P)
    moved = sum(x for p, x in rows if p >= len(rows))
    return dict(bytes=2 * 2 * c["layers"] * row * (sum(c["len"]) + moved), flops=0)
