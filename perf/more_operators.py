"""Cases of position rotation and of the cache in 8 bits: what a pass computes, its inputs, its plain form and its floor.

Five operators of a decode loop whose target rotates queries and keys by position and may hold its cache in 8 bits:

rotate  queries and keys of a step's drafted nodes, each at its place behind the request's cached rows
append  keys and values into a paged cache of their own type, the keys rotated on the way (and queries beside them)
append8 the same into a cache of 8-bit values (e4m3) with a scale for each block of tokens and head
tree8   attention of a step's drafted tokens over such a cache
prompt8 causal attention of packed prompts, each behind a cached prefix in 8 bits

A cache is a pool [2 * layers, pages, kv heads, page tokens, dim] (planes 2l and 2l + 1 hold layer l's K and V), a
page table per slot and a length per slot; one in 8 bits also has scales [2 * layers, pages, kv heads, page tokens /
block].  Rows that come into a block without rows before them take the least power of two with which the largest
magnitude is at most 448; where there are rows before, the larger of that and the block's scale, and those rows are
rounded to it.  Keys are rotated in float32: x c - y s and y c + x s with every operation rounded.
"""
import math
import random

import torch

own = False
DEV = "cuda"
TOP = 448.0  # the largest e4m3 value
LEAST = -120  # the least exponent of a scale


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # the drafted tree of one request: latency
        dict(name="rotate-tree-1", op="rotate", B=1, N=16, tree="branches", lo=2048, hi=2048, Hq=32, Hkv=8, D=128, P=64, pairs=64,
             style="half", dtype="bf16", lens=1),
        # a wide batch of bushy trees, half of each row rotated, neighbouring elements paired
        dict(name="rotate-trees-256", op="rotate", B=256, N=32, tree="random", lo=300, hi=4096, Hq=48, Hkv=8, D=128, P=16, pairs=32,
             style="neighbours", dtype="f16", lens=2),
        # one token of plain decoding: its query, its key, its row in the pages
        dict(name="append-token-1", op="append", B=1, packed=False, N=1, lo=2000, hi=2000, clo=1, chi=1, Hq=32, Hkv=8, D=128, P=64,
             pairs=64, style="half", layers=1, dtype="bf16", lens=3),
        # one layer of 16 packed prompts of 100 to 2,000 tokens behind what is cached
        dict(name="append-prompts-16", op="append", B=16, packed=True, N=0, lo=0, hi=8192, clo=100, chi=2000, Hq=32, Hkv=8, D=128, P=64,
             pairs=64, style="half", layers=1, dtype="bf16", lens=4),
        # the end of a mixed batch's step in 8 bits: the accepted nodes of every request, four layers at once
        dict(name="append8-step-64", op="append8", B=64, packed=False, N=16, lo=500, hi=8000, clo=1, chi=16, Hq=0, Hkv=8, D=128, P=64,
             pairs=64, style="half", layers=4, block=16, dtype="bf16", lens=5),
        # prompts of 64 requests, one layer, rows of 64, odd lengths, scales for 32 tokens
        dict(name="append8-prompts-64", op="append8", B=64, packed=True, N=0, lo=0, hi=300, clo=100, chi=2000, Hq=24, Hkv=4, D=64, P=32,
             pairs=32, style="half", layers=1, block=32, dtype="f16", lens=6),
        # one request, one token over 2,048 rows: latency
        dict(name="tree8-token-2k", op="tree8", B=1, N=1, tree="chain", lo=2048, hi=2048, Hq=32, Hkv=8, D=128, P=64, block=64,
             dtype="bf16", lens=7),
        # the mixed serving batch: 64 requests of 2,000 to 32,000 tokens, blocks of 16 and of 8
        dict(name="tree8-mixed-64", op="tree8", B=64, N=16, tree="branches", lo=2000, hi=32000, Hq=32, Hkv=8, D=128, P=64, block=16,
             dtype="bf16", lens=8),
        # eight very long requests, few heads of keys, chains of 16
        dict(name="tree8-long-262k", op="tree8", B=8, N=16, tree="chain", lo=262100, hi=262144, Hq=16, Hkv=2, D=128, P=128, block=128,
             dtype="f16", lens=9),
        # a wide batch of short requests, an odd number of heads a group, bushy trees, small pages
        dict(name="tree8-wide-256", op="tree8", B=256, N=13, tree="random", lo=300, hi=4096, Hq=24, Hkv=4, D=64, P=16, block=16,
             dtype="f16", lens=10),
        # chunks of prompts behind cached prefixes (a shared document, or the prompt's earlier chunks)
        dict(name="prompt8-chunks-8", op="prompt8", B=8, lo=100, hi=1500, clo=0, chi=8192, Hq=24, Hkv=4, D=64, P=32, block=32,
             dtype="f16", lens=11),
        # a long question about a document that is in the cache
        dict(name="prompt8-document", op="prompt8", B=1, lo=4000, hi=4000, clo=25000, chi=25000, Hq=32, Hkv=8, D=128, P=64, block=64,
             dtype="bf16", lens=12),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rotate", "append", "append8", "tree8", "tree8", "prompt8"])
    Hkv, D, P = rng.choice([1, 2, 4, 8]), rng.choice([64, 128]), rng.choice([16, 32, 64, 128])
    c = dict(op=op, Hkv=Hkv, D=D, P=P, dtype=rng.choice(["bf16", "f16"]), lens=rng.randrange(1 << 20))
    if op in ("rotate", "append", "append8"):
        c.update(pairs=rng.choice([D // 2, D // 2, D // 4]), style=rng.choice(["half", "neighbours"]))
    if op not in ("rotate", "append"):
        c["block"] = rng.choice([t for t in (16, 32, 64, 128) if t <= P])
    trees = ["chain", "branches", "random"]
    if op == "rotate":
        hi = _log(rng, 64, 8192)
        c.update(B=_log(rng, 1, 256), N=_log(rng, 1, 32), tree=rng.choice(trees), lo=hi // 8, hi=hi, Hq=Hkv * rng.choice([1, 3, 4, 6]))
    elif op in ("append", "append8"):
        packed = rng.random() < 0.5
        if packed:
            hi, chi, B = _log(rng, 16, 8192), _log(rng, 16, 2000), _log(rng, 1, 32)
            c.update(B=B, packed=True, N=0, lo=hi // 8, hi=hi, clo=chi // 8, chi=chi, Hq=Hkv * rng.choice([1, 3, 4]), layers=1)
        else:
            hi, N = _log(rng, 64, 4096), _log(rng, 1, 32)
            layers = rng.randint(1, 8)
            c.update(B=_log(rng, 1, 64), packed=False, N=N, lo=hi // 8, hi=hi, clo=0, chi=N, Hq=Hkv * 4 if layers == 1 else 0, layers=layers)
    elif op == "tree8":
        B, N, G = _log(rng, 1, 256), _log(rng, 1, 64), rng.choice([1, 3, 4, 5, 6, 8])
        hi = _log(rng, 64, min(262144, 1e9 / (B * Hkv * D), 1.5e10 / (B * Hkv * G * N * 4)))
        c.update(B=B, N=N, tree=rng.choice(trees), lo=max(0, hi // 8), hi=hi, Hq=G * Hkv)
    else:
        B, G, hi = _log(rng, 1, 16), rng.choice([1, 2, 4, 6, 8]), _log(rng, 16, 4000)
        hi = min(hi, 8000 // B)
        c.update(B=B, lo=max(1, hi // 8), hi=hi, clo=0, chi=_log(rng, 64, 16000 // B), Hq=G * Hkv)
    return c


def _sizes(case):
    """Everything that the case alone fixes, whatever the seed: lengths, counts, trees, packing offsets."""
    r = random.Random(case["lens"])
    c = dict(case)
    B, op = c["B"], c["op"]
    c["len"] = [r.randint(case["lo"], case["hi"]) for _ in range(B)]  # cached rows (prompt8: new ones)
    c["ctx"] = c["len"]
    if op == "prompt8":
        c["ctx"] = [r.randint(case["clo"], case["chi"]) for _ in range(B)]
    elif op in ("append", "append8"):
        c["count"] = [r.randint(case["clo"], case["chi"]) for _ in range(B)]
    c["off"] = [0]
    for n in c["count"] if "count" in c else c["len"]:
        c["off"].append(c["off"][-1] + n)
    if "tree" in c:
        N = c["N"]
        # every other block is a long one, as in a batch where half of the requests copy
        c["nodes"] = [N if b % 2 == 0 else max(1, N // 2) for b in range(B)]
        if c["tree"] == "chain":
            par = [list(range(-1, N - 1)) for _ in range(B)]
        elif c["tree"] == "branches":
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


def _ints(v, dtype=torch.int32):
    return torch.tensor(v, dtype=dtype, device=DEV)


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
    return _ints(rows, torch.int64)


def _cache(s, c, held, r):
    """Slots of `held` rows, grown in shuffled rounds, so that their pages lie in between one another's; free pages
    are handed out lowest number first."""
    B, P = c["B"], c["P"]
    pages = sum(_pages(n, P) for n in held)
    most = max(1, max(_pages(n, P) for n in held))
    slots = r.sample(range(B), B)
    s.update(P=P, pages=pages + pages // 8 + 8, slots=_ints(slots))
    if own:
        import context_lookup_speculative_gb300 as clk

        s["clk"] = clk
        s["cache"] = clk.Cache(max_slots=B, max_pages=most, num_pages=s["pages"], page_tokens=P)
    length, table, taken, left = [0] * B, [[] for _ in range(B)], 0, list(held)
    for part in (3, 2, 1):
        order = list(range(B))
        r.shuffle(order)
        for b in order:
            n = left[b] // part
            left[b] -= n
            length[slots[b]] += n
            need = _pages(length[slots[b]], P) - len(table[slots[b]])
            table[slots[b]] += range(taken, taken + need)
            taken += need
            held[b] = n
        if own:
            s["clk"].cache_grow(s["cache"], _ints([slots[b] for b in order]), _ints([held[b] for b in order]))
    s["length"] = _ints(length)
    s["table"] = _ints([t + [-1] * (most - len(t)) for t in table])


def _table(c):
    """cos and sin of every position's angles, [positions, 2, pairs]."""
    freq = 10000.0 ** (-torch.arange(c["pairs"], dtype=torch.float64, device=DEV) / c["pairs"])
    most = max(n + (c["count"][b] if "count" in c else c["N"]) for b, n in enumerate(c["len"]))
    a = torch.arange(most + 1, dtype=torch.float64, device=DEV)[:, None] * freq
    return torch.stack([a.cos(), a.sin()], 1).float()


def _pool8(s, c, planes, seed):
    """Normal values as appended rows leave them, of another size from block to block."""
    shape = (planes, s["pages"], c["Hkv"], c["P"], c["D"])
    blocks = shape[:3] + (c["P"] // c["block"],)
    s["pool"] = torch.empty(shape, dtype=torch.float8_e4m3fn, device=DEV)
    for i in range(planes):
        x = _normal(shape[1:], torch.bfloat16, seed * 64 + i, 0)
        s["pool"][i] = x.mul_(100.0).clamp_(-TOP, TOP).to(torch.float8_e4m3fn)
    s["scale"] = torch.exp2(torch.randint(-8, -5, blocks, generator=_gen(seed, 5), device=DEV).float())


def prepare(case, seed):
    c = _sizes(case)
    op, B, D, Hq, Hkv, dt = c["op"], c["B"], c["D"], c["Hq"], c["Hkv"], _dtype(c)
    r = random.Random(seed)
    s = dict(op=op, c=c)
    held = list(c["ctx"]) if op in ("rotate", "tree8", "prompt8") else [n + m for n, m in zip(c["len"], c["count"])]
    _cache(s, c, held, r)
    if op in ("rotate", "append", "append8"):
        s["table_cs"] = _table(c)
        if own:
            s["rotary"] = s["clk"].Rotary(s["table_cs"], neighbours=c["style"] == "neighbours")
    if op in ("rotate", "tree8", "prompt8"):
        rows = (c["off"][-1],) if op == "prompt8" else (B, c["N"])
        # queries, keys and values are slices of one projection's output
        qkv = _normal(rows + (Hq + 2 * Hkv, D), dt, seed, 1)
        qkv[..., :Hq, :] *= 1.5
        s.update(q=qkv[..., :Hq, :], k=qkv[..., Hq:Hq + Hkv, :], v=qkv[..., Hq + Hkv:, :])
        if op == "prompt8":
            s.update(off=_ints(c["off"], torch.int64), ctx=_ints(c["ctx"]))
        else:
            s.update(nodes=_ints(c["nodes"]), mask=_mask_bits(c))
        if op == "rotate":
            # rows past a tree's nodes are left as they are
            s.update(q_out=torch.zeros(rows + (Hq, D), dtype=dt, device=DEV), k_out=torch.zeros(rows + (Hkv, D), dtype=dt, device=DEV))
        else:
            _pool8(s, c, 2, seed)
            s.update(scale_qk=1 / math.sqrt(D), out=torch.empty(rows + (Hq, D), dtype=dt, device=DEV))
            if own:
                s["pool8"] = s["clk"].ScaledPool(s["pool"], s["scale"])
                s["scratch"] = s["clk"].attend_scratch(Hq, Hkv, D)
        return s
    L, N = c["layers"], c["N"]
    rows = (c["off"][-1],) if c["packed"] else (B, N)
    s["count"] = _ints(c["count"])
    if c["packed"]:
        s["off"] = _ints(c["off"], torch.int64)
    elif Hq == 0:
        # accepted nodes, ascending; rows past a count are not looked at
        s["path"] = _ints([sorted(r.sample(range(N), n)) + [-1] * (N - n) for n in c["count"]])
    if Hq:
        qkv = _normal((L,) + rows + (Hq + 2 * Hkv, D), dt, seed, 1)
        s.update(q=qkv[0][..., :Hq, :], k=qkv[..., Hq:Hq + Hkv, :], v=qkv[..., Hq + Hkv:, :],
                 q_out=torch.zeros(rows + (Hq, D), dtype=dt, device=DEV), k_out=torch.zeros((L,) + rows + (Hkv, D), dtype=dt, device=DEV))
    else:
        s.update(k=_normal((L,) + rows + (Hkv, D), dt, seed, 1), v=_normal((L,) + rows + (Hkv, D), dt, seed, 4))
    if op == "append":
        s["pool"] = _normal((2 * L, s["pages"], Hkv, c["P"], D), dt, seed, 0)
    else:
        _pool8(s, c, 2 * L, seed)
        if own:
            s["pool8"] = s["clk"].ScaledPool(s["pool"], s["scale"])
    return s


# ---------------------------------------------------------------------------
# Plain forms: rotation and appending
# ---------------------------------------------------------------------------
def _rotate(x, cs, style):
    """Rows x [..., heads, dim] by cs [..., 2, pairs], in float32."""
    x = x.float()
    n = cs.shape[-1]
    c, s = cs[..., 0, :].unsqueeze(-2), cs[..., 1, :].unsqueeze(-2)
    a, b = (x[..., :n], x[..., n:2 * n]) if style == "half" else (x[..., 0:2 * n:2], x[..., 1:2 * n:2])
    u, v = a * c - b * s, b * c + a * s
    turned = torch.cat([u, v], -1) if style == "half" else torch.stack([u, v], -1).flatten(-2)
    return torch.cat([turned, x[..., 2 * n:]], -1)


def _rotate_trees(s):
    q, k, mask = s["q"], s["k"], s["mask"]
    N = q.shape[1]
    at = torch.arange(N, device=DEV)
    bits = (mask[:, :, None] >> at) & 1
    pos = s["length"][s["slots"].long()].long()[:, None] + (bits.sum(2) - 1).clamp(min=0)
    cs, style = s["table_cs"][pos], s["c"]["style"]
    real = (at < s["nodes"][:, None])[:, :, None, None]
    s["q_out"].copy_(torch.where(real, _rotate(q, cs, style).to(q.dtype), s["q_out"]))
    s["k_out"].copy_(torch.where(real, _rotate(k, cs, style).to(k.dtype), s["k_out"]))
    return dict(q=s["q_out"], k=s["k_out"])


def _append_rows(s):
    """For every appended row: its request, source row, slot and position; and the rotated keys and the values, [layers, rows, heads, dim]."""
    count = s["count"].long()
    who = torch.repeat_interleave(torch.arange(count.numel(), device=DEV), count)
    i = torch.arange(who.numel(), device=DEV) - (torch.cumsum(count, 0) - count)[who]
    if "off" in s:
        row = s["off"][who] + i
    else:
        row = who * s["k"].shape[2] + (i if "path" not in s else s["path"][who, i].long())
    slot = s["slots"].long()[who]
    pos = (s["length"][slot].long() - count[who]) + i
    flat = (lambda x: x) if "off" in s else (lambda x: x.flatten(1, 2))
    cs, style = s["table_cs"][pos], s["c"]["style"]
    k = _rotate(flat(s["k"])[:, row], cs, style)
    if "q" in s:
        q_out, k_out = s["q_out"].view(-1, *s["q_out"].shape[-2:]), s["k_out"].view(s["k"].shape[0], -1, *s["k"].shape[-2:])
        q_out[row] = _rotate(flat(s["q"][None])[0][row], cs, style).to(q_out.dtype)
        k_out[:, row] = k.to(k_out.dtype)
    return who, slot, pos, k, flat(s["v"])[:, row]


def _outputs(s):
    more = dict(q=s["q_out"], k=s["k_out"]) if "q" in s else {}
    if "scale" in s:
        more["scale"] = s["scale"]
    return dict(more, pool=s["pool"])


def _append(s):
    P = s["P"]
    who, slot, pos, k, v = _append_rows(s)
    page = s["table"][slot, pos // P].long()
    s["pool"][0::2][:, page, :, pos % P] = k.transpose(0, 1).to(s["pool"].dtype)
    s["pool"][1::2][:, page, :, pos % P] = v.transpose(0, 1).to(s["pool"].dtype)
    return _outputs(s)


def _append8(s):
    P, T = s["P"], s["c"]["block"]
    who, slot, pos, k, v = _append_rows(s)
    x = torch.stack([k, v.float()], 1).flatten(0, 1)  # [planes, rows, heads, dim]
    planes, _, heads, dim = x.shape
    # the blocks that are written to, in the rows' order, and each row's place in them
    new = torch.ones_like(pos, dtype=torch.bool)
    new[1:] = (who[1:] != who[:-1]) | (pos[1:] // T != pos[:-1] // T)
    blk = torch.cumsum(new, 0) - 1
    at, n = pos % T, new.nonzero().flatten()
    page, part = s["table"][slot[n], pos[n] // P].long(), pos[n] % P // T
    first = at[n]  # rows before the first written one
    fresh = torch.zeros((n.numel(), T), dtype=torch.bool, device=DEV)
    fresh[blk, at] = True
    body = s["pool"].view(torch.uint8).unflatten(3, (P // T, T))
    held = body[:, page, :, part].view(torch.float8_e4m3fn).float()  # [blocks, planes, heads, T, dim]
    rows = torch.zeros_like(held)
    rows.transpose(2, 3)[blk, :, at] = x.transpose(0, 1)
    top = rows.abs().amax((3, 4))
    m, e = torch.frexp(top)
    e = torch.where(top > 0, torch.where(m <= TOP / 512, e - 9, e - 8), LEAST).clamp(min=LEAST)
    least = torch.ldexp(torch.ones_like(top), e)
    old = s["scale"][:, page, :, part]
    before = (first > 0)[:, None, None]
    scale = torch.where(before & (old > least) & (old < math.inf), old, least)
    f = scale[..., None, None]
    kept = torch.arange(T, device=DEV) < first[:, None]
    grown = (before & (scale > old))[..., None, None] & kept[:, None, None, :, None]
    held = torch.where(grown, held * old[..., None, None] / f, held)
    rows = torch.where(fresh[:, None, None, :, None], (rows / f).clamp(-TOP, TOP), held).to(torch.float8_e4m3fn)
    body[:, page, :, part] = rows.view(torch.uint8)
    s["scale"][:, page, :, part] = scale
    return _outputs(s)


# ---------------------------------------------------------------------------
# Plain forms: attention
# ---------------------------------------------------------------------------
def _softmax_product(scores, seen, v):
    """softmax over the seen places, times v; a row that sees nothing gives 0."""
    scores.masked_fill_(~seen, -math.inf)
    top = scores.amax(-1, keepdim=True).clamp(min=torch.finfo(torch.float32).min)
    scores.sub_(top).exp_()
    return torch.matmul(scores, v) / scores.sum(-1, keepdim=True).clamp(min=torch.finfo(torch.float32).tiny)


def _values(s, plane, at):
    """Pages `at` of a plane as the values that they stand for: [..., kv heads, page tokens, dim]."""
    T = s["c"]["block"]
    x = s["pool"][plane].view(torch.uint8)[at].view(torch.float8_e4m3fn).float().unflatten(-2, (-1, T))
    return (x * s["scale"][plane][at][..., None, None]).flatten(-3, -2)


def _tree_attend(s):
    q, k, v = s["q"], s["k"], s["v"]
    B, N, Hq, D = q.shape
    Hkv = k.shape[2]
    pages = s["table"][s["slots"].long()].clamp(min=0).long()
    keys = torch.cat([_values(s, 0, pages).permute(0, 2, 1, 3, 4).flatten(2, 3), k.transpose(1, 2).float()], 2)
    vals = torch.cat([_values(s, 1, pages).permute(0, 2, 1, 3, 4).flatten(2, 3), v.transpose(1, 2).float()], 2)
    rows = q.float().view(B, N, Hkv, Hq // Hkv, D).permute(0, 2, 1, 3, 4).flatten(2, 3)
    scores = torch.matmul(rows, keys.transpose(2, 3)).mul_(s["scale_qk"])
    at = torch.arange(keys.shape[2] - N, device=DEV)
    near = (s["mask"][:, :, None] >> torch.arange(N, device=DEV)) & 1
    valid = torch.arange(N, device=DEV) < s["nodes"][:, None]
    ctx = s["length"][s["slots"].long()]
    seen = torch.cat([(at < ctx[:, None])[:, None, :].expand(B, N, -1), (near > 0) & valid[:, None, :]], 2) & valid[:, :, None]
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
    every = torch.arange(s["pages"], device=DEV)
    keys = torch.cat([_values(s, 0, every)[page, :, opos % P], k.float()]).transpose(0, 1)
    vals = torch.cat([_values(s, 1, every)[page, :, opos % P], v.float()]).transpose(0, 1)
    seen = (who[:, None] == torch.cat([old, who])) & (torch.cat([opos, pos]) <= pos[:, None])
    rows = q.float().view(T, Hkv, Hq // Hkv, D).permute(1, 2, 0, 3)
    out = _softmax_product(torch.matmul(rows, keys[:, None].transpose(2, 3)).mul_(s["scale_qk"]), seen, vals[:, None])
    return out.permute(2, 0, 1, 3).reshape(T, Hq, D).to(q.dtype)


def _run_own(s):
    clk, h, op = s["clk"], s["cache"], s["op"]
    if op == "rotate":
        clk.tree_rotate(h, s["slots"], s["q"], s["k"], s["nodes"], s["mask"], s["rotary"], s["q_out"], s["k_out"])
        return dict(q=s["q_out"], k=s["k_out"])
    if op == "tree8":
        clk.tree_attend(h, s["slots"], s["pool8"], 0, s["q"], s["k"], s["v"], s["nodes"], s["mask"], s["scale_qk"], s["out"], s["scratch"])
        return s["out"]
    if op == "prompt8":
        clk.prompt_attend(s["q"], s["k"], s["v"], s["off"], s["scale_qk"], s["out"], s["scratch"], cache=h, slots=s["slots"],
                          pool=s["pool8"], layer=0, ctx=s["ctx"])
        return s["out"]
    clk.cache_append_rotary(h, s["slots"], s["pool8"] if op == "append8" else s["pool"], s["k"], s["v"], s["count"], rotary=s["rotary"],
                            path=s.get("path"), offsets=s.get("off"), q=s.get("q"), q_out=s.get("q_out"), k_out=s.get("k_out"))
    return _outputs(s)


def run(s):
    if own:
        return _run_own(s)
    return {"rotate": _rotate_trees, "append": _append, "append8": _append8, "tree8": _tree_attend, "prompt8": _prompt_attend}[s["op"]](s)


# ---------------------------------------------------------------------------
# The definition in 64 bits, request by request
# ---------------------------------------------------------------------------
def _turned(x, pos, c):
    """Rows [rows, heads, dim] at positions pos as complex numbers times e^(i angle)."""
    n = c["pairs"]
    angle = torch.as_tensor(pos, dtype=torch.float64, device=DEV)[:, None] * 10000.0 ** (-torch.arange(n, dtype=torch.float64, device=DEV) / n)
    y = x.double().clone()
    lo, hi = (slice(0, n), slice(n, 2 * n)) if c["style"] == "half" else (slice(0, 2 * n, 2), slice(1, 2 * n, 2))
    z = torch.complex(y[..., lo], y[..., hi]) * torch.polar(torch.ones_like(angle), angle)[:, None]
    y[..., lo], y[..., hi] = z.real, z.imag
    return y


def _exact_append(s, c):
    eight, P, slots, table = c["op"] == "append8", c["P"], s["slots"].tolist(), s["table"]
    pool = s["pool"].double()
    out = dict(pool=pool)
    if eight:
        out["scale"] = s["scale"].double()
    if "q" in s:
        out.update(q=s["q_out"].double(), k=s["k_out"].double())
    for b, (n, m) in enumerate(zip(c["len"], c["count"])):
        if m == 0:
            continue
        row = range(c["off"][b], c["off"][b] + m) if c["packed"] else (s["path"][b, :m].tolist() if "path" in s else range(m))
        row = torch.tensor(list(row), device=DEV)
        at = (row,) if c["packed"] else (b, row)
        pos = torch.arange(n, n + m, device=DEV)
        if "q" in s:
            out["q"][at] = _turned(s["q"][at], pos, c)
        page, line = table[slots[b], pos // P].long(), pos % P
        for layer in range(c["layers"]):
            for x, plane in ((_turned(s["k"][layer][at], pos, c), 2 * layer), (s["v"][layer][at].double(), 2 * layer + 1)):
                if plane == 2 * layer and "q" in s:
                    out["k"][layer][at] = x
                if not eight:
                    pool[plane][page, :, line] = x
                    continue
                T = c["block"]
                for first in range(n // T * T, n + m, T):
                    lo, hi = max(first, n), min(first + T, n + m)
                    new = x[lo - n:hi - n].transpose(0, 1)  # [heads, rows, dim]
                    p, y = int(table[slots[b], first // P]), first % P
                    need = torch.exp2(torch.ceil(torch.log2(new.abs().amax((1, 2)) / TOP)).clamp(min=LEAST))
                    old = out["scale"][plane, p, :, y // T].clone()
                    got = torch.maximum(need, old) if lo > first else need
                    pool[plane, p, :, y:y + lo - first] *= (old / got)[:, None, None]
                    pool[plane, p, :, y + lo - first:y + hi - first] = new / got[:, None, None]
                    out["scale"][plane, p, :, y // T] = got
    return out


def exact(case, seed):
    global own
    c, was = _sizes(case), own
    # blocks (or requests and layers) are gone through one by one
    if c["op"] == "append8" and c["layers"] * sum(m // c["block"] + 2 for m in c["count"]) > 12000:
        return None
    own = False
    s = prepare(case, seed)
    own = was
    op, slots = c["op"], s["slots"].tolist()
    if op in ("append", "append8"):
        return _exact_append(s, c)
    if op == "rotate":
        out = dict(q=s["q_out"].double(), k=s["k_out"].double())
        for b, (par, m, n) in enumerate(zip(c["parent"], c["nodes"], c["len"])):
            pos = [n + len(a) - 1 for a in _ancestors(par, m)]
            for x in "qk":
                out[x][b, :m] = _turned(s[x][b, :m], pos, c)
        return out
    G, P, T = c["Hq"] // c["Hkv"], c["P"], c["block"]
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device=DEV)
    for b in range(c["B"]):
        n, N = c["ctx"][b], c["nodes"][b] if op == "tree8" else c["len"][b]
        pages = s["table"][slots[b], :_pages(n, P)].long()
        new = (b, slice(0, N)) if op == "tree8" else (slice(c["off"][b], c["off"][b] + N),)
        if op == "tree8":
            sees = torch.zeros((N, N), dtype=torch.bool)
            for i, a in enumerate(_ancestors(c["parent"][b], N)):
                sees[i, a] = True
            sees = sees.to(DEV)
        else:
            sees = torch.ones((N, N), dtype=torch.bool, device=DEV).tril()
        for h in range(c["Hkv"]):
            kv = []
            for x in (0, 1):
                size = s["scale"][x][pages, h].double().repeat_interleave(T, 1)[..., None]
                codes = s["pool"][x, :, h].view(torch.uint8)[pages].view(torch.float8_e4m3fn)
                kv.append(torch.cat([(codes.double() * size).reshape(-1, c["D"])[:n], s["kv"[x]][new][:, h].double()]))
            for g in range(h * G, h * G + G):
                e = (s["q"][new][:, g].double() @ kv[0].T) * s["scale_qk"]
                e[:, n:][~sees] = -math.inf
                out[new + (g,)] = torch.softmax(e, 1) @ kv[1]
    return out


# ---------------------------------------------------------------------------
# The floor
# ---------------------------------------------------------------------------
def work(case):
    c = _sizes(case)
    op, B, P, D, Hq, Hkv = c["op"], c["B"], c["P"], c["D"], c["Hq"], c["Hkv"]
    row = Hkv * D  # elements of a token's K (or V)
    if op == "rotate":
        rows = sum(c["nodes"])
        return dict(bytes=rows * (4 * (Hq + Hkv) * D + 8 * c["pairs"] + 8), flops=rows * (Hq + Hkv) * c["pairs"] * 6)
    if op in ("append", "append8"):
        rows, L = sum(c["count"]), c["layers"]
        size = 2 if op == "append" else 1
        each = 2 * L * row * (2 + size) + 8 * c["pairs"] + (4 * Hq * D + 2 * L * row if Hq else 0)
        more = 0
        if op == "append8":
            # a scale for each block that is written to, read too where it has rows before
            T = c["block"]
            more = sum(8 * L * Hkv * ((n + m - 1) // T - n // T + 1 + (n % T > 0)) for n, m in zip(c["len"], c["count"]) if m)
        return dict(bytes=rows * each + more, flops=rows * (L * Hkv + Hq) * c["pairs"] * 6)
    cached = sum(c["ctx"])
    scales = 8 * Hkv * sum(_pages(n, c["block"]) for n in c["ctx"])
    if op == "tree8":
        pairs = sum(n * m + sum(map(len, _ancestors(p, m))) for n, m, p in zip(c["ctx"], c["nodes"], c["parent"]))
        rows = sum(c["nodes"])
        return dict(bytes=2 * row * (cached + 2 * rows) + scales + 2 * D * Hq * (rows + B * c["N"]) + 4 * sum(_pages(n, P) for n in c["ctx"]),
                    flops=4 * D * Hq * pairs)
    pairs = sum(n * m + m * (m + 1) // 2 for n, m in zip(c["ctx"], c["len"]))
    return dict(bytes=2 * row * (cached + 2 * sum(c["len"])) + scales + 4 * D * Hq * sum(c["len"]), flops=4 * D * Hq * pairs)
