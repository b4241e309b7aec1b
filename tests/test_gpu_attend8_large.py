"""A cache in 8 bits of more than 2^32 bytes in a plane, and one of several hundred heads and layers: rows that are
appended, read by trees and prompts in both kernels, forked and moved.  GPU."""
import numpy as np
import pytest
import torch

import context_lookup_speculative_gb300 as clk
from cache_model import attend_row
from rotary_model import Eight, angles, same, turned
from test_gpu_append8 import Case
from test_gpu_attend import DT, compare, f64, ints
from test_gpu_attend8 import Prompt8, Tree8

pytestmark = pytest.mark.gpu


def test_a_plane_of_more_than_two_to_the_32_bytes():
    pages, P, H, D, T, n = 17400, 128, 16, 128, 64, 300
    cache = clk.Cache(4, pages, pages, P)
    pool = clk.ScaledPool(torch.empty((2, pages, H, P, D), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn),
                          torch.ones((2, pages, H, P // T), device="cuda"))
    assert pool.data[0].numel() > 1 << 32
    clk.cache_grow(cache, ints([0]), ints([(pages - 8) * P]))
    clk.cache_grow(cache, ints([2]), ints([n]))
    far = cache.table[2, :3].tolist()
    assert far == [pages - 8, pages - 7, pages - 6]
    pool.data.view(torch.uint8)[:, far] = 0
    model = Eight(pool.data[:, far], pool.scale[:, far])
    g = torch.Generator(device="cuda").manual_seed(5)
    table = angles(n + 8, 64)
    rot = clk.Rotary(table.cuda())
    k, v = (torch.empty((1, n, H, D), device="cuda").normal_(generator=g).bfloat16() for _ in range(2))
    clk.cache_append_rotary(cache, ints([2]), pool, k, v, ints([n]), rotary=rot, offsets=ints([0, n], torch.int64))
    torch.cuda.synchronize()
    for plane, rows in ((0, turned(k[0].cpu(), range(n), table, False)), (1, v[0].cpu().float())):
        model.append(plane, [0, 1, 2], 0, rows)
    assert same(pool.data[:, far], model.codes) and same(pool.scale[:, far], model.scale)
    values = (model.codes.double().unflatten(3, (P // T, T)) * model.scale[..., None, None].double()).flatten(3, 4).numpy()
    held = [values[x].transpose(1, 0, 2, 3).reshape(H, 3 * P, D)[:, :n] for x in (0, 1)]
    for kind in ("bf16", "f16"):
        qkv = torch.empty((1, 2, 3 * H, D), device="cuda").normal_(generator=g).to(DT[kind])
        q, nk, nv = qkv.split(H, 2)
        for scale in (0.09, -0.09):  # a negative one goes through the general kernel
            out, flat = (torch.zeros((1, 2, H, D), dtype=DT[kind], device="cuda") for _ in range(2))
            scratch = clk.attend_scratch(H, H, D)
            clk.tree_attend(cache, ints([2]), pool, 0, q, nk, nv, ints([2]), ints([[1, 3]], torch.int64), scale, out, scratch)
            clk.prompt_attend(q[0], nk[0], nv[0], ints([0, 2], torch.int64), scale, flat[0], scratch, cache=cache, slots=ints([2]), pool=pool,
                              ctx=ints([n]))
            torch.cuda.synchronize()
            for h in (0, H - 1):
                for t in range(2):
                    keys, vals = np.concatenate([held[0][h], f64(nk)[0, :t + 1, h]]), np.concatenate([held[1][h], f64(nv)[0, :t + 1, h]])
                    want, size = attend_row(f64(q)[0, t, h], keys, vals, scale)
                    for o in (out, flat):
                        compare(f64(o)[0, t, h], want, size, kind, len(keys), np.abs(vals).max(), (kind, scale, h, t))
    # forked to the pages behind, then moved to the front
    clk.cache_fork(cache, ints([2]), ints([3]), pool)
    tail = cache.table[3, 2].item()
    assert tail == pages - 5
    assert same(pool.data[:, tail, :, :n - 2 * P], pool.data[:, far[2], :, :n - 2 * P]) and same(pool.scale[:, tail], pool.scale[:, far[2]])
    clk.cache_free(cache, ints([0]))
    clk.cache_compact(cache, pool)
    torch.cuda.synchronize()
    assert cache.status()[0] == 0 and cache.table[2, :3].tolist() == [0, 1, 2] and cache.table[3, :3].tolist() == [0, 1, 3]
    for page, rows in ((0, P), (1, P), (2, n - 2 * P)):
        assert same(pool.data[:, page, :, :rows], model.codes[:, page, :, :rows]) and same(pool.scale[:, page], model.scale[:, page])


def test_hundreds_of_heads_and_layers():
    c = Case(11, 2, 48, 64, 16, "bf16", P=16, layers=8, pages=5, pairs=32)
    c.add([1, 0], [40, 17])
    c.add([0, 1], [3, 20], "dense", size=3.0)
    c.check()
    for D, kind in ((64, "f16"), (128, "bf16")):
        Tree8(12, 2, 3, [150, 40], 2, 48, D, 16, kind, nodes=[3, 2], layers=8, layer=7).run().check()
        Prompt8(13, [5, 20], 2, 96, D, kind, ctx=[140, 30]).run().check(rows=3)
