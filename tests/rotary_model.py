"""Plain models of position rotation and of a cache in 8 bits, for the tests:
rows in float32 with every operation rounded, block by block, on the CPU."""
import math

import torch

TOP, LEAST = 448.0, -120


def angles(positions, pairs, seed=0):
    """A table [positions, 2, pairs] of turns that differ from pair to pair and position to position."""
    f = 10000.0 ** (-torch.arange(pairs, dtype=torch.float64) / pairs)
    a = (torch.arange(positions, dtype=torch.float64)[:, None] + seed) * f
    return torch.stack([a.cos(), a.sin()], 1).float()


def turned(x, pos, table, neighbours):
    """Rows x [rows, heads, dim] at positions pos, in float32."""
    x = x.float().clone()
    n = table.shape[2]
    cs = table[torch.as_tensor(pos, dtype=torch.int64)]
    c, s = cs[:, None, 0], cs[:, None, 1]
    i = torch.arange(n)
    lo, hi = (2 * i, 2 * i + 1) if neighbours else (i, i + n)
    a, b = x[..., lo], x[..., hi]
    x[..., lo], x[..., hi] = a * c - b * s, b * c + a * s
    return x


def codes(x):
    """float32 values as the e4m3 values next to them (a tie to the even one), the largest for those beyond."""
    return x.clamp(-TOP, TOP).to(torch.float8_e4m3fn).float()


def scale_of(rows):
    """The least power of two with which the largest finite magnitude is at most 448."""
    a = rows.abs()
    a = a[torch.isfinite(a)]
    top = float(a.max()) if a.numel() else 0.0
    if top == 0.0:
        return 2.0 ** LEAST
    m, e = math.frexp(top)  # 448 = 0.875 * 2^9
    return 2.0 ** max(LEAST, e - 9 if m <= 0.875 else e - 8)


class Eight:
    """Codes (as float32 values) [planes, pages, heads, page tokens, dim] and scales [planes, pages, heads, blocks]."""

    def __init__(self, data, scale):
        self.codes, self.scale = data.float().cpu(), scale.cpu().clone()
        self.P = self.codes.shape[3]
        self.T = self.P // scale.shape[3]

    def append(self, plane, pages, p0, rows):
        """rows [n, heads, dim] (float32) to positions p0 .. of a slot that holds these pages."""
        n, T, P = rows.shape[0], self.T, self.P
        for start in range(p0 // T * T, p0 + n, T):
            lo, hi = max(start, p0), min(start + T, p0 + n)
            page, line = pages[start // P], start % P
            for h in range(rows.shape[1]):
                new = rows[lo - p0:hi - p0, h]
                need = torch.tensor(scale_of(new), dtype=torch.float32)
                had = self.scale[plane, page, h, line // T].clone()
                if lo > start and 0 < float(had) < math.inf:
                    if had < need:
                        old = self.codes[plane, page, h, line:line + lo - start]
                        self.codes[plane, page, h, line:line + lo - start] = codes(old * had / need)
                    need = torch.maximum(need, had)
                self.scale[plane, page, h, line // T] = need
                self.codes[plane, page, h, line + lo - start:line + hi - start] = codes(new / need)


def same(got, want):
    """Equal bit for bit, any NaN for a NaN."""
    got, want = got.float().cpu(), want.float().cpu()
    if got.shape != want.shape:
        return False
    nan = torch.isnan(want)
    return torch.equal(torch.isnan(got), nan) and torch.equal(got[~nan], want[~nan]) \
        and torch.equal(torch.signbit(got[~nan]), torch.signbit(want[~nan]))
