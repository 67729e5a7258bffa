"""Plain float64 definitions of the 8-bit cache, the page tables and the rotary positions, and
seeded caches for the tests."""

from __future__ import annotations

import math

import numpy as np
import torch

from cache_reference import Case, f64

LOWEST, HIGHEST = 10, 246  # exponent bytes


def decoded():
    """The values of the 256 E4M3 codes."""
    out = np.empty(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        out[c] = (m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)) * (-1.0 if c & 128 else 1.0)
        if c & 127 == 127:
            out[c] = math.nan
    return out


VALUES = decoded()


def encoded(x):
    """Codes of float64 x, to nearest, ties to even codes; beyond the largest the largest; NaN is 127."""
    x = np.asarray(x, np.float64)
    grid = VALUES[:127]  # 0 … 448, code c's value, ascending
    a = np.minimum(np.abs(np.nan_to_num(x, nan=0.0, posinf=448.0, neginf=448.0)), 448.0)
    hi = np.minimum(np.searchsorted(grid, a), 126)
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - grid[lo], grid[hi] - a
    up = (dh < dl) | ((dh == dl) & (hi % 2 == 0)) | (hi == 0)
    c = np.where(up, hi, lo) | np.where(np.signbit(x), 128, 0)
    return np.where(np.isnan(x), 127, c).astype(np.uint8)


def byte_for(x):
    """Exponent byte of a block's finite values."""
    x = np.abs(x[np.isfinite(x)])
    top = x.max() if x.size else 0.0
    if top == 0.0:
        return LOWEST
    m, p = math.frexp(top / 448.0)  # top / 448 = m 2^p; a quotient of 8 bits and 7 is no power of two unless exact
    return min(max((p - 1 if m == 0.5 else p) + 127, LOWEST), HIGHEST)


def append(codes, scales, table, lens, cu, new, rows=None):
    """codes [pages, page, hkv, d] and scales [pages, hkv, page / 16] (numpy, changed in place) after
    the append of `new` [total, hkv, d]; lens after it."""
    page = codes.shape[1]
    for s, n in enumerate(lens):
        t = cu[s + 1] - cu[s]
        fresh = {}
        for i in range(t):
            src = cu[s] + i if rows is None else int(rows[cu[s] + i])
            if n - t + i >= 0 and 0 <= src < len(new):
                fresh[n - t + i] = src
        for blk in sorted({j // 16 for j in fresh}):
            at = int(table[s, blk * 16 // page])
            if not 0 <= at < codes.shape[0]:
                continue
            js = [j for j in fresh if j // 16 == blk]
            old = [j for j in range(blk * 16, n - t)]
            old = [j for j in old if j // 16 == blk]
            for h in range(codes.shape[2]):
                x = np.stack([new[fresh[j], h] for j in js])
                sc = scales[at, h]
                b, before = blk * 16 % page // 16, min(max(int(sc[blk * 16 % page // 16]), LOWEST), HIGHEST)
                e = byte_for(x)
                if old:
                    e = max(e, before)
                    if e > before:
                        for j in old:
                            codes[at, j % page, h] = encoded(VALUES[codes[at, j % page, h]] * 2.0 ** (before - e))
                if not old or e > before:
                    sc[b] = e
                for j, row in zip(js, x):
                    codes[at, j % page, h] = encoded(row * 2.0 ** (127 - e))


def values(codes, scales):
    """What the codes stand for."""
    e = np.clip(scales.astype(np.float64), LOWEST, HIGHEST) - 127.0
    per = np.repeat(np.swapaxes(e, 1, 2), 16, axis=1)[..., None]  # [pages, page, hkv, 1]
    return VALUES[codes] * np.exp2(per)


class Fp8Case(Case):
    """A Case whose cache is also held in codes: k and v become what the codes stand for, unused slots
    hold NaN codes, unused blocks the scale byte 255."""

    def __init__(self, *a, spread=0, **kw):
        super().__init__(*a, **kw)
        g = np.random.default_rng(kw.get("seed", 0) + 1)
        for name in ("k", "v"):
            x = f64(getattr(self, name))
            if spread:  # blocks of very different sizes
                x *= 2.0 ** g.integers(-spread, spread + 1, (x.shape[0], x.shape[1] // 16, x.shape[2])).repeat(16, 1)[..., None]
            codes = np.full(x.shape, 127, np.uint8)
            scales = np.full((x.shape[0], x.shape[2], x.shape[1] // 16), 255, np.uint8)
            blocks = x.reshape(x.shape[0], -1, 16, *x.shape[2:])
            for p, b, h in np.ndindex(*scales.swapaxes(1, 2).shape):
                rows = ~np.isnan(blocks[p, b, :, h, 0])
                if rows.any():
                    scales[p, h, b] = byte_for(blocks[p, b, rows, h])
                    codes[p, 16 * b:16 * b + 16, h][rows] = encoded(blocks[p, b, rows, h] * 2.0 ** (127 - int(scales[p, h, b])))
            setattr(self, name + "_codes", torch.from_numpy(codes))
            setattr(self, name + "_scales", torch.from_numpy(scales))
            setattr(self, name, torch.from_numpy(values(codes, scales)).bfloat16())  # (exact)

    def cuda(self):
        super().cuda()
        for name in ("k_codes", "v_codes", "k_scales", "v_scales"):
            setattr(self, name, getattr(self, name).cuda())
        return self

    def pages(self):
        return self.k_codes, self.v_codes, self.k_scales, self.v_scales


def resize(table, held, free, top, lens, page):
    """Lists after cache_pages; (missing, top)."""
    n, width = len(table), len(table[0])
    for s in range(n):
        want = -(-max(lens[s], 0) // page)
        for j in range(want, held[s]):
            if top < len(free):
                free[top] = table[s][j]
                top += 1
            table[s][j] = -1
        held[s] = min(held[s], want)
    asked, there, missing = 0, top, []
    for s in range(n):
        want = -(-max(lens[s], 0) // page)
        if want <= width:
            asked += want - held[s]
            if want > held[s] and asked <= there:
                for j in range(held[s], want):
                    top -= 1
                    table[s][j] = free[top]
                held[s] = want
        missing.append(want - held[s])
    return missing, top


def rotary(x, positions, inv_freq, interleaved, magnitude, inverse=False):
    """x [batch, rows, heads, d] float64, positions [batch, rows]."""
    part = 2 * len(inv_freq)
    # (a position times a frequency in Python's integers: 2^-80 turns)
    unit = [int(round(f / (2 * math.pi) * 2.0 ** 80)) for f in inv_freq]
    turn = np.array([[[(int(p) * u) % (1 << 80) / 2.0 ** 80 for u in unit] for p in row] for row in positions])
    a = 2 * math.pi * turn[:, :, None, :] * (-1.0 if inverse else 1.0)
    c, s = np.cos(a) * magnitude, np.sin(a) * magnitude
    y = x.copy()
    u, w = (slice(0, part, 2), slice(1, part, 2)) if interleaved else (slice(0, part // 2), slice(part // 2, part))
    y[..., u], y[..., w] = x[..., u] * c - x[..., w] * s, x[..., w] * c + x[..., u] * s
    return y
