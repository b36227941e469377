"""CPU oracle of the operators around a serving cache: norms with the rotation and
their gradients, rows of the 4-bit cache, pages; in float64 and plain Python from
their definitions.

TEST INFRASTRUCTURE ONLY; shares no code with the CUDA library.
"""
from __future__ import annotations

from fractions import Fraction

import numpy as np

from oracle import serving_oracle as S

F64 = np.float64


def norm_rope(x, w, pos, inv_freq, begin, half=False, eps=1e-6):
    """x [rows, heads, dim]: w x / sqrt(mean x^2 + eps), rotated; and the same before its rotation."""
    x = np.asarray(x, F64)
    u = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    if w is not None:
        u = u * np.asarray(w, F64)
    return (S.rope(u, pos, inv_freq, begin, half) if len(inv_freq) else u.copy()), u


def norm_rope_grad(x, w, dy, pos, inv_freq, begin, half=False, eps=1e-6):
    """dx, dw, and the turned gradient g with r and m = r^2 mean(w g x)."""
    x, dy = np.asarray(x, F64), np.asarray(dy, F64)
    w = np.ones(x.shape[-1]) if w is None else np.asarray(w, F64)
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    g = S.rope(dy, pos, inv_freq, begin, half, inverse=True) if len(inv_freq) else dy
    m = (w * g * x).mean(-1, keepdims=True) * r * r
    return r * (w * g - x * m), (g * x * r).sum((0, 1)), g, r, m


NIBBLE = (0, 2, 4, 6, 1, 3, 5, 7)      # value of each nibble of a word of eight


def q4_row_bytes(dim):
    return -(-(dim // 2 + dim // 16) // 16) * 16


def q4_scale(byte):
    return Fraction(8 + byte % 8, 8) * Fraction(2) ** (byte // 8 - 20)


def _nearest(v):
    """Rational v to the nearest integer, ties to even."""
    n = v.numerator // v.denominator
    rest = v - n
    return n + (1 if rest > Fraction(1, 2) or (rest == Fraction(1, 2) and n % 2) else 0)


def q4_scale_byte(amax):
    """Byte of the scale nearest to amax / 7 (ties to the even significand), in rationals."""
    want = Fraction(float(amax)) / 7
    if want <= q4_scale(0):
        return 0
    e = 0
    while e < 40 and want >= Fraction(2) ** (e + 1 - 20):
        e += 1
    return min(255, 8 * (e - 1) + _nearest(want * 8 / Fraction(2) ** (e - 20)))


def q4_pack(x):
    """Rows x [n, dim] (finite) as bytes [n, row bytes]."""
    x = np.asarray(x, F64)
    n, dim = x.shape
    out = np.zeros((n, q4_row_bytes(dim)), np.uint8)
    for t in range(n):
        for g in range(dim // 16):
            v = x[t, 16 * g:16 * g + 16]
            b = q4_scale_byte(np.abs(v).max())
            s = q4_scale(b)
            codes = [8 + min(7, max(-8, _nearest(Fraction(float(e)) / s))) for e in v]
            for half in (0, 1):
                word = sum(codes[8 * half + NIBBLE[i]] << (4 * i) for i in range(8))
                out[t, 8 * g + 4 * half:8 * g + 4 * half + 4] = [(word >> (8 * i)) & 255 for i in range(4)]
            out[t, dim // 2 + g] = b
    return out


def q4_unpack(rows, dim):
    """Values [n, dim] of byte rows."""
    rows = np.asarray(rows, np.uint8)
    i = np.arange(dim)
    nib = np.array([NIBBLE.index(k) for k in range(8)])[i % 8]
    code = (rows[:, i // 8 * 4 + nib // 2] >> (4 * (nib % 2)).astype(np.uint8)) & 15
    b = rows[:, dim // 2 + i // 16].astype(F64)
    return (code.astype(F64) - 8.0) * 2.0 ** (b // 8 - 20) * (1.0 + (b % 8) / 8.0)


class Pages:
    """Block tables and counts as lists, with the operations' definitions step by step."""

    def __init__(self, table, ref, page):
        self.table = [list(map(int, r)) for r in table]
        self.ref = [int(v) for v in ref]
        self.page = page

    def take(self):
        for p, n in enumerate(self.ref):
            if n == 0:
                self.ref[p] = 1
                return p
        return -1

    def blocks(self, tokens):
        return -(-tokens // self.page)

    def alloc(self, have, need):
        lack = 0
        for i, row in enumerate(self.table):
            for k in range(self.blocks(have[i]), self.blocks(need[i])):
                if row[k] == -1:
                    row[k] = self.take()
                    lack += row[k] < 0
        return lack

    def fork(self, src, length, out_blocks):
        rows, copies, lack = [], [], 0
        free = [p for p, n in enumerate(self.ref) if n == 0]
        for s, n in zip(src, length):
            row, copy = [-1] * out_blocks, [-1, -1, 0]
            if s >= 0:
                old = self.table[s]
                for k in range(n // self.page):
                    row[k] = old[k]
                    if old[k] >= 0:
                        self.ref[old[k]] += 1
                k = n // self.page
                if n % self.page and old[k] >= 0:
                    if free:
                        row[k] = free.pop(0)
                        self.ref[row[k]] = 1
                        copy = [old[k], row[k], n % self.page]
                    else:
                        lack += 1
            rows.append(row)
            copies.append(copy)
        return rows, copies, lack

    def free(self, lo, hi):
        for i, row in enumerate(self.table):
            for k, p in enumerate(row):
                held = any(lo[i] <= u < hi[i] for u in range(k * self.page, (k + 1) * self.page))
                if p >= 0 and not held:
                    row[k] = -1
                    self.ref[p] -= 1


def compact(cache, table, page, base, keep):
    """cache [layers, pages, page, ...] with row base[i] + keep[i][j] of sequence i at base[i] + j."""
    out = cache.copy()
    for i, kept in enumerate(keep):
        for j, s in enumerate(kept):
            a, b = base[i] + s, base[i] + j
            out[:, table[i][b // page], b % page] = cache[:, table[i][a // page], a % page]
    return out
