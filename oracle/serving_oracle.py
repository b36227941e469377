"""CPU oracle of the serving operators: rotary positions, drafted token trees
over a paged cache and 4-bit projections, in float64 from their definitions.

TEST INFRASTRUCTURE ONLY; shares no code with the CUDA library.  Sequences are
walked one row and one key at a time, so it is slow and meant for small cases.
"""
from __future__ import annotations

import numpy as np

F64 = np.float64


def angles(pos, inv_freq):
    """pos * inv_freq reduced to (-pi, pi], exact to about 1e-9 for any int32 position.

    The product of a 32-bit integer and a 24-bit float fits the 64-bit
    mantissa of a long double; so does the reduction's error."""
    a = np.asarray(pos, np.int64).astype(np.longdouble)[:, None] * np.asarray(inv_freq, np.float32).astype(np.longdouble)
    two_pi = np.longdouble("6.283185307179586476925286766559005768")
    return (a - np.rint(a / two_pi) * two_pi).astype(F64)


def rope(x, pos, inv_freq, begin, half=False, inverse=False, mscale=1.0):
    """x [rows, heads, dim] with dims [begin, begin + R) rotated at pos."""
    y = np.array(x, dtype=F64, copy=True)
    phi = angles(pos, inv_freq)[:, None, :] * (-1.0 if inverse else 1.0)
    c, s, R = np.cos(phi), np.sin(phi), 2 * len(inv_freq)
    ia = begin + (np.arange(R // 2) if half else 2 * np.arange(R // 2))
    ib = ia + (R // 2 if half else 1)
    a, b = np.array(x[..., ia], F64), np.array(x[..., ib], F64)
    y[..., ia] = mscale * (a * c - b * s)
    y[..., ib] = mscale * (a * s + b * c)
    return y


def rope_error(x, inv_freq, begin, half=False, mscale=1.0):
    """Bound of the fp32 rotation's error before the final rounding, per element.

    Angle: at most pi 2^-25 from an fp32 fraction of a half turn (pi 2^-27 from one of
    an eighth of a turn) and 1.5e-9 from the dropped bits; sine and cosine 2^-23; a scale, two products and a sum 2^-24 each:
    below 2^-21 (|a| + |b|) in all."""
    e = np.zeros(np.shape(x), F64)
    R = 2 * len(inv_freq)
    ia = begin + (np.arange(R // 2) if half else 2 * np.arange(R // 2))
    ib = ia + (R // 2 if half else 1)
    m = (np.abs(np.asarray(x[..., ia], F64)) + np.abs(np.asarray(x[..., ib], F64))) * abs(mscale) * 2.0 ** -21
    e[..., ia] = m
    e[..., ib] = m
    return e


def tree_plan(node_begin, seq_len, parent, n_rows):
    """plan [n_rows, 8] (int64 words; the four bit words unsigned), positions [n_rows]."""
    plan = np.zeros((n_rows, 8), np.int64)
    plan[:, 0] = -1
    for b, L in enumerate(seq_len):
        lo, hi = int(node_begin[b]), int(node_begin[b + 1])
        for row in range(lo, hi):
            bits, depth, j = 0, -1, row - lo
            while j >= 0:
                bits |= 1 << j
                depth += 1
                j = int(parent[lo + j]) if parent is not None else j - 1
            plan[row] = [b, row - lo, L + depth, L] + [(bits >> (32 * w)) & 0xFFFFFFFF for w in range(4)]
    return plan, np.where(plan[:, 0] >= 0, plan[:, 2], 0)


def tree_keys(plan, row, tok_rows, ent_rows, idx, ratio, window, K):
    """Key rows of a planned row.  tok_rows(b, at) and ent_rows(b, s) give a cache row or None."""
    b, _, t, L = (int(v) for v in plan[row, :4])
    keys = []
    n_ent = 0
    if ratio:
        n_ent = min((t + 1) // ratio, ent_rows(b, None))
        for s in (range(n_ent) if not K else [int(v) for v in idx[row]]):
            if 0 <= s < n_ent:
                keys.append(ent_rows(b, s))
    if window != 0:
        for u in range(0 if window < 0 else max(0, t - window + 1), min(L, t + 1)):
            keys.append(tok_rows(b, u))
        first = row - int(plan[row, 1])
        for j in range(128):
            if (int(plan[row, 4 + j // 32]) >> (j % 32)) & 1:
                d = t - int(plan[first + j, 2])
                if d >= 0 and (window < 0 or d < window):
                    keys.append(tok_rows(b, L + j))
    return [k for k in keys if k is not None]


def tree_mqa(q, plan, tok_rows, ent_rows, idx, sink, inv_freq, ratio, window, K, scale, o0, lse0):
    """o, lse, and per-element bounds' ingredients: sum_j p_j |key_j| mixed over rotated pairs, and the
    largest sum_c |q_c||key_c| of a row's keys."""
    n, H, D = q.shape
    R = 2 * len(inv_freq)
    o, lse = np.array(o0, F64), np.array(lse0, F64)
    mass, dots = np.zeros((n, H, D)), np.zeros((n, H))
    for row in range(n):
        if plan[row, 0] < 0:
            continue
        t = int(plan[row, 2])
        keys = tree_keys(plan, row, tok_rows, ent_rows, idx, ratio, window, K)
        k = np.array(keys, F64).reshape(len(keys), D)
        qr = rope(q[row:row + 1], [t], inv_freq, D - R)[0] if R else np.asarray(q[row], F64)
        x = qr @ k.T * scale
        cols = x if sink is None else np.concatenate([x, np.asarray(sink, F64)[:, None]], 1)
        if cols.shape[1] == 0:
            o[row], lse[row] = 0.0, -np.inf
            continue
        top = cols.max(1, keepdims=True)
        with np.errstate(divide="ignore", invalid="ignore"):
            total = np.exp(cols - top).sum(1, keepdims=True)
            p = np.exp(x - top) / total
            lse[row] = (top + np.log(total))[:, 0]
        y = p @ k
        a = p @ np.abs(k)
        if R:
            y = rope(y[None], [t], inv_freq, D - R, inverse=True)[0]
            pair = a[:, D - R::2] + a[:, D - R + 1::2]
            a[:, D - R::2], a[:, D - R + 1::2] = pair, pair
        o[row], mass[row] = y, a
        if len(keys):
            dots[row] = (np.abs(qr) @ np.abs(k).T).max(1)
    return o, lse, mass, dots


def w4_order(K):
    """(byte, nibble) of each input within an output's codes."""
    k = np.arange(K)
    blk, c, t, e = k // 128, k % 128 // 32, k % 32 // 8, k % 8
    nib = (e % 2) * 4 + e // 2
    return blk * 64 + (4 * t + c) * 4 + nib // 2, nib % 2


def w4_weights(codes, scales, gs):
    """Codes [G, N, K/2] and scales [G, N, K/gs] as float64 weights [G, N, K]."""
    K = codes.shape[2] * 2
    byte, high = w4_order(K)
    c = (codes[:, :, byte] >> (4 * high).astype(np.uint8)) & 15
    return (c.astype(F64) - 8.0) * np.repeat(np.asarray(scales, F64), gs, axis=2)


def w4_pack(w, gs, to_bf16):
    """Codes and scales of w [G, K, N] (bf16 values): the definition in fp32, as the library takes its decisions."""
    G, K, N = w.shape
    wt = np.ascontiguousarray(np.asarray(w, np.float32).transpose(0, 2, 1))
    amax = np.abs(wt).reshape(G, N, K // gs, gs).max(-1)
    scales = to_bf16(amax / np.float32(7.0)).astype(np.float32)
    s = np.repeat(scales, gs, axis=2)
    with np.errstate(divide="ignore", invalid="ignore"):
        q = np.where(s > 0, np.rint(wt / s), 0.0)
    q = np.clip(q, -8, 7).astype(np.int64) + 8
    codes = np.zeros((G, N, K // 2), np.uint8)
    byte, high = w4_order(K)
    for h in (0, 1):
        sel = np.nonzero(high == h)[0]
        codes[:, :, byte[sel]] |= (q[:, :, sel] << (4 * h)).astype(np.uint8)
    return codes, scales


def w4_proj(x, codes, scales, gs, norm_dim=0, eps=1e-6, norm_w=None):
    """y [rows, G, N] and the sums of magnitudes sum_k |x||w|."""
    w = w4_weights(codes, scales, gs)
    x = np.asarray(x, F64)
    y = np.einsum("tgk,gnk->tgn", x, w)
    mag = np.einsum("tgk,gnk->tgn", np.abs(x), np.abs(w))
    if norm_dim:
        h = y.reshape(y.shape[0], y.shape[1], -1, norm_dim)
        inv = 1.0 / np.sqrt((h * h).mean(-1, keepdims=True) + eps)
        g = np.ones(norm_dim) if norm_w is None else np.asarray(norm_w, F64)
        y = (h * inv * g).reshape(y.shape)
        m = mag.reshape(h.shape)
        # an error e of each sum moves the output by inv g e, and through the norm by at most |y| |e| / |h|
        rel = np.sqrt((m * m).sum(-1, keepdims=True)) * inv / np.sqrt(norm_dim)
        mag = (m * inv * np.abs(g) + np.abs(y).reshape(h.shape) * rel).reshape(y.shape)
    return y, mag
