"""Norms over so many heads that a group takes a run of them: ring slots, angles and exchange strips used again, rows that
change within a run, weight sums over thousands of blocks.  Against the definitions in 64 bits, on the GPU."""
import numpy as np
import pytest
import torch

import sparse_compressed_attention_gb300 as V
from oracle import v4_oracle as O

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: U}


def places(R, begin, half):
    i = begin + (torch.arange(R // 2) if half else 2 * torch.arange(R // 2))
    return i.cuda(), (i + (R // 2 if half else 1)).cuda()


def turned(x, pos, f, begin, half, sign):
    out = x.clone()
    if f is not None:
        i, j = places(2 * f.numel(), begin, half)
        phi = sign * pos.double()[:, None, None] * f.double()
        c, s = torch.cos(phi), torch.sin(phi)
        a, b = x[..., i], x[..., j]
        out[..., i], out[..., j] = a * c - b * s, a * s + b * c
    return out


def pair_sums(x, f, begin, half):
    """|a| + |b| of each rotated pair in both its places, |a| elsewhere."""
    x = x.abs()
    if f is not None:
        i, j = places(2 * f.numel(), begin, half)
        x[..., i] = x[..., j] = x[..., i] + x[..., j]
    return x


def check_fwd(y, x, w, pos, f, begin, half, eps):
    """Squares: at most 32 in a lane's row and five butterfly steps, sums of positives (38 U, half of it in the root); the mean,
    the root, the division, two products: 8 U.  The rotation: 2^-21 (8 U) of a pair.  One rounding."""
    xf = x.double()
    u = xf / torch.sqrt(xf.square().mean(-1, keepdim=True) + eps) * w.double()
    ref = turned(u, pos, f, begin, half, 1.0)
    allow = HALF_STEP[x.dtype] * ref.abs() * (1 + 2.0 ** -8) + 40 * U * pair_sums(u, f, begin, half) + 1e-37
    worst = ((y.double() - ref).abs() / allow).max().item()
    assert worst <= 1, worst


def check_bwd(dx, dw, x, w, dy, pos, f, begin, half, eps, depth):
    """dx: g off by 2^-21 of its pair, its products with w and x and their sum by 48 U of the magnitudes.  dw: each term is off by
    its g and by 40 U, each of `depth` additions that a term goes through by U of the magnitudes."""
    xf = x.double()
    r = 1.0 / torch.sqrt(xf.square().mean(-1, keepdim=True) + eps)
    g = turned(dy.double(), pos, f, begin, half, -1.0)
    eg = 8 * U * pair_sums(dy.double(), f, begin, half) if f is not None else torch.zeros_like(xf)
    wf = w.double()
    m = (wf * g * xf).mean(-1, keepdim=True) * r * r
    ref = r * (wf * g - xf * m)
    dm = r * r * (((wf * xf).abs() * eg).mean(-1, keepdim=True) + 48 * U * (wf * g * xf).abs().mean(-1, keepdim=True)) + 64 * U * m.abs()
    allow = HALF_STEP[x.dtype] * ref.abs() * (1 + 2.0 ** -8) + 1e-37
    allow = allow + r * (wf.abs() * eg + 40 * U * (wf * g).abs() + xf.abs() * dm + 40 * U * (xf * m).abs())
    worst = ((dx.double() - ref).abs() / allow).max().item()
    assert worst <= 1, worst
    u = xf * r
    lim = (u.abs() * eg + (40 + depth) * U * (u * g).abs()).sum((0, 1)) + 1e-37
    worst = ((dw.double() - (u * g).sum((0, 1))).abs() / lim).max().item()
    assert worst <= 1, worst
    assert (lim <= 0.02 * (u * g).square().sum((0, 1)).sqrt()).all()      # a hundredth of the heads left out shows


# Heads for runs of about seven forwards (and more in the gradient, whose waves are smaller): 152 SMs x 8 blocks (3 for wide heads)
# x the heads that 128 threads hold.
SHAPES = [
    # rows, hq, hk, dim, R, begin
    (30011, 8, 1, 24, 16, 8), (9001, 13, 2, 64, 32, 32), (5003, 11, 3, 128, 128, 0), (3001, 9, 2, 512, 64, 448), (34003, 1, 0, 512, 64, 448),
    (2503, 12, 2, 264, 16, 128), (3001, 9, 2, 512, 512, 0), (1801, 5, 2, 1024, 64, 960), (2003, 6, 1, 1000, 0, 0)]
# Additions that a term of dw goes through: its group's run (at most 24 heads), 5 shuffles, 4 warps, then of up to 4864 blocks every
# 1024th (5), 2 + 5 shuffles and 8 blocks of a cluster.
DEPTH = 24 + 5 + 4 + 5 + 7 + 8


def tensors(rows, hq, hk, dim, R, dt, seed, fused):
    g = torch.Generator(device="cuda").manual_seed(seed)
    f = torch.from_numpy(O.make_inv_freq(40000.0, R, 16.0, 4096, 32.0, 1.0)).cuda() if R else None
    pos = torch.randint(-100000, 100000, (rows,), generator=g, device="cuda", dtype=torch.int32)
    w = [1 + 0.3 * torch.randn(dim, generator=g, device="cuda") for _ in range(2)]

    def some():
        t = (torch.randn(rows, hq + hk, dim, generator=g, device="cuda") * 0.7).to(dt)
        if fused:
            return t[:, :hq], t[:, hq:] if hk else None
        return t[:, :hq].contiguous(), t[:, hq:].contiguous() if hk else None
    return some, w, pos, f


@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("shape", SHAPES)
def test_runs_of_heads(shape, dt, half):
    """Strided parts of one projection, forwards in place."""
    rows, hq, hk, dim, R, begin = shape
    lay = V.V4_ROPE_HALF if half else V.V4_ROPE_INTERLEAVED
    some, w, pos, f = tensors(rows, hq, hk, dim, R, dt, dim + R, True)
    (q, k), (gq, gk) = some(), some()
    dq, dk = some()
    dw = [torch.full((dim,), 9.0, device="cuda") for _ in range(2)]
    ws = V.alloc_norm_rope_workspace(dim)
    ws.fill_(255)
    V.v4_norm_rope_bwd(q, k, gq, gk, pos, f, dq, dk, q_w=w[0], k_w=w[1], dq_w=dw[0], dk_w=dw[1] if hk else None, eps=1e-5,
                       rope_begin=begin, layout=lay, workspace=ws)
    check_bwd(dq, dw[0], q, w[0], gq, pos, f, begin, half, 1e-5, DEPTH)
    if hk:
        check_bwd(dk, dw[1], k, w[1], gk, pos, f, begin, half, 1e-5, DEPTH)
    q0, k0 = q.clone(), k.clone() if hk else None
    V.v4_norm_rope_fwd(q, k, pos, f, q, k, q_w=w[0], k_w=w[1], eps=1e-5, rope_begin=begin, layout=lay)
    check_fwd(q, q0, w[0], pos, f, begin, half, 1e-5)
    if hk:
        check_fwd(k, k0, w[1], pos, f, begin, half, 1e-5)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,hq,hk,dim", [
    (9001, 24, 9, 64),             # 1039 and 390 blocks
    (30011, 15, 13, 512),          # 2558 and 2217: as many as there may be, in runs of 44
    (65537, 1, 1, 1024), (400009, 7, 5, 64), (1300003, 5, 4, 8), (50021, 13, 0, 128)])
def test_weight_sums_are_whole(rows, hq, hk, dim, dt):
    """Every value of x is 1 or -1 (so the root is 1 and u = x), those of dy small whole numbers: all sums of a column are whole
    numbers below 2^24, exact in any order, and so are the means' numerators.  A head left out or taken twice shows."""
    g = torch.Generator(device="cuda").manual_seed(rows)
    one = torch.ones(1, 1, dim, device="cuda")
    y = torch.empty_like(one)
    V.v4_norm_rope_fwd(one, None, None, None, y, eps=0.0)
    assert (y == 1).all()                                         # the reciprocal root of one

    def some(lo, hi):
        return torch.randint(lo, hi, (rows, hq + hk, dim), generator=g, device="cuda", dtype=torch.int8)
    x, dy = some(0, 2) * 2 - 1, some(-3, 4)
    q, k = (t.contiguous().to(dt) if t.shape[1] else None for t in (x[:, :hq], x[:, hq:]))
    gq, gk = (t.contiguous().to(dt) if t.shape[1] else None for t in (dy[:, :hq], dy[:, hq:]))
    dq, dk = torch.empty_like(q), torch.empty_like(k) if hk else None
    dw = [torch.full((dim,), 9.0, device="cuda") for _ in range(2)]
    ws = V.alloc_norm_rope_workspace(dim)
    ws.fill_(255)
    V.v4_norm_rope_bwd(q, k, gq, gk, None, None, dq, dk, dq_w=dw[0], dk_w=dw[1] if hk else None, eps=0.0, workspace=ws)
    for part, got, dx in ((slice(0, hq), dw[0], dq), (slice(hq, hq + hk), dw[1], dk)):
        if dx is None:
            continue
        a, b = x[:, part], dy[:, part]
        want = torch.stack([(a[:, h] * b[:, h]).sum(0, dtype=torch.int64) for h in range(a.shape[1])]).sum(0)
        assert int(want.abs().max()) < 2 ** 24 and torch.equal(got.long(), want) and torch.equal(got, got.round())
        for t in range(0, rows, 50000):
            xs, gs = a[t:t + 50000].float(), b[t:t + 50000].float()
            m = (xs * gs).sum(-1, keepdim=True) / dim             # whole over a power of two: exact
            assert torch.equal(dx[t:t + 50000], (gs - xs * m).to(dt))


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_a_run_gives_what_short_calls_give(dt):
    """Rows of a long call against calls of 16 rows each, bit for bit: a head's result depends on the head alone."""
    rows, dim, R = 34000, 512, 64
    some, w, pos, f = tensors(rows, 1, 0, dim, R, dt, 5, False)
    (q, _), (gq, _) = some(), some()
    out, dq = torch.empty_like(q), torch.empty_like(q)
    ws = V.alloc_norm_rope_workspace(dim)
    V.v4_norm_rope_fwd(q, None, pos, f, out, q_w=w[0])
    V.v4_norm_rope_bwd(q, None, gq, None, pos, f, dq, q_w=w[0], workspace=ws)
    o2, d2 = torch.empty_like(q), torch.empty_like(q)
    for t in np.random.default_rng(0).choice(rows // 16, 60, replace=False) * 16:
        s = slice(int(t), int(t) + 16)
        V.v4_norm_rope_fwd(q[s], None, pos[s], f, o2[s], q_w=w[0])
        V.v4_norm_rope_bwd(q[s], None, gq[s], None, pos[s], f, d2[s], q_w=w[0], workspace=ws)
        assert torch.equal(out[s], o2[s]) and torch.equal(dq[s], d2[s])
