"""Per-head norms with the rotation and their gradients (v4_norm_rope_fwd, v4_norm_rope_bwd) against the float64 oracle."""
import numpy as np
import pytest
import torch

import sparse_compressed_attention_gb300 as V
from oracle import cache_oracle as CO
from oracle import v4_oracle as O
from tests.helpers import np64

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: U}


def pairs(a, R, begin, half):
    """|a| + |b| of each rotated pair in both its places, |a| elsewhere."""
    a = np.abs(a)
    out = a.copy()
    if R:
        i = begin + (np.arange(R // 2) if half else 2 * np.arange(R // 2))
        j = i + (R // 2 if half else 1)
        out[..., i] = out[..., j] = a[..., i] + a[..., j]
    return out


def check_fwd(y, x, w, pos, f, begin, half, eps):
    """Squares: at most 32 in a lane's row and five butterfly steps, sums of positives (38 U, half of it in the root); the mean,
    the root, the division, two products: 8 U.  The rotation: 2^-21 (8 U) of a pair.  One rounding."""
    ref, u = CO.norm_rope(np64(x), None if w is None else np64(w), pos, f, begin, half, eps)
    allow = HALF_STEP[x.dtype] * np.abs(ref) * (1 + 2.0 ** -8) + 40 * U * pairs(u, 2 * len(f), begin, half) + 1e-37
    err = np.abs(np64(y) - ref)
    assert np.all(err <= allow), float((err / allow).max())


def check_bwd(dx, dw, x, w, dy, pos, f, begin, half, eps):
    """As the forward; g is off by 2^-21 of its pair, its products with w and x and their sum by 48 U of the magnitudes, and a
    sum of n weight-gradient terms in any order by n U of theirs."""
    xf, R = np64(x), 2 * len(f)
    rdx, rdw, g, r, m = CO.norm_rope_grad(xf, None if w is None else np64(w), np64(dy), pos, f, begin, half, eps)
    wf = np.ones(xf.shape[-1]) if w is None else np64(w)
    eg = 8 * U * pairs(np64(dy), R, begin, half) if R else np.zeros_like(xf)
    mag = np.abs(wf * g * xf)
    dm = r * r * ((np.abs(wf * xf) * eg).mean(-1, keepdims=True) + 48 * U * mag.mean(-1, keepdims=True)) + 64 * U * np.abs(m)
    allow = HALF_STEP[x.dtype] * np.abs(rdx) * (1 + 2.0 ** -8) + 1e-37
    allow = allow + r * (np.abs(wf) * eg + 40 * U * np.abs(wf * g) + np.abs(xf) * dm + 40 * U * np.abs(xf * m))
    err = np.abs(np64(dx) - rdx)
    assert np.all(err <= allow), float((err / allow).max())
    if dw is not None:
        u = np.abs(xf) * r
        n = xf.shape[0] * xf.shape[1]
        lim = (u * eg + (40 + n) * U * u * np.abs(g)).sum((0, 1)) + 1e-37
        err = np.abs(np64(dw) - rdw)
        assert np.all(err <= lim), float((err / lim).max())


def make(rows, hq, hk, dim, R, half, dt, seed, fused=False, far=100000):
    g = torch.Generator().manual_seed(seed)
    rng = np.random.default_rng(seed)
    f = O.make_inv_freq(40000.0, R, 16.0, 4096, 32.0, 1.0) if R else np.zeros(0, np.float32)
    pos = rng.integers(-far, far, rows).astype(np.int32)

    def some():
        t = (torch.randn(rows, hq + hk, dim, generator=g) * 0.7).to(dt).cuda()
        if fused:
            return t[:, :hq], t[:, hq:] if hk else None
        return t[:, :hq].contiguous(), t[:, hq:].contiguous() if hk else None
    w = [(1 + 0.3 * torch.randn(dim, generator=g)).cuda() for _ in range(2)]
    return some, w, pos, torch.from_numpy(pos).cuda(), f, torch.from_numpy(f).cuda() if R else None


SHAPES = [
    # rows, hq, hk, dim, R, begin, half
    (1, 1, 0, 8, 0, 0, False), (1, 64, 1, 512, 64, 448, False), (3, 5, 2, 64, 64, 0, True), (7, 3, 1, 24, 8, 8, False),
    (5, 2, 2, 96, 32, 64, True), (33, 1, 0, 128, 128, 0, True), (2, 7, 3, 200, 48, 40, True), (9, 2, 1, 256, 64, 192, False),
    (4, 3, 1, 264, 16, 128, True), (3, 2, 1, 512, 512, 0, True), (3, 2, 1, 1024, 64, 960, False), (2, 3, 1, 1000, 1000, 0, False),
    (2, 2, 2, 1024, 1024, 0, True), (300, 1, 1, 16, 16, 0, True), (65, 16, 4, 40, 0, 0, False), (40, 64, 1, 512, 64, 448, False)]


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("shape", SHAPES)
def test_norm_with_rotation(shape, dt):
    rows, hq, hk, dim, R, begin, half = shape
    if half and R % 16:
        pytest.skip("half layout needs R % 16 == 0")
    some, w, pos, dpos, f, df = make(rows, hq, hk, dim, R, half, dt, sum(shape[:5]))
    q, k = some()
    qo, ko = torch.full_like(q, 9.0), torch.full_like(k, 9.0) if hk else None
    V.v4_norm_rope_fwd(q, k, dpos, df, qo, ko, q_w=w[0], eps=1e-5, rope_begin=begin,
                       layout=V.V4_ROPE_HALF if half else V.V4_ROPE_INTERLEAVED)
    check_fwd(qo, q, w[0], pos, f, begin, half, 1e-5)
    if hk:
        check_fwd(ko, k, None, pos, f, begin, half, 1e-5)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("shape", SHAPES)
def test_gradients(shape, dt):
    rows, hq, hk, dim, R, begin, half = shape
    if half and R % 16:
        pytest.skip("half layout needs R % 16 == 0")
    some, w, pos, dpos, f, df = make(rows, hq, hk, dim, R, half, dt, sum(shape[:5]) + 1)
    q, k = some()
    gq, gk = some()
    dq, dk = torch.full_like(q, 9.0), torch.full_like(k, 9.0) if hk else None
    dwq, dwk = torch.full((dim,), 9.0, device="cuda"), torch.full((dim,), 9.0, device="cuda")
    ws = V.alloc_norm_rope_workspace(dim)
    ws.fill_(255)
    kw = dict(q_w=w[0], dq_w=dwq, dk_w=dwk if hk else None, eps=1e-5, rope_begin=begin,
              layout=V.V4_ROPE_HALF if half else V.V4_ROPE_INTERLEAVED, workspace=ws)
    V.v4_norm_rope_bwd(q, k, gq, gk, dpos, df, dq, dk, **kw)
    check_bwd(dq, dwq, q, w[0], gq, pos, f, begin, half, 1e-5)
    if hk:
        check_bwd(dk, dwk, k, None, gk, pos, f, begin, half, 1e-5)
    again = [t.clone() for t in (dq, dwq)]
    V.v4_norm_rope_bwd(q, k, gq, gk, dpos, df, dq, dk, **kw)
    assert torch.equal(dq, again[0]) and torch.equal(dwq, again[1])


@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("rows", [70, 1300])
def test_many_rows_over_the_blocks(rows, half):
    """More tiles than blocks: every block walks several, queries and keys apart."""
    dim, R = 64, 32
    some, w, pos, dpos, f, df = make(rows, 96, 5, dim, R, half, torch.float32, rows)
    (q, k), (gq, gk) = some(), some()
    dq, dk, ws = torch.empty_like(q), torch.empty_like(k), V.alloc_norm_rope_workspace(dim)
    dwq, dwk = torch.empty(dim, device="cuda"), torch.empty(dim, device="cuda")
    lay = V.V4_ROPE_HALF if half else V.V4_ROPE_INTERLEAVED
    V.v4_norm_rope_bwd(q, k, gq, gk, dpos, df, dq, dk, q_w=w[0], k_w=w[1], dq_w=dwq, dk_w=dwk, layout=lay, workspace=ws)
    check_bwd(dq, dwq, q, w[0], gq, pos, f, dim - R, half, 1e-6)
    check_bwd(dk, dwk, k, w[1], gk, pos, f, dim - R, half, 1e-6)


@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_parts_of_one_fused_projection_in_place(dt, half):
    some, w, pos, dpos, f, df = make(11, 6, 2, 128, 64, half, dt, 5, fused=True)
    lay = V.V4_ROPE_HALF if half else V.V4_ROPE_INTERLEAVED
    q, k = some()
    gq, gk = some()
    q0, k0, gq0, gk0 = q.clone(), k.clone(), gq.clone(), gk.clone()
    dwq, dwk = torch.empty(128, device="cuda"), torch.empty(128, device="cuda")
    V.v4_norm_rope_bwd(q, k, gq, gk, dpos, df, gq, gk, q_w=w[0], k_w=w[1], dq_w=dwq, dk_w=dwk, layout=lay,
                       workspace=V.alloc_norm_rope_workspace(128))
    check_bwd(gq, dwq, q0, w[0], gq0, pos, f, 64, half, 1e-6)
    check_bwd(gk, dwk, k0, w[1], gk0, pos, f, 64, half, 1e-6)
    V.v4_norm_rope_fwd(q, k, dpos, df, q, k, q_w=w[0], k_w=w[1], layout=lay)
    check_fwd(q, q0, w[0], pos, f, 64, half, 1e-6)
    check_fwd(k, k0, w[1], pos, f, 64, half, 1e-6)


def test_broadcast_and_transposed_inputs():
    """Rows or heads of stride 0, heads outside rows."""
    f = O.make_inv_freq(10000.0, 16, 1.0, 0)
    df = torch.from_numpy(f).cuda()
    pos = np.arange(6, dtype=np.int32) * 1000
    base = torch.randn(1, 1, 64, generator=torch.Generator().manual_seed(3)).cuda()
    x = base.expand(6, 4, 64)
    out = torch.empty(4, 6, 64, device="cuda").transpose(0, 1)
    V.v4_norm_rope_fwd(x, None, torch.from_numpy(pos).cuda(), df, out)
    check_fwd(out, x.contiguous(), None, pos, f, 48, False, 1e-6)
    dy = torch.randn(6, 4, 64, generator=torch.Generator().manual_seed(4)).cuda()
    dx = torch.empty(4, 6, 64, device="cuda").transpose(0, 1)
    V.v4_norm_rope_bwd(x, None, dy, None, torch.from_numpy(pos).cuda(), df, dx, workspace=V.alloc_norm_rope_workspace(64))
    check_bwd(dx, None, x.contiguous(), None, dy, pos, f, 48, False, 1e-6)


def test_no_rows():
    e = torch.empty(0, 2, 64, device="cuda")
    z = torch.empty(0, dtype=torch.int32, device="cuda")
    dw = torch.full((64,), 5.0, device="cuda")
    V.v4_norm_rope_fwd(e, None, z, torch.ones(8, device="cuda"), e)
    V.v4_norm_rope_bwd(e, None, e, None, z, torch.ones(8, device="cuda"), e, dq_w=dw, workspace=V.alloc_norm_rope_workspace(64))
    assert (dw == 0).all()


def test_special_values_stay_in_their_head():
    x = torch.randn(3, 2, 64, generator=torch.Generator().manual_seed(1)).cuda()
    clean = x.clone()
    x[1, 0, 5], x[2, 1, 7] = float("nan"), float("inf")
    pos, f = torch.arange(3, dtype=torch.int32).cuda(), torch.rand(8).cuda()
    out, want = torch.empty_like(x), torch.empty_like(x)
    V.v4_norm_rope_fwd(x, None, pos, f, out)
    V.v4_norm_rope_fwd(clean, None, pos, f, want)
    same = torch.ones(3, 2, dtype=torch.bool)
    same[1, 0] = same[2, 1] = False
    assert torch.equal(out[same], want[same])
    assert torch.isnan(out[1, 0]).all() and torch.isnan(out[2, 1, 7])
    zero = torch.zeros(1, 1, 64, device="cuda")
    V.v4_norm_rope_fwd(zero, None, pos[:1], f, zero)
    assert (zero == 0).all()


def test_special_values_of_the_gradient_stay_in_their_head():
    g = torch.Generator().manual_seed(2)
    x, dy = (torch.randn(5, 2, 64, generator=g).cuda() for _ in range(2))
    pos, f = torch.arange(5, dtype=torch.int32).cuda(), torch.rand(8).cuda()
    ws = V.alloc_norm_rope_workspace(64)
    dx, want, dw = torch.empty_like(x), torch.empty_like(x), torch.empty(64, device="cuda")
    V.v4_norm_rope_bwd(x, None, dy, None, pos, f, want, workspace=ws)
    x[1, 0, 5], x[2, 1, 7], dy[3, 1, 9] = float("nan"), float("inf"), float("-inf")
    V.v4_norm_rope_bwd(x, None, dy, None, pos, f, dx, dq_w=dw, workspace=ws)
    bad = torch.zeros(5, 2, dtype=torch.bool)
    bad[1, 0] = bad[2, 1] = bad[3, 1] = True
    assert torch.equal(dx[~bad], want[~bad])
    assert not torch.isfinite(dx[bad]).all(dim=1).any() and not torch.isfinite(dw).all()


def test_gradient_against_differences_of_the_forward():
    """Central differences of the fp32 kernel's own forward: the step's error is about h^2 of the third derivative (1e-6
    here), the difference's 2 U / h of the sum (6e-5 of values of one)."""
    some, w, pos, dpos, f, df = make(2, 1, 0, 32, 16, True, torch.float32, 8, far=50)
    q, _ = some()
    dy, _ = some()
    dq, dw = torch.empty_like(q), torch.empty(32, device="cuda")
    kw = dict(layout=V.V4_ROPE_HALF)
    V.v4_norm_rope_bwd(q, None, dy, None, dpos, df, dq, q_w=w[0], dq_w=dw, workspace=V.alloc_norm_rope_workspace(32), **kw)
    h = 2.0 ** -9

    def total(x, weight):
        out = torch.empty_like(x)
        V.v4_norm_rope_fwd(x, None, dpos, df, out, q_w=weight, **kw)
        return float((out.double() * dy.double()).sum())
    for t, c in ((0, 3), (1, 20), (0, 31)):
        a, b = q.clone(), q.clone()
        a[t, 0, c] += h
        b[t, 0, c] -= h
        assert abs((total(a, w[0]) - total(b, w[0])) / (2 * h) - float(dq[t, 0, c])) < 3e-3
    for c in (0, 17):
        a, b = w[0].clone(), w[0].clone()
        a[c] += h
        b[c] -= h
        assert abs((total(q, a) - total(q, b)) / (2 * h) - float(dw[c])) < 3e-3
