"""Rotary positions and the paged cache write against the float64 oracle:
layouts, parts of the head, strides, far positions, the gradient, refusals."""
import numpy as np
import pytest
import torch

import sparse_compressed_attention_gb300 as V
from oracle import serving_oracle as S
from oracle import v4_oracle as O
from tests.helpers import np64

pytestmark = pytest.mark.gpu
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def freqs(R, theta=40000.0, yarn=16.0):
    return O.make_inv_freq(theta, R, yarn, 4096, 32.0, 1.0)


def check(out, x, pos, f, begin, half=False, inverse=False, mscale=1.0):
    ref = S.rope(np64(x), np64(pos).astype(np.int64), f, begin, half, inverse, mscale)
    allow = HALF_STEP[out.dtype] * np.abs(ref) + S.rope_error(np64(x), f, begin, half, mscale) * (1 + 2 ** -8)
    err = np.abs(np64(out) - ref)
    assert np.all(err <= allow), (err - allow).max()
    R = 2 * len(f)
    keep = np.ones(x.shape[-1], bool)
    keep[begin:begin + R] = False
    assert np.array_equal(np64(out)[..., keep], np64(x)[..., keep])


def draw(rows, heads, dim, dt, seed=0, far=1 << 20):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, heads, dim, generator=g).to(dt).cuda()
    pos = torch.randint(0, far, (rows,), generator=g, dtype=torch.int32).cuda()
    return x, pos


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("rows,heads,dim,R,begin", [
    (1, 1, 8, 8, 0), (1, 64, 512, 64, 448), (3, 7, 512, 64, 448), (129, 1, 512, 64, 448), (257, 2, 64, 64, 0),
    (5, 3, 136, 32, 40), (33, 5, 128, 128, 0), (2, 1, 2048, 1024, 1024), (1000, 9, 24, 16, 8)])
def test_rotation_matches_oracle(rows, heads, dim, R, begin, half, dt):
    if half and R % 16:
        pytest.skip("the half layout takes multiples of 16")
    x, pos = draw(rows, heads, dim, dt, seed=rows)
    f = freqs(R)
    out = torch.full_like(x, float("nan"))
    V.v4_rope(x, pos, torch.from_numpy(f).cuda(), out, rope_begin=begin,
              layout=V.V4_ROPE_HALF if half else V.V4_ROPE_INTERLEAVED)
    check(out, x, pos, f, begin, half)


@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("inverse", [False, True])
def test_extreme_positions_and_scaling(half, inverse):
    x, _ = draw(8, 2, 128, torch.float32, seed=4)
    pos = torch.tensor([0, 1, -1, 2 ** 31 - 1, -2 ** 31, 123456789, -987654321, 1 << 30], dtype=torch.int32).cuda()
    f = freqs(64)
    f[3] = 0.0
    f[5] = -f[5]
    f[7] = 1.5
    out = torch.empty_like(x)
    V.v4_rope(x, pos, torch.from_numpy(f).cuda(), out, rope_begin=64, inverse=inverse, mscale=1.2772588,
              layout=V.V4_ROPE_HALF if half else V.V4_ROPE_INTERLEAVED)
    check(out, x, pos, f, 64, half, inverse, float(np.float32(1.2772588)))


def test_strided_views_in_place_and_head_major():
    g = torch.Generator().manual_seed(9)
    f = freqs(64)
    fd = torch.from_numpy(f).cuda()
    pos = torch.randint(0, 70000, (37,), generator=g, dtype=torch.int32).cuda()
    fused = torch.randn(37, 10, 192, generator=g).to(torch.bfloat16).cuda()
    before = fused.clone()
    out = torch.empty(37, 4, 128, dtype=torch.bfloat16, device="cuda")
    V.v4_rope(fused[:, 2:6, 64:], pos, fd, out)                       # a part of a fused buffer
    check(out, before[:, 2:6, 64:].contiguous(), pos, f, 64)
    V.v4_rope(fused[:, 2:6, 64:], pos, fd, fused[:, 2:6, 64:])        # the same part in place
    assert torch.equal(fused[:, 2:6, 64:], out)
    fused[:, 2:6, 64:] = before[:, 2:6, 64:]
    assert torch.equal(fused, before)
    hm = torch.empty(4, 37, 128, dtype=torch.bfloat16, device="cuda")  # heads outermost
    V.v4_rope(before[:, 2:6, 64:], pos, fd, hm.transpose(0, 1))
    assert torch.equal(hm.transpose(0, 1), out)
    one = before[:, 2:3, 64:].expand(37, 5, 128)                      # a broadcast head
    wide = torch.empty(37, 5, 128, dtype=torch.bfloat16, device="cuda")
    V.v4_rope(one, pos, fd, wide)
    assert all(torch.equal(wide[:, i], out[:, 0]) for i in range(5))
    V.v4_rope(before[:, 0:4, :128], pos, fd, before[:, 4:8, :128])     # two parts of one buffer, side by side
    check(before[:, 4:8, :128].contiguous(), before[:, 0:4, :128].contiguous(), pos, f, 64)


@pytest.mark.parametrize("order", ["rows", "heads"])
def test_strides_beyond_32_bits(order):
    """Rows, or heads, 2^30 elements apart: a tile of them does not fit 32-bit offsets."""
    f = freqs(16)
    x, pos = draw(4, 3, 64, torch.bfloat16, seed=9)
    shape, far = (4, 3, 64), 1 << 30
    stride = (far, 64, 1) if order == "rows" else (64, far, 1)
    big = torch.empty(5 * far, dtype=torch.bfloat16, device="cuda")
    src = big.as_strided(shape, stride)
    src.copy_(x)
    out = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
    V.v4_rope(src, pos, torch.from_numpy(f).cuda(), out)
    check(out, x, pos, f, 48)
    V.v4_rope(x, pos, torch.from_numpy(f).cuda(), src)
    check(src, x, pos, f, 48)
    V.v4_rope(src, pos, torch.from_numpy(f).cuda(), src, inverse=True)
    check(src, out, pos, f, 48, inverse=True)


def test_cache_write_beyond_32_bits():
    f = freqs(64)
    x, pos = draw(70, 1, 512, torch.bfloat16, seed=10)
    n = (1 << 23) + 200
    cache = torch.empty(n // 8, 8, 512, dtype=torch.bfloat16, device="cuda")
    slot = (torch.randperm(100)[:70] + (1 << 23) + 50).to(torch.int32).cuda()
    V.v4_cache_append(x[:, 0], pos, torch.from_numpy(f).cuda(), slot, cache)
    check(cache.view(-1, 512)[slot.long()][:, None], x, pos, f, 448)


@pytest.mark.parametrize("half", [False, True])
def test_gradient_is_the_inverse_call(half):
    """Against central differences of sum(dout * rope(x)) in fp32 (the map is linear: the difference quotient is exact up
    to rounding), and against the formula."""
    x, pos = draw(6, 2, 64, torch.float32, seed=11)
    f = freqs(32)
    fd = torch.from_numpy(f).cuda()
    lay = V.V4_ROPE_HALF if half else V.V4_ROPE_INTERLEAVED
    dout, _ = draw(6, 2, 64, torch.float32, seed=12)
    dx = torch.empty_like(x)
    V.v4_rope(dout, pos, fd, dx, layout=lay, inverse=True, mscale=1.25)
    check(dx, dout, pos, f, 32, half, True, 1.25)
    g = torch.Generator().manual_seed(13)
    for _ in range(8):
        d = torch.randn(x.shape, generator=g).cuda()
        hi, lo = torch.empty_like(x), torch.empty_like(x)
        V.v4_rope(x + d, pos, fd, hi, layout=lay, mscale=1.25)
        V.v4_rope(x - d, pos, fd, lo, layout=lay, mscale=1.25)
        lhs = float(((hi.double() - lo.double()) / 2 * dout.double()).sum())
        rhs = float((d.double() * dx.double()).sum())
        # 768 products of rotated values (each within 2^-21 of sums below 16) and of rounded x +- d (2^-24 of values below 8)
        assert abs(lhs - rhs) < 768 * 4 * (2 ** -21 * 16 + 2 ** -24 * 16)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,dim,R,page", [(1, 512, 64, 64), (77, 512, 64, 16), (300, 128, 64, 128), (5, 64, 16, 1)])
def test_cache_write(rows, dim, R, page, dt):
    x, pos = draw(rows, 1, dim, dt, seed=rows + 1)
    x = x[:, 0]
    f = freqs(R)
    fd = torch.from_numpy(f).cuda()
    pages = (2 * rows + page - 1) // page + 1
    g = torch.Generator().manual_seed(3)
    cache = torch.randn(pages, page, dim, generator=g).to(dt).cuda()
    before = cache.clone()
    slot = torch.randperm(pages * page, generator=g)[:rows].to(torch.int32)
    if rows > 4:
        slot[2] = -1
    V.v4_cache_append(x, pos, fd, slot.cuda(), cache)
    keep = np.ones(pages * page, bool)
    live = slot[slot >= 0].long()
    keep[live.numpy()] = False
    flat, old = cache.view(-1, dim), before.view(-1, dim)
    assert torch.equal(flat[torch.from_numpy(keep).cuda()], old[torch.from_numpy(keep).cuda()])
    sel = (slot >= 0).cuda()
    check(flat[live.cuda()][:, None], x[sel][:, None], pos[sel], f, dim - R)
    # rows that are rotated already
    V.v4_cache_append(x, None, None, slot.cuda(), cache)
    assert torch.equal(flat[live.cuda()], x[sel])
    assert V.v4_get_device_status() == 0


def test_cache_write_flags_and_skips_bad_slots():
    x, pos = draw(4, 1, 64, torch.bfloat16)
    fd = torch.from_numpy(freqs(16)).cuda()
    cache = torch.zeros(2, 4, 64, dtype=torch.bfloat16, device="cuda")
    slot = torch.tensor([8, -2, 3, 2 ** 31 - 1], dtype=torch.int32).cuda()
    V.v4_cache_append(x[:, 0], pos, fd, slot, cache)
    assert V.v4_get_device_status() == 6
    V.v4_reset_device_status()
    live = cache.view(8, 64).abs().sum(1) > 0
    assert live.tolist() == [i == 3 for i in range(8)]


def test_empty_calls_and_captured_replay():
    x, pos = draw(16, 4, 128, torch.bfloat16)
    fd = torch.from_numpy(freqs(64)).cuda()
    V.v4_rope(x[:0], pos[:0], fd, torch.empty_like(x[:0]))
    V.v4_cache_append(x[:0, 0], pos[:0], fd, pos[:0], torch.empty(1, 4, 128, dtype=torch.bfloat16, device="cuda"))
    out = torch.empty_like(x)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        V.v4_rope(x, pos, fd, out)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=s):
        V.v4_rope(x, pos, fd, out)
    x2, pos2 = draw(16, 4, 128, torch.bfloat16, seed=5)
    x.copy_(x2)
    pos.copy_(pos2)
    graph.replay()
    torch.cuda.synchronize()
    check(out, x2, pos2, freqs(64), 64)
