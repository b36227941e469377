"""4-bit projections against the float64 oracle: packing bit for bit, row counts
around the kernel's tiles, scale groups, the norm, slices of many rows."""
import numpy as np
import pytest
import torch

import sparse_compressed_attention_gb300 as V
from oracle import serving_oracle as S
from tests.helpers import np64, rel_l2

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def to_bf16(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(torch.bfloat16).float().numpy()


def operands(rows, G, K, N, gs, seed=0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, G, K, generator=g).to(torch.bfloat16).cuda()
    codes = torch.randint(0, 256, (G, N, K // 2), generator=g, dtype=torch.uint8).cuda()
    scales = (torch.rand(G, N, K // gs, generator=g) * 0.01 + 1e-4).to(torch.bfloat16).cuda()
    return x, codes, scales


def check(y, x, codes, scales, gs, norm_dim=0, eps=1e-6, norm_w=None):
    K = x.shape[2]
    ref, mag = S.w4_proj(np64(x), codes.cpu().numpy(), np64(scales), gs, norm_dim, eps,
                         None if norm_w is None else np64(norm_w))
    # one rounding to bf16, and fp32 sums of K products (and of the groups' scaled sums)
    allow = 2.0 ** -8 * np.abs(ref) + (K + 64) * U * mag * (1 + 2.0 ** -8) + 1e-30
    err = np.abs(np64(y) - ref)
    assert np.all(err <= allow), float((err - allow).max())
    assert rel_l2(np64(y), ref) < 2.0 ** -8


@pytest.mark.parametrize("rows", [1, 2, 7, 8, 9, 16, 17, 31, 32, 33, 64])
@pytest.mark.parametrize("G,K,N,gs", [(1, 128, 64, 32), (3, 384, 128, 128), (2, 1024, 192, 64), (1, 2176, 64, 32)])
def test_projection_matches_oracle(rows, G, K, N, gs):
    x, codes, scales = operands(rows, G, K, N, gs, seed=rows)
    y = torch.full((rows, G, N), float("nan"), dtype=torch.bfloat16, device="cuda")
    V.v4_w4_proj(x, codes, scales, y)
    check(y, x, codes, scales, gs)


@pytest.mark.parametrize("rows", [1, 5, 12, 20, 64])
@pytest.mark.parametrize("N,norm,weighted", [(64, 64, True), (512, 512, True), (1024, 512, False), (768, 256, True),
                                             (384, 128, False)])
def test_projection_with_norm(rows, N, norm, weighted):
    x, codes, scales = operands(rows, 2, 512, N, 64, seed=N + rows)
    w = (torch.rand(norm) + 0.5).cuda() if weighted else None
    y = torch.empty(rows, 2, N, dtype=torch.bfloat16, device="cuda")
    V.v4_w4_proj(x, codes, scales, y, norm_dim=norm, eps=1e-5, norm_w=w)
    check(y, x, codes, scales, 64, norm, 1e-5, w)


@pytest.mark.parametrize("rows,G,K,N,gs,norm", [
    (1, 1, 8192, 64, 128, 0), (8, 2, 4096, 192, 32, 0), (3, 1, 2048, 256, 64, 0),              # inputs split in 16 and 8
    (2, 1, 1024, 8192, 128, 512), (2, 1, 1024, 16384, 64, 128), (2, 1, 512, 4096, 32, 256),    # norms of wide and narrow blocks
    (24, 8, 512, 128, 32, 0), (40, 1, 1024, 256, 64, 0), (48, 1, 384, 1024, 128, 512)])        # three and six tiles of rows
def test_projection_at_every_split(rows, G, K, N, gs, norm):
    x, codes, scales = operands(rows, G, K, N, gs, seed=K + rows)
    y = torch.full((rows, G, N), float("nan"), dtype=torch.bfloat16, device="cuda")
    V.v4_w4_proj(x, codes, scales, y, norm_dim=norm)
    check(y, x, codes, scales, gs, norm)


@pytest.mark.parametrize("rows,K,N", [(1, 1024, 32768), (8, 512, 16384), (20, 1024, 8192)])
def test_norm_over_blocks_that_finish_apart(rows, K, N):
    """A norm's blocks exchange sums while others still stream their codes, some from a cold cache."""
    x, codes, scales = operands(rows, 1, K, N, 128, seed=rows)
    y = torch.empty(rows, 1, N, dtype=torch.bfloat16, device="cuda")
    V.v4_w4_proj(x, codes, scales, y, norm_dim=512)
    check(y, x, codes, scales, 128, 512)
    flush = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    again = torch.empty_like(y)
    for i in range(40):
        if i % 2:
            flush.fill_(i)
        V.v4_w4_proj(x, codes, scales, again, norm_dim=512)
        assert torch.equal(y, again), i


@pytest.mark.parametrize("rows", [65, 130])
def test_more_rows_than_a_slice(rows):
    x, codes, scales = operands(rows, 1, 256, 512, 128, seed=rows)
    for norm in (0, 512):
        y = torch.full((rows + 3, 1, 512), 7.0, dtype=torch.bfloat16, device="cuda")
        V.v4_w4_proj(x, codes, scales, y[:rows], norm_dim=norm)
        check(y[:rows], x, codes, scales, 128, norm)
        assert torch.all(y[rows:] == 7.0)


def test_zero_rows_scales_and_inputs():
    x, codes, scales = operands(4, 1, 256, 64, 32)
    y = torch.empty(4, 1, 64, dtype=torch.bfloat16, device="cuda")
    V.v4_w4_proj(x[:0], codes, scales, y[:0])
    scales.zero_()
    V.v4_w4_proj(x, codes, scales, y, norm_dim=64, eps=1e-6)
    assert torch.all(y == 0)
    # an infinite input row does not reach the other rows
    x, codes, scales = operands(9, 1, 256, 64, 32, seed=3)
    y0, y1 = (torch.empty(9, 1, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    V.v4_w4_proj(x, codes, scales, y0)
    x[3] = float("inf")
    V.v4_w4_proj(x, codes, scales, y1)
    keep = [i for i in range(9) if i != 3]
    assert torch.equal(y0[keep], y1[keep])


@pytest.mark.parametrize("G,K,N,gs", [(1, 128, 64, 32), (2, 384, 192, 64), (1, 256, 128, 128)])
def test_packing_is_the_definition(G, K, N, gs):
    g = torch.Generator().manual_seed(K)
    w = (torch.randn(G, K, N, generator=g) * 0.02).to(torch.bfloat16)
    w[0, :gs, 3] = 0.0                                  # a group of zeros
    w[0, gs - 1, 5] = 8.0                               # one large weight
    codes = torch.empty(G, N, K // 2, dtype=torch.uint8, device="cuda")
    scales = torch.empty(G, N, K // gs, dtype=torch.bfloat16, device="cuda")
    V.v4_w4_pack(w.cuda(), gs, codes, scales)
    rc, rs = S.w4_pack(np64(w), gs, to_bf16)
    assert np.array_equal(np64(scales), rs.astype(np.float64))
    assert np.array_equal(codes.cpu().numpy(), rc)
    back = S.w4_weights(rc, rs, gs).transpose(0, 2, 1)
    # half a code, and the scale's own rounding at the ends of the range
    step = np.repeat(rs.astype(np.float64), gs, axis=2).transpose(0, 2, 1)
    assert np.all(np.abs(back - np64(w)) <= step * (0.5 + 7 * 2.0 ** -8) + 1e-30)


def test_captured_replay():
    x, codes, scales = operands(3, 2, 512, 512, 64)
    y, ref = (torch.empty(3, 2, 512, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        V.v4_w4_proj(x, codes, scales, y, norm_dim=512)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        V.v4_w4_proj(x, codes, scales, y, norm_dim=512)
    x.mul_(-2)
    graph.replay()
    torch.cuda.synchronize()
    V.v4_w4_proj(x, codes, scales, ref, norm_dim=512)
    assert torch.equal(y, ref)
