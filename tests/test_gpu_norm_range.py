"""Norms at the ends of fp32's range: what the header says of heads whose sum of squares passes it."""
import numpy as np
import pytest
import torch

import sparse_compressed_attention_gb300 as V

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("dim", [8, 128, 512, 1024])
def test_both_sides_of_the_largest_sum_of_squares(dim, dt, half):
    """Heads 0 and 2 ordinary, head 1 all x with dim x^2 below or above 2^128.  Below, out is +-1 (square, mean, root and
    product: 8 U, one rounding); above, out, dx and the head's part of dw are zero, whatever the sum of w g x is."""
    pos, f = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.rand(8).cuda() if dim > 8 else None
    lay = V.V4_ROPE_HALF if half else V.V4_ROPE_INTERLEAVED
    ws = V.alloc_norm_rope_workspace(dim)
    top = (2.0 ** 128 / dim) ** 0.5
    g = torch.Generator().manual_seed(dim)
    base = torch.randn(1, 3, dim, generator=g)
    grad = torch.randn(1, 3, dim, generator=g)
    for x1, dy1, over in ((0.98 * top, 1.0, False), (1.02 * top, 1.0, True), (1.02 * top, 1e19, True), (1e30, 1e8, True),
                          (1e38, 1.0, True)):
        x, dy = base.clone(), grad.clone()
        x[:, 1], dy[:, 1] = x1, dy1
        x[:, 1, ::2] *= -1
        dy[:, 1, ::2] *= -1
        x, dy = x.to(dt).cuda(), dy.to(dt).cuda()
        out, dx, dw = torch.empty_like(x), torch.empty_like(x), torch.empty(dim, device="cuda")
        V.v4_norm_rope_fwd(x, None, pos, f, out, eps=1e-6, layout=lay)
        V.v4_norm_rope_bwd(x, None, dy, None, pos, f, dx, dq_w=dw, eps=1e-6, layout=lay, workspace=ws)
        two, dwant = x[:, [0, 2]].contiguous(), torch.empty(dim, device="cuda")
        o2, d2 = torch.empty_like(two), torch.empty_like(two)
        V.v4_norm_rope_fwd(two, None, pos, f, o2, eps=1e-6, layout=lay)
        V.v4_norm_rope_bwd(two, None, dy[:, [0, 2]].contiguous(), None, pos, f, d2, dq_w=dwant, eps=1e-6, layout=lay, workspace=ws)
        assert torch.equal(out[:, [0, 2]], o2) and torch.equal(dx[:, [0, 2]], d2)
        if over:
            assert (out[:, 1] == 0).all() and (dx[:, 1] == 0).all()
            # two terms in another order of partial sums
            assert ((dw - dwant).abs() <= 4 * U * (dwant.abs() + 40)).all()
        else:
            assert ((out[:, 1].float().abs() - 1).abs() <= 2.0 ** -8 + 8 * U if dt == torch.bfloat16 else
                    (out[:, 1].float().abs() - 1).abs() <= 8 * U).all()
            assert torch.isfinite(dx[:, 1].float()).all() and torch.isfinite(dw).all()


def test_sums_of_products_that_pass_the_range_stay_in_their_head():
    """A head whose sum of w g x overflows while its squares do not: dx of that head is not finite, the others' are untouched."""
    x = torch.randn(1, 3, 64, generator=torch.Generator().manual_seed(1)).cuda()
    dy = torch.randn(1, 3, 64, generator=torch.Generator().manual_seed(2)).cuda()
    pos, f, ws = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.rand(8).cuda(), V.alloc_norm_rope_workspace(64)
    want, dx = torch.empty_like(x), torch.empty_like(x)
    V.v4_norm_rope_bwd(x, None, dy, None, pos, f, want, workspace=ws)
    x[:, 1], dy[:, 1] = 1e18, 1e21
    V.v4_norm_rope_bwd(x, None, dy, None, pos, f, dx, workspace=ws)
    assert torch.equal(dx[:, [0, 2]], want[:, [0, 2]])
    assert not torch.isfinite(dx[:, 1]).any()
