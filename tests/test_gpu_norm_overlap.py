"""Norms whose weights lie between the rows of an output: not refused, and right."""
import pytest
import torch

import sparse_compressed_attention_gb300 as V

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("heads_outer", [False, True])
def test_weights_between_an_outputs_rows(heads_outer):
    g = torch.Generator().manual_seed(1)
    x = torch.randn(5, 2, 64, generator=g).cuda()
    buf = torch.zeros(10, 256, device="cuda")
    out = buf[:, :64].view(2, 5, 64).transpose(0, 1) if heads_outer else buf[:5, :128].view(5, 2, 64)
    w, pos, f = buf[1, 128:192], buf.view(torch.int32)[2, 192:197], buf[3, 200:208]
    w.copy_(torch.rand(64, generator=g)), pos.copy_(torch.arange(5, dtype=torch.int32)), f.copy_(torch.rand(8, generator=g))
    want = torch.empty_like(x)
    V.v4_norm_rope_fwd(x, None, pos.clone(), f.clone(), want, q_w=w.clone())
    kept = w.clone()
    V.v4_norm_rope_fwd(x, None, pos, f, out, q_w=w)
    assert torch.equal(out, want) and torch.equal(w, kept)
    with pytest.raises(V.V4Error, match="weights, positions"):
        V.v4_norm_rope_fwd(x, None, pos, f, out, q_w=out[2, 1])
