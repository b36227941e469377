"""Seeded 4-bit caches for the tree attention's tests: tree_cases.Case with its caches quantised."""
import numpy as np
import torch

import sparse_compressed_attention_gb300 as V
from oracle import cache_oracle as CO
from tests.helpers import np64
from tests.tree_cases import Case


def fast_pack(x):
    """cache_oracle.q4_pack for normal values in float64 (quotients that close to a tie do not occur in it)."""
    n, dim = x.shape
    g = x.reshape(n, dim // 16, 16)
    want = np.maximum(np.abs(g).max(-1) / 7.0, 2.0 ** -20)
    e = np.floor(np.log2(want))
    m = np.rint(want * 2.0 ** (3 - e))
    byte = np.clip(8 * (e + 20) + m - 8, 0, 255).astype(np.int64)
    scale = 2.0 ** (byte // 8 - 20) * (1 + (byte % 8) / 8.0)
    code = (np.clip(np.rint(g / scale[..., None]), -8, 7) + 8).astype(np.int64).reshape(n, dim // 8, 8)[..., list(CO.NIBBLE)]
    out = np.zeros((n, CO.q4_row_bytes(dim)), np.uint8)
    out[:, :dim // 2] = (code[..., 0::2] | (code[..., 1::2] << 4)).reshape(n, dim // 2)
    out[:, dim // 2:dim // 2 + dim // 16] = byte
    return out


class Q4Case(Case):
    """rows that nothing may read hold the largest code and scale."""

    def __init__(self, *a, **kw):
        super().__init__(*a, fill=float("nan"), **kw)
        self.tok_rows, self.tok = self.quantised(self.tok)
        if self.ratio:
            self.ent_rows, self.ent = self.quantised(self.ent)

    def quantised(self, t):
        flat = np64(t).reshape(-1, self.D)
        unread = np.isnan(flat).any(1)
        rows = fast_pack(np.where(unread[:, None], 0.0, flat))
        values = CO.q4_unpack(rows, self.D)
        rows[unread] = 255
        return (torch.from_numpy(rows).view(t.shape[0], t.shape[1], -1),
                torch.from_numpy(np.ascontiguousarray(values)).to(self.dt).view(t.shape))

    def device_inputs(self):
        x = super().device_inputs()
        x["tok_cache"] = self.tok_rows.cuda()
        if self.ratio:
            x["ent_cache"] = self.ent_rows.cuda()
        return x

    def dense_inputs(self):
        x = super().device_inputs()
        return x

    def run(self, x=None, mark=3.0):
        x = x or self.device_inputs()
        o = torch.full((self.n, self.H, self.D), mark, dtype=self.dt, device="cuda")
        lse = torch.full((self.n, self.H), mark, device="cuda")
        ws = V.alloc_tree_workspace(self.cfg, self.n)
        ws.fill_(255)
        V.v4_tree_mqa_fwd_q4(self.cfg, x, o, lse, ws)
        torch.cuda.synchronize()
        return o, lse
