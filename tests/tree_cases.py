"""Seeded paged caches, drafted trees and the derived error bounds of the tree attention's tests."""
import numpy as np
import torch

import sparse_compressed_attention_gb300 as V
from oracle import serving_oracle as S
from oracle import v4_oracle as O
from tests.helpers import np64

U = 2.0 ** -24


def random_parents(rng, n):
    return [-1 if i == 0 or rng.random() < 0.15 else int(rng.integers(max(-1, i - 4), i)) for i in range(n)]


class Case:
    """Inputs of one call (device tensors) and its oracle."""

    def __init__(self, lens, nodes, H=64, D=512, R=64, window=128, ratio=0, K=0, tok_page=64, ent_page=32, dt=torch.bfloat16,
                 sink=False, pad=(0, 0), parents=None, seed=0, q_scale=1.0, path=0, holes=True, fill=0.0, pool=0):
        rng = np.random.default_rng(seed)
        g = torch.Generator().manual_seed(seed)
        B = len(lens)
        self.H, self.D, self.R, self.window, self.ratio, self.K = H, D, R, window, ratio, K
        self.lens, self.nodes = lens, nodes
        begin = np.concatenate([[0], np.cumsum(nodes)]) + pad[0]
        n = int(begin[-1]) + pad[1]
        if parents is None:
            parents = [random_parents(rng, m) for m in nodes]
        par = np.full(n, -7, np.int32)                 # padding rows hold nonsense
        for b in range(B):
            par[begin[b]:begin[b + 1]] = parents[b]
        self.begin, self.parent, self.n = begin, par, n
        self.plan_ref, self.pos_ref = S.tree_plan(begin, lens, par, n)
        f = O.make_inv_freq(40000.0, R, 16.0, 4096, 32.0, 1.0) if R else np.zeros(0, np.float32)
        self.f = f

        # paged caches; pages and rows that nothing may read hold `fill` (the tests put NaN there)
        def cache(counts, page, lo):
            blocks = max(1, max((c + page - 1) // page for c in counts))
            table = np.full((B, blocks), -1, np.int32)
            used = [(b, k) for b in range(B) for k in range(lo[b] // page, (counts[b] + page - 1) // page)]
            pages = max(len(used) + 3, pool)
            perm = rng.permutation(pages)
            for i, (b, k) in enumerate(used):
                table[b, k] = perm[i]
            data = torch.full((pages, page, D), fill, dtype=dt)
            for b, k in used:
                first, last = max(lo[b], k * page), min(counts[b], (k + 1) * page)
                data[table[b, k], first - k * page:last - k * page] = torch.randn(last - first, D, generator=g).to(dt)
            return data, table

        counts = [l + m for l, m in zip(lens, nodes)]
        lo = [0 if window < 0 else max(0, l - window + 1) if window else c for l, c in zip(lens, counts)]
        self.tok, self.tok_table = cache(counts, tok_page, lo)
        self.tok_page, self.ent_page = tok_page, ent_page
        if ratio:
            self.ent_counts = [l // ratio for l in lens]
            self.ent, self.ent_table = cache(self.ent_counts, ent_page, [0] * B)
        self.q = (torch.randn(n, H, D, generator=g) * q_scale).to(dt)
        self.sink = torch.randn(H, generator=g) if sink else None
        self.idx = None
        if K:
            idx = np.full((n, K), -1, np.int64)
            for row in range(n):
                if self.plan_ref[row, 0] < 0:
                    idx[row] = 10 ** 6                 # padding rows hold nonsense
                    continue
                nv = min((int(self.plan_ref[row, 2]) + 1) // ratio, self.ent_counts[self.plan_ref[row, 0]])
                take = rng.permutation(nv)[:K]
                at = rng.permutation(K)[:len(take)] if holes else np.arange(len(take))
                idx[row, at] = take
            self.idx = torch.from_numpy(idx.astype(np.int32))
        self.dt = dt
        self.cfg = V.make_config(B, 1, H, D, R, ratio=ratio, window=window, topk=K,
                                 dtype="bf16" if dt == torch.bfloat16 else "f32", path=path)
        self.scale = D ** -0.5

    def device_inputs(self):
        i32 = torch.int32
        self.plan = torch.empty(self.n, 8, dtype=i32, device="cuda")
        self.pos = torch.empty(self.n, dtype=i32, device="cuda")
        self.slot = torch.empty(self.n, dtype=i32, device="cuda")
        V.v4_tree_plan(torch.from_numpy(self.begin.astype(np.int32)).cuda(), torch.tensor(self.lens, dtype=i32).cuda(),
                       torch.from_numpy(self.parent).cuda(), self.plan, pos=self.pos, slot=self.slot,
                       block_table=torch.from_numpy(self.tok_table).cuda(), page_size=self.tok_page,
                       n_slots=self.tok.shape[0] * self.tok_page)
        x = dict(q=self.q.cuda(), plan=self.plan, tok_cache=self.tok.cuda(), tok_table=torch.from_numpy(self.tok_table).cuda())
        if self.ratio:
            x.update(ent_cache=self.ent.cuda(), ent_table=torch.from_numpy(self.ent_table).cuda(),
                     ent_len=torch.tensor(self.ent_counts, dtype=i32).cuda())
        if self.K:
            x["idx"] = self.idx.cuda()
        if self.sink is not None:
            x["sink"] = self.sink.cuda()
        if self.R:
            x["inv_freq"] = torch.from_numpy(self.f).cuda()
        return x

    def run(self, x=None, mark=3.0):
        x = x or self.device_inputs()
        o = torch.full((self.n, self.H, self.D), mark, dtype=self.dt, device="cuda")
        lse = torch.full((self.n, self.H), mark, device="cuda")
        ws = V.alloc_tree_workspace(self.cfg, self.n)
        ws.fill_(255)                                  # NaN wherever a float is read before it is written
        V.v4_tree_mqa_fwd(self.cfg, x, o, lse, ws)
        torch.cuda.synchronize()
        return o, lse

    def oracle(self, mark=3.0):
        tok, D = np64(self.tok).reshape(-1, self.D), self.D
        ent = np64(self.ent).reshape(-1, D) if self.ratio else None

        def tok_rows(b, u):
            return tok[int(self.tok_table[b, u // self.tok_page]) * self.tok_page + u % self.tok_page]

        def ent_rows(b, s):
            if s is None:
                return self.ent_counts[b]
            return ent[int(self.ent_table[b, s // self.ent_page]) * self.ent_page + s % self.ent_page]

        return S.tree_mqa(np64(self.q), self.plan_ref, tok_rows, ent_rows if self.ratio else None,
                          None if self.idx is None else self.idx.numpy(), None if self.sink is None else np64(self.sink),
                          self.f, self.ratio, self.window, self.K, self.scale,
                          np.full((self.n, self.H, D), mark), np.full((self.n, self.H), mark))

    def check(self, o, lse, ref=None):
        """Every element within the kernel's roundings.

        Logits: fp32 sums of D + R products (the rotated part of q enters as two bf16 terms, leaving 2^-17 of it) and
        the exponent's argument; e bounds their error.  Probabilities are rounded to bf16 (2^-8) on the tensor-core
        path, sums over keys are fp32; the output is rounded once."""
        ro, rl, mass, dots = ref or self.oracle()
        b16 = self.dt == torch.bfloat16
        fin = np.where(np.isfinite(rl), np.abs(rl), 0.0)
        e = self.scale * dots * ((self.D + 70) * U + (2.0 ** -17 if b16 else 0.0)) + 16 * U * (fin + 40.0)
        keys = 256 + 16 * np.log2(2.0 + max(self.lens))    # fp32 sums run over at most 128-key tiles, then over tiles
        p_err = (2.0 ** -8 if b16 else 0.0) + 2 * e[..., None] + keys * U
        allow = (2.0 ** -8 if b16 else U) * np.abs(ro) * (1 + 2.0 ** -8) + p_err * mass * 1.01 + 1e-30
        go, gl = np64(o), np64(lse)
        live = self.plan_ref[:, 0] >= 0
        assert np.array_equal(go[~live], ro[~live]) and np.array_equal(gl[~live], rl[~live])
        bad = np.abs(go[live] - ro[live]) > allow[live]
        assert not bad.any(), (int(bad.sum()), float((np.abs(go - ro) - allow)[live].max()))
        inf = ~np.isfinite(rl)
        assert np.array_equal(gl[inf], rl[inf])
        d = np.abs(gl - rl)[~inf & live[:, None]]
        lim = (e + keys * U + 4 * U * fin)[~inf & live[:, None]]
        assert np.all(d <= lim), float((d - lim).max())
        assert V.v4_get_device_status() == 0
