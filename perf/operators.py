"""Workloads of the serving operators: rotary positions and the paged cache they
fill, attention of drafted token trees over that cache, and the projections of
single tokens with 4-bit weights.

``listed()`` names the fixed cases, ``draw(rng)`` makes more of the same ranges,
``prepare(case, seed)`` makes one case's inputs on the GPU and ``run(state)`` is
one pass: through the framework's entry points where ``own`` is true, in
elementary torch operations in 32 bits (angles in 64) where it is false.
``exact(case, seed)`` evaluates the definitions in 64 bits.
"""
from __future__ import annotations

import math
import random

import numpy as np
import torch

own = False

YARN_LEN = 4096          # original context of the scaled frequency table


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # one decode step of a small batch: the query heads of 16 tokens, latency only
        dict(name="rope_step", op="rope", rows=16, heads=64, dim=512, R=64, begin=448, half=False, inverse=False,
             far=1000000, dtype="bf16", fused=0),
        # queries of a 4096-token prefill chunk, last 64 of 512 dims, scaled for long contexts
        dict(name="rope_chunk", op="rope", rows=4096, heads=64, dim=512, R=64, begin=448, half=False, inverse=False,
             far=65536, dtype="bf16", fused=0),
        # gradient of the half layout over whole 128-wide heads, read out of a wider fused buffer, fp32
        dict(name="rope_grad_half", op="rope", rows=5003, heads=64, dim=128, R=128, begin=0, half=True, inverse=True,
             far=131072, dtype="f32", fused=64),
        # the latent rows of a decode step of 64 sequences go into their pages
        dict(name="append_step", op="append", rows=64, D=512, R=64, far=131072, page=64, dtype="bf16"),
        # the latent rows of a 16384-token prompt go into shuffled pages
        dict(name="append_prompt", op="append", rows=16384, D=512, R=64, far=0, page=64, dtype="bf16"),
        # one token of one sequence: 512 selected entries and the 128-token window
        dict(name="tree_one_token", op="tree", B=1, T=1, length=16384, H=64, W=128, ratio=4, K=512, page=64,
             sink=False, ragged=False, pad=0, shape=1),
        # speculative decoding of 32 ragged sequences, up to 8 drafted tokens each, selected entries, padded batch
        dict(name="tree_selected", op="tree", B=32, T=8, length=65536, H=64, W=128, ratio=4, K=512, page=64,
             sink=True, ragged=True, pad=8, shape=2),
        # drafted trees over every entry of million-token contexts (ratio 128), plus the window
        dict(name="tree_entries_1m", op="tree", B=8, T=8, length=1000003, H=64, W=128, ratio=128, K=0, page=64,
             sink=False, ragged=False, pad=0, shape=3),
        # single tokens of 16 sequences over their whole token caches, ragged lengths
        dict(name="tree_all_tokens", op="tree", B=16, T=1, length=49152, H=64, W=-1, ratio=0, K=0, page=32,
             sink=False, ragged=True, pad=0, shape=4),
        # trees of 16 drafted tokens over whole token caches: the largest
        dict(name="tree_all_tokens_16", op="tree", B=4, T=16, length=32768, H=64, W=-1, ratio=0, K=0, page=64,
             sink=False, ragged=False, pad=0, shape=5),
        # query projection of one token from the rank-1024 latent, per-head RMSNorm
        dict(name="w4_q_one", op="w4", rows=1, groups=1, K=1024, N=32768, gs=128, norm=512),
        # grouped output projection of 24 drafted tokens, finer scales
        dict(name="w4_o_24", op="w4", rows=24, groups=8, K=4096, N=1024, gs=32, norm=0),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "append", "tree", "tree", "tree", "w4", "w4"])
    if op == "rope":
        dim = rng.choice([64, 128, 256, 512])
        half = rng.random() < 0.5
        R = dim if rng.random() < 0.3 else rng.choice([32, 64])
        begin = rng.choice([0, dim - R])
        heads = rng.choice([1, 2, 7, 16, 64])
        rows = _log(rng, 1, max(2, 4096 * 64 * 512 // (heads * dim * 2)))
        return dict(op=op, rows=min(rows, 100000), heads=heads, dim=dim, R=R, begin=begin, half=half,
                    inverse=rng.random() < 0.5, far=rng.choice([4096, 65536, 1000000]),
                    dtype=rng.choice(["bf16", "f32"]), fused=rng.choice([0, 0, 64]))
    if op == "append":
        return dict(op=op, rows=_log(rng, 1, 16384), D=rng.choice([128, 512]), R=64, far=_log(rng, 1000, 1000000),
                    page=rng.choice([16, 32, 64, 128]), dtype=rng.choice(["bf16", "f32"]))
    if op == "w4":
        if rng.random() < 0.5:
            return dict(op=op, rows=_log(rng, 1, 64), groups=1, K=rng.choice([512, 1024, 1536]), N=512 * rng.randint(8, 64),
                        gs=rng.choice([32, 64, 128]), norm=rng.choice([0, 512]))
        return dict(op=op, rows=_log(rng, 1, 64), groups=rng.choice([1, 4, 8]), K=128 * rng.randint(4, 32),
                    N=64 * rng.randint(4, 16), gs=rng.choice([32, 64, 128]), norm=0)
    kind = rng.choice(["selected", "entries", "tokens"])
    H = rng.choice([64, 64, 128])
    if kind == "selected":
        return dict(op=op, B=_log(rng, 1, 32), T=rng.randint(1, 8), length=_log(rng, 100, 100000), H=H, W=128, ratio=4,
                    K=rng.choice([512, 1024]), page=rng.choice([16, 64, 128]), sink=rng.random() < 0.5,
                    ragged=rng.random() < 0.5, pad=rng.choice([0, 3]), shape=rng.randint(10, 1000000))
    if kind == "entries":
        return dict(op=op, B=_log(rng, 1, 8), T=rng.randint(1, 8), length=_log(rng, 1000, 1000000), H=H,
                    W=rng.choice([16, 100, 128]), ratio=128, K=0, page=rng.choice([16, 64, 128]),
                    sink=rng.random() < 0.5, ragged=rng.random() < 0.5, pad=rng.choice([0, 3]),
                    shape=rng.randint(10, 1000000))
    B = _log(rng, 1, 8)
    return dict(op=op, B=B, T=rng.randint(1, 8), length=_log(rng, 50, 200000 // B), H=64, W=-1, ratio=0, K=0,
                page=rng.choice([16, 64, 128]), sink=rng.random() < 0.5, ragged=rng.random() < 0.5,
                pad=rng.choice([0, 3]), shape=rng.randint(10, 1000000))


def _shape(case):
    """Committed length and node count of each sequence, the nodes' parents and depths."""
    r = random.Random(case["shape"])
    B, T, L = case["B"], case["T"], case["length"]
    lens = [max(1, int(L * (0.15 + 0.85 * r.random()))) if case["ragged"] else L for _ in range(B)]
    nodes = [r.randint(1, T) if case["ragged"] else T for _ in range(B)]
    parents, depths = [], []
    for n in nodes:
        par, dep = [], []
        for i in range(n):
            # mostly deep trees: a node hangs below one of the last three, sometimes below the prefix
            p = -1 if i == 0 or r.random() < 0.1 else max(-1, i - 1 - r.randint(0, 2))
            par.append(p)
            dep.append(0 if p < 0 else dep[p] + 1)
        parents.append(par)
        depths.append(dep)
    return lens, nodes, parents, depths


def work(case):
    op = case["op"]
    if op == "rope":
        es = 2 if case["dtype"] == "bf16" else 4
        n = case["rows"] * case["heads"]
        return {"bytes": 2.0 * n * case["dim"] * es + 4.0 * case["rows"], "flops": 3.0 * n * case["R"]}
    if op == "append":
        es = 2 if case["dtype"] == "bf16" else 4
        return {"bytes": 2.0 * case["rows"] * case["D"] * es + 8.0 * case["rows"], "flops": 3.0 * case["rows"] * case["R"]}
    if op == "w4":
        w = case["groups"] * case["N"] * case["K"]
        io = case["rows"] * case["groups"] * (case["K"] + case["N"]) * 2
        return {"bytes": w * (0.5 + 2.0 / case["gs"]) + io, "flops": 2.0 * case["rows"] * w}
    lens, nodes, _, depths = _shape(case)
    H, D, W, r, K = case["H"], 512, case["W"], case["ratio"], case["K"]
    rows_read = pairs = 0
    for L, n, dep in zip(lens, nodes, depths):
        ne = L // r if r else 0
        rows_read += (min(ne, n * K) if K else ne) + n + (L if W < 0 else min(L, W - 1))
        for d in dep:
            nv = min((L + d + 1) // r, ne) if r else 0
            pairs += (min(K, nv) if K else nv) + (L + d + 1 if W < 0 else min(L + d + 1, W))
    n = sum(nodes)
    return {"bytes": rows_read * D * 2.0 + n * H * (2 * D * 2.0 + 4) + n * K * 4.0, "flops": 4.0 * H * D * pairs}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _freqs(R, theta=40000.0, factor=16.0):
    """YaRN-scaled inverse frequencies (ramp 1..32 over the original length), as the compressed layers use."""
    j = torch.arange(R // 2, dtype=torch.float64)
    f = theta ** (-2.0 * j / R)
    turns = YARN_LEN * f / (2.0 * math.pi)
    g = ((turns - 1.0) / 31.0).clamp(0.0, 1.0)
    return ((1.0 - g) * f / factor + g * f).to(torch.float32).cuda()


def _type(case):
    return torch.bfloat16 if case.get("dtype", "bf16") == "bf16" else torch.float32


def _unit_rms(x):
    return x / x.square().mean(-1, keepdim=True).sqrt()


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rng = np.random.RandomState(seed % (1 << 31))
    op, dt = case["op"], _type(case)
    s = dict(case)
    if op == "rope":
        wide = case["dim"] + case["fused"]
        base = torch.randn(case["rows"], case["heads"], wide, generator=g, device="cuda", dtype=torch.float32).to(dt)
        s["x"] = base[..., case["fused"]:]
        first = int(rng.randint(0, case["far"]))
        s["pos"] = (torch.arange(case["rows"], device="cuda", dtype=torch.int32) + first
                    if case["rows"] > 512 else
                    torch.from_numpy(rng.randint(0, case["far"], case["rows"]).astype(np.int32)).cuda())
        s["inv_freq"] = _freqs(case["R"])
        s["mscale"] = 1.0 if case["dtype"] == "bf16" else 0.1 * math.log(16.0) + 1.0
        s["out"] = torch.empty(case["rows"], case["heads"], case["dim"], device="cuda", dtype=dt)
        return s
    if op == "append":
        n, D, page = case["rows"], case["D"], case["page"]
        s["x"] = _unit_rms(torch.randn(n, D, generator=g, device="cuda")).to(dt)
        if case["far"]:          # a decode step: one row for each sequence, far apart
            pages = 2 * n + 8
            s["pos"] = torch.from_numpy(rng.randint(0, case["far"], n).astype(np.int32)).cuda()
            s["slot"] = torch.from_numpy((rng.permutation(pages)[:n] * page + rng.randint(0, page, n)).astype(np.int32)).cuda()
        else:                    # a prompt: consecutive tokens fill one page after another
            pages = (n + page - 1) // page + 8
            perm = rng.permutation(pages)
            u = np.arange(n)
            s["pos"] = torch.arange(n, device="cuda", dtype=torch.int32)
            s["slot"] = torch.from_numpy((perm[u // page] * page + u % page).astype(np.int32)).cuda()
        s["inv_freq"] = _freqs(case["R"])
        s["cache"] = torch.zeros(pages, page, D, device="cuda", dtype=dt)
        return s
    if op == "w4":
        G, K, N, gs = case["groups"], case["K"], case["N"], case["gs"]
        s["x"] = _unit_rms(torch.randn(case["rows"], G, K, generator=g, device="cuda")).to(torch.bfloat16)
        # codes 0..15 (value code - 8) of a quantised normal weight, two to a byte in the library's order
        s["codes"] = torch.randint(0, 256, (G, N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
        s["scales"] = (0.004 * (0.5 + torch.rand(G, N, K // gs, generator=g, device="cuda"))).to(torch.bfloat16)
        s["norm_w"] = 1.0 + 0.1 * torch.randn(max(case["norm"], 8), generator=g, device="cuda")
        s["y"] = torch.empty(case["rows"], G, N, device="cuda", dtype=torch.bfloat16)
        return s
    lens, nodes, parents, depths = _shape(case)
    B, H, W, r, K, page, D = case["B"], case["H"], case["W"], case["ratio"], case["K"], case["page"], 512
    n, total = sum(nodes), sum(nodes) + case["pad"]
    plan = np.zeros((total, 8), np.int64)
    plan[:, 0] = -1
    row = 0
    for b in range(B):
        masks = []
        for i in range(nodes[b]):
            m = (1 << i) | (masks[parents[b][i]] if parents[b][i] >= 0 else 0)
            masks.append(m)
            plan[row] = [b, i, lens[b] + depths[b][i], lens[b]] + [(m >> (32 * w)) & 0xFFFFFFFF for w in range(4)]
            row += 1
    s["plan"] = torch.from_numpy(plan.astype(np.uint32).view(np.int32)).cuda()
    # token pages: the blocks that some query of the sequence can see; older ones were given back
    blocks = max((lens[b] + nodes[b] - 1) // page + 1 for b in range(B))
    table = np.full((B, blocks), -1, np.int32)
    at = []
    for b in range(B):
        lo = 0 if W < 0 else max(0, lens[b] - W + 1) // page
        at += [(b, k) for k in range(lo, (lens[b] + nodes[b] - 1) // page + 1)]
    at = np.array(at)
    table[at[:, 0], at[:, 1]] = rng.permutation(len(at))
    s["tok_table"] = torch.from_numpy(table).cuda()
    s["tok_cache"] = torch.randn(len(at), page, D, generator=g, device="cuda", dtype=torch.bfloat16)
    s["q"] = torch.randn(total, H, D, generator=g, device="cuda", dtype=torch.bfloat16)
    s["sinks"] = torch.randn(H, generator=g, device="cuda") if case["sink"] else None
    s["inv_freq"] = _freqs(64)
    s["ent_cache"] = s["ent_table"] = s["ent_len"] = s["idx"] = None
    if r:
        ne = [L // r for L in lens]
        eb = max(1, max((e + page - 1) // page for e in ne))
        pages = B * eb
        s["ent_table"] = torch.from_numpy(rng.permutation(pages).reshape(B, eb).astype(np.int32)).cuda()
        s["ent_cache"] = torch.randn(pages, page, D, generator=g, device="cuda", dtype=torch.bfloat16)
        s["ent_len"] = torch.tensor(ne, dtype=torch.int32, device="cuda")
        s["max_ent"] = max(ne)
        if K:
            # K distinct visible entries of each row in ascending order, -1 behind them
            seq, pos = s["plan"][:, 0].long(), s["plan"][:, 2]
            nv = torch.minimum((pos + 1) // r, s["ent_len"][seq.clamp(min=0)])
            keys = torch.rand(total, max(K, max(ne)), generator=g, device="cuda")
            keys[torch.arange(keys.shape[1], device="cuda")[None, :] >= nv[:, None]] = -1.0
            v, i = keys.topk(K, dim=1)
            i = torch.where(v >= 0, i, 1 << 30).sort(dim=1).values
            s["idx"] = torch.where(i == 1 << 30, -1, i).to(torch.int32).contiguous()
    # which rows belong to each sequence, for forms that treat a sequence at once
    at = np.zeros((B, max(nodes)), np.int64)
    of = np.zeros(total, np.int64)
    row = 0
    for b in range(B):
        at[b] = np.minimum(row + np.arange(max(nodes)), row + nodes[b] - 1)
        of[row:row + nodes[b]] = b * max(nodes) + np.arange(nodes[b])
        row += nodes[b]
    s["rows_of"], s["row_at"] = torch.from_numpy(at).cuda(), torch.from_numpy(of).cuda()
    s["max_len"], s["max_nodes"] = max(lens), max(nodes)
    s["o"] = torch.zeros(total, H, D, device="cuda", dtype=torch.bfloat16)
    s["lse"] = torch.zeros(total, H, device="cuda")
    s["scratch"] = {}
    return s


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------
def _angles(pos, inv_freq, sign=1.0):
    a = pos.double()[:, None] * inv_freq.double()[None, :]
    return torch.cos(a).float(), (sign * torch.sin(a)).float()


def _rotated(x, c, sn, begin, R, half, mscale=1.0):
    """x [rows, heads, dim] fp32 with dims [begin, begin + R) rotated."""
    part = x[..., begin:begin + R]
    c, sn = c[:, None, :] * mscale, sn[:, None, :] * mscale
    if half:
        a, b = part[..., :R // 2], part[..., R // 2:]
        new = torch.cat([a * c - b * sn, a * sn + b * c], -1)
    else:
        a, b = part[..., 0::2], part[..., 1::2]
        new = torch.stack([a * c - b * sn, a * sn + b * c], -1).flatten(-2)
    return torch.cat([x[..., :begin], new, x[..., begin + R:]], -1)


def _plain_rope(s):
    c, sn = _angles(s["pos"], s["inv_freq"], -1.0 if s["inverse"] else 1.0)
    s["out"].copy_(_rotated(s["x"].float(), c, sn, s["begin"], s["R"], s["half"], s["mscale"]))
    return s["out"]


def _plain_append(s):
    c, sn = _angles(s["pos"], s["inv_freq"])
    y = _rotated(s["x"].float()[:, None], c, sn, s["D"] - s["R"], s["R"], False)[:, 0]
    s["cache"].view(-1, s["D"])[s["slot"].long()] = y.to(s["cache"].dtype)
    return s["cache"]


def _plain_weights(codes, scales, gs):
    """Codes in the library's order (64-byte blocks of 128 inputs: word 4 t + c holds inputs 32 c + 8 t ..,
    its nibbles in the order 0, 2, 4, 6, 1, 3, 5, 7) as fp32 weights [groups, N, K]."""
    G, N, half = codes.shape
    nib = torch.stack([codes & 15, codes >> 4], -1).view(G, N, half // 64, 4, 4, 2, 4)     # block, t, c, odd, pair
    k = nib.permute(0, 1, 2, 4, 3, 6, 5).reshape(G, N, 2 * half)                           # block, c, t, pair, odd
    w = (k.float() - 8.0).view(G, N, -1, gs) * scales.float()[..., None]
    return w.view(G, N, 2 * half)


def _plain_w4(s):
    w = _plain_weights(s["codes"], s["scales"], s["gs"])
    y = torch.matmul(s["x"].float().transpose(0, 1), w.transpose(1, 2)).transpose(0, 1)
    if s["norm"]:
        h = y.reshape(y.shape[0], y.shape[1], -1, s["norm"])
        y = (h * torch.rsqrt(h.square().mean(-1, keepdim=True) + 1e-6) * s["norm_w"]).reshape(y.shape)
    s["y"].copy_(y)
    return s["y"]


def _paged(cache, table, seq, at, ok):
    """Rows `at` (logical) of the sequences `seq` through their page table, fp32; zeros where not ok."""
    page = cache.shape[1]
    at = torch.where(ok, at, 0)
    slot = table[seq, at // page].long() * page + at % page
    rows = cache.view(-1, cache.shape[2])[torch.where(ok, slot, 0)].float()
    return torch.where(ok[..., None], rows, 0.0)


def _plain_tree(s):
    plan, W, r, dev = s["plan"], s["W"], s["ratio"], s["q"].device
    live = plan[:, 0] >= 0
    seq, pos, base = plan[:, 0].clamp(min=0).long(), plan[:, 2].long(), plan[:, 3].long()
    n, H, D = s["q"].shape
    scale = D ** -0.5
    c, sn = _angles(pos, s["inv_freq"])
    q = _rotated(s["q"].float(), c, sn, D - 64, 64, False) * scale
    T = s["max_nodes"]
    j = torch.arange(T, device=dev)
    first = s["rows_of"][seq, 0]                                         # row of the sequence's node 0
    inside = j[None, :] < (plan[:, 0:1] == plan[:, 0]).sum(1)[:, None]
    npos = pos[(first[:, None] + j[None, :]).clamp(max=n - 1)]
    word = plan[:, 4:8].gather(1, (j // 32)[None, :].expand(n, T))
    see = (((word >> (j % 32)[None, :]) & 1) != 0) & inside              # drafted ancestors
    see = see & ((pos[:, None] - npos < W) if W >= 0 else True)
    # keys of one row alone: drafted ancestors, window tokens, selected entries
    keys, ok = [_paged(s["tok_cache"], s["tok_table"], seq[:, None], base[:, None] + j[None, :], see)], [see]
    if W >= 0:
        u = pos[:, None] - W + 1 + torch.arange(W, device=dev)[None, :]
        good = (u >= 0) & (u < base[:, None]) & live[:, None]
        keys.append(_paged(s["tok_cache"], s["tok_table"], seq[:, None], u, good))
        ok.append(good)
    nv = torch.minimum((pos + 1) // r, s["ent_len"][seq].long()) if r else None
    if s["idx"] is not None:
        i = s["idx"].long()
        good = (i >= 0) & (i < nv[:, None]) & live[:, None]
        keys.append(_paged(s["ent_cache"], s["ent_table"], seq[:, None], i, good))
        ok.append(good)
    keys, ok = torch.cat(keys, 1), torch.cat(ok, 1)
    logits = torch.matmul(q, keys.transpose(1, 2)).masked_fill(~ok[:, None, :], -math.inf)
    # keys that the rows of a sequence share: every entry, every committed token
    B = s["rows_of"].shape[0]
    shared = None
    if W < 0:
        u = torch.arange(s["max_len"], device=dev)[None, :].expand(B, -1)
        own_len = base[s["rows_of"][:, 0]]
        shared = _paged(s["tok_cache"], s["tok_table"], torch.arange(B, device=dev)[:, None], u, u < own_len[:, None])
        sok = u[seq] < base[:, None]
    elif r and s["idx"] is None:
        u = torch.arange(s["max_ent"], device=dev)[None, :].expand(B, -1)
        shared = _paged(s["ent_cache"], s["ent_table"], torch.arange(B, device=dev)[:, None], u,
                        u < s["ent_len"][:, None])
        sok = u[seq] < nv[:, None]
    if shared is not None:
        qs = q[s["rows_of"]].reshape(B, -1, D)
        more = torch.matmul(qs, shared.transpose(1, 2)).view(-1, H, shared.shape[1])[s["row_at"]]
        logits = torch.cat([logits, more.masked_fill_(~sok[:, None, :], -math.inf)], 2)
    top = logits.amax(2, keepdim=True)
    if s["sinks"] is not None:
        top = torch.maximum(top, s["sinks"][None, :, None])
    p = torch.exp(logits - top)
    total = p.sum(2, keepdim=True)
    if s["sinks"] is not None:
        total = total + torch.exp(s["sinks"][None, :, None] - top)
    o = torch.matmul(p[:, :, :keys.shape[1]], keys)
    if shared is not None:
        ps = p[:, :, keys.shape[1]:][s["rows_of"]].reshape(B, -1, shared.shape[1])
        ps = ps * sok[s["rows_of"]].repeat_interleave(H, 1).reshape(B, -1, shared.shape[1])
        o = o + torch.matmul(ps, shared).view(-1, H, D)[s["row_at"]]
    o = _rotated(o / total, c, -sn, D - 64, 64, False)
    lse = (top + torch.log(total))[..., 0]
    s["o"].copy_(torch.where(live[:, None, None], o.to(torch.bfloat16), s["o"]))
    s["lse"].copy_(torch.where(live[:, None], lse, s["lse"]))
    return s["o"], s["lse"]


# ---------------------------------------------------------------------------
# the framework's calls
# ---------------------------------------------------------------------------
def _own(s):
    import sparse_compressed_attention_gb300 as V
    op = s["op"]
    if op == "rope":
        V.v4_rope(s["x"], s["pos"], s["inv_freq"], s["out"], rope_begin=s["begin"],
                  layout=V.V4_ROPE_HALF if s["half"] else V.V4_ROPE_INTERLEAVED, inverse=s["inverse"], mscale=s["mscale"])
        return s["out"]
    if op == "append":
        V.v4_cache_append(s["x"], s["pos"], s["inv_freq"], s["slot"], s["cache"])
        return s["cache"]
    if op == "w4":
        V.v4_w4_proj(s["x"], s["codes"], s["scales"], s["y"], norm_dim=s["norm"], eps=1e-6,
                     norm_w=s["norm_w"] if s["norm"] else None)
        return s["y"]
    kept = s["scratch"]
    if not kept:                 # a program makes its configuration and workspace once
        kept["cfg"] = V.make_config(s["B"], s["length"] + 128, s["H"], 512, 64, ratio=s["ratio"], window=s["W"], topk=s["K"])
        kept["ws"] = V.alloc_tree_workspace(kept["cfg"], s["q"].shape[0])
    V.v4_tree_mqa_fwd(kept["cfg"], dict(q=s["q"], plan=s["plan"], tok_cache=s["tok_cache"], tok_table=s["tok_table"],
                                        ent_cache=s["ent_cache"], ent_table=s["ent_table"], ent_len=s["ent_len"],
                                        idx=s["idx"], sink=s["sinks"], inv_freq=s["inv_freq"]),
                      s["o"], s["lse"], kept["ws"])
    return s["o"], s["lse"]


def run(s):
    if own:
        return _own(s)
    return {"rope": _plain_rope, "append": _plain_append, "tree": _plain_tree, "w4": _plain_w4}[s["op"]](s)


# ---------------------------------------------------------------------------
# definitions in 64 bits
# ---------------------------------------------------------------------------
def _turn(x, pos, f, sign, begin, R, half):
    """Complex multiplication of the rotated pairs of x [..., heads, dim] (fp64), pos [rows]."""
    phi = sign * pos.double()[:, None, None] * f.double()
    e = torch.polar(torch.ones_like(phi), phi)
    y = x.clone()
    if half:
        z = torch.complex(x[..., begin:begin + R // 2], x[..., begin + R // 2:begin + R]) * e
        y[..., begin:begin + R // 2], y[..., begin + R // 2:begin + R] = z.real, z.imag
    else:
        z = torch.complex(x[..., begin:begin + R:2], x[..., begin + 1:begin + R:2]) * e
        y[..., begin:begin + R:2], y[..., begin + 1:begin + R:2] = z.real, z.imag
    return y


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "rope":
        if s["x"].numel() > 40000000:          # in pieces: 64 bits of the large chunk would be several copies of 1 GB
            out = torch.empty(s["x"].shape, dtype=torch.float64, device="cuda")
            for a in range(0, case["rows"], 512):
                out[a:a + 512] = _turn(s["x"][a:a + 512].double(), s["pos"][a:a + 512], s["inv_freq"],
                                       -1.0 if case["inverse"] else 1.0, case["begin"], case["R"], case["half"])
        else:
            out = _turn(s["x"].double(), s["pos"], s["inv_freq"], -1.0 if case["inverse"] else 1.0, case["begin"],
                        case["R"], case["half"])
        out[..., case["begin"]:case["begin"] + case["R"]] *= s["mscale"]
        return out
    if op == "append":
        out = s["cache"].double()
        y = _turn(s["x"].double()[:, None], s["pos"], s["inv_freq"], 1.0, case["D"] - case["R"], case["R"], False)[:, 0]
        out.view(-1, case["D"])[s["slot"].long()] = y
        return out
    if op == "w4":
        G, N, K = case["groups"], case["N"], case["K"]
        out = torch.empty(case["rows"], G, N, dtype=torch.float64, device="cuda")
        kk = torch.arange(K, device="cuda")
        blk, c, t, e = kk // 128, kk % 128 // 32, kk % 32 // 8, kk % 8
        nib = (e % 2) * 4 + e // 2                                   # nibble of input k within its word
        byte = blk * 64 + (4 * t + c) * 4 + nib // 2
        for g in range(G):
            code = (s["codes"][g][:, byte] >> (4 * (nib % 2)).to(torch.uint8)[None, :]) & 15
            w = (code.double() - 8.0) * s["scales"][g].double()[:, kk // case["gs"]]
            out[:, g] = s["x"][:, g].double() @ w.T
        if case["norm"]:
            h = out.view(case["rows"], G, -1, case["norm"])
            h /= (h.square().mean(-1, keepdim=True) + 1e-6).sqrt()
            h *= s["norm_w"].double()
        return out
    lens, nodes, parents, depths = _shape(case)
    H, D, W, r = case["H"], 512, case["W"], case["ratio"]
    o = s["o"].double()
    lse = s["lse"].double()
    row = 0

    def paged(cache, table, at):
        return cache.view(-1, D)[table[at // case["page"]].long() * case["page"] + at % case["page"]].double()

    for b in range(case["B"]):
        L, ne = lens[b], lens[b] // r if r else 0
        tt = s["tok_table"][b]
        lo = 0 if W < 0 else max(0, L - W + 1)
        toks = paged(s["tok_cache"], tt, torch.arange(lo, L + nodes[b], device="cuda"))
        ents = paged(s["ent_cache"], s["ent_table"][b], torch.arange(ne, device="cuda")) if ne else None
        for i in range(nodes[b]):
            t = L + depths[b][i]
            q = _turn(s["q"][row:row + 1].double(), torch.tensor([t], device="cuda"), s["inv_freq"], 1.0, D - 64, 64,
                      False)[0]
            path, a = [], i
            while a >= 0:
                path.append(a)
                a = parents[b][a]
            at = [L + a for a in path if W < 0 or t - (L + depths[b][a]) < W]
            low = 0 if W < 0 else max(0, t - W + 1)
            keys = [toks[min(low, L) - lo:L - lo], toks[torch.tensor([u - lo for u in at], dtype=torch.long, device="cuda")]]
            nv = min((t + 1) // r, ne) if r else 0
            if case["K"]:
                sel = s["idx"][row]
                keys.append(ents[sel[sel >= 0].long()] if ne else toks[:0])
            elif nv:
                keys.append(ents[:nv])
            keys = torch.cat(keys)
            x = q @ keys.T * D ** -0.5
            full = torch.cat([x, s["sinks"].double()[:, None]], 1) if s["sinks"] is not None else x
            lse[row] = torch.logsumexp(full, 1)
            y = torch.exp(x - lse[row][:, None]) @ keys
            o[row] = _turn(y[None], torch.tensor([t], device="cuda"), s["inv_freq"], -1.0, D - 64, 64, False)[0]
            row += 1
    return o, lse
