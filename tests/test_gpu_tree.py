"""Plans of drafted trees and the tree attention over paged caches against the
float64 oracle: masks that leave nothing, pages that end inside a tile, ragged
lengths from nothing up, padding rows, bad indices, replayed graphs."""
import numpy as np
import pytest
import torch

import seeded_inputs as SI
import sparse_compressed_attention_gb300 as V
from tests.helpers import inv_freq_for, np64, rel_l2
from tests.tree_cases import Case, random_parents

pytestmark = pytest.mark.gpu
NAN = float("nan")
TINY = dict(H=5, D=64, R=16)


# ---------------------------------------------------------------- plan
@pytest.mark.parametrize("nodes", [[1], [2, 0, 1], [128], [127, 3, 64, 33, 0], [5] * 40])
@pytest.mark.parametrize("pad", [(0, 0), (3, 200)])
def test_plan_matches_walk(nodes, pad):
    c = Case([17 * i + 3 for i in range(len(nodes))], nodes, pad=pad, seed=len(nodes), window=-1, **TINY)
    c.device_inputs()
    assert np.array_equal(c.plan.cpu().numpy().astype(np.int64)[:, :4], c.plan_ref[:, :4])
    assert np.array_equal(c.plan.cpu().numpy().view(np.uint32)[:, 4:].astype(np.int64), c.plan_ref[:, 4:])
    assert np.array_equal(c.pos.cpu().numpy(), c.pos_ref)
    slot = np.full(c.n, -1)
    for row in range(c.n):
        b, j, _, L = c.plan_ref[row, :4]
        if b >= 0:
            slot[row] = c.tok_table[b, (L + j) // c.tok_page] * c.tok_page + (L + j) % c.tok_page
    assert np.array_equal(c.slot.cpu().numpy(), slot)
    assert V.v4_get_device_status() == 0


@pytest.mark.parametrize("shape", ["chain", "star", "zigzag"])
def test_plan_of_extreme_trees(shape):
    par = {"chain": list(range(-1, 127)), "star": [-1] + [0] * 127, "zigzag": [-1, -1] + list(range(126))}[shape]
    c = Case([1000], [128], parents=[par], window=-1, **TINY)
    c.device_inputs()
    assert np.array_equal(c.plan.cpu().numpy().view(np.uint32).astype(np.int64), c.plan_ref)
    if shape == "chain":                                # NULL parents are chains
        again = torch.empty_like(c.plan)
        V.v4_tree_plan(torch.tensor([0, 128], dtype=torch.int32).cuda(), torch.tensor([1000], dtype=torch.int32).cuda(),
                       None, again)
        assert torch.equal(again, c.plan)


def test_plan_flags_bad_values():
    i32 = torch.int32
    plan = torch.empty(6, 8, dtype=i32, device="cuda")
    slot = torch.empty(6, dtype=i32, device="cuda")
    t = lambda *v: torch.tensor(v, dtype=i32).cuda()                       # noqa: E731
    V.v4_tree_plan(t(0, 3, 6), t(5, 9), t(-1, 1, -5, 2, 0, 1), plan, slot=slot, block_table=t(0, 9, 1, 7).view(2, 2),
                   page_size=8, n_slots=64)
    assert V.v4_get_device_status() == 6
    V.v4_reset_device_status()
    got = plan.cpu().numpy()
    assert got[:3, 2].tolist() == [5, 5, 5]             # nodes 1 and 2 hang below the prefix
    assert got[3:, 2].tolist() == [9, 10, 11]           # node 0's parent 2 is no earlier node
    assert slot.cpu().tolist() == [5, 6, 7, 57, 58, 59]
    V.v4_tree_plan(t(0, 3, 6), t(7, -1), t(-1, 0, 1, -1, 0, 1), plan, slot=slot, block_table=t(0, 9, 1, 7).view(2, 2),
                   page_size=8, n_slots=64)
    assert V.v4_get_device_status() == 6                # a page outside the cache, and a negative length
    V.v4_reset_device_status()
    assert slot.cpu().tolist() == [7, -1, -1, -1, -1, -1]
    assert plan.cpu()[3:, 0].tolist() == [-1] * 3
    big = torch.empty(200, 8, dtype=i32, device="cuda")
    V.v4_tree_plan(t(0, 129, 150), t(7, 8), None, big)
    assert V.v4_get_device_status() == 6                # 129 nodes
    V.v4_reset_device_status()
    assert big.cpu()[:, 0].tolist() == [-1] * 129 + [1] * 21 + [-1] * 50


# ---------------------------------------------------------------- attention
SHAPES = [
    # window alone: no committed token, one, around the window, far
    dict(lens=[0, 1, 126, 127, 128, 129, 1000], nodes=[1, 3, 2, 1, 1, 2, 5]),
    # every token, lengths around a tile, ragged nodes
    dict(lens=[0, 1, 127, 128, 255, 513], nodes=[2, 1, 1, 7, 3, 1], window=-1, tok_page=16),
    # no token at all: entries only
    dict(lens=[0, 5, 300, 1024], nodes=[1, 2, 2, 1], window=0, ratio=4),
    # every entry and a window; pages that end inside a tile
    dict(lens=[3, 700, 1537], nodes=[2, 4, 3], ratio=4, tok_page=48, ent_page=80, sink=True),
    dict(lens=[100, 5000], nodes=[3, 2], ratio=128, window=17, tok_page=1, ent_page=3),
    # selections with unused slots anywhere, rows with fewer visible entries than slots, rows with none
    dict(lens=[2, 40, 2200], nodes=[2, 3, 4], ratio=4, K=96, sink=True),
    dict(lens=[30, 900], nodes=[1, 6], ratio=4, K=200, window=5, ent_page=16),
    # long trees: drafted ancestors fall out of the window
    dict(lens=[50, 3], nodes=[128, 60], window=16, tok_page=32),
    # padding before and behind
    dict(lens=[10, 200], nodes=[3, 4], ratio=4, pad=(2, 5)),
    # nothing to see: o = 0 and lse = -inf, or the sink alone
    dict(lens=[0, 100], nodes=[2, 1], window=0, ratio=128),
    dict(lens=[0, 100], nodes=[2, 1], window=0, ratio=128, sink=True),
]


@pytest.mark.parametrize("i", range(len(SHAPES)))
@pytest.mark.parametrize("kind", ["bf16", "bf16_128_heads", "f32_tiny", "bf16_odd", "f32_no_rotation"])
def test_attention_matches_oracle(i, kind):
    over = {"bf16": {}, "bf16_128_heads": dict(H=128), "f32_tiny": dict(TINY, dt=torch.float32),
            "bf16_odd": dict(H=9, D=96, R=32), "f32_no_rotation": dict(H=3, D=32, R=0, dt=torch.float32)}[kind]
    c = Case(seed=i, fill=NAN, **{**SHAPES[i], **over})
    c.check(*c.run())


@pytest.mark.parametrize("i", [1, 3, 5])
def test_forced_paths(i):
    c = Case(seed=i, fill=NAN, path=V.V4_PATH_SIMT, **SHAPES[i])
    c.check(*c.run())
    c = Case(seed=i, fill=NAN, path=V.V4_PATH_TC, **SHAPES[i])
    c.check(*c.run())


@pytest.mark.parametrize("q_scale", [8.0, 64.0])
@pytest.mark.parametrize("sink", [False, True])
def test_large_logits(q_scale, sink):
    """Logits that outgrow those of earlier tiles by far: the running maximum has to follow."""
    c = Case([1500, 300], [2, 1], window=-1, tok_page=64, sink=sink, q_scale=q_scale, seed=2)
    for k in range(24):                                # keys grow along the sequence
        c.tok[c.tok_table[0, k]] = (c.tok[c.tok_table[0, k]].float() * (0.25 + 0.25 * k)).to(c.dt)
    c.check(*c.run())


def test_masked_rows_may_hold_anything():
    """Infinities and NaN in cache rows that no key list names, and the lowest values in ones that it does."""
    c = Case([400, 90], [3, 2], ratio=4, K=64, fill=float("inf"), seed=5)
    c.check(*c.run())
    # a NaN key reaches its own sequence's rows alone
    c = Case([300, 90], [1, 1], window=-1, seed=6)
    x = c.device_inputs()
    b = int(c.tok_table[0, 1])
    x["tok_cache"][b, 3] = NAN
    o, lse = c.run(x)
    assert torch.isnan(o[0].float()).all() and torch.isnan(lse[0]).all()
    assert torch.isfinite(o[1].float()).all() and torch.isfinite(lse[1]).all()


def test_long_rows_split_and_joined():
    c = Case([20011, 7], [1, 1], window=-1, tok_page=128, sink=True, seed=8)
    c.check(*c.run())
    c = Case([33000], [2], window=100, ratio=4, ent_page=64, seed=9)
    c.check(*c.run())


def test_many_rows():
    rng = np.random.default_rng(1)
    lens = [int(v) for v in rng.integers(0, 400, 60)]
    nodes = [int(v) for v in rng.integers(1, 7, 60)]
    c = Case(lens, nodes, ratio=4, K=40, seed=10, pad=(0, 3))
    c.check(*c.run())


@pytest.mark.parametrize("page", [8, 20, 24, 96, 100, 256])
@pytest.mark.parametrize("over", ["tokens", "entries"])
def test_whole_page_runs_of_any_page_size(page, over):
    """Every token, or every entry: leading tiles come page by page where the page has a power of two from 8 in it."""
    if over == "tokens":
        c = Case([700, 257, 3], [2, 1, 4], window=-1, tok_page=page, seed=13)
    else:
        c = Case([3000, 1030, 9], [2, 1, 4], window=64, ratio=4, ent_page=page, seed=14)
    c.check(*c.run())


def test_more_items_than_threads_of_a_block():
    rng = np.random.default_rng(2)
    lens = [int(v) for v in rng.integers(0, 300, 70)]
    nodes = [int(v) for v in rng.integers(1, 7, 70)]
    c = Case(lens, nodes, H=192, ratio=4, K=24, window=16, seed=15, pad=(2, 5))
    assert c.n * 3 > 448
    c.check(*c.run())


def test_long_rows_of_several_head_slices():
    """Items in few and in many parts in one call, with sinks."""
    c = Case([9000, 40, 2500], [1, 2, 1], H=128, window=-1, tok_page=16, sink=True, seed=16)
    c.check(*c.run())


@pytest.mark.parametrize("kind", ["bf16", "f32_tiny"])
def test_call_of_padding_alone_writes_nothing(kind):
    kw = dict(H=4, D=64, R=16, dt=torch.float32) if kind == "f32_tiny" else {}
    c = Case([50], [1], seed=17, **kw)
    x = c.device_inputs()
    x["plan"].zero_()
    x["plan"][:, 0] = -1
    o = torch.full((c.n, c.H, c.D), 3.0, dtype=c.dt, device="cuda")
    lse = torch.full((c.n, c.H), 3.0, device="cuda")
    V.v4_tree_mqa_fwd(c.cfg, x, o, lse, V.alloc_tree_workspace(c.cfg, c.n))
    assert (o == 3).all() and (lse == 3).all()


def test_chain_of_calls_in_a_forked_graph():
    """Every call starts while the one before drains, and waits for what it reads: a chain of short calls that feed one
    another, in one stream and over two streams of one captured graph, against the same chain with a wait after each."""
    g = torch.Generator().manual_seed(33)
    c = Case([300, 77, 5000], [3, 2, 1], ratio=4, K=48, sink=True, seed=20)
    x = c.device_inputs()
    n, H = c.n, 64
    w = (torch.randn(1, 512, 64 * 512, generator=g) * 0.05).to(torch.bfloat16).cuda()
    codes, scales = torch.empty(1, 64 * 512, 256, dtype=torch.uint8, device="cuda"), torch.empty(
        1, 64 * 512, 4, dtype=torch.bfloat16, device="cuda")
    V.v4_w4_pack(w, 128, codes, scales)
    lat = torch.randn(n, 1, 512, generator=g).to(torch.bfloat16).cuda()
    kv = torch.randn(n, 512, generator=g).to(torch.bfloat16).cuda()
    begin = torch.from_numpy(c.begin.astype(np.int32)).cuda()
    lens, par = torch.tensor(c.lens, dtype=torch.int32).cuda(), torch.from_numpy(c.parent).cuda()
    table = x["tok_table"]
    ws = V.alloc_tree_workspace(c.cfg, n)
    q, o = (torch.empty(n, H, 512, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    lse = torch.empty(n, H, device="cuda")

    def layer(norm, wait, side=None):
        here = torch.cuda.current_stream()
        V.v4_tree_plan(begin, lens, par, x["plan"], pos=c.pos, slot=c.slot, block_table=table, page_size=c.tok_page,
                       n_slots=c.tok.shape[0] * c.tok_page)
        wait()
        if side is not None:
            side.wait_stream(here)
        with torch.cuda.stream(side or here):
            V.v4_cache_append(kv, c.pos, x["inv_freq"], c.slot, x["tok_cache"])
            wait()
        V.v4_w4_proj(lat, codes, scales, q.view(n, 1, -1), norm_dim=norm)
        wait()
        V.v4_rope(q, c.pos, x["inv_freq"], q, inverse=True)
        wait()
        if side is not None:
            here.wait_stream(side)
        V.v4_tree_mqa_fwd(c.cfg, dict(x, q=q), o, lse, ws)
        wait()
        lat.copy_(o[:, 3][:, None])                    # a kernel of another library in the chain
        V.v4_rope(o, c.pos, x["inv_freq"], o)
        wait()
        kv.copy_(o[:, 7])

    def run(wait, side=None):
        for norm in (512, 64, 0, 512):
            layer(norm, wait, side)

    start = [t.clone() for t in (lat, kv, x["tok_cache"])]

    def reset():
        for t, s in zip((lat, kv, x["tok_cache"]), start):
            t.copy_(s)
        torch.cuda.synchronize()

    live = torch.from_numpy(c.plan_ref[:, 0] >= 0).cuda()
    outs = []
    run(torch.cuda.synchronize)
    outs.append((o[live].clone(), lse[live].clone(), x["tok_cache"].clone()))
    side, main = torch.cuda.Stream(), torch.cuda.Stream()
    for other in (None, side):
        reset()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=main):
            run(lambda: None, other)
        for _ in range(3):
            reset()
            graph.replay()
            torch.cuda.synchronize()
            outs.append((o[live].clone(), lse[live].clone(), x["tok_cache"].clone()))
    for other in (None, side):
        reset()
        run(lambda: None, other)
        torch.cuda.synchronize()
        outs.append((o[live].clone(), lse[live].clone(), x["tok_cache"].clone()))
    for got in outs[1:]:
        assert all(torch.equal(u, v) for u, v in zip(got, outs[0]))
    assert V.v4_get_device_status() == 0


@pytest.mark.parametrize("over", ["selected", "tokens", "entries"])
def test_offsets_beyond_32_bits(over):
    """Pages more than 2^32 bytes (and 2^32 elements) into their caches, gathered and as page runs."""
    c = {"selected": lambda: Case([300, 77], [3, 2], ratio=4, K=48, seed=22),
         "tokens": lambda: Case([700, 257], [2, 1], window=-1, seed=23),
         "entries": lambda: Case([3000, 1030], [2, 1], window=64, ratio=4, ent_page=64, seed=24)}[over]()
    x = c.device_inputs()
    for kind in ("tok", "ent") if c.ratio else ("tok",):
        small, table = x[kind + "_cache"], x[kind + "_table"]
        pages, page, D = small.shape
        far = (1 << 32) // (page * D) + 5
        big = torch.empty(far + pages, page, D, dtype=small.dtype, device="cuda")
        big[far:] = small
        x[kind + "_cache"], x[kind + "_table"] = big, torch.where(table < 0, table, table + far)
    c.check(*c.run(x))


def test_two_calls_at_once():
    """Calls on two streams, each with its own workspace."""
    cases = [Case([9000, 30], [2, 3], window=-1, seed=18), Case([5000, 700], [4, 1], ratio=4, seed=19)]
    ins = [c.device_inputs() for c in cases]
    want = [c.run(x) for c, x in zip(cases, ins)]
    ws = [V.alloc_tree_workspace(c.cfg, c.n) for c in cases]
    outs = [(torch.empty_like(o), torch.empty_like(s)) for o, s in want]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(10):
        for c, x, w, (o, s), st in zip(cases, ins, ws, outs, streams):
            V.v4_tree_mqa_fwd(c.cfg, x, o, s, w, stream=st)
    torch.cuda.synchronize()
    live = [torch.from_numpy(c.plan_ref[:, 0] >= 0).cuda() for c in cases]
    for (o, s), (wo, wl), m in zip(outs, want, live):
        assert torch.equal(o[m], wo[m]) and torch.equal(s[m], wl[m])


def test_repeats_bit_for_bit_and_replays():
    c = Case([700, 1900, 20], [3, 4, 1], ratio=4, K=128, sink=True, seed=11, pool=60)
    x = c.device_inputs()
    o, lse = c.run(x)
    again = c.run(x)
    assert torch.equal(o, again[0]) and torch.equal(lse, again[1])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    ws = V.alloc_tree_workspace(c.cfg, c.n)
    o2, lse2 = torch.zeros_like(o), torch.zeros_like(lse)
    with torch.cuda.stream(s):
        V.v4_tree_mqa_fwd(c.cfg, x, o2, lse2, ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        V.v4_tree_mqa_fwd(c.cfg, x, o2, lse2, ws)
    # the captured call follows lengths, trees and pages that change between replays
    d = Case([650, 1890, 3], [2, 2, 4], ratio=4, K=128, sink=True, seed=12, pool=60)
    y = d.device_inputs()
    for name in ("q", "plan", "idx", "sink"):
        x[name].copy_(y[name])
    x["ent_len"].copy_(y["ent_len"])
    for kind in ("tok", "ent"):
        if x[kind + "_cache"].shape != y[kind + "_cache"].shape or x[kind + "_table"].shape != y[kind + "_table"].shape:
            pytest.fail("the two cases must share their buffers' shapes")
        x[kind + "_cache"].copy_(y[kind + "_cache"])
        x[kind + "_table"].copy_(y[kind + "_table"])
    o2.fill_(3.0)
    lse2.fill_(3.0)
    graph.replay()
    torch.cuda.synchronize()
    d.check(o2, lse2)


def test_bad_indices_are_flagged_and_skipped():
    c = Case([300, 200], [2, 2], ratio=4, K=32, seed=13)
    x = c.device_inputs()
    x["idx"][0, 5] = 10 ** 6
    x["idx"][2, 0] = -3
    x["tok_table"][1, 2] = 99                           # a page outside the cache
    o, lse = c.run(x)
    assert V.v4_get_device_status() == 6
    V.v4_reset_device_status()
    c.idx[0, 5] = -1
    c.idx[2, 0] = -1
    tok = c.tok_table.copy()
    flat = np64(c.tok).reshape(-1, c.D)
    ent = np64(c.ent).reshape(-1, c.D)
    from oracle import serving_oracle as S

    def tok_rows(b, u):
        if b == 1 and u // c.tok_page == 2:
            return None
        return flat[int(tok[b, u // c.tok_page]) * c.tok_page + u % c.tok_page]

    def ent_rows(b, s):
        if s is None:
            return c.ent_counts[b]
        return ent[int(c.ent_table[b, s // c.ent_page]) * c.ent_page + s % c.ent_page]

    ref = S.tree_mqa(np64(c.q), c.plan_ref, tok_rows, ent_rows, c.idx.numpy(), None, c.f, 4, 128, 32, c.scale,
                     np.full((c.n, c.H, c.D), 3.0), np.full((c.n, c.H), 3.0))
    c.check(o, lse, ref)
    # plan rows that cannot be used are left out like padding
    x = c.device_inputs()
    x["plan"][1, 0] = 2
    x["plan"][3, 2] = -4
    o, lse = c.run(x)
    assert V.v4_get_device_status() == 6
    V.v4_reset_device_status()
    assert torch.all(o[[1, 3]] == 3.0) and torch.all(lse[[1, 3]] == 3.0)


def test_chain_equals_the_rows_of_a_whole_sequence():
    """A chain of drafted tokens at the end of a cache is the last rows of v4_sparse_mqa_fwd."""
    p = SI.preset("csa_bf16_4k", S=600, q_mode="direct", K=64)
    x = SI.make_layer_inputs(p, "cuda", seed=3, sink=True)
    f = torch.from_numpy(inv_freq_for(p)).cuda()
    n, L, S_ = 10, 590, 600
    cfg = V.config_from_preset(p, q_begin=L)
    full = V.config_from_preset(p)
    N = S_ // 4
    ent = torch.empty(1, N, 512, dtype=torch.bfloat16, device="cuda")
    V.v4_compress(full, x["ckv"], x["cscore"], x["ape"], x.get("norm_w"), f, 512, 0, ent)
    idx = SI.random_topk_indices(1, S_, 4, 64, "cuda", seed=5)[:, L:].contiguous()
    o_ref = torch.empty(1, n, 64, 512, dtype=torch.bfloat16, device="cuda")
    l_ref = torch.empty(1, n, 64, device="cuda")
    V.v4_sparse_mqa_fwd(cfg, x["q"][:, L:].contiguous(), x["kv"], ent, idx, x["sink"], f, o_ref, l_ref,
                        V.alloc_workspace(cfg))
    # the same through the serving calls: plan, paged writes of the committed and drafted tokens, attention
    i32 = torch.int32
    page, pages = 16, 40
    perm = torch.randperm(pages, generator=torch.Generator().manual_seed(1))
    table = perm[:38].to(i32).view(1, 38).cuda()
    tok = torch.zeros(pages, page, 512, dtype=torch.bfloat16, device="cuda")
    ents = torch.zeros(pages, page, 512, dtype=torch.bfloat16, device="cuda")
    u = torch.arange(S_)
    slots = (perm[u // page] * page + u % page).to(i32).cuda()
    V.v4_cache_append(x["kv"][0, :L], torch.arange(L, dtype=i32, device="cuda"), f, slots[:L].contiguous(), tok)
    V.v4_cache_append(ent[0], None, None, slots[:N].contiguous(), ents)
    plan, pos, slot = (torch.empty(n, 8, dtype=i32, device="cuda"), torch.empty(n, dtype=i32, device="cuda"),
                       torch.empty(n, dtype=i32, device="cuda"))
    V.v4_tree_plan(torch.tensor([0, n], dtype=i32).cuda(), torch.tensor([L], dtype=i32).cuda(), None, plan, pos=pos,
                   slot=slot, block_table=table, page_size=page, n_slots=pages * page)
    assert torch.equal(slot, slots[L:])
    V.v4_cache_append(x["kv"][0, L:], pos, f, slot, tok)
    tcfg = V.make_config(1, S_, 64, 512, 64, ratio=4, window=128, topk=64)
    o, lse = torch.empty_like(o_ref[0]), torch.empty_like(l_ref[0])
    # every entry of the sequence is in the cache: entries that the drafted tokens complete included
    V.v4_tree_mqa_fwd(tcfg, dict(q=x["q"][0, L:].contiguous(), plan=plan, tok_cache=tok, tok_table=table, ent_cache=ents,
                                 ent_table=table, ent_len=torch.tensor([N], dtype=i32).cuda(), idx=idx[0], sink=x["sink"],
                                 inv_freq=f), o, lse, V.alloc_tree_workspace(tcfg, n))
    assert V.v4_get_device_status() == 0
    assert rel_l2(np64(o), np64(o_ref[0])) < 1e-2
    assert np.max(np.abs(np64(lse) - np64(l_ref[0]))) < 2e-2


def test_decode_step_as_used():
    """One step of a layer as a server runs it: 4-bit query projection with its norm, plan, cache write, attention,
    4-bit grouped output projection; against the oracles chained."""
    from oracle import serving_oracle as S
    g = torch.Generator().manual_seed(21)
    c = Case([300, 77], [3, 2], ratio=4, K=48, sink=True, seed=14)
    x = c.device_inputs()
    n = c.n
    wq = (torch.randn(1, 256, 64 * 512, generator=g) * 0.06).to(torch.bfloat16).cuda()
    wo = (torch.randn(8, 4096, 128, generator=g) * 0.015).to(torch.bfloat16).cuda()
    packed = []
    for w, gs in ((wq, 64), (wo, 128)):
        G, K, N = w.shape
        codes = torch.empty(G, N, K // 2, dtype=torch.uint8, device="cuda")
        scales = torch.empty(G, N, K // gs, dtype=torch.bfloat16, device="cuda")
        V.v4_w4_pack(w, gs, codes, scales)
        packed.append((codes, scales, gs))
    qlat = torch.randn(n, 1, 256, generator=g).to(torch.bfloat16).cuda()
    kv = torch.randn(n, 512, generator=g).to(torch.bfloat16).cuda()
    q = torch.empty(n, 1, 64 * 512, dtype=torch.bfloat16, device="cuda")
    y = torch.empty(n, 8, 128, dtype=torch.bfloat16, device="cuda")
    V.v4_w4_proj(qlat, packed[0][0], packed[0][1], q, norm_dim=512)
    V.v4_cache_append(kv, c.pos, x["inv_freq"], c.slot, x["tok_cache"])
    x["q"] = q.view(n, 64, 512)
    o, lse = c.run(x)
    V.v4_w4_proj(o.view(n, 8, 4096), packed[1][0], packed[1][1], y)
    # oracle chain from the library's stored q (bf16) and cache rows
    rq, _ = S.w4_proj(np64(qlat), packed[0][0].cpu().numpy(), np64(packed[0][1]), 64, 512)
    assert rel_l2(np64(q), rq) < 2.0 ** -8
    c.q = q.view(n, 64, 512).cpu()
    c.tok = x["tok_cache"].cpu()
    c.check(o, lse)
    ry, _ = S.w4_proj(np64(o).reshape(n, 8, 4096), packed[1][0].cpu().numpy(), np64(packed[1][1]), 128)
    assert rel_l2(np64(y), ry) < 2.0 ** -8
