"""The 4-bit cache: its write and read bit for bit, and the tree attention over it."""
import numpy as np
import pytest
import torch

import sparse_compressed_attention_gb300 as V
from oracle import cache_oracle as CO
from tests.helpers import np64
from tests.q4_cases import Q4Case

pytestmark = pytest.mark.gpu


def special_rows(dim, dt, seed, n=24):
    """Rows with ties, tiny and huge groups, zeros, one large value among small ones."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(n, dim, generator=g)
    x[0] = 0.0
    x[1] *= 1e-9
    x[2] *= 1e6
    x[3] = torch.arange(dim).float() % 15 - 7                     # codes themselves, scale one
    x[4] = (torch.arange(dim).float() % 15 - 7) * 0.5 + 0.25      # halfway between
    x[5, 16:32] = 0.0
    x[6, 3] = 1000.0
    x[7] = torch.where(torch.arange(dim) % 16 == 0, 7 * 17 / 16, 0.9)      # scales halfway between two
    x[8] = torch.where(torch.arange(dim) % 16 == 5, -7 * 19 / 16, 2.0)
    x[9] *= 2.0 ** -21
    x[10] = -0.0
    return x.to(dt)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("dim", [32, 64, 128, 160, 512, 576])
def test_write_and_read_bit_for_bit(dim, dt):
    x = special_rows(dim, dt, dim)
    n = x.shape[0]
    perm = np.random.default_rng(dim).permutation(64)[:n].astype(np.int32)
    perm[11] = -1
    cache = torch.full((4, 16, V.v4_q4_row_bytes(dim)), 77, dtype=torch.uint8, device="cuda")
    slot = torch.from_numpy(perm).cuda()
    V.v4_cache_append_q4(x.cuda(), slot, cache)
    want = np.full((64, CO.q4_row_bytes(dim)), 77, np.uint8)
    live = perm >= 0
    want[perm[live]] = CO.q4_pack(np64(x))[live]
    assert np.array_equal(cache.cpu().numpy().reshape(64, -1), want)
    for out_dt in (torch.bfloat16, torch.float32):
        out = torch.full((n, dim), 3.0, dtype=out_dt, device="cuda")
        V.v4_cache_read_q4(cache, slot, out)
        ref = CO.q4_unpack(want[np.where(live, perm, 0)], dim)
        ref[~live] = 0.0
        assert np.array_equal(np64(out), ref)
    assert V.v4_get_device_status() == 0


def test_every_code_and_scale_reads_exactly():
    rows = np.zeros((256, 48), np.uint8)                          # 64 values: 32 code bytes, 4 scales
    rows[:, :32] = np.random.default_rng(0).integers(0, 256, (256, 32))
    rows[:, 32:36] = (np.arange(256)[:, None] + 64 * np.arange(4)) % 256
    cache = torch.from_numpy(rows).cuda()
    slot = torch.arange(256, dtype=torch.int32).cuda()
    for dt in (torch.bfloat16, torch.float32):
        out = torch.empty(256, 64, dtype=dt, device="cuda")
        V.v4_cache_read_q4(cache, slot, out)
        assert np.array_equal(np64(out), CO.q4_unpack(rows, 64))


@pytest.mark.parametrize("rows", [1, 1000, 40000])
def test_many_rows(rows):
    """A read row written again is the same row: its largest code is 7 where the group's maximum was not rounded down."""
    x = torch.randn(rows, 512, generator=torch.Generator().manual_seed(rows)).to(torch.bfloat16).cuda()
    wide = torch.zeros(rows, 640, dtype=torch.bfloat16, device="cuda")
    wide[:, 64:576] = x
    cache = torch.zeros(rows, V.v4_q4_row_bytes(512), dtype=torch.uint8, device="cuda")
    slot = torch.randperm(rows, generator=torch.Generator().manual_seed(1)).to(torch.int32).cuda()
    V.v4_cache_append_q4(wide[:, 64:576], slot, cache)            # a strided view
    out = torch.zeros(rows, 576, dtype=torch.bfloat16, device="cuda")
    V.v4_cache_read_q4(cache, slot, out[:, 64:])
    assert (out[:, :64] == 0).all()
    got, xf = out[:, 64:].float(), x.float()
    step = cache[slot.long(), 256:].to(torch.int32)
    scale = (((step << 20) + (107 << 23)).view(torch.float32)).repeat_interleave(16, 1)
    assert ((got - xf).abs() <= 0.5 * scale).all()                # max|x| / 7 rounds by less than one part in 16: no code is cut
    some = slice(0, min(rows, 40))
    assert np.array_equal(cache[slot[some].long()].cpu().numpy(), CO.q4_pack(np64(x[some])))


def test_values_that_are_no_numbers():
    x = torch.ones(3, 32, device="cuda")
    x[0, 3], x[1, 4], x[2, 5] = float("nan"), float("inf"), float("-inf")
    cache = torch.zeros(3, V.v4_q4_row_bytes(32), dtype=torch.uint8, device="cuda")
    slot = torch.arange(3, dtype=torch.int32).cuda()
    V.v4_cache_append_q4(x, slot, cache)
    out = torch.empty_like(x)
    V.v4_cache_read_q4(cache, slot, out)
    assert out[0, 3] == 0 and out[1, 4] == 7 * 3840 and out[2, 5] == -8 * 3840
    assert torch.isfinite(out).all() and ((out[:, 16:] - 1).abs() <= 0.5 / 7 * 17 / 16).all()


def test_bad_slots_are_flagged():
    V.v4_reset_device_status()
    cache = torch.zeros(4, 48, dtype=torch.uint8, device="cuda")
    x = torch.ones(3, 64, device="cuda")
    V.v4_cache_append_q4(x, torch.tensor([4, -2, 1], dtype=torch.int32).cuda(), cache)
    assert V.v4_get_device_status() == 6
    assert (cache[[0, 2, 3]] == 0).all() and (cache[1] != 0).any()
    V.v4_reset_device_status()
    out = torch.ones(3, 64, device="cuda")
    V.v4_cache_read_q4(cache, torch.tensor([4, 2 ** 31 - 1, 1], dtype=torch.int32).cuda(), out)
    assert V.v4_get_device_status() == 6 and (out[:2] == 0).all() and (out[2] != 0).all()
    V.v4_reset_device_status()


CASES = {
    "one_token": dict(lens=[700], nodes=[1], ratio=4, K=64),
    "nothing_committed": dict(lens=[0, 0], nodes=[1, 3], window=128),
    "lengths_one": dict(lens=[1, 2, 3], nodes=[1, 1, 2], ratio=4, K=32),
    "ragged_trees": dict(lens=[5, 300, 64, 129], nodes=[3, 8, 1, 5], ratio=4, K=32, sink=True, pad=(2, 3)),
    "all_tokens": dict(lens=[1000, 63, 64, 65, 127, 128, 129], nodes=[1, 2, 1, 1, 1, 1, 1], window=-1),
    "entries": dict(lens=[5000, 100, 127], nodes=[2, 1, 1], ratio=8, tok_page=16, ent_page=48),
    "odd_pages": dict(lens=[517, 91], nodes=[4, 2], window=77, ratio=4, tok_page=7, ent_page=5),
    "window_zero": dict(lens=[517, 3], nodes=[2, 1], window=0, ratio=4),
    "two_slices": dict(lens=[300, 40], nodes=[2, 1], H=128, ratio=4, K=32, sink=True),
    "large_logits": dict(lens=[400, 30], nodes=[3, 1], window=-1, q_scale=20.0),
}


@pytest.mark.parametrize("path", ["auto", "cuda_cores", "f32"])
@pytest.mark.parametrize("name", list(CASES))
def test_attention(name, path):
    kw = dict(CASES[name])
    if path == "f32":
        kw.update(H=9, D=64, R=16, dt=torch.float32)
    elif path == "cuda_cores":
        kw.update(path=V.V4_PATH_SIMT)
    c = Q4Case(seed=sum(map(ord, name)), **kw)
    c.check(*c.run())


@pytest.mark.parametrize("D,R", [(32, 8), (96, 32), (128, 64), (1024, 64)])
def test_attention_of_other_widths(D, R):
    c = Q4Case([90, 7], [2, 1], H=5, D=D, R=R, dt=torch.bfloat16, ratio=4, seed=D)
    c.check(*c.run())


@pytest.mark.parametrize("kw", [dict(lens=[20000], nodes=[1], window=-1), dict(lens=[9000, 31, 4000], nodes=[4, 1, 2], window=-1),
                                dict(lens=[3000] * 20, nodes=[1] * 20, ratio=4, K=512)])
def test_attention_against_the_dense_cache(kw):
    """The same values in a bf16 cache: logits are sums of the same products, so lse agrees to the sums' order, and outputs to
    one rounding of the probabilities and one of the output on each side."""
    c = Q4Case(seed=9, **kw)
    o, lse = c.run()
    dense = c.dense_inputs()
    do, dl = torch.zeros_like(o), torch.zeros_like(lse)
    V.v4_tree_mqa_fwd(c.cfg, dense, do, dl, V.alloc_tree_workspace(c.cfg, c.n))
    assert (lse - dl).abs().max() <= 2.0 ** -16 * (1 + dl.abs().max())
    rel = (o.float() - do.float()).norm() / do.float().norm()
    assert rel <= 2 * (2.0 ** -8 + 2.0 ** -8)
    assert V.v4_get_device_status() == 0


def test_attention_repeats_in_graphs_and_streams():
    cases = [Q4Case([5000, 3], [2, 1], window=-1, seed=3), Q4Case([900, 70], [3, 2], ratio=4, K=64, seed=4)]
    ins = [c.device_inputs() for c in cases]
    want = [c.run(x) for c, x in zip(cases, ins)]
    outs = [(torch.full_like(o, 3.0), torch.full_like(s, 3.0)) for o, s in want]
    ws = [V.alloc_tree_workspace(c.cfg, c.n) for c in cases]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for c, x, (o, s), w in zip(cases, ins, outs, ws):
            V.v4_tree_mqa_fwd_q4(c.cfg, x, o, s, w)
    for o, s in outs:
        o.fill_(3.0), s.fill_(3.0)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    for (o, s), (wo, wl) in zip(outs, want):
        assert torch.equal(o, wo) and torch.equal(s, wl)
    streams = [torch.cuda.Stream() for _ in cases]
    for st, c, x, (o, s), w in zip(streams, cases, ins, outs, ws):
        o.fill_(3.0), s.fill_(3.0)
        st.wait_stream(torch.cuda.current_stream())
        for _ in range(5):
            V.v4_tree_mqa_fwd_q4(c.cfg, x, o, s, w, stream=st)
    torch.cuda.synchronize()
    for (o, s), (wo, wl) in zip(outs, want):
        assert torch.equal(o, wo) and torch.equal(s, wl)


def test_bad_pages_and_indices_are_skipped_and_flagged():
    V.v4_reset_device_status()
    c = Q4Case([300, 200], [1, 1], ratio=4, K=32, seed=12)
    x = c.device_inputs()
    x["tok_table"] = x["tok_table"].clone()
    x["tok_table"][0, 4] = 10 ** 6                                # tokens 256..299 of sequence 0
    o, lse = c.run(x)
    assert V.v4_get_device_status() == 6
    V.v4_reset_device_status()
    ref_o, ref_l = c.run()
    assert torch.equal(o[1], ref_o[1]) and torch.equal(lse[1], ref_l[1])
    assert torch.isfinite(o.float()).all() and not torch.equal(o[0], ref_o[0])


def test_rows_of_no_values_are_refused():
    none = torch.empty(4, 0, dtype=torch.uint8, device="cuda")
    x, slot = torch.empty(2, 0, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError, match="cache"):
        V.v4_cache_append_q4(x, slot, none)
    with pytest.raises(ValueError, match="cache"):
        V.v4_cache_read_q4(none, slot, x)
