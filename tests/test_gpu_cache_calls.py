"""The norm, 4-bit cache and page operators together, as a serving program calls them, and calls that the other files do not make."""
from types import SimpleNamespace

import numpy as np
import pytest
import torch

import sparse_compressed_attention_gb300 as V
from oracle import cache_oracle as CO
from oracle import serving_oracle as S
from oracle import v4_oracle as O
from tests.helpers import np64
from tests.q4_cases import Q4Case
from tests.tree_cases import Case

pytestmark = pytest.mark.gpu

H, D, R, PAGE = 64, 512, 64, 16


def i32(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32).cuda()


class Server:
    """Three sequences over one pool of 4-bit pages; `keys` mirrors on the host what every cache row has to hold."""

    def __init__(self, lens, window=-1, blocks=12, pages=40, seed=0):
        self.g = torch.Generator().manual_seed(seed)
        self.lens, self.window = list(lens), window
        self.f = O.make_inv_freq(40000.0, R, 16.0, 4096, 32.0, 1.0)
        self.df = torch.from_numpy(self.f).cuda()
        self.w = (1 + 0.1 * torch.randn(D, generator=self.g)).cuda()
        self.table = torch.full((len(lens), blocks), -1, dtype=torch.int32, device="cuda")
        self.ref = torch.zeros(pages, dtype=torch.int32, device="cuda")
        self.cache = torch.zeros(pages, PAGE, V.v4_q4_row_bytes(D), dtype=torch.uint8, device="cuda")
        self.keys = [[] for _ in lens]

    def latents(self, n, pos):
        """n rows, normed and rotated on the GPU; checked against the oracle."""
        x = torch.randn(n, 1, D, generator=self.g).to(torch.bfloat16).cuda()
        k = torch.empty_like(x)
        V.v4_norm_rope_fwd(x, None, pos, self.df, k, q_w=self.w)
        ref, u = CO.norm_rope(np64(x), np64(self.w), pos.cpu().numpy(), self.f, D - R)
        assert np.all(np.abs(np64(k) - ref) <= 2.0 ** -8 * np.abs(ref) * 1.01 + 2.0 ** -18 * (np.abs(u) + 1))
        return k[:, 0]

    def store(self, k, slot):
        V.v4_cache_append_q4(k, slot, self.cache)
        rows = CO.q4_pack(np64(k))
        got = self.cache.view(-1, self.cache.shape[-1])[slot.long()].cpu().numpy()
        assert np.array_equal(got, rows)
        return CO.q4_unpack(rows, D)

    def prompt(self):
        V.v4_pages_alloc(self.table, self.ref, i32(self.lens), PAGE)
        for b, n in enumerate(self.lens):
            u = np.arange(n)
            t = self.table[b].cpu().numpy()
            values = self.store(self.latents(n, i32(u)), i32(t[u // PAGE] * PAGE + u % PAGE))
            self.keys[b] = list(values)

    def step(self, parents, graph=False):
        """Drafted trees of every sequence: attention of their nodes against the oracle's."""
        B, nodes = len(self.lens), [len(p) for p in parents]
        begin, n = np.concatenate([[0], np.cumsum(nodes)]), sum(nodes)
        V.v4_pages_alloc(self.table, self.ref, i32([a + b for a, b in zip(self.lens, nodes)]), PAGE, have=i32(self.lens))
        plan, pos, slot = (torch.empty(n, *d, dtype=torch.int32, device="cuda") for d in ((8,), (), ()))
        V.v4_tree_plan(i32(begin), i32(self.lens), i32(np.concatenate(parents)), plan, pos=pos, slot=slot, block_table=self.table,
                       page_size=PAGE, n_slots=self.cache.shape[0] * PAGE)
        drafted = self.store(self.latents(n, pos), slot)
        q = torch.randn(n, H, D, generator=self.g).to(torch.bfloat16).cuda()
        sink = torch.randn(H, generator=self.g).cuda()
        cfg = V.make_config(B, 1, H, D, R, window=self.window)
        o, lse = torch.zeros(n, H, D, dtype=torch.bfloat16, device="cuda"), torch.zeros(n, H, device="cuda")
        x = dict(q=q, plan=plan, tok_cache=self.cache, tok_table=self.table, sink=sink, inv_freq=self.df)
        ws = V.alloc_tree_workspace(cfg, n)
        V.v4_tree_mqa_fwd_q4(cfg, x, o, lse, ws)
        plan_ref, _ = S.tree_plan(begin, self.lens, np.concatenate(parents), n)
        now = [self.keys[b] + list(drafted[begin[b]:begin[b + 1]]) for b in range(B)]
        ref = S.tree_mqa(np64(q), plan_ref, lambda b, u: now[b][u], None, None, np64(sink), self.f, 0, self.window, 0, D ** -0.5,
                         np.zeros((n, H, D)), np.zeros((n, H)))
        ns = SimpleNamespace(dt=torch.bfloat16, scale=D ** -0.5, D=D, lens=self.lens, plan_ref=plan_ref)
        Case.check(ns, o, lse, ref)
        return now, begin

    def accept(self, now, accepted):
        """The accepted nodes of each sequence become its next tokens; pages that nothing needs go back."""
        wide = max(1, max(len(a) for a in accepted))
        keep = np.zeros((len(accepted), wide))
        for b, a in enumerate(accepted):
            keep[b, :len(a)] = a
        V.v4_pages_compact(self.cache, self.table, i32(self.lens), i32([len(a) for a in accepted]), i32(keep))
        for b, a in enumerate(accepted):
            self.keys[b] = now[b][:self.lens[b]] + [now[b][self.lens[b] + j] for j in a]
            self.lens[b] = len(self.keys[b])
        V.v4_pages_free(self.table, self.ref, PAGE, hi=i32(self.lens))

    def check_cache(self):
        for b, rows in enumerate(self.keys):
            u = np.arange(len(rows))
            t = self.table[b].cpu().numpy()
            out = torch.empty(len(rows), D, device="cuda")
            V.v4_cache_read_q4(self.cache, i32(t[u // PAGE] * PAGE + u % PAGE), out)
            assert np.array_equal(np64(out), np.array(rows).reshape(len(rows), D))
            assert (t[-(-len(rows) // PAGE):] == -1).all()
        held = self.table[self.table >= 0].cpu().numpy()
        assert np.array_equal(np.bincount(held, minlength=self.ref.numel()), self.ref.cpu().numpy())


@pytest.mark.parametrize("window", [-1, 20])
def test_serving_as_used(window):
    """Prompt, drafted trees, acceptance, beams of the result, a further step of the beams."""
    s = Server([37, 16, 1], window=window, seed=1)
    s.prompt()
    now, _ = s.step([[-1, 0, 0, 1, 3, 2], [-1, 0], [-1, -1, 1]])
    s.accept(now, [[0, 1, 3, 4], [], [1, 2]])
    s.check_cache()
    # two beams of sequence 0, one of sequence 2, cut two tokens back
    src, lens = [0, 0, 2], [s.lens[0], s.lens[0], s.lens[2] - 2]
    beams = torch.full_like(s.table, -1)
    copies, lack = torch.zeros(3, 3, dtype=torch.int32, device="cuda"), i32([5])
    V.v4_pages_fork(s.table, i32(src), i32(lens), beams, s.ref, PAGE, copies, lack=lack)
    V.v4_pages_copy(s.cache, copies)
    V.v4_pages_free(s.table, s.ref, PAGE)
    assert int(lack) == 0
    s.table, s.keys, s.lens = beams, [list(s.keys[b][:n]) for b, n in zip(src, lens)], lens
    s.check_cache()
    now, _ = s.step([[-1], [-1, 0], [-1]])          # the beams of one sequence go different ways
    s.accept(now, [[0], [0, 1], [0]])
    s.check_cache()
    now, _ = s.step([[-1], [-1], [-1]])
    assert V.v4_get_device_status() == 0


def test_a_captured_step_replays():
    """Pages given, latents normed, rotated and stored, attention, release: captured once and replayed over new inputs."""
    c = Q4Case([300, 60], [1, 1], window=-1, seed=5)
    x = c.device_inputs()
    ws = V.alloc_tree_workspace(c.cfg, c.n)
    lat = torch.randn(c.n, 1, D, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16).cuda()
    k, o, lse = torch.empty_like(lat), torch.zeros(c.n, H, D, dtype=torch.bfloat16, device="cuda"), torch.zeros(c.n, H, device="cuda")
    table, ref = torch.full((2, 8), -1, dtype=torch.int32, device="cuda"), torch.zeros(20, dtype=torch.int32, device="cuda")
    need, lack = i32([100, 30]), i32([0])
    f = torch.from_numpy(c.f).cuda()

    def step():
        V.v4_pages_alloc(table, ref, need, 16, lack=lack)
        V.v4_norm_rope_fwd(lat, None, c.pos, f, k)
        V.v4_cache_append_q4(k[:, 0], c.slot, x["tok_cache"])
        V.v4_tree_mqa_fwd_q4(c.cfg, x, o, lse, ws)
    step()
    torch.cuda.synchronize()
    first = table.clone(), o.clone(), lse.clone()
    V.v4_pages_free(table, ref, 16)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(2):
        o.zero_(), table.fill_(-1), ref.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(table, first[0]) and torch.equal(o, first[1]) and torch.equal(lse, first[2])
    lat.mul_(-1)
    graph.replay()
    torch.cuda.synchronize()
    assert not torch.equal(o, first[1]) and V.v4_get_device_status() == 0


def test_gradients_captured_and_eager_share_nothing():
    """Two graphs with a workspace each, an eager call between their replays."""
    g = torch.Generator().manual_seed(3)
    q, dy = (torch.randn(300, 8, 128, generator=g).cuda() for _ in range(2))
    pos, f = torch.arange(300, dtype=torch.int32).cuda(), torch.rand(32, generator=g).cuda()
    outs = [(torch.empty_like(q), torch.empty(128, device="cuda"), V.alloc_norm_rope_workspace(128)) for _ in range(3)]

    def call(i, stream=None):
        dq, dw, ws = outs[i]
        V.v4_norm_rope_bwd(q, None, dy, None, pos, f, dq, dq_w=dw, workspace=ws, stream=stream)
    call(0)
    torch.cuda.synchronize()
    want = outs[0][0].clone(), outs[0][1].clone()
    graphs = []
    for i in (1, 2):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            call(i)
    streams = [torch.cuda.Stream() for _ in graphs]
    for dq, dw, _ in outs:
        dq.zero_(), dw.zero_()
    torch.cuda.synchronize()
    for _ in range(3):
        for st, gr in zip(streams, graphs):
            with torch.cuda.stream(st):
                gr.replay()
        call(0)
    torch.cuda.synchronize()
    for dq, dw, _ in outs:
        assert torch.equal(dq, want[0]) and torch.equal(dw, want[1])


def test_calls_on_a_stream_of_their_own():
    x = torch.randn(64, 1, D, generator=torch.Generator().manual_seed(4)).to(torch.bfloat16).cuda()
    pos, f, slot = torch.arange(64, dtype=torch.int32).cuda(), torch.rand(32).cuda(), torch.arange(64, dtype=torch.int32).cuda()
    want, got = [], []
    for st, res in ((None, want), (torch.cuda.Stream(), got)):
        k, cache, out = torch.empty_like(x), torch.zeros(64, 288, dtype=torch.uint8, device="cuda"), torch.empty(64, D, device="cuda")
        torch.cuda.synchronize()
        V.v4_norm_rope_fwd(x, None, pos, f, k, stream=st)
        V.v4_cache_append_q4(k[:, 0], slot, cache, stream=st)
        V.v4_cache_read_q4(cache, slot, out, stream=st)
        torch.cuda.synchronize()
        res += [k, cache, out]
    assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_offsets_beyond_32_bits():
    """A cache of 4.3 GB: rows at its far end written, read, copied and moved together."""
    pages, page = 235000, 64
    cache = torch.empty(pages, page, 288, dtype=torch.uint8, device="cuda")
    last = pages * page - 1
    x = torch.randn(3, D, generator=torch.Generator().manual_seed(5)).cuda()
    slot = i32([last, last - 1, last - page])
    V.v4_cache_append_q4(x, slot, cache)
    out = torch.empty_like(x)
    V.v4_cache_read_q4(cache, slot, out)
    assert np.array_equal(np64(out), CO.q4_unpack(CO.q4_pack(np64(x)), D))
    V.v4_pages_copy(cache, i32([[pages - 1, 3, page], [pages - 2, pages - 5, page]]))
    assert torch.equal(cache[3], cache[pages - 1]) and torch.equal(cache[pages - 5], cache[pages - 2])
    V.v4_pages_compact(cache, i32([[pages - 1]]), i32([0]), i32([2]), i32([[page - 2, page - 1]]))
    assert torch.equal(cache[pages - 1, :2], cache[3, page - 2:])
    table = i32([[pages - 2, pages - 1]])
    plan = torch.empty(1, 8, dtype=torch.int32, device="cuda")
    V.v4_tree_plan(i32([0, 1]), i32([2 * page - 1]), None, plan)
    q, f = torch.randn(1, H, D).to(torch.bfloat16).cuda(), torch.rand(32).cuda()
    cfg = V.make_config(1, 1, H, D, R, window=2)
    res = []
    for c, t in ((cache, table), (cache[pages - 2:].clone(), i32([[0, 1]]))):
        o, lse = torch.empty_like(q), torch.empty(1, H, device="cuda")
        V.v4_tree_mqa_fwd_q4(cfg, dict(q=q, plan=plan, tok_cache=c, tok_table=t, inv_freq=f), o, lse, V.alloc_tree_workspace(cfg, 1))
        res.append((o, lse))
    assert torch.equal(res[0][0], res[1][0]) and torch.equal(res[0][1], res[1][1]) and V.v4_get_device_status() == 0


def test_strided_norms_beyond_32_bits():
    base = torch.empty((1 << 31) + 4096, dtype=torch.bfloat16, device="cuda")
    far = base.as_strided((2, 1, 64), (1 << 31, 64, 1))
    x = torch.randn(2, 1, 64, generator=torch.Generator().manual_seed(6)).to(torch.bfloat16).cuda()
    far.copy_(x)
    pos, f = i32([3, 9]), torch.rand(8).cuda()
    want = torch.empty_like(x)
    V.v4_norm_rope_fwd(x, None, pos, f, want)
    V.v4_norm_rope_fwd(far, None, pos, f, far)
    assert torch.equal(far.contiguous(), want)


@pytest.mark.parametrize("op", ["norm", "norm_rope_bwd", "pages", "pages_copy", "pages_compact", "q4"])
def test_stages_are_timed(op):
    from sparse_compressed_attention_gb300 import _lib
    x = torch.randn(2, 1, 64).cuda()
    pos, f, t, ref = i32([0, 1]), torch.rand(8).cuda(), i32([[-1, -1]]), i32([0, 0, 0])
    cache = torch.zeros(2, 2, 48, dtype=torch.uint8, device="cuda")
    _lib.lib().v4_profile_enable(1)
    if op == "norm":
        V.v4_norm_rope_fwd(x, None, pos, f, x)
    elif op == "norm_rope_bwd":
        V.v4_norm_rope_bwd(x, None, x, None, pos, f, torch.empty_like(x), workspace=V.alloc_norm_rope_workspace(64))
    elif op == "pages":
        V.v4_pages_alloc(t, ref, i32([3]), 2)
        V.v4_pages_free(t, ref, 2)
    elif op == "pages_copy":
        V.v4_pages_copy(cache, i32([[0, 1, 2]]))
    elif op == "pages_compact":
        V.v4_pages_compact(cache, i32([[0, 1]]), i32([0]), i32([1]), i32([[2]]))
    else:
        V.v4_cache_append_q4(x[:, 0], i32([0, 1]), cache)
        V.v4_cache_read_q4(cache, i32([0, 1]), x[:, 0])
    _lib.lib().v4_profile_enable(0)
    kinds = [k for k, ms in V.v4_profile_records() if ms > 0]
    assert kinds == {"norm": ["norm_rope"], "pages": ["pages"] * 2, "q4": ["cache_append_q4", "cache_read_q4"]}.get(op, [op])
