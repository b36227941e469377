"""Calls of the serving operators that a program may make and the other files do not."""
import ctypes
import threading

import numpy as np
import pytest
import torch

import sparse_compressed_attention_gb300 as V
from oracle import serving_oracle as S
from sparse_compressed_attention_gb300 import _lib
from tests.helpers import np64
from tests.tree_cases import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["whole", "few_parts", "many_parts", "nothing_to_see", "f32", "bf16_cuda_cores"])
def test_sinks_that_are_no_numbers(kind):
    """A NaN sink makes its head NaN, one of +inf takes all of it (o = 0, lse = +inf), one of -inf is none; the other heads
    and rows are as without."""
    kw = {"whole": dict(lens=[20] * 100, nodes=[1] * 100),
          "few_parts": dict(lens=[700, 30], nodes=[1, 1], window=-1),
          "many_parts": dict(lens=[20000], nodes=[1], window=-1),
          "nothing_to_see": dict(lens=[0, 9], nodes=[1, 1], window=0, ratio=128),
          "f32": dict(lens=[300, 40], nodes=[2, 1], H=9, D=64, R=16, dt=torch.float32),
          "bf16_cuda_cores": dict(lens=[300, 40], nodes=[2, 1], H=9)}[kind]
    c = Case(sink=True, seed=31, **kw)
    x = c.device_inputs()
    o0, l0 = c.run(x)
    x["sink"] = x["sink"].clone()
    x["sink"][1], x["sink"][4], x["sink"][6] = float("nan"), float("inf"), float("-inf")
    o, lse = c.run(x)
    assert torch.isnan(o[:, 1].float()).all() and torch.isnan(lse[:, 1]).all()
    assert (o[:, 4] == 0).all() and (lse[:, 4] == float("inf")).all()
    rest = [h for h in range(c.H) if h not in (1, 4, 6)]
    assert torch.equal(o[:, rest], o0[:, rest]) and torch.equal(lse[:, rest], l0[:, rest])
    none = c.run({k: v for k, v in x.items() if k != "sink"})
    assert torch.equal(o[:, 6], none[0][:, 6]) and torch.equal(lse[:, 6], none[1][:, 6])
    assert V.v4_get_device_status() == 0


@pytest.mark.parametrize("half", [False, True])
def test_angles_keep_their_precision_at_every_part_of_a_turn(half):
    """Rows of ones and zeros come out as the cosines and sines themselves.

    The angle reaches sincospif within an eighth of a turn of a quarter, in half turns below 1/4: half a step of fp32 is
    2^-27 of them, pi 2^-27 as an angle.  The 64-bit fraction of a turn behind it is off by less than 2^-31 turns for
    tables up to 1.  sincospif is within one step (2^-23 relative at most), products with one and zero are exact."""
    rows, R = 4096, 64
    rng = np.random.default_rng(5)
    f = (10.0 ** rng.uniform(-6, 0, R // 2)).astype(np.float32)
    pos = rng.integers(-2 ** 31, 2 ** 31, rows).astype(np.int32)
    pos[:1024] = rng.integers(0, 4096, 1024)
    x = torch.zeros(rows, 1, R, device="cuda")
    out = torch.empty_like(x)
    first = slice(0, R // 2) if half else slice(0, R, 2)
    second = slice(R // 2, R) if half else slice(1, R, 2)
    x[..., first] = 1.0
    V.v4_rope(x, torch.from_numpy(pos).cuda(), torch.from_numpy(f).cuda(), out,
              layout=V.V4_ROPE_HALF if half else V.V4_ROPE_INTERLEAVED)
    phi = S.angles(pos, f)
    got = np64(out)[:, 0]
    for part, ref in ((first, np.cos(phi)), (second, np.sin(phi))):
        err = np.abs(got[:, part] - ref)
        allow = 2.0 ** -23 * np.abs(ref) + np.pi * 2.0 ** -27 + 2 * np.pi * 2.0 ** -31
        assert np.all(err <= allow), float((err / allow).max())


def library_call(call, stream):
    """The library function and the arguments of the last call that `call` makes on `stream`."""
    real, made = _lib.lib(), []

    class Spy:
        def __getattr__(self, name):
            fn = getattr(real, name)

            def go(*args):
                made.append((fn, args))
                return fn(*args)
            return go

    _lib._lib = Spy()
    try:
        call(stream)
    finally:
        _lib._lib = real
    return made[-1]


def at_once(*calls, times=20000):
    """Each call `times` times in a host thread and on a stream of its own, through the library alone; what was refused."""
    made, refused, done = [library_call(c, torch.cuda.Stream()) for c in calls], [], []
    gate = threading.Barrier(len(calls))

    def work(fn, args):
        torch.cuda.set_device(0)
        gate.wait()
        for _ in range(times):
            if fn(*args) != 0:
                refused.append(_lib.lib().v4_last_error().decode())
                return
        done.append(fn)

    threads = [threading.Thread(target=work, args=m) for m in made]
    torch.cuda.synchronize()
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert len(done) + len(refused) == len(calls)
    return refused


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_tree_calls_of_two_host_threads_with_other_widths(dt):
    cases = [Case([9], [1], H=3, D=512, R=64, dt=dt, seed=1), Case([5], [1], H=2, D=32, R=16, dt=dt, seed=2)]
    ins = [c.device_inputs() for c in cases]
    want = [c.run(x) for c, x in zip(cases, ins)]
    outs = [(torch.empty_like(o), torch.empty_like(s)) for o, s in want]
    ws = torch.empty(256, dtype=torch.uint8, device="cuda")

    def call(c, x, o, s):
        return lambda stream: V.v4_tree_mqa_fwd(c.cfg, x, o, s, ws, stream=stream)

    assert at_once(*(call(c, x, o, s) for c, x, (o, s) in zip(cases, ins, outs))) == []
    for (o, s), (wo, wl) in zip(outs, want):
        assert torch.equal(o, wo) and torch.equal(s, wl)


def sequence_call(op, big):
    """One call of an operator over a short sequence whose kernel takes much (or little) shared memory."""
    g = torch.Generator().manual_seed(int(big))
    f32 = lambda *shape: torch.randn(*shape, generator=g).cuda()        # noqa: E731
    D, R = (512, 64) if big else (32, 16)
    if op == "attention":
        cfg = V.make_config(1, 4, 2, D, R, window=4, dtype="f32", path=V.V4_PATH_SIMT)
        q, kv, f, o = f32(1, 4, 2, D), f32(1, 4, D), f32(R // 2).abs(), torch.empty(1, 4, 2, D, device="cuda")
        return lambda ws, s: V.v4_sparse_mqa_fwd(cfg, q, kv, None, None, None, f, o, None, ws, stream=s), cfg, o
    if op == "compressor":
        cfg = V.make_config(1, 64, 2, D, R, ratio=32, dtype="f32", path=V.V4_PATH_SIMT)
        kv, sc, ape, f = f32(1, 64, D), f32(1, 64, D), f32(32, D), f32(R // 2).abs()
        o = torch.empty(1, 2, D, device="cuda")
        return lambda ws, s: V.v4_compress(cfg, kv, sc, ape, None, f, D, 0, o, stream=s), cfg, o
    Hi, Di, n = (64, 128, 64) if big else (1, 16, 8)
    n = 400 if big else n
    cfg = V.make_config(1, n, 2, 32, 16, ratio=4, topk=4, Hi=Hi, Di=Di, dtype="f32", path=V.V4_PATH_SIMT)
    iq, ik, w, f = f32(1, n, Hi, Di), f32(1, n // 4, Di), f32(1, n, Hi), f32(8).abs()
    o = torch.empty(1, n, 4, dtype=torch.int32, device="cuda")
    return lambda ws, s: V.v4_indexer_topk(cfg, iq, 1, ik, w, f, o, None, ws, stream=s), cfg, o


@pytest.mark.parametrize("op", ["attention", "compressor", "indexer"])
def test_sequence_calls_of_two_host_threads_with_other_widths(op):
    made = [sequence_call(op, big) for big in (True, False)]
    ws = [V.alloc_workspace(cfg) for _, cfg, _ in made]
    want = []
    for (call, _, o), w in zip(made, ws):
        call(w, None)
        want.append(o.clone())
        o.zero_()

    def bound(call, w):
        return lambda stream: call(w, stream)

    assert at_once(*(bound(call, w) for (call, _, _), w in zip(made, ws))) == []
    for (_, _, o), wo in zip(made, want):
        assert torch.equal(o, wo)


def test_a_call_after_one_that_could_not_be_launched():
    """A launch that the runtime refuses (the legacy stream, while a blocking stream is captured) is reported by its own call
    and by no later one."""
    rt = ctypes.CDLL("libcudart.so.13")
    x = torch.randn(4, 2, 64).cuda()
    pos, f = torch.arange(4, dtype=torch.int32).cuda(), torch.rand(8).cuda()
    out, want = torch.empty_like(x), torch.empty_like(x)
    V.v4_rope(x, pos, f, want)
    torch.cuda.synchronize()
    stream, graph = ctypes.c_void_p(), ctypes.c_void_p()
    assert rt.cudaStreamCreate(ctypes.byref(stream)) == 0
    try:
        assert rt.cudaStreamBeginCapture(stream, 0) == 0
        with pytest.raises(V.V4Error, match="rotation kernel"):
            V.v4_rope(x, pos, f, out, stream=0)
    finally:
        rt.cudaStreamEndCapture(stream, ctypes.byref(graph))
        rt.cudaStreamDestroy(stream)
        rt.cudaGetLastError()
    V.v4_rope(x, pos, f, out)
    assert torch.equal(out, want)


@pytest.mark.parametrize("kind", ["tensor_cores", "cuda_cores"])
def test_stages_of_the_tree_attention_are_apart(kind):
    """The attention's record ends before the join's begins: records come in the order in which stages end."""
    c = Case([5000, 3], [1, 1], window=-1, seed=3) if kind == "tensor_cores" else Case([90], [2], H=3, seed=4)
    x = c.device_inputs()
    c.run(x)
    k, ms = ctypes.c_int32(), ctypes.c_float()
    L = _lib.lib()
    assert L.v4_profile_enable(1) == 0
    c.run(x)
    assert L.v4_profile_enable(0) == 0
    n = L.v4_profile_count()
    kinds = []
    for i in range(n):
        assert L.v4_profile_get(i, ctypes.byref(k), ctypes.byref(ms)) == 0 and ms.value > 0
        kinds.append(_lib.PROFILE_KINDS[k.value])
    assert kinds == (["tree_attention", "tree_join"] if kind == "tensor_cores" else ["tree_attention"])


def test_workspace_may_be_left_out_where_none_is_needed():
    c = Case([90, 7], [2, 1], H=3, D=64, R=16, seed=6)
    x = c.device_inputs()
    o, lse = c.run(x)
    o2, lse2 = torch.full_like(o, 3.0), torch.full_like(lse, 3.0)
    assert V.v4_tree_workspace_size(c.cfg, c.n) == 0
    V.v4_tree_mqa_fwd(c.cfg, x, o2, lse2, None)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    c = Case([90, 7], [2, 1], seed=6)
    with pytest.raises(V.V4Error, match="workspace"):
        V.v4_tree_mqa_fwd(c.cfg, c.device_inputs(), *(torch.empty(c.n, 64, *d, dtype=t, device="cuda") for d, t in
                                                      (((512,), torch.bfloat16), ((), torch.float32))), None)


@pytest.mark.parametrize("order", ["rows", "heads"])
def test_views_of_one_buffer_that_do_not_meet(order):
    """Two views that step alike are refused exactly where an element belongs to both."""
    pos, f = torch.arange(3, dtype=torch.int32).cuda(), torch.tensor([0.5, 0.01, 1.0, 0.3]).cuda()
    base = torch.randn(400, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    seen = [0, 0]
    for rows in (1, 2, 3):
        for heads in (1, 2, 3):
            inner = rows if order == "heads" else heads
            outer = heads if order == "heads" else rows
            for s_in in (8, 16, 24, 32):
                for s_out in ((inner - 1) * s_in + 8, (inner - 1) * s_in + 16, (inner - 1) * s_in + 40):
                    span = (outer - 1) * s_out + (inner - 1) * s_in + 8
                    st = (s_in, s_out) if order == "heads" else (s_out, s_in)
                    at = np.array([t * st[0] + h * st[1] + c for t in range(rows) for h in range(heads) for c in range(8)])
                    for shift in range(-64, 72, 8):
                        if not shift or 100 + abs(shift) + span > 400 or 100 + shift < 0:
                            continue
                        buf = base.clone()
                        x = buf.as_strided((rows, heads, 8), (*st, 1), 100 - 100 % 8)
                        out = buf.as_strided((rows, heads, 8), (*st, 1), 100 - 100 % 8 + shift)
                        meet = np.intersect1d(at, at + shift).size > 0
                        seen[meet] += 1
                        if meet:
                            with pytest.raises(V.V4Error, match="overlap"):
                                V.v4_rope(x, pos[:rows], f, out)
                            continue
                        want = torch.empty(rows, heads, 8, dtype=torch.bfloat16, device="cuda")
                        V.v4_rope(x.clone(memory_format=torch.contiguous_format), pos[:rows], f, want)
                        V.v4_rope(x, pos[:rows], f, out)
                        assert torch.equal(out, want), (rows, heads, st, shift)
    assert min(seen) > 100
