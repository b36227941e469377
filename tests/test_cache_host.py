"""Refusals of the norm, 4-bit cache and page entry points on the host (no kernel runs), and CPU pins of their oracle."""
import ctypes as C
from fractions import Fraction

import numpy as np
import pytest
import torch

from oracle import cache_oracle as CO
from oracle import serving_oracle as S
from oracle import v4_oracle as O
from sparse_compressed_attention_gb300 import _lib as L
from sparse_compressed_attention_gb300 import build as B


@pytest.fixture(scope="module")
def lib():
    B.build()
    return L.lib()


def refused(lib, st, status, text):
    assert st == status, (st, lib.v4_last_error().decode())
    assert text in lib.v4_last_error().decode()


def part(base, **over):
    a = dict(x=base, w=16, dy=base + (1 << 20), out=base + (2 << 20), dw=16, heads=2)
    for n in ("x", "dy", "out"):
        a[n + "_row_stride"], a[n + "_head_stride"] = 128, 64
    a.update(over)
    p = L.v4_norm_rope_part()
    for n, v in a.items():
        setattr(p, n, v)
    return p


def norm(lib, grad=False, q=None, k=None, ws=(256, 1 << 30), **over):
    a = dict(rows=4, dim=64, pos=16, f=16, R=16, begin=48, layout=0, eps=1e-6, dtype=1)
    a.update(over)
    head = (None if q == 0 else C.byref(q or part(1 << 24)), None if k is None else C.byref(k), a["rows"], a["dim"], a["pos"],
            a["f"], a["R"], a["begin"], a["layout"], a["eps"], a["dtype"])
    return lib.v4_norm_rope_bwd(*head, *ws, None) if grad else lib.v4_norm_rope_fwd(*head, None)


@pytest.mark.parametrize("grad", [False, True])
@pytest.mark.parametrize("over,status,text", [
    (dict(q=0), 1, "q struct"), (dict(rows=-1), 1, "rows"), (dict(dim=60), 1, "dim"), (dict(dim=1032), 2, "1024"),
    (dict(R=12), 1, "rope_dim"), (dict(R=24, layout=1), 1, "rope_dim"), (dict(begin=52), 1, "rope_begin"),
    (dict(begin=56), 1, "rope_begin"), (dict(layout=2), 1, "layout"), (dict(dtype=3), 1, "dtype"),
    (dict(eps=-1.0), 1, "eps"), (dict(eps=float("nan")), 1, "eps"), (dict(eps=float("inf")), 1, "eps"),
    (dict(pos=None), 1, "pos"), (dict(pos=20), 1, "aligned"), (dict(f=None), 1, "inv_freq"), (dict(rows=1 << 30), 2, "2^30"),
    (dict(q=part(1 << 24, x=None)), 1, "q.x is NULL"), (dict(q=part(1 << 24, x=(1 << 24) + 8)), 1, "aligned"),
    (dict(q=part(1 << 24, out=None)), 1, "q.out"), (dict(q=part(1 << 24, heads=0)), 1, "q.heads"),
    (dict(q=part(1 << 24, w=20)), 1, "weight"), (dict(k=part(1 << 28, heads=70000)), 1, "k.heads"),
    (dict(q=part(1 << 24, x_row_stride=132)), 1, "q.x row stride"), (dict(q=part(1 << 24, out_head_stride=-64)), 1, "head stride"),
    (dict(q=part(1 << 24, out_head_stride=0)), 1, "overlap"), (dict(q=part(1 << 24, out_row_stride=64)), 1, "overlap"),
    (dict(q=part(1 << 24, x_row_stride=1 << 40), rows=1 << 20), 1, "reaches"),
    (dict(q=part(1 << 24, out=(1 << 24) + 128)), 1, "not the same tensor"),
    (dict(q=part(1 << 24, out=1 << 24, out_row_stride=256)), 1, "not the same tensor"),
    (dict(k=part(1 << 28, out=(1 << 28) + 64, dw=4096)), 1, "overlaps an input"),
    (dict(q=part(1 << 24), k=part(1 << 28, out=(1 << 24) + (2 << 20), dw=4096)), 1, "the outputs overlap"),
    (dict(q=part(1 << 24), k=part(1 << 28, out=1 << 24, dw=4096)), 1, "other part")])
def test_norm_refusals(lib, grad, over, status, text):
    refused(lib, norm(lib, grad, **over), status, text)


def test_norm_gradient_refusals(lib):
    for over, status, text in ((dict(q=part(1 << 24, dy=None)), 1, "q.dy"), (dict(q=part(1 << 24, dw=24)), 1, "weight gradient"),
                               (dict(k=part(1 << 28, dw=32)), 1, "weight gradients overlap"), (dict(ws=(256, 100)), 3, "needed"), (dict(ws=(None, 1 << 30)), 3, "NULL"),
                               (dict(ws=(128, 1 << 30)), 3, "256-byte"),
                               (dict(q=part(1 << 24, out=(1 << 24) + (1 << 20) + 64)), 1, "not the same tensor")):
        refused(lib, norm(lib, True, **over), status, text)
    n = C.c_size_t(0)
    for dim in (0, 60, 1032):
        refused(lib, lib.v4_norm_rope_workspace_size(dim, C.byref(n)), 1, "dim")
    refused(lib, lib.v4_norm_rope_workspace_size(64, None), 1, "bytes")


def test_norm_of_no_rows_does_nothing(lib):
    assert norm(lib, rows=0, pos=None, q=part(1 << 24, x=None, out=None)) == L.V4_OK


def append(lib, **over):
    a = dict(x=1 << 24, rows=4, dim=64, xr=64, slot=16, n=32, dtype=1, cache=1 << 28)
    a.update(over)
    return lib.v4_cache_append_q4(a["x"], a["rows"], a["dim"], a["xr"], a["slot"], a["n"], a["dtype"], a["cache"], None)


def read(lib, **over):
    a = dict(cache=1 << 28, n=32, slot=16, rows=4, dim=64, dtype=1, out=1 << 24, yr=64)
    a.update(over)
    return lib.v4_cache_read_q4(a["cache"], a["n"], a["slot"], a["rows"], a["dim"], a["dtype"], a["out"], a["yr"], None)


@pytest.mark.parametrize("call,over,text", [
    (append, dict(x=None), "x is NULL"), (append, dict(x=(1 << 24) + 8), "aligned"), (append, dict(slot=None), "slot"),
    (append, dict(cache=None), "cache"), (append, dict(dim=48), "dim"), (append, dict(dim=8224), "dim"),
    (append, dict(dtype=2), "dtype"), (append, dict(xr=60), "stride"), (append, dict(rows=-1), "rows"),
    (append, dict(rows=(1 << 24) + 1), "rows"), (append, dict(rows=1 << 24, dim=8192), "2^35"),
    (append, dict(n=1 << 31), "n_slots"), (append, dict(cache=(1 << 24) + 256), "overlap"),
    (read, dict(out=None), "out is NULL"), (read, dict(out=(1 << 28) + 64), "overlap"), (read, dict(yr=32), "overlap"),
    (read, dict(dim=40), "dim"), (read, dict(slot=20), "aligned")])
def test_q4_refusals(lib, call, over, text):
    refused(lib, call(lib, **over), L.V4_ERR_INVALID_ARG, text)


def test_q4_sizes(lib):
    for dim, n in ((32, 32), (64, 48), (96, 64), (128, 80), (512, 288), (1024, 576), (8192, 4608)):
        assert L.v4_q4_row_bytes(dim) == n == CO.q4_row_bytes(dim) == L._q4_width(dim)
    with pytest.raises(L.V4Error, match="dim"):
        L.v4_q4_row_bytes(48)
    assert append(lib, rows=0, x=None) == L.V4_OK and read(lib, rows=0, out=None) == L.V4_OK


def test_q4_attention_refusals(lib):
    def tree(cfg=None, **over):
        v = L.v4_tree_inputs()
        for n in ("q", "plan", "tok_cache", "tok_table", "ent_cache", "ent_table", "ent_len", "idx", "inv_freq"):
            setattr(v, n, 32)
        v.tok_slots = v.ent_slots = 640
        v.n_rows, v.tok_blocks, v.tok_page, v.ent_blocks, v.ent_page = 3, 10, 64, 10, 64
        for n, x in over.items():
            setattr(v, n, x)
        cfg = cfg or L.make_config(2, 1, 64, 512, 64, ratio=4, window=128, topk=512)
        return lib.v4_tree_mqa_fwd_q4(C.byref(cfg), C.byref(v), 16, 16, 256, 1 << 32, None)
    for over, text in ((dict(q=None), "q is NULL"), (dict(tok_cache=48), "32-byte"), (dict(ent_cache=16), "32-byte"),
                       (dict(tok_cache=None), "tok_cache"), (dict(idx=None), "idx"), (dict(tok_page=0), "tok_page"),
                       (dict(n_rows=-1), "n_rows")):
        refused(lib, tree(**over), L.V4_ERR_INVALID_ARG, text)
    refused(lib, tree(L.make_config(2, 1, 32, 512, 64, window=128, path=L.V4_PATH_TC)), L.V4_ERR_UNSUPPORTED, "tensor-core")
    assert tree(n_rows=0, q=None) == L.V4_OK


def pages(lib, op, **over):
    a = dict(n=2, table=1 << 20, blocks=8, page=16, have=None, need=16, ref=16, pages=64, lack=None, B=2, src=16, length=16,
             out=1 << 24, out_blocks=8, copies=16, lo=None, hi=None, cache=1 << 28, layers=2, stride=64 * 16 * 288, row=288,
             base=16, count=16, keep=16, width=4)
    a.update(over)
    g = a.get
    if op == "alloc":
        return lib.v4_pages_alloc(g("n"), g("table"), g("blocks"), g("page"), g("have"), g("need"), g("ref"), g("pages"), g("lack"), None)
    if op == "fork":
        return lib.v4_pages_fork(g("B"), g("table"), g("blocks"), g("n"), g("src"), g("length"), g("out"), g("out_blocks"), g("page"),
                                 g("ref"), g("pages"), g("copies"), g("lack"), None)
    if op == "free":
        return lib.v4_pages_free(g("n"), g("table"), g("blocks"), g("page"), g("lo"), g("hi"), g("ref"), g("pages"), None)
    if op == "copy":
        return lib.v4_pages_copy(g("cache"), g("layers"), g("stride"), g("pages"), g("page"), g("row"), g("copies"), g("n"), None)
    return lib.v4_pages_compact(g("cache"), g("layers"), g("stride"), g("pages"), g("page"), g("row"), g("n"), g("table"), g("blocks"),
                                g("base"), g("count"), g("keep"), g("width"), None)


@pytest.mark.parametrize("op,over,status,text", [
    ("alloc", dict(n=-1), 1, "sequences"), ("alloc", dict(n=8193), 2, "8192"), ("alloc", dict(table=None), 1, "table"),
    ("alloc", dict(blocks=0), 1, "blocks"), ("alloc", dict(page=0), 1, "page_size"), ("alloc", dict(need=None), 1, "need"),
    ("alloc", dict(have=20), 1, "have"), ("alloc", dict(ref=None), 1, "ref"), ("alloc", dict(pages=0), 1, "pages"),
    ("alloc", dict(lack=20), 1, "lack"), ("alloc", dict(n=8192, blocks=1 << 20), 1, "entries"),
    ("fork", dict(n=8193), 2, "8192"), ("fork", dict(src=None), 1, "src"), ("fork", dict(length=None), 1, "len"),
    ("fork", dict(copies=None), 1, "copies"), ("fork", dict(out=None), 1, "out_table"), ("fork", dict(out=(1 << 20) + 32), 1, "overlap"),
    ("fork", dict(out_blocks=0), 1, "blocks"), ("free", dict(table=24), 1, "aligned"), ("free", dict(lo=8), 1, "lo"),
    ("free", dict(ref=None), 1, "ref"), ("copy", dict(cache=None), 1, "cache"), ("copy", dict(layers=0), 1, "layers"),
    ("copy", dict(row=24), 1, "row_bytes"), ("copy", dict(stride=100), 1, "layer_stride"), ("copy", dict(stride=16), 1, "layer_stride"),
    ("copy", dict(copies=None), 1, "copies"), ("copy", dict(n=-1), 1, "copies"), ("copy", dict(page=1 << 24), 1, "2^30"),
    ("copy", dict(pages=1 << 28), 1, "2^31"), ("compact", dict(base=None), 1, "base"), ("compact", dict(count=None), 1, "count"),
    ("compact", dict(keep=None), 1, "keep"), ("compact", dict(width=-1), 1, "keep"), ("compact", dict(table=None), 1, "table")])
def test_page_refusals(lib, op, over, status, text):
    refused(lib, pages(lib, op, **over), status, text)


def test_calls_that_have_nothing_to_do(lib):
    assert pages(lib, "free", n=0, table=None) == L.V4_OK
    assert pages(lib, "copy", n=0, copies=None) == L.V4_OK
    assert pages(lib, "compact", n=0) == L.V4_OK and pages(lib, "compact", width=0, keep=None) == L.V4_OK


def test_binding_refuses_host_tensors_and_wrong_shapes():
    x = torch.zeros(2, 2, 64)
    with pytest.raises(ValueError, match="CUDA"):
        L.v4_norm_rope_fwd(x, None, None, None, x)
    with pytest.raises(ValueError, match="CUDA"):
        L.v4_cache_append_q4(x[0], torch.zeros(2, dtype=torch.int32), torch.zeros(4, 48, dtype=torch.uint8))
    with pytest.raises(ValueError, match="CUDA"):
        L.v4_pages_alloc(torch.zeros(2, 2, dtype=torch.int32), None, None, 16)
    with pytest.raises(TypeError, match="tensor"):
        L.v4_pages_copy(None, None)


# ---------------------------------------------------------------------------
# the oracle
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("half", [False, True])
def test_norm_oracle_gradients_against_differences(half):
    """Central differences in fp64: h = 1e-5 leaves 1e-10 of the third derivative and 1e-11 of rounding."""
    rng = np.random.default_rng(1)
    x, w, dy = rng.standard_normal((2, 2, 32)), rng.standard_normal(32), rng.standard_normal((2, 2, 32))
    f, pos = O.make_inv_freq(10000.0, 16, 1.0, 0), np.array([3, 77])
    dx, dw, _, _, _ = CO.norm_rope_grad(x, w, dy, pos, f, 8, half, 1e-3)

    def total(a, b):
        return float((CO.norm_rope(a, b, pos, f, 8, half, 1e-3)[0] * dy).sum())
    h = 1e-5
    for i in ((0, 0, 3), (1, 1, 12), (0, 1, 20), (1, 0, 31)):
        a, b = x.copy(), x.copy()
        a[i] += h
        b[i] -= h
        assert abs((total(a, w) - total(b, w)) / (2 * h) - dx[i]) < 1e-7
    for c in (0, 9, 30):
        a, b = w.copy(), w.copy()
        a[c] += h
        b[c] -= h
        assert abs((total(x, a) - total(x, b)) / (2 * h) - dw[c]) < 1e-7


def test_norm_oracle_is_the_rotation_of_unit_rms_rows():
    rng = np.random.default_rng(2)
    x, f, pos = rng.standard_normal((3, 2, 32)) * 5, O.make_inv_freq(10000.0, 16, 1.0, 0), np.array([0, 1, 9])
    y, u = CO.norm_rope(x, None, pos, f, 16, eps=0.0)
    assert np.allclose((y * y).mean(-1), 1.0) and np.allclose(u, x / np.sqrt((x * x).mean(-1, keepdims=True)))
    assert np.allclose(S.rope(y, pos, f, 16, inverse=True), u) and np.array_equal(y[0], u[0])


def test_q4_oracle_scales_and_codes():
    assert CO.q4_scale(0) == Fraction(1, 2 ** 20) and CO.q4_scale(255) == 3840 and CO.q4_scale(160) == 1
    every = [CO.q4_scale(b) for b in range(256)]
    assert every == sorted(set(every))
    for b in range(1, 255):                                       # a scale is its own nearest, ties go to the even significand
        assert CO.q4_scale_byte(float(7 * every[b])) == b
        mid = float(7 * (every[b] + every[b + 1]) / 2)
        assert CO.q4_scale_byte(mid) == b + b % 2
        assert CO.q4_scale_byte(np.nextafter(mid, np.inf)) == b + 1 and CO.q4_scale_byte(np.nextafter(mid, 0)) == b
    assert CO.q4_scale_byte(0.0) == 0 and CO.q4_scale_byte(1e30) == 255
    x = np.zeros((1, 32))
    x[0, :15] = np.arange(-7, 8)
    x[0, 16] = 7 * 1.0625                                         # halfway between scales 1 and 1.125: the even significand, 8
    x[0, 17], x[0, 18], x[0, 19] = 0.5, 1.5, -2.5                 # halves go to even codes
    rows = CO.q4_pack(x)
    v = CO.q4_unpack(rows, 32)
    assert np.array_equal(v[0, :16], x[0, :16])
    assert list(v[0, 16:20]) == [7.0, 0.0, 2.0, -2.0] and rows.shape[1] == 32 and rows[0, 16] == rows[0, 17] == 160
    word = int.from_bytes(rows[0, :4].tobytes(), "little")        # values -7 .. 0: codes 1 .. 8
    assert [(word >> (4 * i)) & 15 for i in range(8)] == [1, 3, 5, 7, 2, 4, 6, 8]


def test_q4_values_are_exact_in_bf16():
    rows = np.zeros((256, 32), np.uint8)
    rows[:, :16] = np.random.default_rng(0).integers(0, 256, (256, 16))
    rows[:, 16], rows[:, 17] = np.arange(256), np.arange(256)[::-1]
    v = torch.from_numpy(np.ascontiguousarray(CO.q4_unpack(rows, 32)))
    assert torch.equal(v.to(torch.bfloat16).double(), v)


def test_quotients_by_markstein_and_by_division_round_alike():
    """The kernel's quotient, in fp32 arithmetic here: one step of the exact remainder with the rounded reciprocal."""
    rng = np.random.default_rng(3)
    f32 = np.float32
    for m in range(8, 16):
        s = f32(m) * f32(2.0) ** f32(int(rng.integers(-12, 5)))
        k = np.arange(-16, 15) * 0.5
        x = np.concatenate([rng.uniform(-8, 7, 20000), k]) * float(s)
        x = x.astype(f32)
        x = np.concatenate([x, np.nextafter(x, f32(np.inf)), np.nextafter(x, f32(-np.inf))])
        x = np.clip(x, f32(-8) * s, f32(7) * s)
        inv = f32(1) / s
        q0 = (x * inv).astype(f32)
        rem = (x.astype(np.float64) - q0.astype(np.float64) * float(s)).astype(f32)      # exact in 64 bits, one rounding
        q = (q0.astype(np.float64) + rem.astype(np.float64) * float(inv)).astype(f32)
        assert np.array_equal(np.rint(q), np.rint(x / s))
        assert np.array_equal(np.rint(x / s), [float(round(Fraction(float(a)) / Fraction(float(s)))) for a in x])


def test_page_oracle():
    p = CO.Pages([[-1, -1, -1], [-1, -1, -1]], [0, 1, 0, 0, 0], 4)
    assert p.alloc([0, 0], [5, 8]) == 0
    assert p.table == [[0, 2, -1], [3, 4, -1]] and p.ref == [1, 1, 1, 1, 1]
    p.free([4, 0], [5, 4])
    assert p.table == [[-1, 2, -1], [3, -1, -1]] and p.ref == [0, 1, 1, 1, 0]
    rows, copies, lack = p.fork([1, 1, 0], [3, 4, 6], 3)
    assert rows == [[0, -1, -1], [3, -1, -1], [-1, 4, -1]] and copies == [[3, 0, 3], [-1, -1, 0], [2, 4, 2]] and lack == 0
    c = np.arange(5 * 4).reshape(1, 5, 4, 1)
    got = CO.compact(c, [[3, 1]], 4, [1], [[0, 2, 5]])
    assert list(got[0, 3, :, 0]) == [12, 13, 15, 6] and list(got[0, 1, :, 0]) == [4, 5, 6, 7]
