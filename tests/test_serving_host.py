"""Refusals of the serving operators on the host (no kernel runs), and CPU pins of their oracle."""
import ctypes as C

import numpy as np
import pytest
import torch

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


def rope(lib, **over):
    a = dict(x=1 << 20, rows=4, heads=2, dim=64, xr=128, xh=64, pos=16, f=16, R=16, begin=48, layout=0, inverse=0, mscale=1.0,
             dtype=1, out=1 << 24, yr=128, yh=64)
    a.update(over)
    return lib.v4_rope(a["x"], a["rows"], a["heads"], a["dim"], a["xr"], a["xh"], a["pos"], a["f"], a["R"], a["begin"],
                       a["layout"], a["inverse"], a["mscale"], a["dtype"], a["out"], a["yr"], a["yh"], None)


@pytest.mark.parametrize("over,text", [
    (dict(x=None), "x is NULL"), (dict(x=(1 << 20) + 8), "aligned"), (dict(pos=None), "pos"), (dict(f=None), "inv_freq"),
    (dict(dim=60), "dim"), (dict(R=12), "rope_dim"), (dict(R=24, layout=1), "rope_dim"), (dict(begin=52), "rope_begin"),
    (dict(begin=56), "rope_begin"), (dict(layout=2), "layout"), (dict(inverse=2), "inverse"), (dict(dtype=3), "dtype"),
    (dict(heads=0), "heads"), (dict(heads=70000), "heads"), (dict(rows=-1), "rows"), (dict(mscale=float("inf")), "mscale"),
    (dict(xr=132), "x_row_stride"), (dict(yh=-64), "out_head_stride"), (dict(yh=0), "overlap"), (dict(yr=64), "overlap"),
    (dict(out=(1 << 20) + 128), "overlap"), (dict(out=1 << 20, yr=256), "overlap")])
def test_rope_refusals(lib, over, text):
    refused(lib, rope(lib, **over), L.V4_ERR_INVALID_ARG, text)


def test_rope_of_no_rows_does_nothing(lib):
    assert rope(lib, rows=0, x=None, out=None, pos=None) == L.V4_OK


def append(lib, **over):
    a = dict(x=1 << 20, rows=4, dim=64, xr=64, pos=16, f=16, R=16, slot=16, n_slots=32, dtype=1, cache=1 << 24)
    a.update(over)
    return lib.v4_cache_append(a["x"], a["rows"], a["dim"], a["xr"], a["pos"], a["f"], a["R"], a["slot"], a["n_slots"],
                               a["dtype"], a["cache"], None)


@pytest.mark.parametrize("over,text", [
    (dict(x=None), "x is NULL"), (dict(slot=None), "slot"), (dict(cache=None), "cache"), (dict(f=None), "inv_freq"),
    (dict(R=72), "rope_begin"), (dict(dim=12), "dim"), (dict(xr=60), "x_row_stride"), (dict(n_slots=1 << 31), "n_slots"),
    (dict(dtype=2), "dtype"), (dict(cache=(1 << 20) + 256), "overlap")])
def test_cache_write_refusals(lib, over, text):
    refused(lib, append(lib, **over), L.V4_ERR_INVALID_ARG, text)


def test_plan_refusals(lib):
    ok = [2, 8, 16, 16, 16, 16, 4, 16, 64, 16, 16, 16, None]

    def call(i, v):
        a = list(ok)
        a[i] = v
        return lib.v4_tree_plan(*a)
    for i, v, text in ((0, 0, "batch"), (1, -1, "n_rows"), (2, None, "node_begin"), (3, None, "seq_len"),
                       (5, None, "block_table"), (6, 0, "max_blocks"), (7, 0, "page_size"), (8, -1, "n_slots"),
                       (9, None, "plan"), (9, 24, "aligned")):
        refused(lib, call(i, v), L.V4_ERR_INVALID_ARG, text)
    assert call(1, 0) == L.V4_OK


def tree(lib, cfg=None, ws=(256, 1 << 32), o=16, lse=16, **over):
    cfg = cfg or L.make_config(2, 1, 64, 512, 64, ratio=4, window=128, topk=512)
    v = L.v4_tree_inputs()
    for n in ("q", "plan", "tok_cache", "tok_table", "ent_cache", "ent_table", "ent_len", "idx", "inv_freq"):
        setattr(v, n, 16)
    v.tok_slots = v.ent_slots = 640
    v.n_rows, v.tok_blocks, v.tok_page, v.ent_blocks, v.ent_page = 3, 10, 64, 10, 64
    for n, x in over.items():
        setattr(v, n, x)
    return lib.v4_tree_mqa_fwd(C.byref(cfg), C.byref(v), o, lse, ws[0], ws[1], None)


@pytest.mark.parametrize("over,text", [
    (dict(q=None), "q is NULL"), (dict(q=20), "aligned"), (dict(plan=None), "plan"), (dict(tok_cache=None), "tok_cache"),
    (dict(tok_table=None), "tok_table"), (dict(ent_cache=None), "ent_cache"), (dict(ent_len=None), "ent_len"),
    (dict(idx=None), "idx"), (dict(inv_freq=None), "inv_freq"), (dict(o=None), "o is NULL"), (dict(n_rows=-1), "n_rows"),
    (dict(tok_page=0), "tok_page"), (dict(ent_blocks=0), "ent_blocks"), (dict(tok_slots=0), "tok_slots"),
    (dict(ent_slots=1 << 31), "ent_slots")])
def test_tree_refusals(lib, over, text):
    refused(lib, tree(lib, **over), L.V4_ERR_INVALID_ARG, text)


def test_tree_refuses_unsupported_calls_and_workspaces(lib):
    cfg = L.make_config(2, 9, 64, 512, 64, window=128, q_begin=1)
    refused(lib, tree(lib, cfg), L.V4_ERR_UNSUPPORTED, "q_begin")
    cfg = L.make_config(2, 1, 32, 512, 64, window=128, path=L.V4_PATH_TC)
    refused(lib, tree(lib, cfg), L.V4_ERR_UNSUPPORTED, "tensor-core")
    cfg = L.make_config(2, 1, 64, 512, 64, window=-2)
    refused(lib, tree(lib, cfg), L.V4_ERR_INVALID_ARG, "window")
    cfg = L.make_config(2, 1, 64, 512, 64, window=128)
    need = L.v4_tree_workspace_size(cfg, 3)
    if need:
        refused(lib, tree(lib, cfg, ws=(256, need - 1)), L.V4_ERR_WORKSPACE, "needed")
        refused(lib, tree(lib, cfg, ws=(None, need)), L.V4_ERR_WORKSPACE, "NULL")
    refused(lib, tree(lib, cfg, ws=(128, need)), L.V4_ERR_WORKSPACE, "256-byte")
    assert tree(lib, n_rows=0, q=None) == L.V4_OK
    with pytest.raises(L.V4Error, match="n_rows"):
        L.v4_tree_workspace_size(cfg, -1)


def w4(lib, **over):
    a = dict(x=16, rows=3, G=2, K=256, N=512, gs=64, codes=16, scales=16, norm=512, eps=1e-6, w=16, y=16)
    a.update(over)
    return lib.v4_w4_proj(a["x"], a["rows"], a["G"], a["K"], a["N"], a["gs"], a["codes"], a["scales"], a["norm"], a["eps"],
                          a["w"], a["y"], None)


def test_w4_refusals(lib):
    for over, text in ((dict(x=None), "x"), (dict(codes=24), "codes"), (dict(scales=None), "scales"), (dict(y=None), "y"),
                       (dict(w=8), "norm_w"), (dict(rows=-1), "rows"), (dict(eps=-1.0), "eps"), (dict(eps=float("nan")), "eps"),
                       (dict(G=0), "groups")):
        refused(lib, w4(lib, **over), L.V4_ERR_INVALID_ARG, text)
    for over, text in ((dict(K=192), "K a multiple"), (dict(N=96), "N a multiple"), (dict(gs=16), "group_size"),
                       (dict(norm=96), "norm_dim"), (dict(norm=512, N=256), "norm_dim")):
        refused(lib, w4(lib, **over), L.V4_ERR_UNSUPPORTED, text)
    assert w4(lib, rows=0, x=None, y=None) == L.V4_OK
    refused(lib, lib.v4_w4_pack(None, 1, 128, 64, 32, 16, 16, None), L.V4_ERR_INVALID_ARG, "w is NULL")
    refused(lib, lib.v4_w4_pack(16, 1, 128, 63, 32, 16, 16, None), L.V4_ERR_UNSUPPORTED, "N a multiple")


def test_binding_refuses_host_tensors():
    x = torch.zeros(2, 1, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        L.v4_rope(x, torch.zeros(2, dtype=torch.int32), torch.zeros(8), x)
    with pytest.raises(ValueError, match="codes"):
        L.v4_w4_proj(x, None, None, x)


# ---------------------------------------------------------------- oracle pins
def test_rotation_of_the_oracle():
    f = O.make_inv_freq(40000.0, 16)
    x = np.random.default_rng(0).standard_normal((5, 3, 40))
    pos = [0, 1, 7, 100000, -3]
    y = S.rope(x, pos, f, 24)
    ref = np.stack([O.rope_rotate(x[i], pos[i], f) for i in range(5)])
    assert np.allclose(y, ref, atol=1e-9)
    assert np.allclose(S.rope(y, pos, f, 24, inverse=True), x, atol=1e-12)
    # the half layout is the interleaved one under the permutation of its pairs
    perm = np.arange(40)
    perm[24:40:2], perm[25:40:2] = np.arange(24, 32), np.arange(32, 40)
    assert np.allclose(S.rope(x, pos, f, 24, half=True)[..., perm], S.rope(x[..., perm], pos, f, 24), atol=1e-12)


def test_tree_of_the_oracle_is_the_sequence_attention():
    """A chain at the end of a cache equals the oracle's rows of a whole sequence."""
    rng = np.random.default_rng(1)
    S_, n, H, D, R, W, r = 40, 6, 3, 32, 8, 9, 4
    f = O.make_inv_freq(10000.0, R)
    q, kv = rng.standard_normal((1, S_, H, D)), rng.standard_normal((1, S_, D))
    ent, sink = rng.standard_normal((1, S_ // r, D)), rng.standard_normal(H)
    ro, rl = O.sparse_mqa(q, kv, ent, None, sink, f, r, W)
    rot = np.stack([O.rope_rotate(kv[0, u], u, f) for u in range(S_)])
    plan, _ = S.tree_plan([0, n], [S_ - n], None, n)
    o, lse, _, _ = S.tree_mqa(q[0, S_ - n:], plan, lambda b, u: rot[u], lambda b, s: S_ // r if s is None else ent[0, s],
                              None, sink, f, r, W, 0, D ** -0.5, np.zeros((n, H, D)), np.zeros((n, H)))
    assert np.allclose(o, ro[0, S_ - n:], atol=1e-9) and np.allclose(lse, rl[0, S_ - n:], atol=1e-9)


def test_tree_siblings_do_not_see_each_other():
    plan, pos = S.tree_plan([0, 4], [10], [-1, 0, 0, 2], 4)
    assert pos.tolist() == [10, 11, 11, 12]
    assert plan[:, 4].tolist() == [0b1, 0b11, 0b101, 0b1101]


def test_codes_of_the_oracle_round_trip():
    rng = np.random.default_rng(2)
    w = rng.integers(-8, 8, (2, 256, 64)).astype(np.float32)
    w[:, ::32] = 7.0                                  # every group's maximum: the scale is one
    w[w < -7] = -7.0
    codes, scales = S.w4_pack(w, 32, lambda a: a)
    assert np.all(scales == 1.0)
    assert np.array_equal(S.w4_weights(codes, scales, 32).transpose(0, 2, 1), w)
    # the order as the header words it: word 4 t + c, inputs 32 c + 8 t + e, nibbles 0 2 4 6 1 3 5 7
    words = codes[0, 0].view("<u4")
    for k in (0, 1, 9, 37, 127, 128, 255):
        word = words[(k // 128) * 16 + 4 * (k % 32 // 8) + k % 128 // 32]
        at = [0, 2, 4, 6, 1, 3, 5, 7].index(k % 8)
        assert int(word >> np.uint32(4 * at)) & 15 == int(w[0, k, 0]) + 8


def test_tree_refuses_overlaps_and_counts_beyond_32_bits(lib):
    refused(lib, tree(lib), L.V4_ERR_INVALID_ARG, "overlap")
    refused(lib, tree(lib, o=16 + 3 * 64 * 512), L.V4_ERR_INVALID_ARG, "overlap")
    big = dict(o=1 << 40)
    cfg = L.make_config(2, 1, 64, 512, 64, window=-1)
    refused(lib, tree(lib, cfg, n_rows=1 << 18, tok_blocks=16384, **big), L.V4_ERR_UNSUPPORTED, "2^30 tiles")
    refused(lib, tree(lib, cfg, n_rows=1, tok_blocks=1 << 30, tok_page=1 << 30, **big), L.V4_ERR_UNSUPPORTED, "2^30 tiles")
    refused(lib, tree(lib, n_rows=(1 << 24) + 1, **big), L.V4_ERR_INVALID_ARG, "n_rows")
    with pytest.raises(L.V4Error, match="n_rows"):
        L.v4_tree_workspace_size(cfg, (1 << 24) + 1)
    refused(lib, lib.v4_tree_plan(2, 1 << 30, 16, 16, 16, 16, 4, 16, 64, 16, 16, 16, None), L.V4_ERR_INVALID_ARG, "n_rows")


def test_w4_refuses_overlap(lib):
    refused(lib, w4(lib), L.V4_ERR_INVALID_ARG, "overlap")
    refused(lib, w4(lib, y=16 + 3 * 2 * 256 * 2 - 16), L.V4_ERR_INVALID_ARG, "overlap")


@pytest.mark.parametrize("swap", ["sign", "window", "order"])
def test_planted_mistakes_are_seen(swap):
    """The comparisons of this file tell a wrong oracle from a right one."""
    rng = np.random.default_rng(3)
    f = O.make_inv_freq(10000.0, 8)
    if swap == "sign":
        x = rng.standard_normal((3, 1, 8))
        assert not np.allclose(S.rope(x, [5, 6, 7], f, 0, inverse=True),
                               np.stack([O.rope_rotate(x[i], 5 + i, f) for i in range(3)]), atol=1e-3)
    elif swap == "window":
        plan, _ = S.tree_plan([0, 1], [20], None, 1)
        rows = lambda b, u: np.full(8, float(u))            # noqa: E731
        a = S.tree_keys(plan, 0, rows, None, None, 0, 5, 0)
        b = S.tree_keys(plan, 0, rows, None, None, 0, 6, 0)
        assert [k[0] for k in a] == [16, 17, 18, 19, 20] and len(b) == 6
    else:
        codes = rng.integers(0, 256, (1, 64, 64)).astype(np.uint8)
        w = S.w4_weights(codes, np.ones((1, 64, 1)), 128)
        naive = np.stack([codes & 15, codes >> 4], -1).reshape(1, 64, 128).astype(float) - 8
        assert not np.array_equal(w, naive)
