"""The norm, 4-bit cache and page calls of two host threads at once, each with sizes and kernels of its own, and what a refused
launch leaves behind."""
import ctypes

import numpy as np
import pytest
import torch

import sparse_compressed_attention_gb300 as V
from tests.q4_cases import Q4Case
from tests.test_gpu_serving_calls import at_once

pytestmark = pytest.mark.gpu


def i32(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32).cuda()


def norm_call(big, grad):
    g = torch.Generator().manual_seed(int(big))
    rows, heads, dim, dt = (40, 3, 1024, torch.float32) if big else (9, 2, 64, torch.bfloat16)
    x, dy = (torch.randn(rows, heads, dim, generator=g).to(dt).cuda() for _ in range(2))
    pos, f = torch.arange(rows, dtype=torch.int32).cuda(), torch.rand(8, generator=g).cuda()
    lay = V.V4_ROPE_HALF if big else V.V4_ROPE_INTERLEAVED
    out, dw, ws = torch.zeros_like(x), torch.zeros(dim, device="cuda"), V.alloc_norm_rope_workspace(dim)
    if grad:
        return lambda s: V.v4_norm_rope_bwd(x, None, dy, None, pos, f, out, dq_w=dw, layout=lay, workspace=ws, stream=s), [out, dw]
    return lambda s: V.v4_norm_rope_fwd(x, None, pos, f, out, layout=lay, stream=s), [out]


def q4_rows_call(big, read):
    rows, dim, dt = (500, 512, torch.bfloat16) if big else (7, 64, torch.float32)
    x = torch.randn(rows, dim, generator=torch.Generator().manual_seed(rows)).to(dt).cuda()
    slot = torch.randperm(rows, generator=torch.Generator().manual_seed(1)).to(torch.int32).cuda()
    cache = torch.zeros(rows, V.v4_q4_row_bytes(dim), dtype=torch.uint8, device="cuda")
    if not read:
        return lambda s: V.v4_cache_append_q4(x, slot, cache, stream=s), [cache]
    V.v4_cache_append_q4(x, slot, cache)
    out = torch.zeros_like(x)
    return lambda s: V.v4_cache_read_q4(cache, slot, out, stream=s), [out]


def attention_call(big, dense):
    c = Q4Case([300, 40], [2, 1], ratio=4, K=32, seed=5) if big else Q4Case([90, 7], [2, 1], H=5, D=96, R=32, dt=torch.float32, seed=6)
    x = c.dense_inputs() if dense else c.device_inputs()
    o, lse = torch.zeros(c.n, c.H, c.D, dtype=c.dt, device="cuda"), torch.zeros(c.n, c.H, device="cuda")
    ws = V.alloc_tree_workspace(c.cfg, c.n)
    call = V.v4_tree_mqa_fwd if dense else V.v4_tree_mqa_fwd_q4
    return lambda s: call(c.cfg, x, o, lse, ws, stream=s), [o, lse]


def pages_call(big, op):
    """Calls whose outcome is the same however often they are made."""
    if op == "alloc":                                             # every wanted entry holds a page: nothing to give
        n = 900 if big else 3
        table, ref, need = i32(np.arange(4 * n).reshape(n, 4)), i32(np.ones(4 * n)), i32(np.full(n, 60))
        lack = i32([7])
        return lambda s: V.v4_pages_alloc(table, ref, need, 16, lack=lack, stream=s), [table, ref, lack]
    if op == "fork":                                              # no whole pages and none free: counts stay
        n = 900 if big else 3
        table, ref, out = i32(np.arange(4).reshape(1, 4)), i32(np.ones(4)), i32(np.zeros((n, 4)))
        src, length, copies, lack = i32(np.zeros(n)), i32(np.full(n, 9)), i32(np.zeros((n, 3))), i32([7])
        return lambda s: V.v4_pages_fork(table, src, length, out, ref, 16, copies, lack=lack, stream=s), [ref, out, copies, lack]
    if op == "free":
        table, ref, hi = i32(np.arange(400).reshape(100, 4) if big else [[0, 1]]), i32(np.ones(400)), i32(np.full(100 if big else 1, 64))
        return lambda s: V.v4_pages_free(table, ref, 16, hi=hi, stream=s), [table, ref]
    cache = torch.randint(0, 255, (3, 40, 16, 288 if big else 32), dtype=torch.uint8, generator=torch.Generator().manual_seed(int(big))).cuda()
    if op == "copy":
        copies = i32([[k, k + 20, 16 - k] for k in range(20 if big else 1)])      # the last three name fewer than no rows
        return lambda s: V.v4_pages_copy(cache, copies, stream=s), [cache]
    keep = np.arange(300 if big else 5)                           # rows that stay
    table, base, count = i32([np.arange(40)]), i32([2]), i32([len(keep)])
    keep = i32([keep])
    return lambda s: V.v4_pages_compact(cache, table, base, count, keep, stream=s), [cache]


PAIRS = {
    "norm": [lambda: norm_call(True, False), lambda: norm_call(False, False)],
    "norm_gradients": [lambda: norm_call(True, True), lambda: norm_call(False, True)],
    "both_directions": [lambda: norm_call(True, True), lambda: norm_call(True, False)],
    "write": [lambda: q4_rows_call(True, False), lambda: q4_rows_call(False, False)],
    "write_and_read": [lambda: q4_rows_call(True, False), lambda: q4_rows_call(True, True)],
    "attention_of_both_paths": [lambda: attention_call(True, False), lambda: attention_call(False, False)],
    "attention_of_both_caches": [lambda: attention_call(True, False), lambda: attention_call(True, True)],
    "alloc": [lambda: pages_call(True, "alloc"), lambda: pages_call(False, "alloc")],
    "fork": [lambda: pages_call(True, "fork"), lambda: pages_call(False, "fork")],
    "alloc_and_fork": [lambda: pages_call(True, "alloc"), lambda: pages_call(True, "fork")],
    "free_and_copy": [lambda: pages_call(True, "free"), lambda: pages_call(True, "copy")],
    "compact": [lambda: pages_call(True, "compact"), lambda: pages_call(False, "compact")],
    "compact_and_norm": [lambda: pages_call(True, "compact"), lambda: norm_call(False, True)],
}


@pytest.mark.parametrize("pair", list(PAIRS))
def test_two_host_threads(pair):
    V.v4_reset_device_status()
    made = [m() for m in PAIRS[pair]]
    want = []
    for call, outs in made:
        call(None)
        want.append([t.clone() for t in outs])
    torch.cuda.synchronize()
    assert at_once(*(c for c, _ in made), times=3000) == []
    for (_, outs), kept in zip(made, want):
        assert all(torch.equal(a, b) for a, b in zip(outs, kept))
    assert V.v4_get_device_status() == (6 if pair == "free_and_copy" else 0)
    V.v4_reset_device_status()


def test_calls_after_ones_that_could_not_be_launched():
    """A launch that the runtime refuses (the legacy stream, while a blocking stream is captured) is reported by its own call
    and by no later one."""
    rt = ctypes.CDLL("libcudart.so.13")
    calls = [(norm_call(False, True), "norm kernel"), (q4_rows_call(False, False), "4-bit write"), (q4_rows_call(False, True), "4-bit read"),
             (attention_call(True, False), "tree attention"), (pages_call(False, "alloc"), "allocation"), (pages_call(False, "fork"), "fork"),
             (pages_call(False, "free"), "release"), (pages_call(False, "copy"), "copy"), (pages_call(False, "compact"), "compaction")]
    want = []
    for (call, outs), _ in calls:
        call(None)
        want.append([t.clone() for t in outs])
    torch.cuda.synchronize()
    for (call, outs), name in calls:
        stream, graph = ctypes.c_void_p(), ctypes.c_void_p()
        assert rt.cudaStreamCreate(ctypes.byref(stream)) == 0
        try:
            assert rt.cudaStreamBeginCapture(stream, 0) == 0
            with pytest.raises(V.V4Error, match=name):
                call(0)
        finally:
            rt.cudaStreamEndCapture(stream, ctypes.byref(graph))
            rt.cudaStreamDestroy(stream)
            rt.cudaGetLastError()
    for ((call, outs), _), kept in zip(calls, want):
        call(None)
        assert all(torch.equal(a, b) for a, b in zip(outs, kept))
