"""ctypes binding of libv4attn.so: the C ABI of include/v4attn.h, same names.

Argument marshalling only: tensors are checked for device, dtype, contiguity
and alignment, then their data pointers and the current CUDA stream are
handed to the library.  Every step of the path runs in the library's CUDA
kernels; there is no fallback.  A missing library raises at first use.
"""
from __future__ import annotations

import ctypes as C
import os

import torch

from . import build as _build

V4_OK, V4_ERR_INVALID_ARG, V4_ERR_UNSUPPORTED, V4_ERR_WORKSPACE, V4_ERR_CUDA, \
    V4_ERR_TIMEOUT, V4_ERR_BAD_INDEX, V4_ERR_BOUND = range(8)
V4_F32, V4_BF16 = 0, 1
V4_PATH_AUTO, V4_PATH_SIMT, V4_PATH_TC = 0, 1, 2
V4_ROPE_INTERLEAVED, V4_ROPE_HALF = 0, 1
V4_TREE_MAX_NODES = 128

STATUS_NAMES = {0: "V4_OK", 1: "V4_ERR_INVALID_ARG", 2: "V4_ERR_UNSUPPORTED", 3: "V4_ERR_WORKSPACE",
                4: "V4_ERR_CUDA", 5: "V4_ERR_TIMEOUT", 6: "V4_ERR_BAD_INDEX", 7: "V4_ERR_BOUND"}

# every symbol include/v4attn.h declares
EXPORTS = ["v4_rope_inv_freq", "v4_workspace_size", "v4_compress", "v4_indexer_prep",
           "v4_indexer_topk", "v4_sparse_mqa_fwd", "v4_grouped_o_proj", "v4_attn_layer_fwd",
           "v4_last_error", "v4_get_device_status", "v4_reset_device_status", "v4_launch_count",
           "v4_profile_enable", "v4_profile_count", "v4_profile_get", "v4_sparse_mqa_fwd_noalloc",
           "v4_bwd_workspace_size", "v4_sparse_mqa_bwd", "v4_quantize_e4m3", "v4_indexer_topk_e4m3",
           "v4_q_proj", "v4_indexer_kl_target", "v4_selftest_wait_timeout", "v4_build_info",
           "v4_rope", "v4_cache_append", "v4_tree_plan", "v4_tree_workspace_size", "v4_tree_mqa_fwd",
           "v4_w4_pack", "v4_w4_proj"]
PROFILE_KINDS = {0: "compress", 1: "window_rotate", 2: "indexer_prep", 3: "indexer_scores", 4: "topk",
                 5: "attention", 6: "o_proj", 7: "bwd_prep", 8: "bwd_attention", 9: "bwd_derotate",
                 10: "indexer_quant", 11: "q_proj", 12: "kl_target", 13: "rope", 14: "cache_append",
                 15: "tree_plan", 16: "tree_attention", 17: "tree_join", 18: "w4_pack", 19: "w4_proj"}


class V4Error(RuntimeError):
    def __init__(self, status, msg):
        super().__init__("%s: %s" % (STATUS_NAMES.get(status, status), msg))
        self.status = status


class v4_config(C.Structure):
    _fields_ = [(n, C.c_int32) for n in (
        "batch", "seqlen", "n_heads", "head_dim", "rope_dim", "ratio", "overlap", "window", "topk",
        "idx_heads", "idx_dim", "o_groups", "o_rank")] + [
        ("softmax_scale", C.c_float), ("rms_eps", C.c_float), ("dtype", C.c_int32), ("path", C.c_int32),
        ("indexer_fp8", C.c_int32), ("q_begin", C.c_int32)]


class v4_layer_inputs(C.Structure):
    _fields_ = [(n, C.c_void_p) for n in (
        "q", "kv", "ckv", "cscore", "ape", "norm_w", "ickv", "icscore", "iape", "inorm_w", "iq", "w",
        "sink", "inv_freq", "wo_a")]


class v4_layer_outputs(C.Structure):
    _fields_ = [(n, C.c_void_p) for n in ("o", "lse", "ent", "ikey", "idx", "iscore", "y")]


class v4_tree_inputs(C.Structure):
    _fields_ = [(n, C.c_void_p) for n in (
        "q", "plan", "tok_cache", "tok_table", "ent_cache", "ent_table", "ent_len", "idx", "sink", "inv_freq")] + [
        (n, C.c_int64) for n in ("tok_slots", "ent_slots")] + [
        (n, C.c_int32) for n in ("n_rows", "tok_blocks", "tok_page", "ent_blocks", "ent_page")]


_lib = None


def lib(path=None):
    """Load the library (once).  Raises if it has not been built.  The
    environment variable V4ATTN_LIB names another build of it (e.g. the
    bound-checking one, build.DEBUG_LIB)."""
    global _lib
    if _lib is not None:
        return _lib
    path = path or os.environ.get("V4ATTN_LIB") or _build.LIB
    if not os.path.exists(path):
        raise RuntimeError("CUDA library %s is missing: build it with "
                           "sparse_compressed_attention_gb300.build.build()" % path)
    L = C.CDLL(path)
    vp, i32, i64, f32, sz = C.c_void_p, C.c_int32, C.c_int64, C.c_float, C.c_size_t
    cfgp = C.POINTER(v4_config)
    sig = {
        "v4_rope_inv_freq": [f32, i32, f32, i32, f32, f32, vp],
        "v4_workspace_size": [cfgp, C.POINTER(sz)],
        "v4_compress": [cfgp, vp, vp, vp, vp, vp, i32, i32, vp, vp],
        "v4_indexer_prep": [cfgp, vp, vp, vp, vp],
        "v4_indexer_topk": [cfgp, vp, i32, vp, vp, vp, vp, vp, vp, sz, vp],
        "v4_quantize_e4m3": [vp, C.c_int64, i32, vp, vp, vp],
        "v4_indexer_topk_e4m3": [cfgp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp],
        "v4_sparse_mqa_fwd": [cfgp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp],
        "v4_sparse_mqa_fwd_noalloc": [cfgp, vp, vp, vp, vp, vp, vp, vp, vp, vp],
        "v4_grouped_o_proj": [cfgp, vp, vp, vp, vp],
        "v4_q_proj": [cfgp, vp, i32, vp, i32, vp, vp, vp, vp, vp],
        "v4_indexer_kl_target": [cfgp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp],
        "v4_bwd_workspace_size": [cfgp, C.POINTER(sz)],
        "v4_sparse_mqa_bwd": [cfgp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp],
        "v4_attn_layer_fwd": [cfgp, C.POINTER(v4_layer_inputs), C.POINTER(v4_layer_outputs), vp, sz, vp],
        "v4_get_device_status": [vp, C.POINTER(i32)],
        "v4_reset_device_status": [vp],
        "v4_profile_enable": [i32],
        "v4_profile_get": [i32, C.POINTER(i32), C.POINTER(f32)],
        "v4_selftest_wait_timeout": [i32, vp],
        "v4_rope": [vp, i64, i32, i32, i64, i64, vp, vp, i32, i32, i32, i32, f32, i32, vp, i64, i64, vp],
        "v4_cache_append": [vp, i64, i32, i64, vp, vp, i32, vp, i64, i32, vp, vp],
        "v4_tree_plan": [i32, i32, vp, vp, vp, vp, i32, i32, i64, vp, vp, vp, vp],
        "v4_tree_workspace_size": [cfgp, i32, C.POINTER(sz)],
        "v4_tree_mqa_fwd": [cfgp, C.POINTER(v4_tree_inputs), vp, vp, vp, sz, vp],
        "v4_w4_pack": [vp, i32, i32, i32, i32, vp, vp, vp],
        "v4_w4_proj": [vp, i64, i32, i32, i32, i32, vp, vp, i32, f32, vp, vp, vp],
    }
    for name, args in sig.items():
        fn = getattr(L, name)
        fn.argtypes = args
        fn.restype = C.c_int
    L.v4_last_error.argtypes = []
    L.v4_last_error.restype = C.c_char_p
    L.v4_build_info.argtypes = []
    L.v4_build_info.restype = C.c_char_p
    L.v4_launch_count.argtypes = []
    L.v4_launch_count.restype = C.c_uint64
    L.v4_profile_count.argtypes = []
    L.v4_profile_count.restype = C.c_int32
    _lib = L
    return L


def _check(status):
    if status != V4_OK:
        raise V4Error(status, lib().v4_last_error().decode())


def make_config(B, S, H, D, R, ratio=0, overlap=0, window=128, topk=0, Hi=64, Di=128,
                o_groups=8, o_rank=1024, scale=0.0, eps=1e-6, dtype="bf16", path=V4_PATH_AUTO,
                indexer_fp8=0, q_begin=0):
    """v4_config; q_begin > 0 restricts the call to query positions q_begin..S-1
    (row tensors then hold S - q_begin rows per sequence)."""
    return v4_config(B, S, H, D, R, ratio, overlap, window, topk, Hi, Di, o_groups, o_rank,
                     scale, eps, V4_BF16 if dtype == "bf16" else V4_F32, path, int(indexer_fp8), int(q_begin))


def config_from_preset(p, **over):
    q = dict(p)
    q.update(over)
    return make_config(q["B"], q["S"], q["H"], q["D"], q["R"], q["ratio"], q["overlap"], q["W"],
                       q["K"], q["Hi"], q["Di"], dtype=q["dtype"], path=q.get("path", V4_PATH_AUTO),
                       eps=q.get("eps", 1e-6), scale=q.get("scale", 0.0),
                       indexer_fp8=q.get("indexer_fp8", 0), q_begin=q.get("q_begin", 0))


def _storage(cfg):
    return torch.bfloat16 if cfg.dtype == V4_BF16 else torch.float32


def _ptr(t, name, dtype=None, optional=False):
    if t is None:
        if optional:
            return None
        raise ValueError("%s is required" % name)
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a tensor" % name)
    if not t.is_cuda:
        raise ValueError("%s must be on a CUDA device" % name)
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    if dtype is not None and t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    return t.data_ptr()


def _stream(stream):
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else stream


def v4_rope_inv_freq(theta, rope_dim, yarn_factor=1.0, original_len=0, beta_fast=32.0, beta_slow=1.0):
    """Host-built inverse-frequency table (float32 CPU tensor of rope_dim/2)."""
    out = (C.c_float * (rope_dim // 2))()
    _check(lib().v4_rope_inv_freq(theta, rope_dim, yarn_factor, original_len, beta_fast, beta_slow, out))
    return torch.tensor(list(out), dtype=torch.float32)


def v4_workspace_size(cfg):
    n = C.c_size_t(0)
    _check(lib().v4_workspace_size(C.byref(cfg), C.byref(n)))
    return n.value


def alloc_workspace(cfg, device=None):
    return torch.empty(max(v4_workspace_size(cfg), 256), dtype=torch.uint8, device=device or "cuda")


def v4_compress(cfg, ckv, cscore, ape, norm_w, inv_freq, dim, hadamard, out, stream=None):
    dt = _storage(cfg)
    _check(lib().v4_compress(C.byref(cfg), _ptr(ckv, "ckv", dt), _ptr(cscore, "cscore", dt),
                             _ptr(ape, "ape", torch.float32),
                             _ptr(norm_w, "norm_w", torch.float32, optional=True),
                             _ptr(inv_freq, "inv_freq", torch.float32, optional=cfg.rope_dim == 0), int(dim), int(hadamard),
                             _ptr(out, "out", dt, optional=out is None), _stream(stream)))
    return out


def v4_indexer_prep(cfg, iq, inv_freq, iq_prep, stream=None):
    dt = _storage(cfg)
    _check(lib().v4_indexer_prep(C.byref(cfg), _ptr(iq, "iq", dt), _ptr(inv_freq, "inv_freq", torch.float32, optional=cfg.rope_dim == 0),
                                 _ptr(iq_prep, "iq_prep", dt), _stream(stream)))
    return iq_prep


def v4_indexer_topk(cfg, iq, iq_prepared, ikey, w, inv_freq, idx, iscore, workspace, stream=None):
    dt = _storage(cfg)
    _check(lib().v4_indexer_topk(C.byref(cfg), _ptr(iq, "iq", dt), int(iq_prepared),
                                 _ptr(ikey, "ikey", dt, optional=True), _ptr(w, "w", torch.float32),
                                 _ptr(inv_freq, "inv_freq", torch.float32, optional=True),
                                 _ptr(idx, "idx", torch.int32),
                                 _ptr(iscore, "iscore", torch.float32, optional=True),
                                 _ptr(workspace, "workspace", torch.uint8), workspace.numel(),
                                 _stream(stream)))
    return idx


def v4_quantize_e4m3(x, codes, scales, stream=None):
    """x [..., dim] bf16 -> codes [..., dim] uint8 (E4M3 bytes), scales [...] fp32."""
    dim = x.shape[-1]
    rows = x.numel() // dim if dim else 0
    _check(lib().v4_quantize_e4m3(_ptr(x, "x", torch.bfloat16), rows, dim, _ptr(codes, "codes", torch.uint8),
                                  _ptr(scales, "scales", torch.float32), _stream(stream)))
    return codes, scales


def v4_indexer_topk_e4m3(cfg, q_codes, q_scales, k_codes, k_scales, w, idx, iscore, workspace, stream=None):
    _check(lib().v4_indexer_topk_e4m3(C.byref(cfg), _ptr(q_codes, "q_codes", torch.uint8),
                                      _ptr(q_scales, "q_scales", torch.float32),
                                      _ptr(k_codes, "k_codes", torch.uint8, optional=True),
                                      _ptr(k_scales, "k_scales", torch.float32, optional=True),
                                      _ptr(w, "w", torch.float32), _ptr(idx, "idx", torch.int32),
                                      _ptr(iscore, "iscore", torch.float32, optional=True),
                                      _ptr(workspace, "workspace", torch.uint8), workspace.numel(),
                                      _stream(stream)))
    return idx


def v4_sparse_mqa_fwd(cfg, q, kv, ent, idx, sink, inv_freq, o, lse, workspace, stream=None):
    dt = _storage(cfg)
    _check(lib().v4_sparse_mqa_fwd(C.byref(cfg), _ptr(q, "q", dt), _ptr(kv, "kv", dt),
                                   _ptr(ent, "ent", dt, optional=True),
                                   _ptr(idx, "idx", torch.int32, optional=True),
                                   _ptr(sink, "sink", torch.float32, optional=True),
                                   _ptr(inv_freq, "inv_freq", torch.float32, optional=cfg.rope_dim == 0),
                                   _ptr(o, "o", dt), _ptr(lse, "lse", torch.float32, optional=True),
                                   _ptr(workspace, "workspace", torch.uint8), workspace.numel(),
                                   _stream(stream)))
    return o


def v4_sparse_mqa_fwd_noalloc(cfg, q, kv, ent, idx, sink, inv_freq, o, lse, stream=None):
    """v4_sparse_mqa_fwd with library-owned scratch (no workspace argument)."""
    dt = _storage(cfg)
    _check(lib().v4_sparse_mqa_fwd_noalloc(C.byref(cfg), _ptr(q, "q", dt), _ptr(kv, "kv", dt),
                                           _ptr(ent, "ent", dt, optional=True),
                                           _ptr(idx, "idx", torch.int32, optional=True),
                                           _ptr(sink, "sink", torch.float32, optional=True),
                                           _ptr(inv_freq, "inv_freq", torch.float32, optional=cfg.rope_dim == 0),
                                           _ptr(o, "o", dt), _ptr(lse, "lse", torch.float32, optional=True),
                                           _stream(stream)))
    return o


def v4_bwd_workspace_size(cfg):
    n = C.c_size_t(0)
    _check(lib().v4_bwd_workspace_size(C.byref(cfg), C.byref(n)))
    return n.value


def alloc_bwd_workspace(cfg, device=None):
    return torch.empty(max(v4_bwd_workspace_size(cfg), 256), dtype=torch.uint8, device=device or "cuda")


def v4_sparse_mqa_bwd(cfg, q, kv, ent, idx, sink, inv_freq, o, lse, dout, dq, dkv, dent, dsink, workspace,
                      stream=None):
    """Gradients of sum(dout * o) for v4_sparse_mqa_fwd; dq, dkv, dent, dsink are written."""
    dt = _storage(cfg)
    _check(lib().v4_sparse_mqa_bwd(C.byref(cfg), _ptr(q, "q", dt), _ptr(kv, "kv", dt),
                                   _ptr(ent, "ent", dt, optional=True),
                                   _ptr(idx, "idx", torch.int32, optional=True),
                                   _ptr(sink, "sink", torch.float32, optional=True),
                                   _ptr(inv_freq, "inv_freq", torch.float32),
                                   _ptr(o, "o", dt), _ptr(lse, "lse", torch.float32), _ptr(dout, "dout", dt),
                                   _ptr(dq, "dq", dt), _ptr(dkv, "dkv", torch.float32),
                                   _ptr(dent, "dent", torch.float32, optional=True),
                                   _ptr(dsink, "dsink", torch.float32, optional=True),
                                   _ptr(workspace, "workspace", torch.uint8), workspace.numel(),
                                   _stream(stream)))
    return dq, dkv, dent, dsink


def v4_q_proj(cfg, qlat, wq, q, q_norm=1, q_norm_w=None, wiq=None, iq=None, stream=None):
    """q = (per-head RMSNorm of) qlat @ wq, and iq = qlat @ wiq when wiq is given."""
    _check(lib().v4_q_proj(C.byref(cfg), _ptr(qlat, "qlat", torch.bfloat16), int(qlat.shape[-1]),
                           _ptr(wq, "wq", torch.bfloat16), int(q_norm),
                           _ptr(q_norm_w, "q_norm_w", torch.float32, optional=True),
                           _ptr(wiq, "wiq", torch.bfloat16, optional=True), _ptr(q, "q", torch.bfloat16),
                           _ptr(iq, "iq", torch.bfloat16, optional=True), _stream(stream)))
    return q, iq


def v4_indexer_kl_target(cfg, q, ent, idx, lse, iscore, inv_freq, target, loss, dscore, workspace, stream=None):
    """Distillation target of the indexer (and, with iscore, the KL loss and its gradient)."""
    dt = _storage(cfg)
    _check(lib().v4_indexer_kl_target(C.byref(cfg), _ptr(q, "q", dt), _ptr(ent, "ent", dt, optional=True),
                                      _ptr(idx, "idx", torch.int32), _ptr(lse, "lse", torch.float32),
                                      _ptr(iscore, "iscore", torch.float32, optional=True),
                                      _ptr(inv_freq, "inv_freq", torch.float32, optional=True),
                                      _ptr(target, "target", torch.float32),
                                      _ptr(loss, "loss", torch.float32, optional=True),
                                      _ptr(dscore, "dscore", torch.float32, optional=True),
                                      _ptr(workspace, "workspace", torch.uint8), workspace.numel(), _stream(stream)))
    return target


def v4_grouped_o_proj(cfg, o, wo_a, y, stream=None):
    dt = _storage(cfg)
    _check(lib().v4_grouped_o_proj(C.byref(cfg), _ptr(o, "o", dt), _ptr(wo_a, "wo_a", dt),
                                   _ptr(y, "y", dt), _stream(stream)))
    return y


_IN_F32 = {"ape", "norm_w", "iape", "inorm_w", "w", "sink", "inv_freq"}


def v4_attn_layer_fwd(cfg, inputs, outputs, workspace, stream=None):
    """inputs / outputs: dicts keyed like v4_layer_inputs / v4_layer_outputs."""
    dt = _storage(cfg)
    vin = v4_layer_inputs()
    for name, _ in v4_layer_inputs._fields_:
        t = inputs.get(name)
        setattr(vin, name, _ptr(t, name, torch.float32 if name in _IN_F32 else dt, optional=True))
    vout = v4_layer_outputs()
    odt = {"lse": torch.float32, "iscore": torch.float32, "idx": torch.int32}
    for name, _ in v4_layer_outputs._fields_:
        t = outputs.get(name)
        setattr(vout, name, _ptr(t, name, odt.get(name, dt), optional=True))
    _check(lib().v4_attn_layer_fwd(C.byref(cfg), C.byref(vin), C.byref(vout),
                                   _ptr(workspace, "workspace", torch.uint8), workspace.numel(),
                                   _stream(stream)))
    return outputs


# The serving calls are short (a few microseconds on the device), so their
# checks are kept cheap: one combined test per tensor, the slow path only to
# say what is wrong, and the raw stream of the current device.
_device = getattr(torch._C, "_cuda_getDevice", None)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream_on(stream, dev):
    if stream is None:
        return _raw_stream(dev)
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else stream


def _current(t, name):
    """Index of the current device; a host tensor is refused before CUDA is touched."""
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a tensor" % name)
    if not t.is_cuda:
        raise ValueError("%s must be on a CUDA device" % name)
    return _device()


def _shaped(t, name, shape, dtype, dev):
    """Pointer of a dense tensor of exactly this shape on device `dev` (the current one)."""
    try:
        if t.dtype is dtype and t.shape == shape and t.get_device() == dev and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    _ptr(t, name, dtype)
    if t.get_device() != dev:
        raise ValueError("%s is on %s, the current device is cuda:%d" % (name, t.device, dev))
    raise ValueError("%s must have shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))


def _strided(t, name, dims, dev):
    """Pointer and strides of a tensor whose last dim is dense; the library checks the strides."""
    if isinstance(t, torch.Tensor) and t.get_device() == dev and t.dim() == dims and t.dtype in _STORAGE_CODE:
        st = t.stride()
        if st[-1] == 1 or t.shape[-1] <= 1:
            return t.data_ptr(), st
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a tensor" % name)
    if not t.is_cuda:
        raise ValueError("%s must be on a CUDA device" % name)
    if t.get_device() != dev:
        raise ValueError("%s is on %s, the current device is cuda:%d" % (name, t.device, dev))
    if t.dim() != dims:
        raise ValueError("%s must have %d dims, got %d" % (name, dims, t.dim()))
    if t.dtype not in _STORAGE_CODE:
        raise TypeError("%s must be bfloat16 or float32, got %s" % (name, t.dtype))
    raise ValueError("%s must be contiguous in its last dim" % name)


_STORAGE_CODE = {torch.bfloat16: V4_BF16, torch.float32: V4_F32}


def v4_rope(x, pos, inv_freq, out, rope_begin=None, layout=V4_ROPE_INTERLEAVED, inverse=False, mscale=1.0,
            stream=None):
    """Rotate dims [rope_begin, rope_begin + R) of x [rows, heads, dim] at pos [rows] into out (or in place).

    R = 2 * len(inv_freq); rope_begin defaults to the last R dims.  x and out may be
    strided views (dense last dim).  The gradient of x is the call on the gradient of out
    with inverse=True and the same mscale."""
    dev = _current(x, "x")
    px, sx = _strided(x, "x", 3, dev)
    po, so = _strided(out, "out", 3, dev)
    if out.shape != x.shape or out.dtype is not x.dtype:
        raise ValueError("out must have x's shape and type")
    rows, heads, dim = x.shape
    half = inv_freq.numel()
    if not rows or not heads or not dim:
        return out
    _check(lib().v4_rope(px, rows, heads, dim, sx[0], sx[1], _shaped(pos, "pos", (rows,), torch.int32, dev),
                         _shaped(inv_freq, "inv_freq", (half,), torch.float32, dev), 2 * half,
                         dim - 2 * half if rope_begin is None else rope_begin, layout, 1 if inverse else 0, mscale,
                         _STORAGE_CODE[x.dtype], po, so[0], so[1], _stream_on(stream, dev)))
    return out


def v4_cache_append(x, pos, inv_freq, slot, cache, stream=None):
    """Store rows x [rows, dim], rotated at pos (None: as they are), at rows slot of cache [..., dim]."""
    dev = _current(x, "x")
    px, sx = _strided(x, "x", 2, dev)
    rows, dim = x.shape
    if not isinstance(cache, torch.Tensor) or cache.dim() < 2 or cache.shape[-1] != dim:
        raise ValueError("cache must be a tensor [..., %d]" % dim)
    pc = _shaped(cache, "cache", cache.shape, x.dtype, dev)
    if not rows or not dim:
        return cache
    half = 0 if pos is None else inv_freq.numel()
    _check(lib().v4_cache_append(px, rows, dim, sx[0],
                                 None if pos is None else _shaped(pos, "pos", (rows,), torch.int32, dev),
                                 None if pos is None else _shaped(inv_freq, "inv_freq", (half,), torch.float32, dev),
                                 2 * half, _shaped(slot, "slot", (rows,), torch.int32, dev), cache.numel() // dim,
                                 _STORAGE_CODE[x.dtype], pc, _stream_on(stream, dev)))
    return cache


def v4_tree_plan(node_begin, seq_len, parent, plan, pos=None, slot=None, block_table=None, page_size=0, n_slots=0,
                 stream=None):
    """Describe drafted trees (see the header): plan [n_rows, 8], and optionally pos and slot [n_rows]."""
    dev = _current(plan, "plan")
    B, n = seq_len.numel(), plan.shape[0]
    i32 = torch.int32
    blocks = 0
    if slot is not None:
        if not isinstance(block_table, torch.Tensor) or block_table.dim() != 2:
            raise ValueError("slot needs block_table [batch, max_blocks]")
        blocks = block_table.shape[1]
    if n == 0:
        return plan
    _check(lib().v4_tree_plan(B, n, _shaped(node_begin, "node_begin", (B + 1,), i32, dev),
                              _shaped(seq_len, "seq_len", (B,), i32, dev),
                              None if parent is None else _shaped(parent, "parent", (n,), i32, dev),
                              None if slot is None else _shaped(block_table, "block_table", (B, blocks), i32, dev),
                              blocks, int(page_size), int(n_slots), _shaped(plan, "plan", (n, 8), i32, dev),
                              None if pos is None else _shaped(pos, "pos", (n,), i32, dev),
                              None if slot is None else _shaped(slot, "slot", (n,), i32, dev),
                              _stream_on(stream, dev)))
    return plan


def v4_tree_workspace_size(cfg, n_rows):
    n = C.c_size_t(0)
    _check(lib().v4_tree_workspace_size(C.byref(cfg), int(n_rows), C.byref(n)))
    return n.value


def alloc_tree_workspace(cfg, n_rows, device=None):
    return torch.empty(max(v4_tree_workspace_size(cfg, n_rows), 256), dtype=torch.uint8, device=device or "cuda")


def _paged(cache, table, kind, D, B, dt, dev):
    """Cache pointer, table pointer, slots, blocks, page size of one paged cache."""
    try:
        pages, page, width = cache.shape
        blocks = table.shape[1]
        if width == D and cache.dtype is dt and cache.get_device() == dev and cache.is_contiguous():
            return (cache.data_ptr(), _shaped(table, kind + "_table", (B, blocks), torch.int32, dev), pages * page, blocks,
                    page)
    except (AttributeError, ValueError, IndexError):
        pass
    if not isinstance(cache, torch.Tensor) or cache.dim() != 3 or cache.shape[2] != D:
        raise ValueError("%s_cache must be a tensor [pages, page_size, %d]" % (kind, D))
    _shaped(cache, kind + "_cache", cache.shape, dt, dev)
    if not isinstance(table, torch.Tensor) or table.dim() != 2:
        raise ValueError("%s_table must be a tensor [batch, blocks]" % kind)
    _shaped(table, kind + "_table", (B, table.shape[1]), torch.int32, dev)
    raise ValueError("%s_cache and %s_table cannot be used" % (kind, kind))


def v4_tree_mqa_fwd(cfg, inputs, o, lse, workspace, stream=None):
    """Attention of planned rows over paged caches.  inputs: a dict keyed like v4_tree_inputs' pointers, with
    tok_cache / ent_cache [pages, page_size, D] and tok_table / ent_table [B, blocks].  workspace may be None where
    v4_tree_workspace_size is 0."""
    i32, f32 = torch.int32, torch.float32
    get = inputs.get
    q, sink = inputs["q"], get("sink")
    dev = _current(q, "q")
    H, D, B, r, K, half, dt = cfg.n_heads, cfg.head_dim, cfg.batch, cfg.ratio, cfg.topk, cfg.rope_dim // 2, _storage(cfg)
    n = q.shape[0]
    shape = (n, H, D)
    tc = tt = ec = et = el = ix = None
    ts = tb = tp = es = eb = ep = 0
    if cfg.window:
        tc, tt, ts, tb, tp = _paged(get("tok_cache"), get("tok_table"), "tok", D, B, dt, dev)
    if r > 0:
        ec, et, es, eb, ep = _paged(get("ent_cache"), get("ent_table"), "ent", D, B, dt, dev)
        el = _shaped(get("ent_len"), "ent_len", (B,), i32, dev)
        if K > 0:
            ix = _shaped(get("idx"), "idx", (n, K), i32, dev)
    vin = v4_tree_inputs(
        _shaped(q, "q", shape, dt, dev), _shaped(inputs["plan"], "plan", (n, 8), i32, dev), tc, tt, ec, et, el, ix,
        None if sink is None else _shaped(sink, "sink", (H,), f32, dev),
        _shaped(get("inv_freq"), "inv_freq", (half,), f32, dev) if half else None, ts, es, n, tb, tp, eb, ep)
    size = 0 if workspace is None else workspace.numel()
    st = lib().v4_tree_mqa_fwd(cfg, vin, _shaped(o, "o", shape, dt, dev),
                               None if lse is None else _shaped(lse, "lse", (n, H), f32, dev),
                               None if workspace is None else _shaped(workspace, "workspace", (size,), torch.uint8, dev),
                               size, _stream_on(stream, dev))
    if st:
        _check(st)
    return o


def v4_w4_pack(w, group_size, codes, scales, stream=None):
    """Quantise w [groups, K, N] bf16 to codes [groups, N, K/2] uint8 and scales [groups, N, K/group_size] bf16."""
    dev = _current(w, "w")
    if w.dim() != 3:
        raise ValueError("w must be a tensor [groups, K, N]")
    G, K, N = w.shape
    gs = int(group_size)
    if gs not in (32, 64, 128):
        raise ValueError("group_size must be 32, 64 or 128")
    _check(lib().v4_w4_pack(_shaped(w, "w", (G, K, N), torch.bfloat16, dev), G, K, N, gs,
                            _shaped(codes, "codes", (G, N, K // 2), torch.uint8, dev),
                            _shaped(scales, "scales", (G, N, K // gs), torch.bfloat16, dev), _stream_on(stream, dev)))
    return codes, scales


def v4_w4_proj(x, codes, scales, y, norm_dim=0, eps=1e-6, norm_w=None, stream=None):
    """y [rows, groups, N] = x [rows, groups, K] . dequantised weights, RMS-normalised over runs of norm_dim outputs."""
    if not isinstance(codes, torch.Tensor) or codes.dim() != 3 or not isinstance(scales, torch.Tensor) or scales.dim() != 3:
        raise ValueError("codes must be [groups, N, K/2] and scales [groups, N, K/group_size]")
    dev = _current(x, "x")
    G, N, half = codes.shape
    K, sg, rows, b16 = 2 * half, scales.shape[2], x.shape[0], torch.bfloat16
    if sg < 1 or K % sg:
        raise ValueError("scales must have shape [groups, N, K/group_size]")
    px, py = _shaped(x, "x", (rows, G, K), b16, dev), _shaped(y, "y", (rows, G, N), b16, dev)
    _check(lib().v4_w4_proj(px, rows, G, K, N, K // sg, _shaped(codes, "codes", (G, N, half), torch.uint8, dev),
                            _shaped(scales, "scales", (G, N, sg), b16, dev), norm_dim, eps,
                            _shaped(norm_w, "norm_w", (norm_dim,), torch.float32, dev) if norm_w is not None and norm_dim
                            else None, py, _stream_on(stream, dev)))
    return y


def v4_last_error():
    return lib().v4_last_error().decode()


def v4_build_info():
    return lib().v4_build_info().decode()


def v4_get_device_status(stream=None):
    v = C.c_int32(0)
    _check(lib().v4_get_device_status(_stream(stream), C.byref(v)))
    return v.value


def v4_reset_device_status(stream=None):
    _check(lib().v4_reset_device_status(_stream(stream)))


def v4_selftest_wait_timeout(limit_us, stream=None):
    """Launch the self-test kernel whose bounded wait runs out (see the header)."""
    _check(lib().v4_selftest_wait_timeout(int(limit_us), _stream(stream)))


def v4_launch_count():
    return int(lib().v4_launch_count())


def v4_profile_enable(on=True):
    _check(lib().v4_profile_enable(1 if on else 0))


def v4_profile_count():
    return int(lib().v4_profile_count())


def v4_profile_get(i):
    """(kind name, milliseconds) of launch record i."""
    k, ms = C.c_int32(0), C.c_float(0.0)
    _check(lib().v4_profile_get(int(i), C.byref(k), C.byref(ms)))
    return PROFILE_KINDS.get(k.value, str(k.value)), float(ms.value)


def v4_profile_records():
    return [v4_profile_get(i) for i in range(v4_profile_count())]
