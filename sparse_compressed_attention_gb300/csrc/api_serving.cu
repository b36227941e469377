// C ABI of the serving operators: rotary positions, the paged cache write,
// drafted token trees and 4-bit projections.  Argument checks and dispatch.
#include <math.h>
#include <stdio.h>

#include "checks.h"
#include "common.cuh"
#include "internal.h"
#include "tree.cuh"

namespace v4 {

// Rows of a call: far above what memory holds, low enough for 32-bit row loops.
constexpr int32_t kMaxRows = 1 << 24;

static v4_status check_rows(int32_t n_rows) {
  if (n_rows < 0 || n_rows > kMaxRows) return bad("n_rows must be in [0, 2^24]");
  return V4_OK;
}

// The configuration as the tree attention reads it.  What it has no use for (the
// length, the compressor's and the indexer's fields) may hold anything.
static v4_status tree_config(const v4_config* cfg, v4_config* c) {
  if (!cfg) return validate_config(cfg);
  *c = *cfg;
  c->seqlen = 1;
  c->overlap = c->indexer_fp8 = c->q_begin = 0;
  c->topk = 0;                                   // with one the indexer's fields are checked
  c->rms_eps = 0.f;
  TRY(validate_config(c));
  if (cfg->topk < 0) return bad("topk must be >= 0");
  if (cfg->topk > 0 && cfg->ratio < 1) return bad("topk needs ratio >= 1");
  c->topk = cfg->topk;
  return V4_OK;
}

static bool tree_on_tc(const v4_config& c) { return tree_tc_supported(c) && c.path != V4_PATH_SIMT; }

}  // namespace v4

using namespace v4;

extern "C" {

v4_status v4_rope(const void* x, int64_t rows, int32_t heads, int32_t dim, int64_t x_row_stride, int64_t x_head_stride,
                  const int32_t* pos, const float* inv_freq, int32_t rope_dim, int32_t rope_begin, int32_t layout,
                  int32_t inverse, float mscale, int32_t dtype, void* out, int64_t out_row_stride,
                  int64_t out_head_stride, void* stream) {
  TRY(check_rotation(rows, dim, rope_dim, rope_begin, layout, dtype));
  if (heads < 1 || heads > 65535) return bad("heads must be in [1, 65535]");
  if (inverse != 0 && inverse != 1) return bad("inverse must be 0 or 1");
  if (!isfinite(mscale)) return bad("mscale must be finite");
  const int es = dtype == V4_BF16 ? 2 : 4;
  TRY(check_stride(x_row_stride, es, "x_row_stride"));
  TRY(check_stride(x_head_stride, es, "x_head_stride"));
  TRY(check_stride(out_row_stride, es, "out_row_stride"));
  TRY(check_stride(out_head_stride, es, "out_head_stride"));
  if (rows == 0) return V4_OK;
  TRY(check_ptr(x, "x"));
  TRY(check_ptr(out, "out"));
  TRY(check_ptr(pos, "pos"));
  if (rope_dim > 0) TRY(check_ptr(inv_freq, "inv_freq"));
  // out's (row, head) runs of dim elements must be apart from each other
  const int64_t rs = out_row_stride, hs = out_head_stride;
  const bool rows_outer = (heads == 1 || hs >= dim) && (rows == 1 || rs >= (heads - 1) * hs + dim);
  const bool heads_outer = (rows == 1 || rs >= dim) && (heads == 1 || hs >= (rows - 1) * rs + dim);
  if (!rows_outer && !heads_outer) return bad("out's rows or heads overlap");
  const bool same = x == out && (rows == 1 || x_row_stride == rs) && (heads == 1 || x_head_stride == hs);
  if (!same && overlap(x, extent(rows, heads, dim, x_row_stride, x_head_stride, es), out,
                       extent(rows, heads, dim, rs, hs, es))) {
    // two views of one buffer that step alike, as parts of a head or runs of heads
    const int64_t step = (intptr_t)out - (intptr_t)x;
    const bool alike = step % es == 0 && (rows == 1 || x_row_stride == rs) && (heads == 1 || x_head_stride == hs);
    const bool apart = alike && !(rows_outer ? views_meet(step / es, rows, rs, heads, hs, dim)
                                             : views_meet(step / es, heads, hs, rows, rs, dim));
    if (!apart) return bad("x and out overlap and are not the same tensor");
  }
  RopeCall c;
  c.x = x;
  c.out = out;
  c.pos = pos;
  c.inv_freq = inv_freq;
  c.slot = nullptr;
  c.n_slots = 0;
  c.rows = rows;
  c.x_row_stride = x_row_stride;
  c.x_head_stride = x_head_stride;
  c.out_row_stride = rs;
  c.out_head_stride = hs;
  c.heads = heads;
  c.dim = dim;
  c.rope_dim = rope_dim;
  c.rope_begin = rope_begin;
  c.layout = layout;
  c.inverse = inverse;
  c.dtype = dtype;
  c.mscale = mscale;
  StageTiming ps(13, (cudaStream_t)stream);
  return cuda_result(launch_rope(c, nullptr, (cudaStream_t)stream), "rotation kernel");
}

v4_status v4_cache_append(const void* x, int64_t rows, int32_t dim, int64_t x_row_stride, const int32_t* pos,
                          const float* inv_freq, int32_t rope_dim, const int32_t* slot, int64_t n_slots, int32_t dtype,
                          void* cache, void* stream) {
  const int32_t R = pos ? rope_dim : 0;
  TRY(check_rotation(rows, dim, R, dim - R, V4_ROPE_INTERLEAVED, dtype));
  const int es = dtype == V4_BF16 ? 2 : 4;
  TRY(check_stride(x_row_stride, es, "x_row_stride"));
  if (n_slots < 0 || n_slots > 0x7FFFFFFF) return bad("n_slots must be in [0, 2^31)");
  if (rows == 0) return V4_OK;
  TRY(check_ptr(x, "x"));
  TRY(check_ptr(slot, "slot"));
  TRY(check_ptr(cache, "cache"));
  TRY(check_ptr(pos, "pos", false));
  if (R > 0) TRY(check_ptr(inv_freq, "inv_freq"));
  if (n_slots > 0 && overlap(x, extent(rows, 1, dim, x_row_stride, 0, es), cache, n_slots * dim * es))
    return bad("x and cache overlap");
  int* status = device_status_ptr();
  if (!status) return set_error(V4_ERR_CUDA, "device status word unavailable");
  RopeCall c;
  c.x = x;
  c.out = cache;
  c.pos = pos;
  c.inv_freq = inv_freq;
  c.slot = slot;
  c.n_slots = n_slots;
  c.rows = rows;
  c.x_row_stride = x_row_stride;
  c.x_head_stride = 0;
  c.out_row_stride = dim;
  c.out_head_stride = 0;
  c.heads = 1;
  c.dim = dim;
  c.rope_dim = R;
  c.rope_begin = dim - R;
  c.layout = V4_ROPE_INTERLEAVED;
  c.inverse = 0;
  c.dtype = dtype;
  c.mscale = 1.f;
  StageTiming ps(14, (cudaStream_t)stream);
  return cuda_result(launch_rope(c, status, (cudaStream_t)stream), "cache write kernel");
}

v4_status v4_tree_plan(int32_t batch, int32_t n_rows, const int32_t* node_begin, const int32_t* seq_len,
                       const int32_t* parent, const int32_t* block_table, int32_t max_blocks, int32_t page_size,
                       int64_t n_slots, int32_t* plan, int32_t* pos, int32_t* slot, void* stream) {
  if (batch < 1 || batch > (1 << 24)) return bad("batch must be in [1, 2^24]");
  TRY(check_rows(n_rows));
  if (slot) {
    TRY(check_ptr(block_table, "block_table"));
    if (max_blocks < 1) return bad("max_blocks must be >= 1");
    if (page_size < 1) return bad("page_size must be >= 1");
    if (n_slots < 0 || n_slots > 0x7FFFFFFF) return bad("n_slots must be in [0, 2^31)");
  }
  if (n_rows == 0) return V4_OK;
  TRY(check_ptr(node_begin, "node_begin"));
  TRY(check_ptr(seq_len, "seq_len"));
  TRY(check_ptr(parent, "parent", false));
  TRY(check_ptr(plan, "plan"));
  TRY(check_ptr(pos, "pos", false));
  TRY(check_ptr(slot, "slot", false));
  int* status = device_status_ptr();
  if (!status) return set_error(V4_ERR_CUDA, "device status word unavailable");
  StageTiming ps(15, (cudaStream_t)stream);
  return cuda_result(launch_tree_plan(batch, n_rows, node_begin, seq_len, parent, block_table, max_blocks, page_size,
                                      n_slots, plan, pos, slot, status, (cudaStream_t)stream),
                     "tree plan kernel");
}

v4_status v4_tree_workspace_size(const v4_config* cfg, int32_t n_rows, size_t* bytes) {
  v4_config c;
  TRY(tree_config(cfg, &c));
  if (!bytes) return bad("bytes is NULL");
  TRY(check_rows(n_rows));
  *bytes = tree_on_tc(c) ? tree_tc_workspace() : 0;
  return V4_OK;
}

static v4_status tree_fwd(const v4_config* cfg, const v4_tree_inputs* in, bool q4, void* o, float* lse,
                          void* workspace, size_t ws_bytes, void* stream) {
  v4_config c;
  TRY(tree_config(cfg, &c));
  if (!in) return bad("inputs struct is NULL");
  if (cfg->q_begin != 0) return set_error(V4_ERR_UNSUPPORTED, "the tree attention needs q_begin = 0");
  TRY(check_rows(in->n_rows));
  const bool tc = tree_on_tc(c);
  if (c.path == V4_PATH_TC && !tc)
    return set_error(V4_ERR_UNSUPPORTED, "tensor-core tree attention needs bf16, H a multiple of 64 up to 512, D=512, R=64");
  if (in->n_rows == 0) return V4_OK;
  TRY(check_ptr(in->q, "q"));
  TRY(check_ptr(in->plan, "plan"));
  TRY(check_ptr(o, "o"));
  TRY(check_ptr(lse, "lse", false));
  TRY(check_ptr(in->sink, "sink", false));
  if (c.rope_dim > 0) TRY(check_ptr(in->inv_freq, "inv_freq"));
  if (c.window != 0) {
    TRY(check_ptr(in->tok_cache, "tok_cache"));
    TRY(check_ptr(in->tok_table, "tok_table"));
    if (in->tok_blocks < 1 || in->tok_page < 1) return bad("tok_blocks and tok_page must be >= 1");
    if (in->tok_slots < 1 || in->tok_slots > 0x7FFFFFFF) return bad("tok_slots must be in [1, 2^31)");
  }
  if (c.ratio > 0) {
    TRY(check_ptr(in->ent_cache, "ent_cache"));
    TRY(check_ptr(in->ent_table, "ent_table"));
    TRY(check_ptr(in->ent_len, "ent_len"));
    if (in->ent_blocks < 1 || in->ent_page < 1) return bad("ent_blocks and ent_page must be >= 1");
    if (in->ent_slots < 1 || in->ent_slots > 0x7FFFFFFF) return bad("ent_slots must be in [1, 2^31)");
    if (c.topk > 0) TRY(check_ptr(in->idx, "idx"));
  }
  if (q4 && (((c.window != 0 ? (uintptr_t)in->tok_cache : 0) | (c.ratio > 0 ? (uintptr_t)in->ent_cache : 0)) & 31u))
    return bad("4-bit caches must be 32-byte aligned");
  size_t need = 0;
  TRY(v4_tree_workspace_size(cfg, in->n_rows, &need));
  if (ws_bytes < need) {
    char buf[128];
    snprintf(buf, sizeof(buf), "workspace of %zu bytes, %zu needed", ws_bytes, need);
    return set_error(V4_ERR_WORKSPACE, buf);
  }
  if (need > 0 && !workspace) return set_error(V4_ERR_WORKSPACE, "workspace is NULL");
  if ((uintptr_t)workspace & 255u) return set_error(V4_ERR_WORKSPACE, "workspace not 256-byte aligned");
  const int64_t out_bytes = (int64_t)in->n_rows * c.n_heads * c.head_dim * (c.dtype == V4_BF16 ? 2 : 4);
  if (overlap(in->q, out_bytes, o, out_bytes)) return bad("q and o overlap");
  if (tc) {
    // the kernel counts tiles of 128 keys in 32 bits
    const int64_t tok = (int64_t)in->tok_blocks * in->tok_page, ent = (int64_t)in->ent_blocks * in->ent_page;
    const int64_t keys = (c.ratio == 0 ? 0 : c.topk > 0 ? c.topk : ent) +
                         (c.window == 0 ? 0 : c.window < 0 || c.window > tok ? tok : c.window) + V4_TREE_MAX_NODES;
    if (keys > (int64_t)1 << 36 || (keys / 128 + 2) * in->n_rows * (c.n_heads / 64) > (int64_t)1 << 30)
      return set_error(V4_ERR_UNSUPPORTED,
                       "n_rows times the longest key list that the tables allow is above 2^30 tiles of 128 keys");
  }
  int* status = device_status_ptr();
  if (!status) return set_error(V4_ERR_CUDA, "device status word unavailable");
  TreeArgs a;
  a.q = in->q;
  a.plan = in->plan;
  a.tok_cache = in->tok_cache;
  a.tok_table = in->tok_table;
  a.ent_cache = in->ent_cache;
  a.ent_table = in->ent_table;
  a.ent_len = in->ent_len;
  a.idx = c.topk > 0 ? in->idx : nullptr;
  a.sink = in->sink;
  a.inv_freq = in->inv_freq;
  a.tok_slots = in->tok_slots;
  a.ent_slots = in->ent_slots;
  a.n_rows = in->n_rows;
  a.tok_blocks = in->tok_blocks;
  a.tok_page = in->tok_page;
  a.ent_blocks = in->ent_blocks;
  a.ent_page = in->ent_page;
  a.o = o;
  a.lse = lse;
  a.status = status;
  a.B = c.batch;
  a.H = c.n_heads;
  a.D = c.head_dim;
  a.R = c.rope_dim;
  a.ratio = c.ratio;
  a.window = c.window;
  a.K = c.ratio > 0 ? c.topk : 0;
  a.scale = c.softmax_scale > 0.f ? c.softmax_scale : 1.0f / sqrtf((float)c.head_dim);
  cudaStream_t st = (cudaStream_t)stream;
  return cuda_result(tc ? launch_tree_tc(a, q4, workspace, st) : launch_tree_simt(a, c.dtype, q4, st),
                     "tree attention kernel");
}

v4_status v4_tree_mqa_fwd(const v4_config* cfg, const v4_tree_inputs* in, void* o, float* lse, void* workspace,
                          size_t ws_bytes, void* stream) {
  return tree_fwd(cfg, in, false, o, lse, workspace, ws_bytes, stream);
}

v4_status v4_tree_mqa_fwd_q4(const v4_config* cfg, const v4_tree_inputs* in, void* o, float* lse, void* workspace,
                             size_t ws_bytes, void* stream) {
  return tree_fwd(cfg, in, true, o, lse, workspace, ws_bytes, stream);
}

static v4_status check_w4(int32_t groups, int32_t K, int32_t N, int32_t group_size) {
  if (groups < 1 || K < 1 || N < 1) return bad("groups, K and N must be >= 1");
  if (K % 128 || N % 64 || (group_size != 32 && group_size != 64 && group_size != 128) || groups > 65535 ||
      K > (1 << 20) || N > (1 << 24))
    return set_error(V4_ERR_UNSUPPORTED, "4-bit weights need K a multiple of 128 up to 2^20, N a multiple of 64 up to "
                                         "2^24, group_size 32, 64 or 128, at most 65535 groups");
  return V4_OK;
}

v4_status v4_w4_pack(const void* w, int32_t groups, int32_t K, int32_t N, int32_t group_size, uint8_t* codes,
                     void* scales, void* stream) {
  TRY(check_w4(groups, K, N, group_size));
  TRY(check_ptr(w, "w"));
  TRY(check_ptr(codes, "codes"));
  TRY(check_ptr(scales, "scales"));
  StageTiming ps(18, (cudaStream_t)stream);
  return cuda_result(launch_w4_pack(w, groups, K, N, group_size, codes, scales, (cudaStream_t)stream),
                     "4-bit packing kernel");
}

v4_status v4_w4_proj(const void* x, int64_t rows, int32_t groups, int32_t K, int32_t N, int32_t group_size,
                     const uint8_t* codes, const void* scales, int32_t norm_dim, float eps, const float* norm_w,
                     void* y, void* stream) {
  TRY(check_w4(groups, K, N, group_size));
  if (rows < 0 || rows > (1 << 21)) return bad("rows must be in [0, 2^21]");
  if (norm_dim != 0 && norm_dim != 64 && norm_dim != 128 && norm_dim != 256 && norm_dim != 512)
    return set_error(V4_ERR_UNSUPPORTED, "norm_dim must be 0, 64, 128, 256 or 512");
  if (norm_dim > 0 && N % norm_dim) return set_error(V4_ERR_UNSUPPORTED, "norm_dim must divide N");
  if (norm_dim > 0 && !(eps >= 0.f)) return bad("eps must be >= 0");
  if (rows == 0) return V4_OK;
  TRY(check_ptr(x, "x"));
  TRY(check_ptr(codes, "codes"));
  TRY(check_ptr(scales, "scales"));
  TRY(check_ptr(norm_w, "norm_w", false));
  TRY(check_ptr(y, "y"));
  if (overlap(x, rows * groups * K * 2, y, rows * groups * N * 2)) return bad("x and y overlap");
  StageTiming ps(19, (cudaStream_t)stream);
  return cuda_result(launch_w4_proj(x, rows, groups, K, N, group_size, codes, scales, norm_dim, eps,
                                    norm_dim > 0 ? norm_w : nullptr, y, (cudaStream_t)stream),
                     "4-bit projection kernel");
}

}  // extern "C"
