// C ABI of the operators around a serving cache: norms with the rotation, rows of
// the 4-bit cache, pages.  Argument checks and dispatch.
#include <math.h>
#include <stdio.h>

#include "checks.h"
#include "common.cuh"
#include "internal.h"
#include "q4.cuh"

namespace v4 {

// A strided tensor [rows, heads, dim] of es-byte elements.
struct View {
  const void* p;
  int64_t rows, heads, dim, rs, hs;
  int es;
  int64_t bytes() const { return extent(rows, heads, dim, rs, hs, es); }
};

static v4_status check_view(const View& v, const char* name) {
  char buf[96];
  snprintf(buf, sizeof(buf), "%s row stride", name);
  TRY(check_stride(v.rs, v.es, buf));
  snprintf(buf, sizeof(buf), "%s head stride", name);
  TRY(check_stride(v.hs, v.es, buf));
  TRY(check_ptr(v.p, name));
  if ((double)(v.rows - 1) * (double)v.rs + (double)(v.heads - 1) * (double)v.hs > 1e15) {
    snprintf(buf, sizeof(buf), "%s reaches above 10^15 elements", name);
    return bad(buf);
  }
  return V4_OK;
}

static bool same_view(const View& a, const View& b) {
  return a.p == b.p && a.heads == b.heads && (a.rows == 1 || a.rs == b.rs) && (a.heads == 1 || a.hs == b.hs);
}

// Whether two views of the same number of rows certainly have no element in common.
static bool apart(const View& a, const View& b) {
  if (!overlap(a.p, a.bytes(), b.p, b.bytes())) return true;
  if (a.rows == 1 || a.rs != b.rs || a.rs == 0) return false;
  // parts of the same rows: each row's part ends before the next row's begins
  const int64_t step = a.rs * a.es, na = ((a.heads - 1) * a.hs + a.dim) * a.es, nb = ((b.heads - 1) * b.hs + b.dim) * b.es;
  const int64_t d = (((int64_t)((intptr_t)b.p - (intptr_t)a.p) % step) + step) % step;
  return na <= step && nb <= step && d >= na && d + nb <= step;
}

// Whether a view has an element among n bytes at p.  Its runs of dim values are nested (the
// inner runs of one outer step end before the next); where they are not, as a broadcast
// input's, everything from the first to the last element counts.
static bool meets(const View& v, const void* p, int64_t n) {
  if (p == nullptr || !overlap(v.p, v.bytes(), p, n)) return false;
  const bool rows_outer = v.rows > 1 && (v.heads == 1 || v.rs >= v.hs);
  const int64_t no = rows_outer ? v.rows : v.heads, so = (rows_outer ? v.rs : v.hs) * v.es;
  const int64_t ni = rows_outer ? v.heads : v.rows, si = (rows_outer ? v.hs : v.rs) * v.es, run = v.dim * v.es;
  if ((ni > 1 && si < run) || (no > 1 && so < (ni - 1) * si + run)) return true;
  const int64_t span = (ni - 1) * si + run, at = (int64_t)((intptr_t)p - (intptr_t)v.p);
  // outer steps whose span reaches behind `at`, the first of them: of three that begin below
  // at + n, the middle one begins among the bytes
  const int64_t o0 = no > 1 && at >= span ? (at - span) / so + 1 : 0;
  for (int64_t o = o0; o < no && o < o0 + 3 && o * so < at + n; ++o) {
    const int64_t from = at - o * so;              // the bytes, relative to this step's first run
    const int64_t i0 = ni > 1 && from >= run ? (from - run) / si + 1 : 0;
    for (int64_t i = i0; i < ni && i < i0 + 1 && i * si < from + n; ++i)
      if (from < i * si + run) return true;
  }
  return false;
}

// An output: its rows and heads must not meet each other.
static v4_status check_out(const View& v, const char* name) {
  const bool rows_outer = (v.heads == 1 || v.hs >= v.dim) && (v.rows == 1 || v.rs >= (v.heads - 1) * v.hs + v.dim);
  const bool heads_outer = (v.rows == 1 || v.rs >= v.dim) && (v.heads == 1 || v.hs >= (v.rows - 1) * v.rs + v.dim);
  if (rows_outer || heads_outer) return V4_OK;
  char buf[96];
  snprintf(buf, sizeof(buf), "%s: rows or heads overlap", name);
  return bad(buf);
}

constexpr int kMaxNormDim = 1024;

static v4_status norm_rope(const v4_norm_rope_part* q, const v4_norm_rope_part* k, int64_t rows, int32_t dim,
                           const int32_t* pos, const float* inv_freq, int32_t rope_dim, int32_t rope_begin,
                           int32_t layout, float eps, int32_t dtype, bool grad, void* workspace, size_t ws_bytes,
                           cudaStream_t st) {
  if (!q) return bad("q struct is NULL");
  TRY(check_rotation(rows, dim, rope_dim, rope_begin, layout, dtype));
  if (dim > kMaxNormDim) return set_error(V4_ERR_UNSUPPORTED, "norms need dim <= 1024");
  if (!(eps >= 0.f) || !isfinite(eps)) return bad("eps must be finite and >= 0");
  const int es = dtype == V4_BF16 ? 2 : 4;
  const v4_norm_rope_part* part[2] = {q, k};
  const char* const names[2][4] = {{"q.x", "q.dy", "q.out", "q.heads"}, {"k.x", "k.dy", "k.out", "k.heads"}};
  for (int i = 0; i < 2; ++i) {
    const v4_norm_rope_part* s = part[i];
    if (s && (s->heads < 1 || s->heads > 65535)) {
      char buf[64];
      snprintf(buf, sizeof(buf), "%s must be in [1, 65535]", names[i][3]);
      return bad(buf);
    }
    if (s && rows * s->heads > (int64_t)1 << 30) return set_error(V4_ERR_UNSUPPORTED, "rows times heads above 2^30");
  }
  if (rows == 0 && !grad) return V4_OK;
  NormCall c;
  c.rows = rows;
  c.dim = dim;
  c.rope_dim = rope_dim;
  c.rope_begin = rope_begin;
  c.dtype = dtype;
  c.half = layout == V4_ROPE_HALF && rope_dim > 0;
  c.grad = grad;
  c.eps = eps;
  c.pos = pos;
  c.inv_freq = inv_freq;
  c.workspace = workspace;
  if (rows > 0 && rope_dim > 0) {
    TRY(check_ptr(pos, "pos"));
    TRY(check_ptr(inv_freq, "inv_freq"));
  }
  View in[4], out[2];
  int n_in = 0, n_out = 0;
  for (int i = 0; i < 2; ++i) {
    const v4_norm_rope_part* s = part[i];
    NormPartCall& d = c.part[i];
    d = NormPartCall();
    if (!s) continue;
    TRY(check_ptr(s->w, "weight", false));
    if (grad) TRY(check_ptr(s->dw, "weight gradient", false));
    d.dw = grad ? s->dw : nullptr;
    if (rows == 0) continue;
    const View x = {s->x, rows, s->heads, dim, s->x_row_stride, s->x_head_stride, es};
    const View dy = {s->dy, rows, s->heads, dim, s->dy_row_stride, s->dy_head_stride, es};
    const View y = {s->out, rows, s->heads, dim, s->out_row_stride, s->out_head_stride, es};
    TRY(check_view(x, names[i][0]));
    if (grad) TRY(check_view(dy, names[i][1]));
    TRY(check_view(y, names[i][2]));
    TRY(check_out(y, names[i][2]));
    d.x = s->x;
    d.dy = grad ? s->dy : nullptr;
    d.w = s->w;
    d.out = s->out;
    d.heads = s->heads;
    d.x_row_stride = x.rs;
    d.x_head_stride = x.hs;
    d.dy_row_stride = dy.rs;
    d.dy_head_stride = dy.hs;
    d.out_row_stride = y.rs;
    d.out_head_stride = y.hs;
    in[n_in++] = x;
    if (grad) in[n_in++] = dy;
    out[n_out++] = y;
  }
  for (int o = 0; o < n_out; ++o)
    for (int i = 0; i < n_in; ++i)
      if (!same_view(out[o], in[i]) && !apart(out[o], in[i]))
        return bad("an output overlaps an input and is not the same tensor");
  if (c.part[0].dw && c.part[1].dw && overlap(c.part[0].dw, (int64_t)dim * 4, c.part[1].dw, (int64_t)dim * 4))
    return bad("the weight gradients overlap");
  // the same tensor is read and written by the same lanes only within its own part
  if (n_out == 2) {
    if (!apart(out[0], out[1])) return bad("the outputs overlap");
    for (int i = 0; i < n_in; ++i) {
      const int own = i / (n_in / 2);
      if (!apart(out[1 - own], in[i])) return bad("an output overlaps an input of the other part");
    }
  }
  if (grad) {
    const size_t need = norm_rope_workspace(dim);
    if (ws_bytes < need) {
      char buf[128];
      snprintf(buf, sizeof(buf), "workspace of %zu bytes, %zu needed", ws_bytes, need);
      return set_error(V4_ERR_WORKSPACE, buf);
    }
    if (!workspace) return set_error(V4_ERR_WORKSPACE, "workspace is NULL");
    if ((uintptr_t)workspace & 255u) return set_error(V4_ERR_WORKSPACE, "workspace not 256-byte aligned");
  }
  // What all blocks read: no output may lie there (dw may, it is written when everything is read).
  const struct {
    const void* p;
    int64_t n;
  } shared[] = {{c.part[0].w, (int64_t)dim * 4}, {c.part[1].w, (int64_t)dim * 4}, {rope_dim > 0 ? pos : nullptr, rows * 4},
                {rope_dim > 0 ? inv_freq : nullptr, (int64_t)rope_dim * 2}};
  const int64_t scratch = grad ? (int64_t)norm_rope_workspace(dim) : 0;
  for (const auto& f : shared) {
    for (int o = 0; o < n_out; ++o)
      if (meets(out[o], f.p, f.n)) return bad("an output overlaps weights, positions or frequencies");
    if (grad && f.p && overlap(f.p, f.n, workspace, scratch)) return bad("the workspace overlaps an input");
  }
  if (grad) {
    for (int i = 0; i < n_in; ++i)
      if (meets(in[i], workspace, scratch)) return bad("the workspace overlaps an input");
    for (int o = 0; o < n_out; ++o)
      if (meets(out[o], workspace, scratch)) return bad("the workspace overlaps an output");
    for (const NormPartCall& d : c.part) {
      if (!d.dw) continue;
      if (overlap(d.dw, (int64_t)dim * 4, workspace, scratch)) return bad("the workspace overlaps a weight gradient");
      for (int o = 0; o < n_out; ++o)
        if (meets(out[o], d.dw, (int64_t)dim * 4)) return bad("an output overlaps a weight gradient");
    }
  }
  StageTiming ps(grad ? 21 : 20, st);
  return cuda_result(launch_norm_rope(c, st), "norm kernel");
}

static v4_status check_q4(int32_t dim, int32_t dtype) {
  if (dtype != V4_F32 && dtype != V4_BF16) return bad("unknown dtype");
  if (dim < 32 || dim > 8192 || dim % 32) return bad("dim must be a multiple of 32 in [32, 8192]");
  return V4_OK;
}

static v4_status q4_rows(const void* x, void* out, int64_t rows, int32_t dim, int64_t stride, const int32_t* slot,
                         int64_t n_slots, int32_t dtype, void* cache, cudaStream_t st) {
  const bool read = x == nullptr && out != nullptr;
  TRY(check_q4(dim, dtype));
  const int es = dtype == V4_BF16 ? 2 : 4;
  if (rows < 0 || rows > (1 << 24)) return bad("rows must be in [0, 2^24]");
  if (rows * (dim / kQ4Group) > 0x7FFFFFFF) return bad("rows times dim above 2^35");
  TRY(check_stride(stride, es, "row stride"));
  if ((double)rows * (double)stride > 1e15) return bad("rows reach above 10^15 elements");
  if (n_slots < 0 || n_slots > 0x7FFFFFFF) return bad("n_slots must be in [0, 2^31)");
  if (read && rows > 1 && stride < dim) return bad("out's rows overlap");
  if (rows == 0) return V4_OK;
  TRY(check_ptr(read ? out : x, read ? "out" : "x"));
  TRY(check_ptr(slot, "slot"));
  TRY(check_ptr(cache, "cache"));
  if (n_slots > 0 && overlap(read ? out : x, extent(rows, 1, dim, stride, 0, es), cache, n_slots * q4_row_bytes(dim)))
    return bad(read ? "out and cache overlap" : "x and cache overlap");
  int* status = device_status_ptr();
  if (!status) return set_error(V4_ERR_CUDA, "device status word unavailable");
  Q4Call c;
  c.x = x;
  c.out = read ? out : nullptr;
  c.cache = cache;
  c.slot = slot;
  c.n_slots = n_slots;
  c.rows = rows;
  c.row_stride = stride;
  c.dim = dim;
  c.dtype = dtype;
  StageTiming ps(read ? 23 : 22, st);
  return cuda_result(launch_q4_rows(c, status, st), read ? "4-bit read kernel" : "4-bit write kernel");
}

static v4_status check_table(const void* table, const char* name, int32_t n, int32_t blocks, int32_t page_size) {
  if (n < 0 || n > (1 << 24)) return bad("the number of sequences must be in [0, 2^24]");
  if (blocks < 1) return bad("blocks must be >= 1");
  if (page_size < 1) return bad("page_size must be >= 1");
  if ((int64_t)n * blocks > 0x7FFFFFFF) return bad("a table has more than 2^31 - 1 entries");
  if (n == 0) return V4_OK;
  return check_ptr(table, name);
}

static v4_status check_pool(const void* ref, int32_t pages) {
  if (pages < 1 || pages > 0x7FFFFFFF - 8192) return bad("pages must be in [1, 2^31 - 8192)");
  return check_ptr(ref, "ref");
}

static v4_status check_cache(const void* cache, int32_t layers, int64_t layer_stride, int32_t pages, int32_t page_size,
                             int32_t row_bytes) {
  if (layers < 1 || layers > 65535) return bad("layers must be in [1, 65535]");
  if (pages < 1 || page_size < 1) return bad("pages and page_size must be >= 1");
  if (row_bytes < 16 || row_bytes % 16) return bad("row_bytes must be a multiple of 16");
  if ((int64_t)page_size * row_bytes > (int64_t)1 << 30) return bad("a page has more than 2^30 bytes");
  if ((int64_t)pages * page_size > 0x7FFFFFFF) return bad("a layer has more than 2^31 - 1 rows");
  if (layers > 1 && (layer_stride % 16 || layer_stride < (int64_t)pages * page_size * row_bytes))
    return bad("layer_stride must be a multiple of 16 that holds a layer");
  return check_ptr(cache, "cache");
}

static v4_status status_word(int** status) {
  *status = device_status_ptr();
  return *status ? V4_OK : set_error(V4_ERR_CUDA, "device status word unavailable");
}

}  // namespace v4

using namespace v4;

extern "C" {

v4_status v4_norm_rope_fwd(const v4_norm_rope_part* q, const v4_norm_rope_part* k, int64_t rows, int32_t dim,
                           const int32_t* pos, const float* inv_freq, int32_t rope_dim, int32_t rope_begin,
                           int32_t layout, float eps, int32_t dtype, void* stream) {
  return norm_rope(q, k, rows, dim, pos, inv_freq, rope_dim, rope_begin, layout, eps, dtype, false, nullptr, 0,
                   (cudaStream_t)stream);
}

v4_status v4_norm_rope_workspace_size(int32_t dim, size_t* bytes) {
  if (dim < 8 || dim > kMaxNormDim || dim % 8) return bad("dim must be a multiple of 8 in [8, 1024]");
  if (!bytes) return bad("bytes is NULL");
  *bytes = norm_rope_workspace(dim);
  return V4_OK;
}

v4_status v4_norm_rope_bwd(const v4_norm_rope_part* q, const v4_norm_rope_part* k, int64_t rows, int32_t dim,
                           const int32_t* pos, const float* inv_freq, int32_t rope_dim, int32_t rope_begin,
                           int32_t layout, float eps, int32_t dtype, void* workspace, size_t ws_bytes, void* stream) {
  return norm_rope(q, k, rows, dim, pos, inv_freq, rope_dim, rope_begin, layout, eps, dtype, true, workspace,
                   ws_bytes, (cudaStream_t)stream);
}

v4_status v4_q4_row_bytes(int32_t dim, int32_t* bytes) {
  TRY(check_q4(dim, V4_BF16));
  if (!bytes) return bad("bytes is NULL");
  *bytes = q4_row_bytes(dim);
  return V4_OK;
}

v4_status v4_cache_append_q4(const void* x, int64_t rows, int32_t dim, int64_t x_row_stride, const int32_t* slot,
                             int64_t n_slots, int32_t dtype, void* cache, void* stream) {
  if (rows > 0 && !x) return bad("x is NULL");
  return q4_rows(x, nullptr, rows, dim, x_row_stride, slot, n_slots, dtype, cache, (cudaStream_t)stream);
}

v4_status v4_cache_read_q4(const void* cache, int64_t n_slots, const int32_t* slot, int64_t rows, int32_t dim,
                           int32_t dtype, void* out, int64_t out_row_stride, void* stream) {
  if (rows > 0 && !out) return bad("out is NULL");
  return q4_rows(nullptr, out, rows, dim, out_row_stride, slot, n_slots, dtype, const_cast<void*>(cache),
                 (cudaStream_t)stream);
}

v4_status v4_pages_alloc(int32_t n, int32_t* table, int32_t blocks, int32_t page_size, const int32_t* have,
                         const int32_t* need, int32_t* ref, int32_t pages, int32_t* lack, void* stream) {
  TRY(check_table(table, "table", n, blocks, page_size));
  if (n > pages_max_sequences()) return set_error(V4_ERR_UNSUPPORTED, "at most 8192 sequences a call");
  TRY(check_pool(ref, pages));
  TRY(check_ptr(lack, "lack", false));
  if (n > 0) TRY(check_ptr(need, "need"));
  TRY(check_ptr(have, "have", false));
  int* status;
  TRY(status_word(&status));
  StageTiming ps(24, (cudaStream_t)stream);
  return cuda_result(launch_pages_alloc(n, table, blocks, page_size, have, need, ref, pages, lack, status,
                                        (cudaStream_t)stream),
                     "page allocation kernel");
}

v4_status v4_pages_fork(int32_t batch, const int32_t* table, int32_t blocks, int32_t n, const int32_t* src,
                        const int32_t* len, int32_t* out_table, int32_t out_blocks, int32_t page_size, int32_t* ref,
                        int32_t pages, int32_t* copies, int32_t* lack, void* stream) {
  TRY(check_table(table, "table", batch, blocks, page_size));
  TRY(check_table(out_table, "out_table", n, out_blocks, page_size));
  if (n > pages_max_sequences()) return set_error(V4_ERR_UNSUPPORTED, "at most 8192 sequences a call");
  TRY(check_pool(ref, pages));
  TRY(check_ptr(lack, "lack", false));
  if (n > 0) {
    TRY(check_ptr(src, "src"));
    TRY(check_ptr(len, "len"));
    TRY(check_ptr(copies, "copies"));
    if (batch > 0 && overlap(table, (int64_t)batch * blocks * 4, out_table, (int64_t)n * out_blocks * 4))
      return bad("table and out_table overlap");
  }
  int* status;
  TRY(status_word(&status));
  StageTiming ps(24, (cudaStream_t)stream);
  return cuda_result(launch_pages_fork(batch, table, blocks, n, src, len, out_table, out_blocks, page_size, ref, pages,
                                       copies, lack, status, (cudaStream_t)stream),
                     "page fork kernel");
}

v4_status v4_pages_free(int32_t n, int32_t* table, int32_t blocks, int32_t page_size, const int32_t* lo,
                        const int32_t* hi, int32_t* ref, int32_t pages, void* stream) {
  TRY(check_table(table, "table", n, blocks, page_size));
  TRY(check_pool(ref, pages));
  TRY(check_ptr(lo, "lo", false));
  TRY(check_ptr(hi, "hi", false));
  if (n == 0) return V4_OK;
  int* status;
  TRY(status_word(&status));
  StageTiming ps(24, (cudaStream_t)stream);
  return cuda_result(launch_pages_free(n, table, blocks, page_size, lo, hi, ref, pages, status, (cudaStream_t)stream),
                     "page release kernel");
}

v4_status v4_pages_copy(void* cache, int32_t layers, int64_t layer_stride, int32_t pages, int32_t page_size,
                        int32_t row_bytes, const int32_t* copies, int32_t n, void* stream) {
  TRY(check_cache(cache, layers, layer_stride, pages, page_size, row_bytes));
  if (n < 0 || n > (1 << 24)) return bad("the number of copies must be in [0, 2^24]");
  if (n == 0) return V4_OK;
  if (((int64_t)page_size * row_bytes / 16384 + 1) * n > 0x7FFFFFFF) return bad("too many copies of pages that large");
  TRY(check_ptr(copies, "copies"));
  int* status;
  TRY(status_word(&status));
  StageTiming ps(25, (cudaStream_t)stream);
  return cuda_result(launch_pages_copy(cache, layers, layer_stride, pages, page_size, row_bytes, copies, n, status,
                                       (cudaStream_t)stream),
                     "page copy kernel");
}

v4_status v4_pages_compact(void* cache, int32_t layers, int64_t layer_stride, int32_t pages, int32_t page_size,
                           int32_t row_bytes, int32_t n, const int32_t* table, int32_t blocks, const int32_t* base,
                           const int32_t* count, const int32_t* keep, int32_t max_keep, void* stream) {
  TRY(check_cache(cache, layers, layer_stride, pages, page_size, row_bytes));
  TRY(check_table(table, "table", n, blocks, page_size));
  if (max_keep < 0 || max_keep > (1 << 30) || (int64_t)n * max_keep > 0x7FFFFFFF)
    return bad("keep must have at most 2^31 - 1 entries, 2^30 for a sequence");
  if (row_bytes / 64 > 65535) return bad("a row has more than 4 MB");
  if (n == 0 || max_keep == 0) return V4_OK;
  TRY(check_ptr(base, "base"));
  TRY(check_ptr(count, "count"));
  TRY(check_ptr(keep, "keep"));
  int* status;
  TRY(status_word(&status));
  StageTiming ps(26, (cudaStream_t)stream);
  return cuda_result(launch_pages_compact(cache, layers, layer_stride, pages, page_size, row_bytes, n, table, blocks,
                                          base, count, keep, max_keep, status, (cudaStream_t)stream),
                     "compaction kernel");
}

}  // extern "C"
