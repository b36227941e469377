// Plan of drafted token trees and the tree attention on CUDA cores (any
// shape, fp32 or bf16 storage); the tensor-core shapes run in tree_tc.cu.
//
// The attention is v4_sparse_mqa_fwd's ([BLOG] "The DeepSeek-V4-Flash
// architecture", "Three attention types, interleaved": 64 heads read one
// latent that is key and value, entries plus a window) for rows that sit at
// the end of a paged cache: row i sees entries, committed window tokens and
// its drafted ancestors.
#include <math.h>

#include "common.cuh"
#include "internal.h"
#include "q4.cuh"
#include "tree.cuh"
#include "turn.cuh"

namespace v4 {

namespace {

// ---------------------------------------------------------------------------
// Plan: one block for each sequence, thread j = node j.  Ancestor bits and
// depths by pointer doubling: after round s a node holds the bits of its 2^s
// nearest path members (itself among them) and points 2^s up, so seven
// rounds cover 128 nodes, against a walk of up to 127 dependent steps.
// Block B marks the rows of no sequence.  A few kilobytes in and out: the launch
// bounds it (1.3 us for one node, 1.8 for 32 trees of 8, 10 for 256 of 128).
// ---------------------------------------------------------------------------
struct PlanArgs {
  const int32_t *node_begin, *seq_len, *parent, *table;
  int32_t *plan, *pos, *slot;
  int* status;
  long long n_slots;
  int B, n_rows, max_blocks, page;
};

__device__ __forceinline__ void plan_padding(const PlanArgs& p, int row) {
  int4* w = reinterpret_cast<int4*>(p.plan + (size_t)row * kPlanWords);
  w[0] = make_int4(-1, 0, 0, 0);
  w[1] = make_int4(0, 0, 0, 0);
  if (p.pos) p.pos[row] = 0;
  if (p.slot) p.slot[row] = -1;
}

__global__ void __launch_bounds__(V4_TREE_MAX_NODES) tree_plan_kernel(const PlanArgs p) {
  __shared__ uint4 s_bits[V4_TREE_MAX_NODES];
  __shared__ int s_up[V4_TREE_MAX_NODES], s_depth[V4_TREE_MAX_NODES];
  const int b = blockIdx.x, j = threadIdx.x;
  after_previous();
  if (b == p.B) {
    const int first = p.node_begin[0], last = p.node_begin[p.B];
    for (int row = j; row < p.n_rows; row += blockDim.x)
      if (row < first || row >= last) plan_padding(p, row);
    if (j == 0 && (first < 0 || last > p.n_rows)) set_status(p.status, kStatusBadIndex);
    return;
  }
  const int begin = p.node_begin[b], end = p.node_begin[b + 1];
  const int L = p.seq_len[b];
  if (begin < 0 || end > p.n_rows || end < begin || end - begin > V4_TREE_MAX_NODES || L < 0 ||
      L > 0x7FFFFFFF - V4_TREE_MAX_NODES) {
    if (j == 0) set_status(p.status, kStatusBadIndex);
    for (long long row = (long long)max(begin, 0) + j; row < min(end, p.n_rows); row += blockDim.x) plan_padding(p, (int)row);
    return;
  }
  const int n = end - begin;
  int up = -1;
  if (j < n) {
    up = p.parent ? p.parent[begin + j] : j - 1;
    if (up < -1 || up >= j) {
      set_status(p.status, kStatusBadIndex);
      up = -1;
    }
  }
  uint4 bits = make_uint4(0, 0, 0, 0);
  const uint32_t bit = 1u << (j & 31);
  if (j < 32) bits.x = bit;
  else if (j < 64) bits.y = bit;
  else if (j < 96) bits.z = bit;
  else bits.w = bit;
  s_bits[j] = bits;
  s_up[j] = up;
  s_depth[j] = up >= 0 ? 1 : 0;                  // steps up that s_up has taken
  __syncthreads();
  for (int s = 1; s < n; s <<= 1) {
    const int u = s_up[j];
    int nu = u, d = s_depth[j];
    bits = s_bits[j];
    if (u >= 0) {
      const uint4 o = s_bits[u];
      bits.x |= o.x;
      bits.y |= o.y;
      bits.z |= o.z;
      bits.w |= o.w;
      nu = s_up[u];
      d += s_depth[u];
    }
    __syncthreads();
    s_bits[j] = bits;
    s_up[j] = nu;
    s_depth[j] = d;
    __syncthreads();
  }
  if (j >= n) return;
  const int row = begin + j;
  const long long t = (long long)L + s_depth[j];
  bits = s_bits[j];
  int4* w = reinterpret_cast<int4*>(p.plan + (size_t)row * kPlanWords);
  w[0] = make_int4(b, j, (int)t, L);
  w[1] = make_int4((int)bits.x, (int)bits.y, (int)bits.z, (int)bits.w);
  if (p.pos) p.pos[row] = (int)t;
  if (p.slot)
    p.slot[row] = (int)paged_row(p.table, p.max_blocks, p.page, p.n_slots, b, (long long)L + j, p.status);
}

// ---------------------------------------------------------------------------
// Attention on CUDA cores.  Block per (row, group of eight heads), one warp
// for each head: the block stages 32 keys at a time as fp32 rows in shared
// memory, lane j scores key j, the running maximum and denominator are kept
// in fp32, and each lane accumulates channels lane, lane + 32, ...  The fallback:
// bound by its fp32 products out of shared memory (one row of 64 heads over 641
// keys 246 us, where the tensor-core kernel takes 16).
// ---------------------------------------------------------------------------
constexpr int kHG = 8, kKT = 32, kSimtThreads = kHG * 32;

// Rows of a cache, dense or 4-bit.
template <typename C>
__device__ __forceinline__ const C* cache_row(const void* cache, long long s, int D) {
  return reinterpret_cast<const C*>(cache) + s * D;
}
template <>
__device__ __forceinline__ const Q4* cache_row<Q4>(const void* cache, long long s, int D) {
  return reinterpret_cast<const Q4*>(cache) + s * q4_row_bytes(D);
}
template <typename C>
__device__ __forceinline__ void load8_key(const C* row, int c8, int, float* v) {
  load8(row + c8, v);
}
__device__ __forceinline__ void load8_key(const Q4* row, int c8, int D, float* v) {
  const uint8_t* b = reinterpret_cast<const uint8_t*>(row);
  q4_values(*reinterpret_cast<const uint32_t*>(b + c8 / 2), q4_scale(b[D / 2 + c8 / kQ4Group]), v);
}

// T: queries and output; C: what the caches hold.
template <typename T, typename C>
__global__ void __launch_bounds__(kSimtThreads) tree_simt_kernel(const TreeArgs a) {
  extern __shared__ float sm[];
  const int D = a.D, R = a.R, ldk = D + 1;
  float* s_q = sm;                               // [kHG][D]
  float* s_k = s_q + kHG * D;                    // [kKT][D + 1]
  float* s_p = s_k + kKT * ldk;                  // [kHG][kKT]
  __shared__ const C* s_ptr[kKT];
  __shared__ float s_cs[2][512];
  __shared__ int s_draft[V4_TREE_MAX_NODES];
  __shared__ int s_count[V4_TREE_MAX_NODES / 32];
  const int row = blockIdx.x, h0 = blockIdx.y * kHG;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int h = h0 + warp;
  const bool head_live = h < a.H;
  const TreeRow r = tree_row(a, row);
  if (!r.live) return;
  // drafted keys in node order
  bool mine = false;
  unsigned vote = 0;
  if (threadIdx.x < V4_TREE_MAX_NODES) {
    mine = tree_draft_key(a, r, row, threadIdx.x, (uint32_t)a.plan[(size_t)row * kPlanWords + 4 + warp]);
    vote = __ballot_sync(0xffffffffu, mine);
    if (lane == 0) s_count[warp] = __popc(vote);
  }
  for (int j = threadIdx.x; j < R / 2; j += kSimtThreads) {
    float c, s;
    turn_cos_sin(r.t, turn_fraction(a.inv_freq[j]), &c, &s);
    s_cs[0][j] = c;
    s_cs[1][j] = s;
  }
  __syncthreads();
  int nd = 0;
  for (int w = 0; w < V4_TREE_MAX_NODES / 32; ++w) {
    if (mine && w == warp) s_draft[nd + __popc(vote & ((1u << lane) - 1u))] = threadIdx.x;
    nd += s_count[w];
  }
  const T* qp = reinterpret_cast<const T*>(a.q) + (size_t)row * a.H * D;
  for (int i = threadIdx.x; i < kHG * D; i += kSimtThreads) {
    const int hh = h0 + i / D, c = i % D;
    float v = 0.f;
    if (hh < a.H) {
      const T* qr = qp + (size_t)hh * D;
      v = to_f(qr[c]);
      if (c >= D - R) {
        const int j = (c - (D - R)) >> 1;
        const float other = to_f(qr[c ^ 1]);
        v = (c & 1) ? (other * s_cs[1][j] + v * s_cs[0][j]) : (v * s_cs[0][j] - other * s_cs[1][j]);
      }
    }
    s_q[i] = v;
  }
  const long long nk = (long long)r.ne + r.nw + nd;
  float m = -INFINITY, l = 0.f;
  if (a.sink != nullptr && head_live) {
    const float s = a.sink[h];
    if (s > -INFINITY) {
      m = s;
      l = 1.f;
    } else if (s != s) {
      l = s;                                     // a NaN sink makes the denominator one
    }
  }
  float acc[32];
#pragma unroll
  for (int i = 0; i < 32; ++i) acc[i] = 0.f;
  const int per_lane = D / 32;
  for (long long k0 = 0; k0 < nk; k0 += kKT) {
    __syncthreads();
    if (threadIdx.x < kKT) {
      const long long j = k0 + threadIdx.x;
      const C* p = nullptr;
      if (j < r.ne) {
        const long long s = tree_entry_row(a, r, row, (int)j);
        if (s >= 0) p = cache_row<C>(a.ent_cache, s, D);
      } else if (j < nk) {
        const long long at = j - r.ne < r.nw ? r.lo + (j - r.ne) : (long long)r.L + s_draft[j - r.ne - r.nw];
        const long long s = tree_token_row(a, r, at);
        if (s >= 0) p = cache_row<C>(a.tok_cache, s, D);
      }
      s_ptr[threadIdx.x] = p;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < kKT * (D / 8); i += kSimtThreads) {
      const int j = i / (D / 8), c8 = (i % (D / 8)) * 8;
      float v[8];
      const C* p = s_ptr[j];
      if (p) {
        load8_key(p, c8, D, v);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = 0.f;
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) s_k[j * ldk + c8 + e] = v[e];
    }
    __syncthreads();
    const bool key = head_live && s_ptr[lane] != nullptr;
    float lg = -INFINITY;
    if (key) {
      const float* qh = s_q + warp * D;
      const float* kr = s_k + lane * ldk;
      float d = 0.f;
      for (int c = 0; c < D; ++c) d = fmaf(qh[c], kr[c], d);
      lg = d * a.scale;
    }
    float tmax = lg;
    for (int off = 16; off > 0; off >>= 1) tmax = fmaxf(tmax, __shfl_xor_sync(0xffffffffu, tmax, off));
    const float mnew = fmaxf(m, tmax);
    float p = 0.f, alpha = 1.f;
    if (key) p = mnew > -INFINITY ? expf(lg - mnew) : (lg == lg ? 0.f : lg);      // a NaN logit stays one
    if (mnew > -INFINITY && !(m == mnew)) alpha = m > -INFINITY ? expf(m - mnew) : 0.f;
    float psum = p;
    for (int off = 16; off > 0; off >>= 1) psum += __shfl_xor_sync(0xffffffffu, psum, off);
    l = l * alpha + psum;
    m = mnew;
    s_p[warp * kKT + lane] = p;
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      if (i < per_lane) {
        const int c = lane + 32 * i;
        float s = acc[i] * alpha;
        for (int j = 0; j < kKT; ++j) s = fmaf(s_p[warp * kKT + j], s_k[j * ldk + c], s);
        acc[i] = s;
      }
    }
  }
  if (!head_live) return;
  const float inv_l = l == 0.f ? 0.f : 1.f / l;       // a NaN sum stays one
  T* orow = reinterpret_cast<T*>(a.o) + ((size_t)row * a.H + h) * D;
#pragma unroll
  for (int i = 0; i < 32; ++i) {
    if (i < per_lane) {
      const int c = lane + 32 * i;
      float v = acc[i] * inv_l;
      const float other = __shfl_xor_sync(0xffffffffu, v, 1);
      if (c >= D - R) {
        const int j = (c - (D - R)) >> 1;
        const float cs = s_cs[0][j], sn = -s_cs[1][j];
        v = (c & 1) ? (other * sn + v * cs) : (v * cs - other * sn);
      }
      from_f(orow + c, v);
    }
  }
  if (a.lse && lane == 0) a.lse[(size_t)row * a.H + h] = l == 0.f ? -INFINITY : m + logf(l);
}

template <typename T, typename C>
cudaError_t tree_simt_t(const TreeArgs& a, cudaStream_t st) {
  const size_t smem = (size_t)(kHG * a.D + kKT * (a.D + 1) + kHG * kKT) * sizeof(float);
  auto kern = tree_simt_kernel<T, C>;
  static OncePerDevice once;
  const cudaError_t e = allow_shared(kern, once);
  if (e != cudaSuccess) return e;
  const dim3 grid(a.n_rows, (a.H + kHG - 1) / kHG);
  StageTiming ps(16, st);
  kern<<<grid, kSimtThreads, smem, st>>>(a);
  note_launch();
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_tree_plan(int B, int n_rows, const int32_t* node_begin, const int32_t* seq_len,
                             const int32_t* parent, const int32_t* table, int max_blocks, int page, long long n_slots,
                             int32_t* plan, int32_t* pos, int32_t* slot, int* status, cudaStream_t st) {
  PlanArgs p;
  p.node_begin = node_begin;
  p.seq_len = seq_len;
  p.parent = parent;
  p.table = table;
  p.plan = plan;
  p.pos = pos;
  p.slot = slot;
  p.status = status;
  p.n_slots = n_slots;
  p.B = B;
  p.n_rows = n_rows;
  p.max_blocks = max_blocks;
  p.page = page;
  const cudaError_t e = launch_overlapped(tree_plan_kernel, dim3(B + 1), dim3(V4_TREE_MAX_NODES), 0, st, p);
  if (e == cudaSuccess) note_launch();
  return e;
}

cudaError_t launch_tree_simt(const TreeArgs& a, int dtype, bool q4, cudaStream_t st) {
  if (q4) return dtype == V4_BF16 ? tree_simt_t<bf16, Q4>(a, st) : tree_simt_t<float, Q4>(a, st);
  return dtype == V4_BF16 ? tree_simt_t<bf16, bf16>(a, st) : tree_simt_t<float, float>(a, st);
}

}  // namespace v4
