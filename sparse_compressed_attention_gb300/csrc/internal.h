// Internal launch interface between the C ABI (api.cu) and the kernels.
// Every launcher enqueues on `stream` and returns the launch error (if any).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <atomic>

#include "v4attn.h"

namespace v4 {

// Counts kernel launches made by the library (reported by v4_launch_count).
void note_launch(int n = 1);

// Query rows per sequence of a call: positions q_begin .. seqlen-1.  Row
// tensors (q, iq, w, o, lse, idx, scores) are indexed by b * q_rows + (t - q_begin);
// sequence tensors (kv, entries) by b * seqlen + t.
inline int q_rows(const v4_config& c) { return c.seqlen - c.q_begin; }

// Argument checks, error text and the device status word (api.cu).
v4_status validate_config(const v4_config* c);
v4_status set_error(v4_status st, const char* msg);
int* device_status_ptr();

// Per-stage timing (v4_profile_*): while timing is on, the launches between
// construction and destruction are bracketed by two CUDA events on `st`
// (api.cu).  `kind` is a stage number of v4_profile_enable's list.
class StageTiming {
 public:
  StageTiming(int kind, cudaStream_t st);
  ~StageTiming();
  StageTiming(const StageTiming&) = delete;
  StageTiming& operator=(const StageTiming&) = delete;

 private:
  void* rec_;
  cudaStream_t st_;
};

// Runs a set-up call once per device (kernel attributes, which stay set for
// the process): the calls it guards cost more than a short kernel's launch.
class OncePerDevice {
 public:
  template <typename F>
  cudaError_t run(F f) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kDevices) return f();
    if (done_[dev].load(std::memory_order_acquire)) return cudaSuccess;
    e = f();                                     // twice in a race: harmless
    if (e == cudaSuccess) done_[dev].store(true, std::memory_order_release);
    return e;
  }

 private:
  static constexpr int kDevices = 128;
  std::atomic<bool> done_[kDevices] = {};
};

// Lets a kernel take what dynamic shared memory a block can have beside its static
// part.  Once: the limit belongs to the process, and one that follows each call's
// own size is taken away by another host thread's smaller call before the launch.
template <typename Kernel>
cudaError_t allow_shared(Kernel kern, OncePerDevice& once) {
  return once.run([&] {
    int dev = 0, most = 0;
    cudaFuncAttributes at;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&most, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev);
    if (e == cudaSuccess) e = cudaFuncGetAttributes(&at, kern);
    if (e != cudaSuccess) return e;
    return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, most - (int)at.sharedSizeBytes);
  });
}

// Launch of a short kernel whose blocks may start while the kernel before it in
// the stream drains (programmatic dependence): 0.2 to 0.5 us a call (16 rotated
// rows 2.1 -> 1.9 us, one token's tree attention 17.1 -> 16.6).  The kernel calls
// after_previous() before it touches global memory.
template <typename... P, typename... A>
cudaError_t launch_overlapped(void (*kern)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t st, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, static_cast<P>(args)...);
}

// Workspace carve-up for one configuration (Sq = q_rows).  Offsets are
// 256-byte aligned.
struct Workspace {
  size_t kv_rot = 0, kv_rot_bytes = 0;     // rotated window keys [B,S,D]
  size_t ent = 0, ent_bytes = 0;           // entries [B,N,D] (layer call)
  size_t ikey = 0, ikey_bytes = 0;         // indexer keys [B,N,Di] (layer call)
  size_t iqp = 0, iqp_bytes = 0;           // prepared indexer queries [B,Sq,Hi,Di]
  size_t scores = 0, scores_bytes = 0;     // indexer scores [B,Sq,N] fp32
  size_t idx = 0, idx_bytes = 0;           // selected entries [B,Sq,K] (layer call)
  size_t counters = 0, counters_bytes = 0; // work counter, redo count, redo list [2 + B*Sq*slices]
  size_t rope = 0, rope_bytes = 0;         // cos/sin table [S][R/2] float2
  size_t qc8 = 0, qc8_bytes = 0;           // E4M3 indexer: query codes [B,Sq,Hi,Di] u8
  size_t qs8 = 0, qs8_bytes = 0;           //   query scales [B,Sq,Hi] fp32
  size_t kc8 = 0, kc8_bytes = 0;           //   key codes [B,N,Di] u8
  size_t ks8 = 0, ks8_bytes = 0;           //   key scales [B,N] fp32
  size_t total = 0;
};
Workspace plan_workspace(const v4_config& c);

// ---- compressor and preparation kernels (compress.cu)
// cs_table: the per-call cos/sin table of positions < S, or null (angles
// computed in place).
cudaError_t launch_compress(const v4_config& c, const void* ckv, const void* cscore,
                            const float* ape, const float* norm_w, const float* inv_freq,
                            const float2* cs_table, int dim, int hadamard, void* out, cudaStream_t st);
cudaError_t launch_rotate_rows(const v4_config& c, const void* kv, const float* inv_freq,
                               void* kv_rot, cudaStream_t st);
// Rotated window keys: token u of kv rotated at u on the last R dims,
// stored in the storage dtype, from the per-call cos/sin table.
cudaError_t launch_key_prep(const v4_config& c, const void* kv, const float2* cs_table, void* kv_rot,
                            cudaStream_t st);
// cos/sin of every (position < S, rotated pair): table[pos * R/2 + j].
cudaError_t launch_rope_table(const v4_config& c, const float* inv_freq, float2* table, cudaStream_t st);

// ---- TMA descriptors (tma_host.cu); returns 0 on success
int make_tmap_bf16_2d(CUtensorMap* map, const void* base, uint64_t cols, uint64_t rows, uint32_t box_cols,
                      uint32_t box_rows, bool swizzle128);
int make_tmap_u8_2d(CUtensorMap* map, const void* base, uint64_t cols, uint64_t rows, uint32_t box_cols,
                    uint32_t box_rows, bool swizzle128);
// cs_table may be null (angles are then computed in the kernel from inv_freq)
cudaError_t launch_indexer_prep(const v4_config& c, const void* iq, const float2* cs_table,
                                const float* inv_freq, void* iqp, cudaStream_t st);
// The same preparation quantised to E4M3 rows in the kernel (bf16, Di = 128):
// codes [B,Sq,Hi,128] and scales [B,Sq,Hi] instead of the bf16 rows.
cudaError_t launch_indexer_prep_e4m3(const v4_config& c, const void* iq, const float2* cs_table,
                                     const float* inv_freq, uint8_t* codes, float* scales, cudaStream_t st);

// ---- indexer (indexer.cu)
cudaError_t launch_indexer_scores_simt(const v4_config& c, const void* iqp, const void* ikey,
                                       const float* w, float* scores, cudaStream_t st);
bool indexer_tc_supported(const v4_config& c);
cudaError_t launch_indexer_scores_tc(const v4_config& c, const void* iqp, const void* ikey, const float* w,
                                     float* scores, int* status, cudaStream_t st);
// Opt-in E4M3 indexer (indexer_tc.cu): per-row absmax quantisation of bf16
// rows (dim a multiple of 128, <= 1024) and the scores of quantised
// operands (Hi = 64, Di = 128): q codes [B,Sq,64,128] with scales [B,Sq,64],
// key codes [B,N,128] with scales [B,N].
cudaError_t launch_quant_e4m3(const void* x, long long rows, int dim, uint8_t* codes, float* scales,
                              cudaStream_t st);
bool indexer_e4m3_supported(const v4_config& c);
cudaError_t launch_indexer_scores_e4m3(const v4_config& c, const uint8_t* qc, const float* qs, const uint8_t* kc,
                                       const float* ks, const float* w, float* scores, int* status,
                                       cudaStream_t st);
cudaError_t launch_topk(const v4_config& c, const float* scores, int32_t* idx, float* iscore,
                        cudaStream_t st);

// ---- attention (mqa.cu)
// `list` (nullable): list[0] = number of queries, list[1..] = b*Sq + (t - q_begin)
// of each (its query row); when given, only those queries are computed.
cudaError_t launch_mqa_simt(const v4_config& c, const void* q, const void* kv_rot,
                            const void* ent, const int32_t* idx, const float* sink,
                            const float* inv_freq, void* o, float* lse, int* status,
                            const int* list, cudaStream_t st);
bool mqa_tc_supported(const v4_config& c);

// ---- grouped output projection (oproj_tc.cu)
bool oproj_tc_supported(const v4_config& c);
cudaError_t launch_oproj_tc(const v4_config& c, const void* o, const void* wo_a, void* y, int* status,
                            cudaStream_t st);
// Query projection y[T, N] = x[T, rank] . w[rank, N] (bf16, fp32 accumulate);
// norm = 1 RMS-normalises every 512-wide column block (N % 512 == 0),
// weight norm_w [512] or ones.  rank % 64 == 0, N % 256 == 0.
cudaError_t launch_qproj_tc(long long T, int rank, const void* x, const void* w, int N, void* y, int norm,
                            float eps, const float* norm_w, int* status, cudaStream_t st);
cudaError_t launch_mqa_tc(const v4_config& c, const void* q, const void* kv_rot, const void* ent,
                          const int32_t* idx, const float* sink, const float2* cs_table, void* o, float* lse,
                          int* counters, int* status, cudaStream_t st);

// ---- sparse indexer distillation target (kl_target_tc.cu)
bool kl_target_tc_supported(const v4_config& c);
// target [B,S,K] (written), loss [B,S] and dscore [B,S,K] nullable (need iscore)
cudaError_t launch_kl_target(const v4_config& c, const void* q, const void* ent, const int32_t* idx,
                             const float* lse, const float* iscore, const float2* cs_table, float* target,
                             float* loss, float* dscore, int* status, cudaStream_t st);

// ---- attention backward (mqa_bwd_tc.cu)
bool mqa_bwd_tc_supported(const v4_config& c);
// qr = rot(q, t), dor = rot(dout, t) (storage dtype), delta = dout . o per
// (query, head); dsink (nullable, pre-zeroed) += -exp(sink - lse) delta.
cudaError_t launch_mqa_bwd_prep(const v4_config& c, const void* q, const void* o, const void* dout,
                                const float* lse, const float* sink, const float2* cs_table, void* qr, void* dor,
                                float* delta, float* dsink, cudaStream_t st);
// dq, and the fp32 reductions into dkv (gradient of the rotated window keys,
// pre-zeroed) and dent (pre-zeroed; nullable when there are no entries).
cudaError_t launch_mqa_bwd_tc(const v4_config& c, const void* qr, const void* dor, const void* kv_rot,
                              const void* ent, const int32_t* idx, const float* lse, const float* delta,
                              const float2* cs_table, void* dq, float* dkv, float* dent, int* status,
                              cudaStream_t st);
// dkv[b, u] = rot(dkv[b, u], -u) in place
cudaError_t launch_mqa_bwd_derotate(const v4_config& c, float* dkv, const float2* cs_table, cudaStream_t st);

// ---- rotary positions and the paged cache write (rope.cu)
struct RopeCall {
  const void* x;
  void* out;
  const int32_t* pos;           // null: rows stored as they are
  const float* inv_freq;
  const int32_t* slot;          // null: row t to row t
  long long n_slots, rows, x_row_stride, x_head_stride, out_row_stride, out_head_stride;
  int heads, dim, rope_dim, rope_begin, layout, inverse, dtype;
  float mscale;
};
cudaError_t launch_rope(const RopeCall& c, int* status, cudaStream_t st);

// ---- norms of queries and keys with the rotation (norm.cu)
struct NormPartCall {
  const void* x;                // null: no such heads
  const void* dy;               // gradient
  const float* w;               // null: ones
  void* out;                    // y, or dx
  float* dw;                    // gradient, null: not wanted
  int heads;
  long long x_row_stride, x_head_stride, dy_row_stride, dy_head_stride, out_row_stride, out_head_stride;
};
struct NormCall {
  NormPartCall part[2];         // queries, keys
  const int32_t* pos;
  const float* inv_freq;
  void* workspace;              // gradient: norm_rope_workspace(dim) bytes
  long long rows;
  int dim, rope_dim, rope_begin, dtype;
  bool half, grad;
  float eps;
};
size_t norm_rope_workspace(int dim);
cudaError_t launch_norm_rope(const NormCall& c, cudaStream_t st);

// ---- rows of the 4-bit cache (cache4.cu)
struct Q4Call {
  const void* x;                // write
  void* out;                    // read; null: write
  void* cache;
  const int32_t* slot;
  long long n_slots, rows, row_stride;
  int dim, dtype;
};
cudaError_t launch_q4_rows(const Q4Call& c, int* status, cudaStream_t st);

// ---- pages of a cache (pages.cu)
int pages_max_sequences();      // of one v4_pages_alloc or v4_pages_fork
cudaError_t launch_pages_alloc(int n, int32_t* table, int blocks, int page, const int32_t* have, const int32_t* need,
                               int32_t* ref, int pages, int32_t* lack, int* status, cudaStream_t st);
cudaError_t launch_pages_fork(int B, const int32_t* table, int blocks, int n, const int32_t* src, const int32_t* len,
                              int32_t* out, int out_blocks, int page, int32_t* ref, int pages, int32_t* copies,
                              int32_t* lack, int* status, cudaStream_t st);
cudaError_t launch_pages_free(int n, int32_t* table, int blocks, int page, const int32_t* lo, const int32_t* hi,
                              int32_t* ref, int pages, int* status, cudaStream_t st);
cudaError_t launch_pages_copy(void* cache, int layers, long long layer_bytes, int pages, int page, int row_bytes,
                              const int32_t* copies, int n, int* status, cudaStream_t st);
cudaError_t launch_pages_compact(void* cache, int layers, long long layer_bytes, int pages, int page, int row_bytes,
                                 int n, const int32_t* table, int blocks, const int32_t* base, const int32_t* count,
                                 const int32_t* keep, int width, int* status, cudaStream_t st);

// ---- drafted token trees (tree.cu, tree_tc.cu)
struct TreeArgs;
cudaError_t launch_tree_plan(int B, int n_rows, const int32_t* node_begin, const int32_t* seq_len,
                             const int32_t* parent, const int32_t* table, int max_blocks, int page, long long n_slots,
                             int32_t* plan, int32_t* pos, int32_t* slot, int* status, cudaStream_t st);
// q4: the caches hold 4-bit rows
cudaError_t launch_tree_simt(const TreeArgs& a, int dtype, bool q4, cudaStream_t st);

// ---- 4-bit projections (w4.cu)
cudaError_t launch_w4_pack(const void* w, int groups, int K, int N, int gs, uint8_t* codes, void* scales,
                           cudaStream_t st);
cudaError_t launch_w4_proj(const void* x, long long rows, int groups, int K, int N, int gs, const uint8_t* codes,
                           const void* scales, int norm_dim, float eps, const float* norm_w, void* y,
                           cudaStream_t st);

}  // namespace v4
