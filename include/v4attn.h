/*
 * v4attn.h - C ABI of the DeepSeek-V4-Flash compressed attention forward
 * (compressor, CSA lightning indexer with top-k, sparse/dense multi-query
 * attention with sliding window and de-rotated output) on one GB300 GPU.
 *
 * Sources of the operations:
 *   [PR]   Primus PR #930 "fix(deepseek-v4): correct V4-Flash attention math,
 *          wire the MoE balance loss", Part 1 (items 1-6, 8).
 *   [BLOG] "Enabling DeepSeek-V4-Flash Training on AMD Instinct MI355X GPUs
 *          with Primus", sections "The DeepSeek-V4-Flash architecture",
 *          "Three attention types, interleaved", "Kernel fusions".
 *
 * Conventions shared by every entry point
 *   - Tensors are dense, row-major, in device memory owned by the caller.
 *     The library never allocates device memory; scratch space is the
 *     caller's workspace (see v4_workspace_size).  One exception:
 *     v4_sparse_mqa_fwd_noalloc keeps its scratch in a library-owned static
 *     device array (see its section).  Every device pointer must be 16-byte
 *     aligned.
 *   - "Storage dtype" (cfg->dtype) is the element type of q, kv, the pooling
 *     projections, entries, indexer keys/queries and the output: V4_F32 or
 *     V4_BF16.  ape, norm weights, indexer weights w, sink, inv_freq, lse
 *     and iscore are always float32.
 *   - Work is enqueued on `stream` (a cudaStream_t; NULL = legacy default
 *     stream) and runs asynchronously.  A non-V4_OK return means nothing was
 *     enqueued; v4_last_error() gives the reason.  Arguments are validated on
 *     the host before any launch.
 *   - Problems found on the device (an out-of-range selected index, a timed
 *     out wait) never trap: they set a sticky status word that
 *     v4_get_device_status() reads.  Offending keys are skipped.
 *   - Entry points may be called from several host threads; the error text
 *     is per thread.
 *
 * Notation: B batch, S sequence length, H query heads, D latent (head) dim,
 * R rotated dims (the last R of D), r compression ratio, ov overlap (0/1),
 * N = S / r entries (floor), Hi / Di indexer heads / dim, K top-k, W window.
 */
#ifndef V4ATTN_H
#define V4ATTN_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  V4_OK = 0,
  V4_ERR_INVALID_ARG = 1,   /* bad pointer, size, alignment or combination */
  V4_ERR_UNSUPPORTED = 2,   /* valid but not implemented (e.g. forced path) */
  V4_ERR_WORKSPACE = 3,     /* workspace missing or smaller than required */
  V4_ERR_CUDA = 4,          /* a CUDA runtime call failed */
  V4_ERR_TIMEOUT = 5,       /* device status: a bounded wait gave up */
  V4_ERR_BAD_INDEX = 6,     /* device status: a selected index was not visible */
  V4_ERR_BOUND = 7          /* device status, V4_DEBUG builds only: an index failed its
                               bound check (gather row, ring slot, TMEM column) and the
                               access was skipped */
} v4_status;

typedef enum { V4_F32 = 0, V4_BF16 = 1 } v4_dtype;

/* Kernel family selection (cfg->path). AUTO picks the tensor-core kernels
 * when the shapes and dtype allow it, otherwise the CUDA-core kernels.
 * Tensor-core attention: bf16, n_heads a multiple of 64 up to 512 (each
 * 64-head slice of a query is one work item), head_dim 512, rope_dim 64,
 * 1 <= window <= 128, topk <= 1024.  Tensor-core indexer: bf16,
 * idx_heads 64, idx_dim 128.  V4_PATH_TC returns V4_ERR_UNSUPPORTED for
 * other shapes. */
typedef enum { V4_PATH_AUTO = 0, V4_PATH_SIMT = 1, V4_PATH_TC = 2 } v4_path;

typedef struct v4_config {
  int32_t batch;          /* B >= 1 */
  int32_t seqlen;         /* S >= 1 */
  int32_t n_heads;        /* H >= 1 (Flash: 64) */
  int32_t head_dim;       /* D, multiple of 32, 32..1024 (Flash: 512) */
  int32_t rope_dim;       /* R, multiple of 8, <= D (Flash: 64) */
  int32_t ratio;          /* r: 0 = window-only layer, 4 = CSA, 128 = HCA; any r >= 1 */
  int32_t overlap;        /* ov: 1 = each entry also pools the previous r tokens (CSA) */
  int32_t window;         /* W: tokens [t-W+1, t]; 0 = no window; -1 = all tokens <= t */
  int32_t topk;           /* K: 0 = attend to every visible entry (HCA); > 0 = CSA selection */
  int32_t idx_heads;      /* Hi (Flash: 64) */
  int32_t idx_dim;        /* Di, power of two, 8..256, >= R (Flash: 128) */
  int32_t o_groups;       /* grouped output projection: groups (Flash: 8) */
  int32_t o_rank;         /* grouped output projection: rank per group (Flash: 1024) */
  float softmax_scale;    /* <= 0 selects D^-0.5, the only value [PR] item 1 allows */
  float rms_eps;          /* entry RMSNorm epsilon (1e-6) */
  int32_t dtype;          /* v4_dtype: storage dtype */
  int32_t path;           /* v4_path */
  int32_t indexer_fp8;    /* 1 = opt-in E4M3 indexer QK (see v4_indexer_topk_e4m3);
                             0 = bf16 operands, fp32 scoring (the default [PR] item 4 asks for) */
  int32_t q_begin;        /* first query position of the call, 0 <= q_begin < seqlen (0 = all).
                             The call computes queries q_begin .. seqlen-1 of every sequence
                             against the whole causal prefix: [BLOG] "Three attention types,
                             interleaved" gives each query its own keys (selected entries and
                             window), so query rows are independent given the prefix.  Row
                             tensors (q, iq, w, o, lse, idx, iscore, y; Sq = seqlen - q_begin
                             rows per sequence, row i = position q_begin + i) hold only these
                             rows; sequence tensors (kv, ckv, cscore, ickv, icscore, entries,
                             indexer keys) hold all seqlen positions.  A chunk [a, b) of a
                             sequence is the call with seqlen = b and q_begin = a: causality
                             means it needs no token past b-1.  The backward and the indexer
                             distillation target take q_begin = 0 only (V4_ERR_UNSUPPORTED). */
} v4_config;

/* ----------------------------------------------------------------------
 * RoPE inverse-frequency table (host function, no GPU).
 * [PR] items 2 and 8: compressed layers rotate with base 40000 paired with a
 * YaRN factor (16) acting on the inverse frequencies.  Base table
 * theta^(-2j/R); YaRN "NTK-by-parts" (Peng et al. 2023, section 3.2) with
 * ramp bounds beta_slow..beta_fast applies when yarn_factor > 1 and
 * original_len > 0.  inv_freq: host array of R/2 floats, written.
 * --------------------------------------------------------------------*/
v4_status v4_rope_inv_freq(float theta, int32_t rope_dim, float yarn_factor,
                           int32_t original_len, float beta_fast, float beta_slow,
                           float* inv_freq);

/* Bytes of workspace that every entry point below needs for `cfg` (the
 * largest of their needs, so one buffer serves them all). */
v4_status v4_workspace_size(const v4_config* cfg, size_t* bytes);

/* ----------------------------------------------------------------------
 * Compressor (one learned pooling operator for CSA and HCA).
 * [BLOG] "Three attention types, interleaved" (softmax over the group biased
 * by a learnable per-position term; CSA groups overlap: own r tokens plus
 * the previous r) and "Kernel fusions", row "Compressor pooling";
 * [PR] item 1 (entries are RMSNormed), item 2 (entry s rotated at r*s),
 * item 6e (indexer keys: RoPE then normalised Hadamard).
 *
 *   ckv, cscore : [B, S, 1+ov, dim] storage dtype. Half 0 is the token's
 *                 projection for its own group, half 1 for the next group
 *                 (used as "previous" members).
 *   ape         : [(1+ov)*r, dim] fp32. Rows are chronological: with
 *                 overlap rows 0..r-1 bias the previous group's tokens,
 *                 rows r..2r-1 the own tokens.
 *   norm_w      : [dim] fp32 RMSNorm weight, NULL = ones.
 *   inv_freq    : [R/2] fp32 device array.
 *   dim         : channel count (D for the attention entries, Di for the
 *                 indexer keys); R <= dim.
 *   hadamard    : 1 = apply the normalised Sylvester Hadamard (dim must be a
 *                 power of two) after the rotation.
 *   out         : [B, N, dim] storage dtype, N = S / r.
 * Per entry s and channel c: pooled = sum_m softmax_m(cscore + ape) * ckv over
 * the members m (entry 0 has no previous group; absent members are left out),
 * then e = pooled / sqrt(mean_c pooled^2 + eps) * g, rotated at position r*s.
 * --------------------------------------------------------------------*/
v4_status v4_compress(const v4_config* cfg, const void* ckv, const void* cscore,
                      const float* ape, const float* norm_w, const float* inv_freq,
                      int32_t dim, int32_t hadamard, void* out, void* stream);

/* ----------------------------------------------------------------------
 * Indexer query preparation.  [PR] item 6e: queries rotated at their own
 * position t (partial RoPE at the compressed base), then the normalised
 * Hadamard.  iq: [B, S, Hi, Di] -> iq_prep: [B, S, Hi, Di], storage dtype.
 * --------------------------------------------------------------------*/
v4_status v4_indexer_prep(const v4_config* cfg, const void* iq, const float* inv_freq,
                          void* iq_prep, void* stream);

/* ----------------------------------------------------------------------
 * Lightning indexer scores and top-k selection (CSA).
 * [PR] item 6a (per-head weights scaled by Hi^-1/2 * Di^-1/2), item 4 (the
 * QK stays in high precision: bf16 operands, fp32 accumulation, fp32
 * scoring and selection); [BLOG] "Kernel fusions", row "Indexer scoring tail"
 * (ReLU, per-head weight, head sum, inline causal mask) and "Three attention
 * types" (keep the best 512).
 *
 *   I[t,s] = sum_h w[t,h] * (Hi*Di)^-1/2 * max(0, iq~[t,h] . ikey[s]),
 *   defined for s < n_vis(t) = (t+1)/r; the best min(K, n_vis(t)) are kept,
 *   equal scores going to the lower index.
 *
 *   iq          : [B, S, Hi, Di]; un-rotated (iq_prepared = 0) or already
 *                 prepared by v4_indexer_prep (iq_prepared = 1).
 *   ikey        : [B, N, Di] from v4_compress(dim = Di, hadamard = 1).
 *   w           : [B, S, Hi] fp32 per-head weights (unscaled).
 *   idx         : [B, S, K] int32 out. The selected entries of row t in
 *                 ascending index order, then -1 padding.
 *   iscore      : [B, S, K] fp32 out, nullable: I[t, idx] (-inf on padding).
 *   workspace   : at least v4_workspace_size bytes.
 * --------------------------------------------------------------------*/
v4_status v4_indexer_topk(const v4_config* cfg, const void* iq, int32_t iq_prepared,
                          const void* ikey, const float* w, const float* inv_freq,
                          int32_t* idx, float* iscore, void* workspace,
                          size_t ws_bytes, void* stream);

/* ----------------------------------------------------------------------
 * Opt-in E4M3 indexer.  [PR] item 4 keeps the indexer QK in high precision
 * by default, because quantisation error there changes which entries are
 * selected, and puts FP8 behind its own switch; [BLOG] closing section: an
 * E4M3 path for the indexer QK ships.  The pages name the format, not the
 * scaling: here every row (one prepared query head, one indexer key) is
 * scaled by its absolute maximum.
 *
 * v4_quantize_e4m3: x [rows, dim] bf16 -> codes [rows, dim] (E4M3 bytes,
 *   OCP "FN" encoding) and scales [rows] fp32 with x ~= code * scale:
 *   scale = amax / 448, code = E4M3(x * (448 / amax)), every step in fp32
 *   rounded to nearest (the conversion saturates at +-448); an all-zero row
 *   gets scale 0 and zero codes.  dim is 128, 256, 512 or 1024; rows >= 0.
 *
 * v4_indexer_topk_e4m3: the selection of v4_indexer_topk from quantised
 *   operands (cfg as for the tensor-core indexer: bf16, Hi = 64, Di = 128):
 *     q_codes [B, S, Hi, Di] with q_scales [B, S, Hi]  (prepared queries),
 *     k_codes [B, N, Di]     with k_scales [B, N]      (indexer keys),
 *     I[t,s] = sum_h w[t,h] (Hi*Di)^-1/2 max(0, (q_code q_scale) . (k_code k_scale)),
 *   E4M3 tensor-core products with fp32 accumulation and fp32 scoring; idx,
 *   iscore, tie rule and workspace as v4_indexer_topk.  Other shapes return
 *   V4_ERR_UNSUPPORTED.
 *
 * With cfg->indexer_fp8 = 1, v4_indexer_topk and v4_attn_layer_fwd prepare
 * the queries in bf16 as before, quantise queries and keys into the
 * workspace with v4_quantize_e4m3's rule and select from the E4M3 scores.
 * --------------------------------------------------------------------*/
v4_status v4_quantize_e4m3(const void* x, int64_t rows, int32_t dim, uint8_t* codes, float* scales,
                           void* stream);
v4_status v4_indexer_topk_e4m3(const v4_config* cfg, const uint8_t* q_codes, const float* q_scales,
                               const uint8_t* k_codes, const float* k_scales, const float* w,
                               int32_t* idx, float* iscore, void* workspace, size_t ws_bytes,
                               void* stream);

/* ----------------------------------------------------------------------
 * Sparse / dense multi-query attention with sliding window, sink and
 * de-rotated output.
 * [BLOG] "The DeepSeek-V4-Flash architecture" (64 heads read one 512-d latent
 * that is both key and value), "Three attention types" (selected entries or
 * all HCA entries, plus the 128-token window), "Kernel fusions", row
 * "SWA / CSA / HCA attention" (window and softmax sink in one kernel);
 * [PR] item 1 (scale exactly D^-0.5), item 3 (output de-rotated at -t).
 *
 * For query t and head h: keys J(t) = idx[t] (K > 0), or every visible entry
 * s < n_vis(t) (K = 0, r > 0), or none (r = 0); plus window tokens u in
 * [max(0,t-W+1), t] rotated at u.  logits = scale * rot(q[t,h], t) . key;
 * softmax over J(t) with the optional sink logit sink[h] in the
 * denominator; o = sum p * key (V = K); o's last R dims rotated at -t.
 *
 *   q    : [B, S, H, D] un-rotated.           kv   : [B, S, D] un-rotated.
 *   ent  : [B, N, D] rotated entries (v4_compress); NULL iff r == 0.
 *   idx  : [B, S, K] int32; -1 = unused slot; NULL = all visible entries.
 *          Values >= n_vis(t) or < -1 are skipped and flagged
 *          (V4_ERR_BAD_INDEX in the device status).
 *   sink : [H] fp32, nullable.
 *   o    : [B, S, H, D] out.   lse : [B, S, H] fp32 out (natural log), nullable.
 * An empty key set without a sink yields o = 0 and lse = -inf.
 * --------------------------------------------------------------------*/
v4_status v4_sparse_mqa_fwd(const v4_config* cfg, const void* q, const void* kv,
                            const void* ent, const int32_t* idx, const float* sink,
                            const float* inv_freq, void* o, float* lse,
                            void* workspace, size_t ws_bytes, void* stream);

/* ----------------------------------------------------------------------
 * v4_sparse_mqa_fwd without a workspace: the method has no counterpart for
 * this entry point; it exists for callers that cannot allocate device memory
 * where they run the attention (a serving stack whose planner owns all
 * device memory up front, a plugin that may not call cudaMalloc inside a
 * host framework, a latency-critical path that cannot absorb an
 * allocation).  Arguments and results are those of v4_sparse_mqa_fwd.
 *
 * Scratch comes from one library-owned device array of about 10 MiB, held by
 * every GPU that loads the library until the process exits.  Limits:
 * batch*seqlen <= 8192, batch*seqlen*head_dim*element size <= 8 MiB and
 * seqlen*rope_dim <= 524288; larger problems return V4_ERR_INVALID_ARG with
 * a message.  The call allocates nothing.  The first call on a device looks
 * up the array's device address (cudaGetSymbolAddress, with that device
 * current), so make that first call before any stream capture.  All calls
 * share the array and it keeps the last call's contents: calls that overlap
 * on the GPU (unordered streams, several host threads) race on it.
 * --------------------------------------------------------------------*/
v4_status v4_sparse_mqa_fwd_noalloc(const v4_config* cfg, const void* q, const void* kv,
                                    const void* ent, const int32_t* idx, const float* sink,
                                    const float* inv_freq, void* o, float* lse, void* stream);

/* ----------------------------------------------------------------------
 * Backward of v4_sparse_mqa_fwd: the gradients of L = sum(dout * o).
 * [BLOG] "Attention kernels for the three layer types", backward: a dQ pass
 * that regathers the keys and recomputes the softmax, the delta
 * rowsum(O * dO), and a head-dimension contraction scattered into the
 * key/value gradient (fused here with dQ; fp32 reductions in L2).
 *
 * With p = softmax probabilities of v4_sparse_mqa_fwd (from lse), g =
 * rot(dout, t), delta = dout . o and ds = p (g . key - delta):
 *   dq   = rot(scale * sum_j ds_j key_j, -t)
 *   dkey = scale * sum_h ds_h rot(q_h, t) + sum_h p_h g_h     (key = value)
 *   dent[b, e] = sum of dkey over every (query, slot) that read entry e
 *   dkv[b, u]  = rot(sum of dkey over queries whose window holds u, -u)
 *   dsink[h]   = -sum_t exp(sink[h] - lse[t, h]) delta[t, h]
 *
 * Inputs are those of the forward call plus its outputs:
 *   o    : [B, S, H, D] the forward output.   lse : [B, S, H] fp32 (required).
 *   dout : [B, S, H, D] gradient of o.
 * Outputs (overwritten):
 *   dq    : [B, S, H, D] (storage dtype).
 *   dkv   : [B, S, D] fp32, gradient of the un-rotated window latent kv.
 *   dent  : [B, N, D] fp32, gradient of the rotated entries; required iff
 *           r > 0 and N > 0, else NULL.
 *   dsink : [H] fp32; required iff sink != NULL.
 * Shapes: those of the tensor-core forward (bf16, H a multiple of 64 up to
 * 512, D = 512, R = 64, 1 <= W <= 128, K <= 1024); others return
 * V4_ERR_UNSUPPORTED.  Reduction order of dkv / dent / dsink follows the
 * GPU's scheduling, so they are not bitwise reproducible.
 * workspace : at least v4_bwd_workspace_size bytes, 256-byte aligned.
 * --------------------------------------------------------------------*/
v4_status v4_bwd_workspace_size(const v4_config* cfg, size_t* bytes);
v4_status v4_sparse_mqa_bwd(const v4_config* cfg, const void* q, const void* kv,
                            const void* ent, const int32_t* idx, const float* sink,
                            const float* inv_freq, const void* o, const float* lse,
                            const void* dout, void* dq, float* dkv, float* dent,
                            float* dsink, void* workspace, size_t ws_bytes, void* stream);

/* ----------------------------------------------------------------------
 * Query projections of the rank-r latent.  [BLOG] "The DeepSeek-V4-Flash
 * architecture": queries arrive through a low-rank path of rank 1024 that
 * the sparse-selection indexer shares.
 *   qlat : [B, S, rank] bf16, the shared latent.
 *   wq   : [rank, H*D] bf16 (row k holds the weights of latent dim k).
 *   q    : [B, S, H, D] out: qlat . wq, and with q_norm = 1 every head
 *          RMS-normalised over its D dims, q / sqrt(mean(q^2) + cfg->rms_eps)
 *          * g with g = q_norm_w [D] fp32 (NULL = ones).
 *   wiq  : [rank, Hi*Di] bf16, nullable; iq : [B, S, Hi, Di] out (required
 *          iff wiq): qlat . wiq.
 * bf16 storage only, fp32 accumulation, one rounding to bf16; rank a
 * multiple of 64 (at most 65536), H*D and Hi*Di multiples of 256, and D =
 * 512 when q_norm = 1; other shapes return V4_ERR_UNSUPPORTED.
 * --------------------------------------------------------------------*/
v4_status v4_q_proj(const v4_config* cfg, const void* qlat, int32_t rank, const void* wq,
                    int32_t q_norm, const float* q_norm_w, const void* wiq, void* q, void* iq,
                    void* stream);

/* ----------------------------------------------------------------------
 * Sparse indexer distillation target.  [PR] item 5: KL(attention ||
 * indexer) over the selected entries, the sparse top-k variant that stays
 * in [B, S, K]; item 11: the target branch is detached and its heads are
 * summed inside the loop, so [B, H, S, K] never exists.
 *
 * With A_h the attention probabilities of v4_sparse_mqa_fwd for head h
 * (window and sink included in the normalisation, given by lse):
 *   target[t,k] = sum_h A_h[idx[t,k]] / sum_k' sum_h A_h[idx[t,k']]
 * over the valid slots (0 on padding and on rows without selections).  With
 * iscore (the indexer scores of the slots, as v4_indexer_topk returns
 * them) and qd = softmax of iscore over the valid slots:
 *   loss[t]     = sum_k target (log target - log qd)     (nullable)
 *   dscore[t,k] = qd - target, the gradient of sum_t loss[t] with respect
 *                 to iscore (0 on padding)                 (nullable)
 *   q    : [B, S, H, D] un-rotated queries.   ent : [B, N, D] rotated entries.
 *   idx  : [B, S, K] selections.              lse : [B, S, H] of the forward.
 * Tensor-core shapes only (bf16, H a multiple of 64 up to 512, D = 512,
 * R = 64, K <= 1024, N <= 65536); others return V4_ERR_UNSUPPORTED.
 * Heads and slices are summed with fp32 atomics (not bitwise reproducible).
 * workspace : at least v4_workspace_size bytes.
 * --------------------------------------------------------------------*/
v4_status v4_indexer_kl_target(const v4_config* cfg, const void* q, const void* ent,
                               const int32_t* idx, const float* lse, const float* iscore,
                               const float* inv_freq, float* target, float* loss, float* dscore,
                               void* workspace, size_t ws_bytes, void* stream);

/* ----------------------------------------------------------------------
 * Grouped low-rank output projection.  [BLOG] "The DeepSeek-V4-Flash
 * architecture": the 64 x 512 output splits into o_groups groups, each
 * through an o_rank bottleneck.  Group g holds heads g*H/G .. (g+1)*H/G-1
 * concatenated along D.
 *   o    : [B, S, H, D];  wo_a : [G, (H/G)*D, o_rank];  y : [B, S, G*o_rank].
 * bf16 storage; (H/G)*D a multiple of 64 and o_rank a multiple of 256 (other
 * shapes return V4_ERR_UNSUPPORTED).  fp32 accumulation, bf16 result.
 * --------------------------------------------------------------------*/
v4_status v4_grouped_o_proj(const v4_config* cfg, const void* o, const void* wo_a,
                            void* y, void* stream);

/* Pointers of one layer call. Nullable fields are marked. */
typedef struct v4_layer_inputs {
  const void* q;         /* [B,S,H,D] */
  const void* kv;        /* [B,S,D] window latent */
  const void* ckv;       /* [B,S,1+ov,D]     (r > 0) */
  const void* cscore;    /* [B,S,1+ov,D]     (r > 0) */
  const float* ape;      /* [(1+ov)r, D]     (r > 0) */
  const float* norm_w;   /* [D], nullable */
  const void* ickv;      /* [B,S,1+ov,Di]    (K > 0) */
  const void* icscore;   /* [B,S,1+ov,Di]    (K > 0) */
  const float* iape;     /* [(1+ov)r, Di]    (K > 0) */
  const float* inorm_w;  /* [Di], nullable */
  const void* iq;        /* [B,S,Hi,Di] un-rotated (K > 0) */
  const float* w;        /* [B,S,Hi]         (K > 0) */
  const float* sink;     /* [H], nullable */
  const float* inv_freq; /* [R/2] */
  const void* wo_a;      /* [G,(H/G)D,o_rank], nullable = no projection */
} v4_layer_inputs;

typedef struct v4_layer_outputs {
  void* o;               /* [B,S,H,D] */
  float* lse;            /* [B,S,H], nullable */
  void* ent;             /* [B,N,D], nullable (kept in the workspace) */
  void* ikey;            /* [B,N,Di], nullable (kept in the workspace) */
  int32_t* idx;          /* [B,S,K], nullable (kept in the workspace) */
  float* iscore;         /* [B,S,K], nullable */
  void* y;               /* [B,S,G*o_rank], required iff wo_a != NULL */
} v4_layer_outputs;

/* ----------------------------------------------------------------------
 * One attention layer: compressor (r > 0), indexer keys + query prep +
 * scores + top-k (K > 0), attention with window and de-rotation, optional
 * grouped output projection; all on `stream`, no host synchronisation.
 * [PR] Part 1 as a whole; [BLOG] "Three attention types, interleaved".
 * --------------------------------------------------------------------*/
v4_status v4_attn_layer_fwd(const v4_config* cfg, const v4_layer_inputs* in,
                            v4_layer_outputs* out, void* workspace, size_t ws_bytes,
                            void* stream);

/* ----------------------------------------------------------------------
 * Rotary positions at given positions (no counterpart of its own on the
 * pages: [PR] items 2 and 8 and [BLOG] "Kernel fusions", row "Interleaved
 * partial RoPE", give the rotation that the other entry points apply inside
 * their kernels).
 *
 *   out[t, h, c] = x[t, h, c] outside [rope_begin, rope_begin + R); inside,
 *   pair j = (a, b) becomes mscale * (a cos p - b sin p, a sin p + b cos p)
 *   with p = pos[t] * inv_freq[j], or -p with inverse = 1.
 *   V4_ROPE_INTERLEAVED: pair j = dims rope_begin + 2j, + 2j + 1;
 *   V4_ROPE_HALF:        pair j = dims rope_begin + j, + j + R/2.
 * The gradient of sum(dout * out) with respect to x is the same call on dout
 * with inverse = 1 and the same mscale.  (Where x was broadcast over heads or
 * rows, the caller sums that result over the broadcast axis.)
 *
 *   x, out   : element (t, h, c) at t * row_stride + h * head_stride + c, in
 *              elements; strides >= 0, multiples of 16 bytes.  x may be
 *              broadcast (a stride of 0); out's rows must not overlap
 *              (refused).  out may be x with the same strides (in place:
 *              only the rotated dims are touched), or another view of x's
 *              buffer with the same strides and no element of x; other
 *              tensors whose extents overlap are refused.
 *   pos      : [rows] int32, any value.   inv_freq : [rope_dim/2] fp32,
 *              finite (the table of v4_rope_inv_freq, or any other scaling).
 *   dim a multiple of 8 up to 8192; rope_dim a multiple of 8 (16 for
 *   V4_ROPE_HALF), <= 1024; rope_begin a multiple of 8, rope_begin +
 *   rope_dim <= dim.  rows = 0 is valid.  dtype: a v4_dtype.
 * Angles are formed from a 64-bit fraction of a turn, for any int32 position:
 * within |pos| (1 + |inv_freq| / 8) 2^-64 + 2^-32 turns, and another 2^-28 for
 * the fp32 remainder that is left of them; the rotation is fp32 with one
 * rounding to the storage type.
 * --------------------------------------------------------------------*/
typedef enum { V4_ROPE_INTERLEAVED = 0, V4_ROPE_HALF = 1 } v4_rope_layout;
v4_status v4_rope(const void* x, int64_t rows, int32_t heads, int32_t dim, int64_t x_row_stride,
                  int64_t x_head_stride, const int32_t* pos, const float* inv_freq, int32_t rope_dim,
                  int32_t rope_begin, int32_t layout, int32_t inverse, float mscale, int32_t dtype,
                  void* out, int64_t out_row_stride, int64_t out_head_stride, void* stream);

/* ----------------------------------------------------------------------
 * Paged cache write: row t of x, its last rope_dim dims rotated at pos[t]
 * (interleaved pairs, the layout of every rotated key here), is stored at
 * row slot[t] of the cache.  Token rows of the window and compressed entries
 * go into their caches this way.
 *   x      : [rows, dim], rows x_row_stride elements apart.
 *   pos    : [rows] int32; NULL = rows stored as they are (rotated already).
 *   slot   : [rows] int32, page * page_size + row within the page; -1 = the
 *            row is not stored.  Values < -1 or >= n_slots are skipped and
 *            flagged (V4_ERR_BAD_INDEX in the device status).  Slots other
 *            than -1 must be distinct: what a slot named twice holds
 *            afterwards is not defined.
 *   cache  : [n_slots, dim], dense.  Must not overlap x.
 * dim, rope_dim, dtype and angles as v4_rope.  Rows of the cache that no slot
 * names keep their values.
 * --------------------------------------------------------------------*/
v4_status v4_cache_append(const void* x, int64_t rows, int32_t dim, int64_t x_row_stride,
                          const int32_t* pos, const float* inv_freq, int32_t rope_dim,
                          const int32_t* slot, int64_t n_slots, int32_t dtype, void* cache,
                          void* stream);

/* ----------------------------------------------------------------------
 * Drafted token trees over a paged cache: decoding (one node for each
 * sequence) and the verification of drafted tokens (a tree of up to
 * V4_TREE_MAX_NODES nodes for each sequence).
 *
 * Sequence b holds seq_len[b] committed tokens; its nodes are the rows
 * node_begin[b] .. node_begin[b+1]-1 of the call, in an order in which a
 * parent precedes its children.  Node j sits at position seq_len[b] +
 * depth(j), depth 0 for a child of the last committed token.
 *
 * v4_tree_plan describes the rows once for all layers of a step:
 *   node_begin  : [B+1] int32, ascending, node_begin[B] <= n_rows <= 2^24.
 *                 Rows before the first sequence and behind the last are
 *                 padding.
 *   seq_len     : [B] int32 in [0, 2^31 - 1 - V4_TREE_MAX_NODES].
 *   parent      : [n_rows] int32, the parent's node number within the
 *                 sequence, -1 = a child of the last committed token; NULL =
 *                 every sequence's nodes form a chain.
 *   block_table : [B, max_blocks] int32, the page of each block of page_size
 *                 tokens; nullable iff slot is NULL.
 *   plan        : [n_rows, 8] int32 out: sequence (-1 = padding), node
 *                 number, position, committed length, and 128 bits (bit j of
 *                 word 4 + j/32): the node itself and its ancestors.
 *   pos         : [n_rows] int32 out, nullable: the positions (0 on padding).
 *   slot        : [n_rows] int32 out, nullable: the cache row of token
 *                 seq_len[b] + node number, where v4_cache_append puts the
 *                 node's key before v4_tree_mqa_fwd reads it (-1 on padding).
 * Bad values are flagged (V4_ERR_BAD_INDEX in the device status): a node
 * whose parent is not an earlier node is treated as a child of the last
 * committed token; a sequence with a bad range, more than V4_TREE_MAX_NODES
 * nodes or a length out of range becomes padding; a slot outside the table or
 * the cache becomes -1.  Where node_begin descends, rows that two sequences
 * then claim hold the plan of one of them or words of both.
 * After acceptance v4_pages_compact moves the accepted nodes' rows to the
 * slots of tokens seq_len[b], seq_len[b] + 1, ...
 * --------------------------------------------------------------------*/
#define V4_TREE_MAX_NODES 128
v4_status v4_tree_plan(int32_t batch, int32_t n_rows, const int32_t* node_begin,
                       const int32_t* seq_len, const int32_t* parent, const int32_t* block_table,
                       int32_t max_blocks, int32_t page_size, int64_t n_slots, int32_t* plan,
                       int32_t* pos, int32_t* slot, void* stream);

/* Pointers and sizes of one call. Nullable fields are marked. */
typedef struct v4_tree_inputs {
  const void* q;             /* [n_rows, H, D] un-rotated */
  const int32_t* plan;       /* [n_rows, 8] of v4_tree_plan */
  const void* tok_cache;     /* [tok_slots, D] rotated token rows; NULL iff window == 0 */
  const int32_t* tok_table;  /* [B, tok_blocks] page of each block of tok_page tokens */
  const void* ent_cache;     /* [ent_slots, D] rotated entries (r > 0) */
  const int32_t* ent_table;  /* [B, ent_blocks] page of each block of ent_page entries */
  const int32_t* ent_len;    /* [B] entries that the cache holds of each sequence (r > 0) */
  const int32_t* idx;        /* [n_rows, K] selected entries (K > 0) */
  const float* sink;         /* [H], nullable */
  const float* inv_freq;     /* [R/2] */
  int64_t tok_slots, ent_slots;                            /* rows of the caches */
  int32_t n_rows;
  int32_t tok_blocks, tok_page, ent_blocks, ent_page;      /* page sizes >= 1 */
} v4_tree_inputs;

/* ----------------------------------------------------------------------
 * v4_tree_mqa_fwd: v4_sparse_mqa_fwd for the planned rows.  Keys of row i
 * (position t, sequence b, committed length L):
 *   - entries s < min((t+1)/r, ent_len[b]): every one (K = 0), or those of
 *     idx[i] (-1 = unused slot; other values outside that range are skipped
 *     and flagged; an entry that is named twice counts twice);
 *   - committed tokens u < L with t - W < u <= t (W = -1: all u <= t);
 *   - the nodes j of its bits with 0 <= t - t_j < W (W = -1: any t_j <= t),
 *     read from token row L + j of the cache.
 * o = softmax-weighted sum (V = K) with the optional sink, de-rotated at -t;
 * lse natural log.  An empty key set yields o = 0 and lse = -inf (with a
 * sink: o = 0, lse = sink).  A sink of -inf is none, one of +inf takes its
 * head whole (o = 0, lse = +inf), a NaN makes its head's o and lse NaN.  Rows of padding (plan sequence -1) keep their o
 * and lse.  Only the rows of the caches named above are read; a token or
 * entry whose page the table does not hold (a negative or too large value)
 * is skipped and flagged.
 *   cfg  : batch, n_heads, head_dim, rope_dim, ratio, window, topk,
 *          softmax_scale, dtype and path are used, the others may hold
 *          anything.  q_begin must be 0.
 *   o    : [n_rows, H, D] out, must not overlap q.
 *   lse  : [n_rows, H] fp32 out, nullable.
 * idx and the entries' cache are the caller's: v4_indexer_topk selects for the
 * rows of whole, equally long sequences and v4_compress makes the entries of
 * whole sequences; neither takes a plan.
 * Logits, sums and lse are fp32 on both paths.  Probabilities are rounded to
 * bf16 on the tensor-core path, as in v4_sparse_mqa_fwd, and fp32 on CUDA
 * cores (path = V4_PATH_SIMT, 15 to 200 times as long at 64 heads).
 * Tensor-core path: bf16, H a multiple of 64 up to 512, D = 512, R = 64;
 * every other shape runs on CUDA cores.  It counts tiles of 128 keys in 32
 * bits: n_rows * H/64 * (longest key list that the tables allow / 128 + 2)
 * above 2^30 returns V4_ERR_UNSUPPORTED.  Workspace: v4_tree_workspace_size
 * bytes, 256-byte aligned; calls that may overlap need one each.  Results do
 * not depend on what the workspace held, and repeat bit for bit on the same
 * inputs.
 * --------------------------------------------------------------------*/
v4_status v4_tree_workspace_size(const v4_config* cfg, int32_t n_rows, size_t* bytes);
v4_status v4_tree_mqa_fwd(const v4_config* cfg, const v4_tree_inputs* in, void* o, float* lse,
                          void* workspace, size_t ws_bytes, void* stream);

/* ----------------------------------------------------------------------
 * Projections of single tokens with 4-bit weights and group scales: the
 * decode form of v4_q_proj and v4_grouped_o_proj, where every weight is read
 * once for a few rows.
 *   y[t, g, n] = sum_k x[t, g, k] * (code[g, n, k] - 8) * scale[g, n, k / gs]
 * and with norm_dim > 0 every block of norm_dim outputs is RMS-normalised:
 * y / sqrt(mean(y^2) + eps) * norm_w (norm_w [norm_dim] fp32, NULL = ones).
 *   x      : [rows, groups, K] bf16.      y : [rows, groups, N] bf16 out, must
 *            not overlap x.
 *   codes  : [groups, N, K/2] bytes.  Each 64-byte block holds 128 inputs:
 *            its little-endian 32-bit word 4 t + c (t, c = 0..3) holds inputs
 *            32 c + 8 t .. + 7 of the block, from the lowest nibble in the
 *            order 0, 2, 4, 6, 1, 3, 5, 7.
 *   scales : [groups, N, K/gs] bf16.
 * K a multiple of 128, N a multiple of 64, gs 32, 64 or 128, norm_dim 0, 64,
 * 128, 256 or 512 dividing N (other shapes return V4_ERR_UNSUPPORTED); rows
 * >= 0.  Products of bf16 inputs and exact codes are summed in fp32 within a
 * scale group, the groups' sums scaled and added in fp32, and rounded to
 * bf16 once (after the norm).  Meant for up to about 64 rows; more are
 * computed in slices of 64 that each read the weights again.
 *
 * v4_w4_pack makes codes and scales of a bf16 weight w [groups, K, N] (the
 * layout of wq and wo_a): scale = bf16(max|w| / 7) over the group's gs
 * inputs, code = 8 + clamp(round_to_even(w / scale), -8, 7); a group whose
 * scale is 0 gets codes 8.  Weights must be finite.
 * --------------------------------------------------------------------*/
v4_status v4_w4_pack(const void* w, int32_t groups, int32_t K, int32_t N, int32_t group_size,
                     uint8_t* codes, void* scales, void* stream);
v4_status v4_w4_proj(const void* x, int64_t rows, int32_t groups, int32_t K, int32_t N,
                     int32_t group_size, const uint8_t* codes, const void* scales,
                     int32_t norm_dim, float eps, const float* norm_w, void* y, void* stream);

/* ----------------------------------------------------------------------
 * RMS norm of each query and key head and the position rotation in one pass
 * (no counterpart of its own on the pages: [PR] items 1 and 2 norm and rotate
 * latents and entries, [BLOG] "The DeepSeek-V4-Flash architecture" norms the
 * queries of each head).
 *
 *   u = x / sqrt(mean(x^2) + eps),  out = R(pos[t]) (w * u)
 * over each head of dim values, R the rotation of v4_rope (mscale 1) on dims
 * [rope_begin, rope_begin + rope_dim).  Queries and keys are two parts of one
 * launch with their own head counts and weights; k may be NULL.  rope_dim = 0
 * leaves the rotation out (pos and inv_freq are then not read).
 *
 * v4_norm_rope_bwd: with g = R(-pos) dy and r = u / x,
 *   dw = sum over rows and heads of g * u (fp32),
 *   out = dx = r (w g - u mean(w g u)),
 * from x and dy alone.  (Where x was broadcast over heads or rows, the caller
 * sums dx over the broadcast axis.)  rows = 0 is valid: dw becomes zero.
 *
 *   x, dy, out : element (t, h, c) at t * row_stride + h * head_stride + c, in
 *                elements; strides >= 0, multiples of 16 bytes.  An output may
 *                be an input of its own part with the same strides (in place);
 *                outputs that meet themselves, each other, any other input (w,
 *                pos and inv_freq among them), dw or the workspace are refused.
 *                Views of one fused projection may be mixed as long as their
 *                row strides are equal.
 *   w          : [dim] fp32, NULL = ones.
 *   dw         : [dim] fp32 out, NULL = not wanted; the parts' must not overlap.
 *                Written when everything has been read.
 * dim a multiple of 8 up to 1024 (above: V4_ERR_UNSUPPORTED); rows times heads
 * up to 2^30; rope_dim, rope_begin, layout, dtype and angles as v4_rope.
 * Squares, sums and products are fp32, results are rounded once.  A head whose
 * sum of squares is 2^128 or more (of 512 values: a root mean square above
 * 8.2e17) becomes zero, and for finite w and dy so do its dx and its part of dw;
 * where the sum of w g x alone passes the range, that head's dx is not finite.
 * With eps = 0 a head of zeros becomes NaN, and one whose mean square is below
 * 2^-126 is inexact or not finite.  NaN and infinities stay within their head, but
 * for dw, which sums all heads.  Sums of dw have a fixed order: results repeat bit
 * for bit on the same device.  Workspace of the gradient:
 * v4_norm_rope_workspace_size(dim) bytes, 256-byte aligned, one for each of the
 * calls that may overlap.
 * --------------------------------------------------------------------*/
typedef struct v4_norm_rope_part {
  const void* x;
  const float* w;            /* nullable */
  const void* dy;            /* v4_norm_rope_bwd alone */
  void* out;                 /* y, or dx */
  float* dw;                 /* v4_norm_rope_bwd alone, nullable */
  int64_t x_row_stride, x_head_stride, dy_row_stride, dy_head_stride, out_row_stride, out_head_stride;
  int32_t heads;
} v4_norm_rope_part;
v4_status v4_norm_rope_fwd(const v4_norm_rope_part* q, const v4_norm_rope_part* k, int64_t rows,
                           int32_t dim, const int32_t* pos, const float* inv_freq, int32_t rope_dim,
                           int32_t rope_begin, int32_t layout, float eps, int32_t dtype, void* stream);
v4_status v4_norm_rope_workspace_size(int32_t dim, size_t* bytes);
v4_status v4_norm_rope_bwd(const v4_norm_rope_part* q, const v4_norm_rope_part* k, int64_t rows,
                           int32_t dim, const int32_t* pos, const float* inv_freq, int32_t rope_dim,
                           int32_t rope_begin, int32_t layout, float eps, int32_t dtype,
                           void* workspace, size_t ws_bytes, void* stream);

/* ----------------------------------------------------------------------
 * A cache held in 4 bits: v4_cache_append and v4_tree_mqa_fwd for rows of
 * 9/16 byte a value.
 *
 * A row of dim values (a multiple of 32) has v4_q4_row_bytes(dim) bytes: dim/2
 * bytes of codes, dim/16 scale bytes, zeros up to a multiple of 16.
 *   value[i] = (code[i] - 8) * scale[i / 16],
 *   scale = 2^(e - 20) * (1 + m / 8) of the byte 8 e + m.
 * The little-endian 32-bit word i of the codes holds values 8 i .. 8 i + 7, from
 * its lowest nibble in the order 0, 2, 4, 6, 1, 3, 5, 7 (as v4_w4_pack's words).
 * Every value is exact in bf16.
 *
 * v4_cache_append_q4 stores row t of x at row slot[t] of the cache, as it is
 * (v4_norm_rope_fwd and v4_rope rotate): scale = max|x| / 7 over 16 values,
 * rounded to the nearest scale (ties to even; at least 2^-20, at most 3840),
 * code = 8 + clamp(round_to_even(x / scale), -8, 7).  Infinities take the
 * largest scale and the last code of their sign; NaN is stored as zero.
 * v4_cache_read_q4 makes dense rows of it, exactly: the rows that
 * v4_sparse_mqa_fwd and v4_sparse_mqa_bwd take, for instance.  A slot of -1
 * reads zeros.
 *   x, out : [rows, dim], rows a stride apart (elements, a multiple of 16
 *            bytes); out's rows must not overlap.  rows up to 2^24.
 *   slot   : [rows] int32 as v4_cache_append's: -1 = none; others outside the
 *            cache are skipped (read: zeros) and flagged.  Written slots must
 *            be distinct.
 *   cache  : [n_slots, row bytes], must not overlap x or out.
 * --------------------------------------------------------------------*/
v4_status v4_q4_row_bytes(int32_t dim, int32_t* bytes);
v4_status v4_cache_append_q4(const void* x, int64_t rows, int32_t dim, int64_t x_row_stride,
                             const int32_t* slot, int64_t n_slots, int32_t dtype, void* cache,
                             void* stream);
v4_status v4_cache_read_q4(const void* cache, int64_t n_slots, const int32_t* slot, int64_t rows,
                           int32_t dim, int32_t dtype, void* out, int64_t out_row_stride, void* stream);

/* ----------------------------------------------------------------------
 * v4_tree_mqa_fwd over 4-bit caches: tok_cache and ent_cache hold rows of
 * v4_q4_row_bytes(D) bytes and are 32-byte aligned, everything else (keys,
 * masks, sinks, padding, bad indices, workspace, dtype of q and o, shapes of
 * either path) is v4_tree_mqa_fwd's.  The values of the rows are exact in bf16, so on the same
 * values both give the same sums but for their order.
 * --------------------------------------------------------------------*/
v4_status v4_tree_mqa_fwd_q4(const v4_config* cfg, const v4_tree_inputs* in, void* o, float* lse,
                             void* workspace, size_t ws_bytes, void* stream);

/* ----------------------------------------------------------------------
 * Pages of a cache.  A block table [n, blocks] int32 names the page of each
 * block of page_size tokens of a sequence (-1: none), as everywhere here;
 * ref [pages] int32 counts the table entries that hold each page, and a page
 * with ref 0 is free.  The lowest free pages are given first, in the order of
 * sequences and blocks, so tables and counts depend on the inputs alone.
 * Tables and counts live on the device and nothing is synchronised; one page
 * number serves the caches of all layers.  Calls that change the same counts
 * must follow each other (one stream, or events).
 *
 * v4_pages_alloc gives sequence i a page for every entry -1 among the blocks
 *   that tokens have[i] .. need[i] - 1 need beyond those of the first have[i]
 *   tokens (blocks ceil(have / page_size) .. ceil(need / page_size) - 1; have
 *   NULL = 0).  Entries of these blocks that hold a page keep it.
 * v4_pages_fork makes out_table[i] a copy of the first len[i] tokens of
 *   sequence src[i] of `table` (src -1: an empty row): whole blocks are shared
 *   (their counts rise), a partly filled last block gets a free page, and
 *   copies[i] = (its page, the new page, its rows), else (-1, -1, 0).  All other
 *   entries become -1: what out_table held before is overwritten, not released.
 *   The tables must not overlap.  An entry -1 of `table` stays one.
 * v4_pages_free releases the entries of sequence i whose blocks hold no token
 *   in [lo[i], hi[i]) (lo NULL = 0; hi NULL: all of them; any int32, so a hi
 *   above every length keeps all from lo on): they become -1 and their pages'
 *   counts fall.
 * v4_pages_copy copies the first copies[i][2] rows of page copies[i][0] to page
 *   copies[i][1] in each layer.  A target may be named once and must be no
 *   source.
 * v4_pages_compact moves rows base[i] + keep[i][j] of sequence i to rows
 *   base[i] + j (j < count[i]) in each layer: accepted nodes of a drafted tree
 *   (base = seq_len, keep = their node numbers), or the tokens that are left
 *   when others are given up.  keep[i] ascends; the pages written must be in
 *   one table row alone.
 *
 *   lack     : int32 out, nullable: entries that got no page for want of free
 *              ones (they stay -1).  NULL: a lack is flagged instead.
 *   cache    : layers of [pages, page_size, row_bytes], layer_stride bytes
 *              apart; row_bytes a multiple of 16, any contents (dense or 4-bit
 *              rows).
 * At most 8192 sequences for v4_pages_alloc and v4_pages_fork (else
 * V4_ERR_UNSUPPORTED).  Bad values are flagged (V4_ERR_BAD_INDEX in the device
 * status) and touch nothing: a length that the table does not hold or a source
 * outside it (that row gets nothing), a page outside the pool (taken for -1), a
 * fork (taken for -1) or a release of a page that is free, a copy outside the pool, a kept row that is
 * not above the one before, below its place in the list or not held, even where it
 * would stay (it is not moved).
 * --------------------------------------------------------------------*/
v4_status v4_pages_alloc(int32_t n, int32_t* table, int32_t blocks, int32_t page_size,
                         const int32_t* have, const int32_t* need, int32_t* ref, int32_t pages,
                         int32_t* lack, void* stream);
v4_status v4_pages_fork(int32_t batch, const int32_t* table, int32_t blocks, int32_t n,
                        const int32_t* src, const int32_t* len, int32_t* out_table,
                        int32_t out_blocks, int32_t page_size, int32_t* ref, int32_t pages,
                        int32_t* copies, int32_t* lack, void* stream);
v4_status v4_pages_free(int32_t n, int32_t* table, int32_t blocks, int32_t page_size,
                        const int32_t* lo, const int32_t* hi, int32_t* ref, int32_t pages, void* stream);
v4_status v4_pages_copy(void* cache, int32_t layers, int64_t layer_stride, int32_t pages,
                        int32_t page_size, int32_t row_bytes, const int32_t* copies, int32_t n,
                        void* stream);
v4_status v4_pages_compact(void* cache, int32_t layers, int64_t layer_stride, int32_t pages,
                           int32_t page_size, int32_t row_bytes, int32_t n, const int32_t* table,
                           int32_t blocks, const int32_t* base, const int32_t* count,
                           const int32_t* keep, int32_t max_keep, void* stream);

/* Text of the last non-OK status returned on this host thread ("" if none). */
const char* v4_last_error(void);

/* Static text naming the build: the target architecture and, for the
 * bound-checking build (compiled with V4_DEBUG), "V4_DEBUG". */
const char* v4_build_info(void);

/* Copy the sticky device status word (a v4_status value, 0 = clean) after
 * synchronising `stream`.  v4_reset_device_status clears it (async). */
v4_status v4_get_device_status(void* stream, int32_t* status);
v4_status v4_reset_device_status(void* stream);

/* Number of kernels this library has launched since it was loaded. */
uint64_t v4_launch_count(void);

/* ----------------------------------------------------------------------
 * Self-test of the device-side failure path (no counterpart in the method).
 * Launches one warp whose lane 0 waits, with the same bounded wait the
 * tensor-core kernels use, on a shared-memory barrier that nothing ever
 * completes; after limit_us microseconds (1 .. 1000000) the wait gives up,
 * records V4_ERR_TIMEOUT in the sticky device status word and the kernel
 * returns.  Nothing traps and no tensor-core or TMA work is in flight, so the
 * context stays usable: the host reads the status with
 * v4_get_device_status and clears it with v4_reset_device_status.
 * --------------------------------------------------------------------*/
v4_status v4_selftest_wait_timeout(int32_t limit_us, void* stream);

/* ----------------------------------------------------------------------
 * Per-stage timing.  While enabled, every stage launch is bracketed by two
 * CUDA events recorded on the stage's stream, so the timing sees exactly the
 * stage's kernels in stream order.  v4_profile_enable(1) discards earlier
 * records and starts recording; v4_profile_enable(0) stops.  Record i
 * (launch order, 0-based) is read with v4_profile_get, which waits for its
 * stop event.  kind: 0 compressor, 1 window-key rotation, 2 indexer query
 * prep, 3 indexer scores, 4 top-k, 5 attention, 6 output projection,
 * 7 backward prep (clears, tables, key rotation, query/gradient rotation and
 * delta), 8 attention backward, 9 window-gradient de-rotation, 10 E4M3
 * quantisation of the indexer operands, 11 query projections, 12 indexer
 * distillation target, 13 rotary positions, 14 paged cache write, 15 tree
 * plan, 16 tree attention, 17 join of split tree attention, 18 4-bit
 * packing, 19 4-bit projection, 20 norms with the rotation, 21 their gradient,
 * 22 4-bit cache write, 23 4-bit cache read, 24 pages given, forked or released,
 * 25 page copies, 26 compaction.
 * --------------------------------------------------------------------*/
v4_status v4_profile_enable(int32_t on);
int32_t v4_profile_count(void);
v4_status v4_profile_get(int32_t i, int32_t* kind, float* ms);

#ifdef __cplusplus
}
#endif
#endif /* V4ATTN_H */
