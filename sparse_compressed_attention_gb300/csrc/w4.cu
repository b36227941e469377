// Projections with 4-bit weights and group scales for few rows (v4_w4_proj),
// and the packing of bf16 weights (v4_w4_pack).
//
// y[t, g, n] = sum_k x[t, g, k] (code - 8) scale[g, n, k / gs], the decode
// form of the query and grouped output projections: every weight is read once
// for a handful of rows, so the bytes of the codes bound it.
#include <math.h>

#include "common.cuh"
#include "internal.h"

namespace v4 {

namespace {

// Byte of a 64-byte block that holds input k (0..127), and its nibble: word
// 4 t + c of the block holds inputs 32 c + 8 t .. + 7 in the nibble order
// 0, 2, 4, 6, 1, 3, 5, 7.
__host__ __device__ constexpr int w4_nibble(int k) {
  const int c = k >> 5, t = (k >> 3) & 3, e = k & 7;
  return (4 * t + c) * 8 + (e & 1) * 4 + (e >> 1);
}

// One thread packs one output's 128 inputs (threads of a warp take
// consecutive outputs, so each row of w is read in whole lines).  Run once for
// a weight, and left simple: 67 us for 1024 x 32768 (1.3 TB/s, floor 12.4; bound by
// the latency of two-byte loads and of the two passes over a group's inputs).
__global__ void __launch_bounds__(128)
w4_pack_kernel(const bf16* __restrict__ w, int K, int N, int gs, uint32_t* __restrict__ codes,
               bf16* __restrict__ scales) {
  const int n = blockIdx.x * blockDim.x + threadIdx.x, kb = blockIdx.y, g = blockIdx.z;
  if (n >= N) return;
  const bf16* src = w + ((size_t)g * K + (size_t)kb * 128) * N + n;
  uint32_t out[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) out[i] = 0;
  float s = 0.f;
  bf16* sdst = scales + ((size_t)g * N + n) * (K / gs);
#pragma unroll
  for (int c = 0; c < 4; ++c) {                    // chunks of 32 inputs
    if ((32 * c) % gs == 0) {                      // a scale group begins
      float amax = 0.f;
      for (int k = 32 * c; k < 32 * c + gs; ++k) amax = fmaxf(amax, fabsf(to_f(src[(size_t)k * N])));
      const bf16 sb = __float2bfloat16_rn(__fdiv_rn(amax, 7.f));
      s = to_f(sb);
      sdst[(kb * 128 + 32 * c) / gs] = sb;
    }
#pragma unroll
    for (int k = 32 * c; k < 32 * c + 32; ++k) {
      float q = s > 0.f ? rintf(__fdiv_rn(to_f(src[(size_t)k * N]), s)) : 0.f;
      q = fminf(fmaxf(q, -8.f), 7.f);
      const int nib = w4_nibble(k);
      out[nib >> 3] |= (uint32_t)((int)q + 8) << (4 * (nib & 7));
    }
  }
  uint4* dst = reinterpret_cast<uint4*>(codes + (((size_t)g * N + n) * K >> 3) + kb * 16);
#pragma unroll
  for (int i = 0; i < 4; ++i) dst[i] = make_uint4(out[4 * i], out[4 * i + 1], out[4 * i + 2], out[4 * i + 3]);
}

// ---------------------------------------------------------------------------
// The projection.  Products run on mma.sync m16n8k16 (bf16 codes x bf16 inputs,
// fp32 sums): at these sizes the codes' bytes are the bound and the legacy
// path's rate is far above it, while a lane can feed its A fragment from the
// very 16 bytes it loaded.  The order of the inputs inside a product is
// free as long as both operands share it, and the code order is chosen for
// that: lane (g, t) of a warp loads bytes 16 t .. + 15 of the 64-byte blocks
// of outputs g and g + 8, whose word c holds inputs 32 c + 8 t .. + 7.  Word c
// is two product steps (inputs 0-3, then 4-7, of every lane's eight), so
// each step stays inside one chunk of 32 inputs and scale groups of 32, 64 and
// 128 end between steps; the matching B fragment is 16 consecutive bytes of
// x.  A nibble pair becomes two bf16 with one mask-or (0x4300 | n is 128 + n)
// and one exact subtraction of 136.
//
// Up to eight rows of x (w4_few_kernel): bound by how fast codes arrive and
// are unpacked.  A warp takes 16 outputs and a contiguous part of the inputs and
// keeps kDepth blocks of 128 inputs in flight through a ring in shared
// memory, where every lane reads back exactly the bytes that it asked for
// (cp.async: no registers wait for them, no barrier).  Scales and x are asked
// for a block ahead: a load waited for where it is used costs its whole
// latency (15.7 us for one row of 1024 x 32768 with scales and x fetched in the
// loop body).  After that the instructions count (306 a warp and block in the
// first streaming version, 96 of them unpacking and products: 9.5 us), so
// pointers are incremented, rows of x beyond the last read the last one (their
// columns are never stored), a scale group's first product starts from zero by
// itself and its sums are folded two an instruction.  One row of 1024 x 32768
// with the norm: 7.5 us with its codes in L2, 8.2 from HBM (2.1 TB/s of codes; nearly
// 2 us of it a launch, about 1 the cluster's exchange).
//
// More rows (w4_rows_kernel): there the rows of x, read again for every 16
// outputs, are the larger traffic (24 rows: six times the codes; 18 us for
// 8 x 4096 x 1024 with the kernel above, 12.1 with this one, 12.7 with the codes in HBM).  Eight warps share
// each 128-input block of x through a ring of stages in shared memory, one
// block barrier a stage; rows lie 256 bytes apart with the halves of odd rows
// exchanged, so that a fragment read touches every bank once.  The issue slots
// are half busy and the tensor pipe a quarter; what is left is the latency of
// a stage, with 13 warps on an SM to cover it.
//
// `ks` warps share an output's inputs and meet in shared memory.  With a norm,
// the blocks of a norm_dim run form a cluster and exchange their sums of
// squares through distributed shared memory.
// ---------------------------------------------------------------------------
constexpr int kMaxCluster = 8;
constexpr int kDepth = 2;                    // blocks in flight, a power of two (see w4_few_kernel)
constexpr uint32_t kStageBytes = 1024;       // codes of 16 outputs x 128 inputs

struct W4Args {
  const bf16* x;
  const uint8_t* codes;
  const bf16* scales;
  const float* norm_w;
  bf16* y;
  long long rows;
  int groups, K, N, gs, norm_dim, log_ks, log_rows;      // warps an output's inputs are split over, outputs of a block
  int sq_at;                                              // shared memory offset of the cluster's sums of squares
  float eps;
};

__device__ __forceinline__ void mma_bf16(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// The same product from zero.
__device__ __forceinline__ void mma_bf16_first(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%10, %10, %10, %10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}

// Nibbles p and p + 4 of a word as bf16 values n - 8.
__device__ __forceinline__ uint32_t w4_pair(uint32_t w) {
  uint32_t u = (w & 0x000F000Fu) | 0x43004300u;                   // 128 + n
  const __nv_bfloat162 off = __floats2bfloat162_rn(136.f, 136.f);
  __nv_bfloat162 v = __hsub2(*reinterpret_cast<__nv_bfloat162*>(&u), off);
  return *reinterpret_cast<uint32_t*>(&v);
}

__device__ __forceinline__ uint32_t word_of(const uint4& v, int c) {
  return c == 0 ? v.x : c == 1 ? v.y : c == 2 ? v.z : v.w;
}

// Scales of one output and one block of 128 inputs: 4 / kFold bf16 values.
template <int kFold>
struct ScaleWord;
template <>
struct ScaleWord<1> { typedef uint2 type; };
template <>
struct ScaleWord<2> { typedef uint32_t type; };
template <>
struct ScaleWord<4> { typedef uint16_t type; };

__device__ __forceinline__ float scale_of(uint2 v, int i) {
  const uint32_t w = i < 2 ? v.x : v.y;
  return __uint_as_float((i & 1) ? (w & 0xFFFF0000u) : (w << 16));
}
__device__ __forceinline__ float scale_of(uint32_t w, int i) {
  return __uint_as_float(i ? (w & 0xFFFF0000u) : (w << 16));
}
__device__ __forceinline__ float scale_of(uint16_t w, int) { return __uint_as_float((uint32_t)w << 16); }

__device__ __forceinline__ void cp_async_16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

__device__ __forceinline__ uint4 lds128(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
  return v;
}

// What a warp's part of the work is.
struct W4Part {
  int warp, lane, gq, t, ks, rw, kw, cta_rows, g, live, n0, peers;
  long long row0;
};

__device__ __forceinline__ W4Part w4_part(const W4Args& p, int tokens) {
  W4Part q;
  // What the kernels before may have written (x; codes and scales, behind a
  // packing) is read by ordinary loads behind this wait: the read-only path wants
  // memory that nothing writes while the kernel lives, and it lives before the wait.
  // The next kernel's blocks may come at once; those of clusters when the sums are
  // done, before the exchange, since clusters that come early can keep the running
  // ones from being placed (clusters of eight blocks: 10.1 us at once for 1024 x 32768
  // with a norm of 512, 8.0 before the exchange; of four, as now: 7.4 and 7.4, 7.6 after it).
  wait_previous();
  if (p.norm_dim <= (1 << p.log_rows)) start_next();
  q.warp = threadIdx.x >> 5;
  q.lane = threadIdx.x & 31;
  q.gq = q.lane >> 2;
  q.t = q.lane & 3;
  q.ks = 1 << p.log_ks;
  q.cta_rows = 1 << p.log_rows;
  q.rw = q.warp >> p.log_ks;
  q.kw = q.warp & (q.ks - 1);
  q.g = blockIdx.y;
  q.row0 = (long long)blockIdx.z * tokens;
  q.live = (int)min((long long)tokens, p.rows - q.row0);
  q.n0 = blockIdx.x << p.log_rows;
  q.peers = p.norm_dim > q.cta_rows ? p.norm_dim >> p.log_rows : 1;
  // the cluster's blocks have all started before one writes to another's
  // shared memory: arrive here, wait before the exchange
  if (q.peers > 1) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  return q;
}

// Partial sums of every warp -> outputs.  The ring (free by now) takes
// [ks][tokens][cta_rows + 4] sums: outputs run along the rows, so that sums
// are stored without bank conflicts (the pitch is 4 modulo 16 words) and leave
// in 16-byte words.  The cluster's sums of squares have a place of their own
// behind the ring: a block that is done writes them to the others while those may
// still be streaming codes through theirs.
template <int NT>
__device__ __forceinline__ void w4_finish(const W4Args& p, const W4Part& q, float (&acc)[NT][4], uint8_t* smem) {
  constexpr int kTok = NT * 8;
  const int threads = blockDim.x, pitch = q.cta_rows + 4, part = kTok * pitch;
  float* red = reinterpret_cast<float*>(smem);
  auto s_sq = reinterpret_cast<float(*)[kTok]>(smem + p.sq_at);
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    float* at = red + q.kw * part + (8 * j + 2 * q.t) * pitch + q.rw * 16 + q.gq;
    at[0] = acc[j][0];
    at[pitch] = acc[j][1];
    at[8] = acc[j][2];
    at[pitch + 8] = acc[j][3];
  }
  __syncthreads();
  if (p.norm_dim > 0) {
    uint32_t rank = 0;
    if (q.peers > 1) {
      asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
      asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    }
    // a warp for each row of x: its sums joined, and their squares to every block
    for (int tok = q.warp; tok < q.live; tok += threads / 32) {
      float s = 0.f;
      for (int r = q.lane; r < q.cta_rows; r += 32) {
        float v = red[tok * pitch + r];
        for (int k = 1; k < q.ks; ++k) v += red[k * part + tok * pitch + r];
        red[tok * pitch + r] = v;
        s = fmaf(v, v, s);
      }
      for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
      if (q.lane < q.peers) {
        if (q.peers > 1) {
          const uint32_t here = (uint32_t)__cvta_generic_to_shared(&s_sq[rank][tok]);
          uint32_t there;
          asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(there) : "r"(here), "r"(q.lane));
          asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(there), "f"(s) : "memory");
        } else {
          s_sq[0][tok] = s;
        }
      }
    }
    if (q.peers > 1) {
      asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
      asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    } else {
      __syncthreads();
    }
  }
  const int log8 = p.log_rows - 3, joined = p.norm_dim > 0 ? 1 : q.ks;
  for (int o = threadIdx.x; o < q.live << log8; o += threads) {
    const int r = (o & ((1 << log8) - 1)) * 8, tok = o >> log8;
    float v[8];
    load8(red + tok * pitch + r, v);
    for (int k = 1; k < joined; ++k) {
      float w[8];
      load8(red + k * part + tok * pitch + r, w);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] += w[e];
    }
    if (p.norm_dim > 0) {
      float s = 0.f;
      for (int k = 0; k < q.peers; ++k) s += s_sq[k][tok];
      const float inv = 1.0f / sqrtf(s / (float)p.norm_dim + p.eps);
      const float* w = p.norm_w ? p.norm_w + ((q.n0 + r) & (p.norm_dim - 1)) : nullptr;
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] *= w ? inv * w[e] : inv;
    }
    store8(p.y + ((size_t)(q.row0 + tok) * p.groups + q.g) * p.N + q.n0 + r, v);
  }
}

// Products of one chunk of 32 inputs: words wl, wh of outputs g and g + 8, x
// of NT tiles.  kParts sums a scale group (shorter chains of products).
template <int NT, int kParts>
__device__ __forceinline__ void w4_chunk(float (&part)[kParts][NT][4], uint32_t wl, uint32_t wh, const uint4* x,
                                         bool first) {
  const uint32_t a0[4] = {w4_pair(wl), w4_pair(wh), w4_pair(wl >> 4), w4_pair(wh >> 4)};
  const uint32_t a1[4] = {w4_pair(wl >> 8), w4_pair(wh >> 8), w4_pair(wl >> 12), w4_pair(wh >> 12)};
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    if (first) mma_bf16_first(part[0][j], a0, x[j].x, x[j].y);
    else mma_bf16(part[0][j], a0, x[j].x, x[j].y);
    if (kParts == 2 && first) mma_bf16_first(part[kParts - 1][j], a1, x[j].z, x[j].w);
    else mma_bf16(part[kParts - 1][j], a1, x[j].z, x[j].w);
  }
}

// acc += part * scale, two sums an instruction.
__device__ __forceinline__ void w4_fma2(float& a0, float& a1, float p0, float p1, float s) {
  asm("{\n\t.reg .b64 a, p, s;\n\t"
      "mov.b64 a, {%0, %1};\n\tmov.b64 p, {%2, %3};\n\tmov.b64 s, {%4, %4};\n\t"
      "fma.rn.f32x2 a, p, s, a;\n\t"
      "mov.b64 {%0, %1}, a;\n\t}"
      : "+f"(a0), "+f"(a1)
      : "f"(p0), "f"(p1), "f"(s));
}

template <int NT, int kParts>
__device__ __forceinline__ void w4_fold(float (&acc)[NT][4], const float (&part)[kParts][NT][4], float s0, float s1) {
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    float v[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = kParts == 1 ? part[0][j][e] : part[0][j][e] + part[kParts - 1][j][e];
    w4_fma2(acc[j][0], acc[j][1], v[0], v[1], s0);
    w4_fma2(acc[j][2], acc[j][3], v[2], v[3], s1);
  }
}

// Up to eight rows.  kFold chunks of 32 inputs in a scale group.  Two blocks of
// codes in flight: with four, one row of 1024 x 32768 takes 8.6 us instead of 8.2 with
// the norm and 8.5 instead of 8.3 without (codes in HBM; in L2 7.4 and 7.4, 7.6 and
// 7.3), 8192 x 1024 4.4 instead of 4.3, but 8 x 4096 x 1024 8.4 instead of 9.4.
template <int kFold>
__global__ void __launch_bounds__(512) w4_few_kernel(const W4Args p) {
  typedef typename ScaleWord<kFold>::type Scales;
  extern __shared__ __align__(16) uint8_t smem[];
  const W4Part q = w4_part(p, 8);
  const int nkb = p.K >> 7;
  const int kb0 = (nkb * q.kw) >> p.log_ks, kb1 = (nkb * (q.kw + 1)) >> p.log_ks;
  const size_t out0 = (size_t)q.g * p.N + q.n0 + q.rw * 16 + q.gq;
  const size_t kbytes = (size_t)p.K >> 1;
  const uint8_t* cp0 = p.codes + out0 * kbytes + (size_t)kb0 * 64 + q.t * 16;
  const uint8_t* cp1 = cp0 + 8 * kbytes;
  const Scales* sp0 = reinterpret_cast<const Scales*>(p.scales) + out0 * nkb + kb0;
  const Scales* sp1 = sp0 + (size_t)8 * nkb;
  const uint4* xp = reinterpret_cast<const uint4*>(
      p.x + ((size_t)(q.row0 + min(q.gq, q.live - 1)) * p.groups + q.g) * p.K + (size_t)kb0 * 128 + 8 * q.t);
  float acc[1][4] = {{0.f, 0.f, 0.f, 0.f}};
  // this lane's 16 bytes of outputs g and g + 8 in each stage
  const uint32_t ring = (uint32_t)__cvta_generic_to_shared(smem) + q.warp * (kDepth * kStageBytes) + q.lane * 16;
  int left = kb1 - kb0;
  auto ask = [&](uint32_t at) {
    cp_async_16(at, cp0);
    cp_async_16(at + 512, cp1);
    cp0 += 64;
    cp1 += 64;
  };
#pragma unroll
  for (int d = 0; d < kDepth; ++d) {
    if (d < left) ask(ring + d * kStageBytes);
    asm volatile("cp.async.commit_group;" ::: "memory");
  }
  Scales s0n = *sp0, s1n = *sp1;
  uint4 xb[4], xc[4];                          // 32 inputs are four 16-byte words
#pragma unroll
  for (int i = 0; i < 4; ++i) xb[i] = xp[4 * i];
  uint32_t stage = ring;
  // one block of 128 inputs; `now` holds its x, `then` takes the next block's
  auto block = [&](uint4 (&now)[4], uint4 (&then)[4]) {
    asm volatile("cp.async.wait_group %0;" ::"n"(kDepth - 1) : "memory");
    const uint4 lo = lds128(stage), hi = lds128(stage + 512);
    // the next block's scales and x before its codes are asked for: behind them, one
    // row of 1024 x 32768 takes 9.1 us instead of 7.5 with the norm, 6.5 instead of 7.4 without
    const Scales slo = s0n, shi = s1n;
    xp += 16;
    if (left > 1) {
      s0n = *++sp0;
      s1n = *++sp1;
#pragma unroll
      for (int c = 0; c < 4; ++c) then[c] = xp[4 * c];
    }
    if (left > kDepth) ask(stage);
    asm volatile("cp.async.commit_group;" ::: "memory");
    stage = ring + ((stage + kStageBytes - ring) & (kDepth * kStageBytes - 1));
    float part[2][1][4];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      w4_chunk<1, 2>(part, word_of(lo, c), word_of(hi, c), &now[c], c % kFold == 0);
      if ((c + 1) % kFold == 0) w4_fold<1, 2>(acc, part, scale_of(slo, c / kFold), scale_of(shi, c / kFold));
    }
    --left;
  };
#pragma unroll 1
  while (left > 1) {
    block(xb, xc);
    block(xc, xb);
  }
  if (left > 0) block(xb, xc);
  asm volatile("cp.async.wait_all;" ::: "memory");
  __syncthreads();                              // every ring is read: partial sums take its place
  if (q.peers > 1) start_next();
  w4_finish<1>(p, q, acc, smem);
}

constexpr int kRowWarps = 8;

__host__ __device__ __forceinline__ uint32_t w4_stage_bytes(int ks, int tok) {
  return (uint32_t)(ks * tok * 256) + kRowWarps * kStageBytes;
}

// More than eight rows: NT tiles of 8 at a time.
template <int NT, int kFold, int kStages>
__global__ void __launch_bounds__(kRowWarps * 32, 2) w4_rows_kernel(const W4Args p) {
  constexpr int kTok = NT * 8;
  typedef typename ScaleWord<kFold>::type Scales;
  extern __shared__ __align__(16) uint8_t smem[];
  const W4Part q = w4_part(p, kTok);
  const int nkb = p.K >> 7;
  // blocks of 128 inputs of this warp's part of the inputs; every part takes
  // `steps` steps of the shared ring
  const int steps = (nkb + q.ks - 1) >> p.log_ks;
  const int kb0 = q.kw * steps, mine = min(steps, nkb - kb0);
  const size_t out0 = (size_t)q.g * p.N + q.n0 + q.rw * 16 + q.gq;
  const size_t kbytes = (size_t)p.K >> 1;
  const uint8_t* cp0 = p.codes + out0 * kbytes + (size_t)kb0 * 64 + q.t * 16;
  const uint8_t* cp1 = cp0 + 8 * kbytes;
  const Scales* sp0 = reinterpret_cast<const Scales*>(p.scales) + out0 * nkb + kb0;
  const Scales* sp1 = sp0 + (size_t)8 * nkb;
  const uint32_t base = (uint32_t)__cvta_generic_to_shared(smem), stage_bytes = w4_stage_bytes(q.ks, kTok);
  const uint32_t xt = q.kw * kTok * 256;                             // this part's x within a stage
  const uint32_t ct = q.ks * kTok * 256 + q.warp * kStageBytes + q.lane * 16;
  // x: the part's warps copy 16-byte units, unit u of a row at u ^ 4 in odd rows
  const int filler = q.rw * 32 + q.lane, fillers = (kRowWarps * 32) >> p.log_ks;
  const int fu = filler & 15, ft = filler >> 4;
  const bf16* x0 = p.x + ((size_t)q.row0 * p.groups + q.g) * p.K + (size_t)kb0 * 128 + fu * 8;
  const size_t xrow = (size_t)p.groups * p.K;
  const uint32_t xdst = xt + ft * 256 + ((fu ^ ((ft & 1) << 2)) << 4);      // rows step by an even number
  auto ask = [&](int step) {
    if (step < mine) {
      const uint32_t at = base + (step % kStages) * stage_bytes;
      cp_async_16(at + ct, cp0 + (size_t)step * 64);
      cp_async_16(at + ct + 512, cp1 + (size_t)step * 64);
      for (int tok = ft; tok < kTok; tok += fillers >> 4)
        cp_async_16(at + xdst + (tok - ft) * 256, x0 + min(tok, q.live - 1) * xrow + step * 128);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  float acc[NT][4];
#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[j][e] = 0.f;
  for (int i = 0; i < kStages - 1; ++i) ask(i);
  Scales s0n = {}, s1n = {};
  if (mine > 0) {
    s0n = *sp0;
    s1n = *sp1;
  }
#pragma unroll 1
  for (int i = 0; i < steps; ++i) {
    asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
    __syncthreads();                            // step i has landed, step i - 1 is read
    ask(i + kStages - 1);
    if (i >= mine) continue;
    const uint32_t at = base + (i % kStages) * stage_bytes;
    const uint4 lo = lds128(at + ct), hi = lds128(at + ct + 512);
    const Scales slo = s0n, shi = s1n;
    if (i + 1 < mine) {
      s0n = sp0[i + 1];
      s1n = sp1[i + 1];
    }
    float part[1][NT][4];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      uint4 x[NT];
#pragma unroll
      for (int j = 0; j < NT; ++j)
        x[j] = lds128(at + xt + (8 * j + q.gq) * 256 + ((c ^ (q.gq & 1)) << 6) + (q.t << 4));
      w4_chunk<NT, 1>(part, word_of(lo, c), word_of(hi, c), x, c % kFold == 0);
      if ((c + 1) % kFold == 0) w4_fold<NT, 1>(acc, part, scale_of(slo, c / kFold), scale_of(shi, c / kFold));
    }
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  __syncthreads();
  if (q.peers > 1) start_next();
  w4_finish<NT>(p, q, acc, smem);
}

// Larger of the ring and the sums that w4_finish puts in its place; the sums of
// squares follow.
size_t w4_ring(size_t ring, int ks, int cta_rows, int tok) {
  const size_t fin = (size_t)ks * (cta_rows + 4) * tok * 4;
  return ring > fin ? ring : fin;
}

template <typename Kernel>
cudaError_t w4_go(Kernel kern, OncePerDevice& once, size_t most, size_t ring, int tok, int threads, W4Args p, int ks,
                  int cta_rows, cudaStream_t st) {
  cudaError_t e =
      once.run([&] { return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most); });
  if (e != cudaSuccess) return e;
  p.log_ks = 0;
  while (1 << p.log_ks < ks) ++p.log_ks;
  p.log_rows = cta_rows == 128 ? 7 : cta_rows == 64 ? 6 : cta_rows == 32 ? 5 : 4;
  p.sq_at = (int)ring;
  cudaLaunchConfig_t cfg = {};
  cfg.dynamicSmemBytes = ring + (size_t)kMaxCluster * tok * 4;
  cfg.gridDim = dim3(p.N / cta_rows, p.groups, (unsigned)((p.rows + tok - 1) / tok));
  cfg.blockDim = dim3(threads);
  cfg.stream = st;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  if (p.norm_dim > cta_rows) {
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = p.norm_dim / cta_rows;
    at[1].val.clusterDim.y = 1;
    at[1].val.clusterDim.z = 1;
    cfg.numAttrs = 2;
  }
  e = cudaLaunchKernelEx(&cfg, kern, (const W4Args)p);
  if (e == cudaSuccess) note_launch();
  return e;
}

template <int kFold>
cudaError_t w4_few(const W4Args& p, cudaStream_t st) {
  static OncePerDevice once;
  const int nkb = p.K / 128;
  const long long tiles = (long long)p.N / 16 * p.groups;             // warps without a split of the inputs
  // split the inputs until about twelve warps an SM (1824 on 152 SMs) stream codes,
  // each with a few blocks to itself (up to 16 of them for 16 outputs: 8192 x 1024
  // 5.7 us split in four, 4.4 in 16).  With a norm a split in four takes an SM for
  // each block; of clusters of eight such blocks 12 run at once, 16 do not (1024 x
  // 8192 with a norm of 512: 6.8 us in four, 5.0 in two; 1024 x 4096: 3.8 and 5.0).
  const int most_ks = p.norm_dim == 0 ? 16 : p.norm_dim > 256 && tiles > 4 * 96 ? 2 : 4;
  int ks = 1;
  while (ks < most_ks && tiles * ks < 1824 && nkb >= 4 * ks) ks *= 2;
  // without a norm a block is four warps; with one it takes 64 outputs, or 128
  // where the norm covers them and the block stays within 16 warps: smaller clusters
  // (1024 x 32768 with a norm of 512: 8.3 us in clusters of eight, 7.4 of four)
  const int wide = p.norm_dim >= 128 && ks <= 2 ? 8 : 4;
  const int cta_rows = 16 * (p.norm_dim > 0 ? wide : (ks < 4 ? 4 / ks : 1));
  const int warps = ks * (cta_rows / 16);
  constexpr size_t most = 16 * kDepth * kStageBytes + kMaxCluster * 8 * 4;
  return w4_go(w4_few_kernel<kFold>, once, most, w4_ring((size_t)warps * kDepth * kStageBytes, ks, cta_rows, 8), 8,
               32 * warps, p, ks, cta_rows, st);
}

template <int NT, int kFold, int kStages>
cudaError_t w4_rows_go(const W4Args& p, int ks, int cta_rows, cudaStream_t st) {
  static OncePerDevice once;
  constexpr int kTok = NT * 8;
  constexpr size_t most = 116 * 1024;                                 // two blocks an SM
  const size_t ring = w4_ring((size_t)kStages * w4_stage_bytes(ks, kTok), ks, cta_rows, kTok);
  return w4_go(w4_rows_kernel<NT, kFold, kStages>, once, most, ring, kTok, kRowWarps * 32, p, ks, cta_rows, st);
}

template <int NT, int kFold>
cudaError_t w4_rows(const W4Args& p, cudaStream_t st) {
  const int nkb = p.K / 128;
  // A block takes 128 outputs; fewer, with the inputs split, while there are
  // not one and a half blocks for each of 152 SMs (or N is an odd number of 64): two warps on a
  // scheduler leave it idle two cycles of three (8 x 4096 x 1024, 24 rows:
  // 13.9 us split in two, 12.5 in four).  The norm needs 64 outputs a block and
  // more than 32 rows of x the room of two stages.
  int ks = p.N % 128 ? 2 : 1;
  const int most = p.norm_dim > 0 || NT > 4 ? 2 : 4;
  while (ks < most && (long long)p.N / 128 * ks * p.groups < 228 && nkb >= 4 * ks) ks *= 2;
  if (p.norm_dim == 64) ks = 2;
  const int cta_rows = 128 / ks;
  // as many stages as leave room for a second block and for L1 (48 rows of
  // 8 x 4096 x 1024, ks 2: 31.1 us with three, 21.4 with two)
  if constexpr (NT > 2)
    if (ks * NT > 8) return w4_rows_go<NT, kFold, 2>(p, ks, cta_rows, st);
  if constexpr (8 % NT == 0)
    if (ks * NT == 8) return w4_rows_go<NT, kFold, 3>(p, ks, cta_rows, st);
  return w4_rows_go<NT, kFold, NT < 8 ? 4 : 3>(p, ks, cta_rows, st);
}

template <int kFold>
cudaError_t w4_by_rows(const W4Args& p, cudaStream_t st) {
  // As few tiles of eight rows as hold them, where it shows: products and sums are
  // what bounds the larger counts (24 rows of 8 x 4096 x 1024: 15.2 us in four
  // tiles, 12.5 in three; 48 rows: 26.5 in eight, 21.4 in six).
  if (p.rows <= 8) return w4_few<kFold>(p, st);
  if (p.rows <= 16) return w4_rows<2, kFold>(p, st);
  if (p.rows <= 24) return w4_rows<3, kFold>(p, st);
  if (p.rows <= 32) return w4_rows<4, kFold>(p, st);
  if (p.rows <= 48) return w4_rows<6, kFold>(p, st);
  return w4_rows<8, kFold>(p, st);
}

}  // namespace

cudaError_t launch_w4_pack(const void* w, int groups, int K, int N, int gs, uint8_t* codes, void* scales,
                           cudaStream_t st) {
  const dim3 grid((N + 127) / 128, K / 128, groups);
  w4_pack_kernel<<<grid, 128, 0, st>>>((const bf16*)w, K, N, gs, (uint32_t*)codes, (bf16*)scales);
  note_launch();
  return cudaGetLastError();
}

cudaError_t launch_w4_proj(const void* x, long long rows, int groups, int K, int N, int gs, const uint8_t* codes,
                           const void* scales, int norm_dim, float eps, const float* norm_w, void* y,
                           cudaStream_t st) {
  W4Args p;
  p.x = (const bf16*)x;
  p.codes = codes;
  p.scales = (const bf16*)scales;
  p.norm_w = norm_w;
  p.y = (bf16*)y;
  p.rows = rows;
  p.groups = groups;
  p.K = K;
  p.N = N;
  p.gs = gs;
  p.norm_dim = norm_dim;
  p.eps = eps;
  p.log_ks = p.log_rows = p.sq_at = 0;
  if (gs == 32) return w4_by_rows<1>(p, st);
  if (gs == 64) return w4_by_rows<2>(p, st);
  return w4_by_rows<4>(p, st);
}

}  // namespace v4
