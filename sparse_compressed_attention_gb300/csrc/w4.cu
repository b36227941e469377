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
// consecutive outputs, so each row of w is read in whole lines).
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
// A warp takes RT tiles of 16 outputs and a contiguous part of the inputs,
// kDepth blocks of 128 inputs ahead in registers: the bytes in flight, not the
// arithmetic, set the speed of few rows.  `ks` warps share an output's inputs
// and meet in shared memory.  With a norm, a block takes 64 outputs and the
// blocks of a norm_dim run form a cluster and exchange their sums of squares
// through distributed shared memory.
// ---------------------------------------------------------------------------
constexpr int kMaxCluster = 8;

struct W4Args {
  const bf16* x;
  const uint8_t* codes;
  const bf16* scales;
  const float* norm_w;
  bf16* y;
  long long rows;
  int groups, K, N, gs, norm_dim, ks, cta_rows;
  float eps;
};

__device__ __forceinline__ void mma_bf16(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
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

// NT tiles of 8 rows of x, RT tiles of 16 outputs of a warp, kFold chunks of 32
// inputs in a scale group.
template <int NT, int RT, int kDepth, int kFold>
__global__ void __launch_bounds__(RT == 1 ? 512 : 256) w4_kernel(const W4Args p) {
  constexpr int kTok = NT * 8;
  extern __shared__ __align__(16) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, threads = blockDim.x;
  auto s_red = reinterpret_cast<float(*)[kTok]>(smem);                         // [ks][cta_rows]: partial sums
  auto s_sq = reinterpret_cast<float(*)[kTok]>(s_red + p.ks * p.cta_rows);     // [block of the cluster]
  const int gq = lane >> 2, t = lane & 3;
  const int g = blockIdx.y;
  const long long row0 = (long long)blockIdx.z * kTok;
  const int live = (int)min((long long)kTok, p.rows - row0);
  const int n0 = blockIdx.x * p.cta_rows;
  const int rw = warp / p.ks, kw = warp - rw * p.ks;
  const int nkb = p.K >> 7;
  const int kb0 = (int)((long long)nkb * kw / p.ks), kb1 = (int)((long long)nkb * (kw + 1) / p.ks);
  const size_t kbytes = (size_t)p.K >> 1;
  typedef typename ScaleWord<kFold>::type Scales;
  const int sgroups = nkb * (4 / kFold);
  const int nw = rw * RT * 16;                                       // first output of this warp within the block
  const uint8_t* cbase = p.codes + ((size_t)g * p.N + n0 + nw + gq) * kbytes + t * 16;
  const bf16* sbase = p.scales + ((size_t)g * p.N + n0 + nw + gq) * sgroups;
  const bf16* xbase = p.x + ((size_t)row0 * p.groups + g) * p.K + 8 * t;
  const size_t xrow = (size_t)p.groups * p.K;
  const int peers = p.norm_dim > p.cta_rows ? p.norm_dim / p.cta_rows : 1;
  // the cluster's blocks have all started before one writes to another's
  // shared memory: arrive here, wait before the exchange
  if (peers > 1) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");

  // Everything a block of inputs needs is asked for ahead: codes and scales
  // kDepth blocks, the rows of x a block (few rows) or a chunk ahead.  A load
  // in the loop that is waited for at once costs its whole latency: with
  // scales and x fetched where they are used, one row of 1024 x 32768 took
  // 15.7 us.
  uint4 lo[kDepth][RT], hi[kDepth][RT];
  Scales slo[kDepth][RT], shi[kDepth][RT];
  auto fetch = [&](int d, int kb) {
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      const uint8_t* src = cbase + (size_t)(16 * i) * kbytes + (size_t)kb * 64;
      lo[d][i] = __ldg(reinterpret_cast<const uint4*>(src));
      hi[d][i] = __ldg(reinterpret_cast<const uint4*>(src + 8 * kbytes));
      const bf16* sp = sbase + (size_t)(16 * i) * sgroups + kb * (4 / kFold);
      slo[d][i] = __ldg(reinterpret_cast<const Scales*>(sp));
      shi[d][i] = __ldg(reinterpret_cast<const Scales*>(sp + (size_t)8 * sgroups));
    }
  };
  constexpr int kAhead = NT <= 2 ? 4 : 1;                            // chunks of x in flight
  uint4 xb[kAhead][NT];
  auto fetch_x = [&](int slot, int chunk) {                          // chunk: 4 kb + c
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const int tok = 8 * j + gq;
      xb[slot][j] = tok < live ? __ldg(reinterpret_cast<const uint4*>(xbase + tok * xrow + 32 * chunk))
                               : make_uint4(0, 0, 0, 0);
    }
  };
#pragma unroll
  for (int d = 0; d < kDepth; ++d)
    if (kb0 + d < kb1) fetch(d, kb0 + d);
#pragma unroll
  for (int i = 0; i < kAhead; ++i) fetch_x(i, 4 * kb0 + i);
  float acc[RT][NT][4];
#pragma unroll
  for (int i = 0; i < RT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[i][j][e] = 0.f;
  for (int base = kb0; base < kb1; base += kDepth) {
#pragma unroll
    for (int d = 0; d < kDepth; ++d) {
      const int kb = base + d;
      if (kb < kb1) {
        uint4 cl[RT], ch[RT];
        Scales sl[RT], sh[RT];
#pragma unroll
        for (int i = 0; i < RT; ++i) {
          cl[i] = lo[d][i];
          ch[i] = hi[d][i];
          sl[i] = slo[d][i];
          sh[i] = shi[d][i];
        }
        if (kb + kDepth < kb1) fetch(d, kb + kDepth);
        // few rows: two sums a scale group (first and second halves of the
        // words), two shorter chains of products
        constexpr int kParts = NT > 2 ? 1 : 2;
        float part[kParts][RT][NT][4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint4 b[NT];
#pragma unroll
          for (int j = 0; j < NT; ++j) b[j] = xb[c % kAhead][j];
          if (4 * kb + c + kAhead < 4 * kb1) fetch_x(c % kAhead, 4 * kb + c + kAhead);
          if (c % kFold == 0) {
#pragma unroll
            for (int h = 0; h < kParts; ++h)
#pragma unroll
              for (int i = 0; i < RT; ++i)
#pragma unroll
                for (int j = 0; j < NT; ++j)
#pragma unroll
                  for (int e = 0; e < 4; ++e) part[h][i][j][e] = 0.f;
          }
#pragma unroll
          for (int i = 0; i < RT; ++i) {
            const uint32_t wl = word_of(cl[i], c), wh = word_of(ch[i], c);
            const uint32_t a0[4] = {w4_pair(wl), w4_pair(wh), w4_pair(wl >> 4), w4_pair(wh >> 4)};
            const uint32_t a1[4] = {w4_pair(wl >> 8), w4_pair(wh >> 8), w4_pair(wl >> 12), w4_pair(wh >> 12)};
#pragma unroll
            for (int j = 0; j < NT; ++j) {
              mma_bf16(part[0][i][j], a0, b[j].x, b[j].y);
              mma_bf16(part[kParts - 1][i][j], a1, b[j].z, b[j].w);
            }
          }
          if ((c + 1) % kFold == 0) {
#pragma unroll
            for (int i = 0; i < RT; ++i) {
              const float s0 = scale_of(sl[i], c / kFold), s1 = scale_of(sh[i], c / kFold);
#pragma unroll
              for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  const float v = kParts == 1 ? part[0][i][j][e] : part[0][i][j][e] + part[kParts - 1][i][j][e];
                  acc[i][j][e] = fmaf(v, e < 2 ? s0 : s1, acc[i][j][e]);
                }
            }
          }
        }
      }
    }
  }
#pragma unroll
  for (int i = 0; i < RT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      float* at = s_red[kw * p.cta_rows + nw + 16 * i + gq] + 8 * j + 2 * t;
      *reinterpret_cast<float2*>(at) = make_float2(acc[i][j][0], acc[i][j][1]);
      *reinterpret_cast<float2*>(at + 8 * kTok) = make_float2(acc[i][j][2], acc[i][j][3]);
    }
  __syncthreads();
  if (p.ks > 1) {
    float* red = &s_red[0][0];
    const int n = p.cta_rows * kTok;
    for (int o = threadIdx.x; o < n; o += threads) {
      float v = red[o];
      for (int k = 1; k < p.ks; ++k) v += red[k * n + o];
      red[o] = v;
    }
    __syncthreads();
  }
  if (p.norm_dim > 0) {
    uint32_t rank = 0;
    if (peers > 1) {
      asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
      asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    }
    // a warp for each row of x: this block's sum of squares, to every block
    for (int tok = warp; tok < live; tok += threads / 32) {
      float q = 0.f;
      for (int r = lane; r < p.cta_rows; r += 32) q = fmaf(s_red[r][tok], s_red[r][tok], q);
      for (int o = 16; o > 0; o >>= 1) q += __shfl_xor_sync(0xffffffffu, q, o);
      if (lane < peers) {
        if (peers > 1) {
          const uint32_t here = (uint32_t)__cvta_generic_to_shared(&s_sq[rank][tok]);
          uint32_t there;
          asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(there) : "r"(here), "r"(lane));
          asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(there), "f"(q) : "memory");
        } else {
          s_sq[0][tok] = q;
        }
      }
    }
    if (peers > 1) {
      asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
      asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    } else {
      __syncthreads();
    }
  }
  for (int o = threadIdx.x; o < p.cta_rows * live; o += threads) {
    const int r = o % p.cta_rows, tok = o / p.cta_rows;
    float v = s_red[r][tok];
    if (p.norm_dim > 0) {
      float q = 0.f;
      for (int k = 0; k < peers; ++k) q += s_sq[k][tok];
      v *= 1.0f / sqrtf(q / (float)p.norm_dim + p.eps);
      if (p.norm_w) v *= p.norm_w[(n0 + r) % p.norm_dim];
    }
    p.y[((size_t)(row0 + tok) * p.groups + g) * p.N + n0 + r] = __float2bfloat16_rn(v);
  }
}

template <int NT, int RT, int kDepth, int kFold>
cudaError_t w4_launch_fold(W4Args p, cudaStream_t st) {
  constexpr int kMaxSmem = 16 * 16 * NT * 8 * 4 * RT + kMaxCluster * NT * 8 * 4;
  static OncePerDevice once;
  cudaError_t e = once.run([&] {
    return cudaFuncSetAttribute(w4_kernel<NT, RT, kDepth, kFold>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem);
  });
  if (e != cudaSuccess) return e;
  const int nkb = p.K / 128;
  const long long tiles = (long long)p.N / (16 * RT) * p.groups;      // warps without a split of the inputs
  // split the inputs until about twelve warps an SM stream codes
  p.ks = 1;
  while (p.ks < 4 && tiles * p.ks < 1824 && nkb >= 4 * p.ks) p.ks *= 2;
  // a norm's blocks take 64 outputs (eight blocks cover 512); without one a
  // block is four warps
  const int rt = p.norm_dim > 0 ? 4 / RT : (p.ks < 4 ? 4 / p.ks : 1);
  p.cta_rows = 16 * RT * rt;
  while (p.N % p.cta_rows) p.cta_rows /= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.dynamicSmemBytes = (size_t)p.ks * p.cta_rows * NT * 8 * 4 + kMaxCluster * NT * 8 * 4;
  cfg.gridDim = dim3(p.N / p.cta_rows, p.groups, (unsigned)((p.rows + NT * 8 - 1) / (NT * 8)));
  cfg.blockDim = dim3(32 * p.ks * (p.cta_rows / (16 * RT)));
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  if (p.norm_dim > p.cta_rows) {
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = p.norm_dim / p.cta_rows;
    at[0].val.clusterDim.y = 1;
    at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
  }
  e = cudaLaunchKernelEx(&cfg, w4_kernel<NT, RT, kDepth, kFold>, (const W4Args)p);
  if (e != cudaSuccess) return e;
  note_launch();
  return cudaGetLastError();
}

template <int NT, int RT, int kDepth>
cudaError_t w4_launch(const W4Args& p, cudaStream_t st) {
  if (p.gs == 32) return w4_launch_fold<NT, RT, kDepth, 1>(p, st);
  if (p.gs == 64) return w4_launch_fold<NT, RT, kDepth, 2>(p, st);
  return w4_launch_fold<NT, RT, kDepth, 4>(p, st);
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
  p.ks = p.cta_rows = 0;
  if (rows <= 8) return w4_launch<1, 1, 4>(p, st);
  if (rows <= 16) return w4_launch<2, 1, 4>(p, st);
  if (rows <= 32) return w4_launch<4, 2, 2>(p, st);
  return w4_launch<8, 2, 2>(p, st);
}

}  // namespace v4
