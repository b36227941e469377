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
// A block takes `cta_rows` outputs; its eight warps split the inputs `ks`
// ways (128-input blocks dealt round robin) and the outputs 8 / ks ways, and the
// partial sums meet in shared memory.  With a norm, the blocks of a
// norm_dim run form a cluster and exchange their sums of squares through
// distributed shared memory.
// ---------------------------------------------------------------------------
constexpr int kW4Warps = 8, kW4Threads = kW4Warps * 32;
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

// NT tiles of 8 rows of x, RT tiles of 16 outputs of a warp.
template <int NT, int RT>
__global__ void __launch_bounds__(kW4Threads) w4_kernel(const W4Args p) {
  constexpr int kTok = NT * 8;
  extern __shared__ __align__(16) uint8_t smem[];
  auto s_red = reinterpret_cast<float(*)[RT * 16][kTok]>(smem);    // [warp]: partial sums of one pass
  auto s_out = reinterpret_cast<float(*)[kTok + 1]>(s_red + kW4Warps);         // [64]
  auto s_sq = reinterpret_cast<float(*)[kTok]>(s_out + 64);        // [block of the cluster]: sums of squares
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int gq = lane >> 2, t = lane & 3;
  const int g = blockIdx.y;
  const long long row0 = (long long)blockIdx.z * kTok;
  const int live = (int)min((long long)kTok, p.rows - row0);
  const int n0 = blockIdx.x * p.cta_rows;
  const int kw = warp % p.ks, rw = warp / p.ks, nrw = kW4Warps / p.ks;
  const int nkb = p.K >> 7;
  const int per_pass = nrw * RT * 16;
  const size_t kbytes = (size_t)p.K >> 1;
  const int sgroups = p.K / p.gs;
  const int fold = p.gs >> 5;                                        // chunks of a scale group: 1, 2 or 4
  const uint8_t* cbase = p.codes + (size_t)g * p.N * kbytes + t * 16;
  const bf16* sbase = p.scales + (size_t)g * p.N * sgroups;
  const bf16* xbase = p.x + ((size_t)row0 * p.groups + g) * p.K + 8 * t;
  const size_t xrow = (size_t)p.groups * p.K;
  const int peers = p.norm_dim > p.cta_rows ? p.norm_dim / p.cta_rows : 1;
  // the cluster's blocks have all started before one writes to another's
  // shared memory: arrive here, wait before the exchange
  if (peers > 1) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");

  for (int pass = 0; pass < p.cta_rows; pass += per_pass) {
    const int nw = n0 + pass + rw * RT * 16;                        // first output of this warp
    float acc[RT][NT][4];
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[i][j][e] = 0.f;
    for (int kb = kw; kb < nkb; kb += p.ks) {
      uint4 lo[RT], hi[RT];
#pragma unroll
      for (int i = 0; i < RT; ++i) {
        const uint8_t* src = cbase + (size_t)(nw + 16 * i + gq) * kbytes + (size_t)kb * 64;
        lo[i] = __ldg(reinterpret_cast<const uint4*>(src));
        hi[i] = __ldg(reinterpret_cast<const uint4*>(src + 8 * kbytes));
      }
      float part[RT][NT][4];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        if (c % fold == 0) {
#pragma unroll
          for (int i = 0; i < RT; ++i)
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
              for (int e = 0; e < 4; ++e) part[i][j][e] = 0.f;
        }
        uint4 b[NT];
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          const int tok = 8 * j + gq;
          b[j] = tok < live ? __ldg(reinterpret_cast<const uint4*>(xbase + tok * xrow + kb * 128 + 32 * c))
                            : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int i = 0; i < RT; ++i) {
          const uint32_t wl = c == 0 ? lo[i].x : c == 1 ? lo[i].y : c == 2 ? lo[i].z : lo[i].w;
          const uint32_t wh = c == 0 ? hi[i].x : c == 1 ? hi[i].y : c == 2 ? hi[i].z : hi[i].w;
          const uint32_t a0[4] = {w4_pair(wl), w4_pair(wh), w4_pair(wl >> 4), w4_pair(wh >> 4)};
          const uint32_t a1[4] = {w4_pair(wl >> 8), w4_pair(wh >> 8), w4_pair(wl >> 12), w4_pair(wh >> 12)};
#pragma unroll
          for (int j = 0; j < NT; ++j) {
            mma_bf16(part[i][j], a0, b[j].x, b[j].y);
            mma_bf16(part[i][j], a1, b[j].z, b[j].w);
          }
        }
        if ((c + 1) % fold == 0) {
#pragma unroll
          for (int i = 0; i < RT; ++i) {
            const bf16* sp = sbase + (size_t)(nw + 16 * i + gq) * sgroups + (kb * 128 + 32 * c) / p.gs;
            const float s0 = to_f(sp[0]), s1 = to_f(sp[(size_t)8 * sgroups]);
#pragma unroll
            for (int j = 0; j < NT; ++j) {
              acc[i][j][0] = fmaf(part[i][j][0], s0, acc[i][j][0]);
              acc[i][j][1] = fmaf(part[i][j][1], s0, acc[i][j][1]);
              acc[i][j][2] = fmaf(part[i][j][2], s1, acc[i][j][2]);
              acc[i][j][3] = fmaf(part[i][j][3], s1, acc[i][j][3]);
            }
          }
        }
      }
    }
    __syncthreads();                                                // the previous pass's sums are read
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        *reinterpret_cast<float2*>(&s_red[warp][16 * i + gq][8 * j + 2 * t]) = make_float2(acc[i][j][0], acc[i][j][1]);
        *reinterpret_cast<float2*>(&s_red[warp][16 * i + gq + 8][8 * j + 2 * t]) =
            make_float2(acc[i][j][2], acc[i][j][3]);
      }
    __syncthreads();
    for (int o = threadIdx.x; o < per_pass * kTok; o += kW4Threads) {
      const int tok = o % kTok, r = o / kTok;                        // r: output of the pass
      const int w0 = (r / (RT * 16)) * p.ks, rr = r % (RT * 16);
      float v = 0.f;
      for (int k = 0; k < p.ks; ++k) v += s_red[w0 + k][rr][tok];
      s_out[pass + r][tok] = v;
    }
  }
  __syncthreads();
  if (p.norm_dim > 0) {
    uint32_t rank = 0;
    if (peers > 1) {
      asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
      asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    }
    // a warp for each row of x: this block's sum of squares
    for (int tok = warp; tok < kTok; tok += kW4Warps) {
      float q = 0.f;
      for (int r = lane; r < p.cta_rows; r += 32) q = fmaf(s_out[r][tok], s_out[r][tok], q);
      for (int o = 16; o > 0; o >>= 1) q += __shfl_xor_sync(0xffffffffu, q, o);
      if (lane < peers) {
        const uint32_t here = (uint32_t)__cvta_generic_to_shared(&s_sq[rank][tok]);
        if (peers > 1) {
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
    for (int o = threadIdx.x; o < p.cta_rows * live; o += kW4Threads) {
      const int r = o % p.cta_rows, tok = o / p.cta_rows;
      float q = 0.f;
      for (int k = 0; k < peers; ++k) q += s_sq[k][tok];
      const float inv = 1.0f / sqrtf(q / (float)p.norm_dim + p.eps);
      const float w = p.norm_w ? p.norm_w[(n0 + r) % p.norm_dim] : 1.f;
      p.y[((size_t)(row0 + tok) * p.groups + g) * p.N + n0 + r] = __float2bfloat16_rn(s_out[r][tok] * inv * w);
    }
    return;
  }
  for (int o = threadIdx.x; o < p.cta_rows * live; o += kW4Threads) {
    const int r = o % p.cta_rows, tok = o / p.cta_rows;
    p.y[((size_t)(row0 + tok) * p.groups + g) * p.N + n0 + r] = __float2bfloat16_rn(s_out[r][tok]);
  }
}

template <int NT, int RT>
cudaError_t w4_launch(W4Args p, cudaStream_t st) {
  const int nkb = p.K / 128;
  // inputs split as many ways as divide their blocks evenly, at most eight
  p.ks = nkb % 8 == 0 ? 8 : nkb % 4 == 0 ? 4 : nkb % 2 == 0 ? 2 : 1;
  if (nkb > 16 && p.ks < 8) p.ks = 8;                               // long rows: an uneven eight-way split
  while (kW4Warps / p.ks * RT * 16 > 64) p.ks *= 2;
  const int per_pass = kW4Warps / p.ks * RT * 16;
  // a norm's blocks take 64 outputs (eight blocks cover 512); without one, the
  // most outputs a block that still give two blocks an SM
  p.cta_rows = 64;
  if (p.norm_dim == 0)
    while (p.cta_rows > per_pass && (long long)p.N / p.cta_rows * p.groups < 304) p.cta_rows /= 2;
  constexpr size_t smem = (size_t)(kW4Warps * RT * 16 * NT * 8 + 64 * (NT * 8 + 1) + kMaxCluster * NT * 8) * 4;
  cudaError_t e = cudaFuncSetAttribute(w4_kernel<NT, RT>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.dynamicSmemBytes = smem;
  cfg.gridDim = dim3(p.N / p.cta_rows, p.groups, (unsigned)((p.rows + NT * 8 - 1) / (NT * 8)));
  cfg.blockDim = dim3(kW4Threads);
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
  e = cudaLaunchKernelEx(&cfg, w4_kernel<NT, RT>, (const W4Args)p);
  if (e != cudaSuccess) return e;
  note_launch();
  return cudaGetLastError();
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
  if (rows <= 8) return w4_launch<1, 4>(p, st);
  if (rows <= 16) return w4_launch<2, 2>(p, st);
  if (rows <= 32) return w4_launch<4, 2>(p, st);
  return w4_launch<8, 1>(p, st);
}

}  // namespace v4
