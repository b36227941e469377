// RMS norm of each query and key head with the position rotation in the same
// pass, and its gradients (v4_norm_rope_fwd, v4_norm_rope_bwd).
//
//   u = x r, r = 1 / sqrt(mean(x^2) + eps);   y = R(pos) (w u)
//   g = R(-pos) dy;   dw = sum g u;   dx = r (w g - x r^2 mean(w g x))
//
// Memory bound: x is read and y written once, the gradient reads x and dy and
// writes dx.  A head belongs to a group of 1 to 32 lanes that keeps it in
// registers, so the mean is a butterfly over the group and nothing is read
// twice; the weight stays in registers over all heads of a block, which are
// queries or keys alone.  The block forms the angles of its rows once in shared
// memory while the first heads are in flight.  Weight gradients are summed in
// registers over all heads of a block, then over its warps; a second kernel adds
// the blocks' sums in a fixed order, so results repeat bit for bit.
#include <math.h>

#include "common.cuh"
#include "fastdiv.cuh"
#include "internal.h"
#include "turn.cuh"

namespace v4 {

namespace {

constexpr int kThreads = 128;
constexpr int kMaxAngles = 1024;                 // (row, pair) angles of a tile
constexpr int kGradBlocks = 912;                 // six for each of 152 SMs

struct Part {
  const void* x;
  const void* dy;                                // gradient
  const float* w;                                // null: ones
  void* out;                                     // y or dx
  long long xr, xh, gr, gh, yr, yh;              // strides in elements
  int heads, rb, hb;                             // rows and heads of a tile
  int head_tiles, tiles, blocks;
  FastDiv by_tiles, by_hb;
};

struct Args {
  Part part[2];
  const int32_t* pos;
  const float* inv_freq;
  float* partial;                                // [blocks of both parts][dim]
  long long rows;
  float eps, inv_dim;
  int dim, units, lg;                            // units of eight, log2 of a group's lanes
  int R, begin;                                  // in elements
  FastDiv by_half;
};

// Heads that a group has in flight: up to 64 bytes a lane of each input.
template <typename T, int U, bool kGrad>
constexpr int ahead() {
  const int n = 8 / (U * (int)sizeof(T)) / (kGrad ? 2 : 1);
  return n < 1 ? 1 : n;
}

// U: units of a lane.  kHalf: pairs half a rotation apart.
template <typename T, int U, bool kHalf, bool kGrad>
__global__ void __launch_bounds__(kThreads) norm_rope_kernel(const Args p) {
  constexpr int K = ahead<T, U, kGrad>();
  __shared__ float2 s_cs[kMaxAngles];
  __shared__ __align__(16) float s_x[kHalf || kGrad ? kThreads * 8 * U : 4];
  after_previous();
  const int G = 1 << p.lg;
  const int lane = threadIdx.x & (G - 1), grp = threadIdx.x >> p.lg, groups = kThreads >> p.lg;
  const bool second = blockIdx.x >= (unsigned)p.part[0].blocks;
  const Part& q = p.part[second];
  const int half = p.R >> 1;
  const int v0 = p.begin >> 3, nv = p.R >> 3;    // rotated units
  float* strip = s_x + (kHalf ? grp * (G * 8 * U) : 0);

  float w[U][8], dw[kGrad ? U : 1][8];
  int rot[U];                                    // number of a rotated unit, -1: not rotated
#pragma unroll
  for (int s = 0; s < U; ++s) {
    const int u = lane + G * s;
    rot[s] = u >= v0 && u < v0 + nv ? u - v0 : -1;
    if (q.w != nullptr && u < p.units) {
      load8(q.w + 8 * u, w[s]);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) w[s][e] = 1.f;
    }
    if (kGrad) {
#pragma unroll
      for (int e = 0; e < 8; ++e) dw[s][e] = 0.f;
    }
  }

  for (int tile = blockIdx.x - (second ? p.part[0].blocks : 0); tile < q.tiles; tile += q.blocks) {
    const int rt = (int)q.by_tiles.div((uint32_t)tile);
    const int head0 = (tile - rt * q.head_tiles) * q.hb;
    const long long row0 = (long long)rt * q.rb;
    const int nr = (int)min((long long)q.rb, p.rows - row0), nh = min(q.hb, q.heads - head0);
    const int n = nr * q.hb;
    const T* x = reinterpret_cast<const T*>(q.x) + row0 * q.xr + (long long)head0 * q.xh;
    const T* dy = kGrad ? reinterpret_cast<const T*>(q.dy) + row0 * q.gr + (long long)head0 * q.gh : nullptr;
    T* out = reinterpret_cast<T*>(q.out) + row0 * q.yr + (long long)head0 * q.yh;
    bool angles = half == 0;                     // formed once the first loads are in flight
    if (kGrad) __syncthreads();                  // the tile before has used its angles
    for (int base = 0; base < n; base += groups * K) {
      Raw<T> a[K][U], d[kGrad ? K : 1][U];
      int row[K], head[K];
      bool live[K];
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const int i = base + k * groups + grp;
        row[k] = (int)q.by_hb.div((uint32_t)i);
        head[k] = i - row[k] * q.hb;
        live[k] = i < n && head[k] < nh;
#pragma unroll
        for (int s = 0; s < U; ++s) {
          const int u = lane + G * s;
          if (live[k] && u < p.units) {
            a[k][s].load(x + row[k] * q.xr + head[k] * q.xh + 8 * u);
            if (kGrad) d[k][s].load(dy + row[k] * q.gr + head[k] * q.gh + 8 * u);
          } else {
#pragma unroll
            for (int e = 0; e < (int)(sizeof(T) / 2); ++e) {
              a[k][s].w[e] = make_uint4(0, 0, 0, 0);
              if (kGrad) d[k][s].w[e] = make_uint4(0, 0, 0, 0);
            }
          }
        }
      }
      if (!angles) {
        angles = true;
        for (int j = threadIdx.x; j < nr * half; j += kThreads) {
          const int r = (int)p.by_half.div((uint32_t)j), c = j - r * half;
          float cs, sn;
          turn_cos_sin(p.pos[row0 + r], turn_fraction(p.inv_freq[c]), &cs, &sn);
          s_cs[j] = make_float2(cs, kGrad ? -sn : sn);
        }
        __syncthreads();
      }
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const float2* cs = s_cs + (live[k] ? row[k] : 0) * half;
        // the tensor that is turned: y before its rotation, or the gradient
        auto turn = [&](float (*v)[8]) {
          if (kHalf) {
            __syncwarp();
#pragma unroll
            for (int s = 0; s < U; ++s)
              if (rot[s] >= 0) store8(strip + 8 * rot[s], v[s]);
            __syncwarp();
          }
#pragma unroll
          for (int s = 0; s < U; ++s) {
            if (rot[s] < 0) continue;
            if (kHalf) {
              const bool low = rot[s] < nv / 2;
              const int j = low ? rot[s] : rot[s] - nv / 2;
              float o[8];
              load8(strip + 8 * (low ? rot[s] + nv / 2 : j), o);
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const float2 c = cs[8 * j + e];
                v[s][e] = low ? v[s][e] * c.x - o[e] * c.y : o[e] * c.y + v[s][e] * c.x;
              }
            } else {
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const float2 c = cs[4 * rot[s] + e];
                rot_pair(v[s][2 * e], v[s][2 * e + 1], c.x, c.y);
              }
            }
          }
        };
        float v[U][8], g[kGrad ? U : 1][8];
        float sq = 0.f, dot = 0.f;
#pragma unroll
        for (int s = 0; s < U; ++s) {
          a[k][s].floats(v[s]);
#pragma unroll
          for (int e = 0; e < 8; ++e) sq = fmaf(v[s][e], v[s][e], sq);
        }
        if (kGrad) {
#pragma unroll
          for (int s = 0; s < U; ++s) d[k][s].floats(g[s]);
          turn(g);
#pragma unroll
          for (int s = 0; s < U; ++s)
#pragma unroll
            for (int e = 0; e < 8; ++e) dot = fmaf(w[s][e] * g[s][e], v[s][e], dot);
        }
        for (int o = G >> 1; o > 0; o >>= 1) {
          sq += __shfl_xor_sync(0xffffffffu, sq, o);
          if (kGrad) dot += __shfl_xor_sync(0xffffffffu, dot, o);
        }
        const float r = 1.f / sqrtf(fmaf(sq, p.inv_dim, p.eps));
        if (kGrad) {
          const float m = dot * p.inv_dim * (r * r);
#pragma unroll
          for (int s = 0; s < U; ++s)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              if (live[k]) dw[s][e] = fmaf(g[s][e], v[s][e] * r, dw[s][e]);
              v[s][e] = r * (w[s][e] * g[s][e] - v[s][e] * m);
            }
        } else {
#pragma unroll
          for (int s = 0; s < U; ++s)
#pragma unroll
            for (int e = 0; e < 8; ++e) v[s][e] *= r * w[s][e];
          turn(v);
        }
        if (!live[k]) continue;
#pragma unroll
        for (int s = 0; s < U; ++s) {
          const int u = lane + G * s;
          if (u < p.units) store8(out + row[k] * q.yr + head[k] * q.yh + 8 * u, v[s]);
        }
      }
    }
  }

  if (kGrad) {
    // a lane's sums over the groups of its warp, then over the warps
#pragma unroll
    for (int s = 0; s < U; ++s)
#pragma unroll
      for (int e = 0; e < 8; ++e)
        for (int o = G; o < 32; o <<= 1) dw[s][e] += __shfl_xor_sync(0xffffffffu, dw[s][e], o);
    __syncthreads();                             // the strips are free
    const int warp = threadIdx.x >> 5, width = G * 8 * U;
    if ((threadIdx.x & 31) < G) {
#pragma unroll
      for (int s = 0; s < U; ++s) store8(s_x + warp * width + 8 * (lane + G * s), dw[s]);
    }
    __syncthreads();
    float* to = p.partial + (size_t)blockIdx.x * p.dim;
    for (int c = threadIdx.x; c < p.dim; c += kThreads) {
      float t = 0.f;
#pragma unroll
      for (int i = 0; i < kThreads / 32; ++i) t += s_x[i * width + c];
      to[c] = t;
    }
  }
}

// dw[c] = sum of the blocks' sums: 32 columns a block, a warp every 32nd row.
struct SumArgs {
  const float* partial;
  float* out[2];
  int first[2], blocks[2];
  int dim;
};

__global__ void __launch_bounds__(1024) norm_weight_kernel(const SumArgs p) {
  __shared__ float s_t[32][33];
  after_previous();
  const int part = blockIdx.y;
  if (p.out[part] == nullptr) return;
  const int cx = threadIdx.x & 31, ry = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + cx;
  float t = 0.f;
  if (c < p.dim) {
    const float* from = p.partial + (size_t)p.first[part] * p.dim + c;
#pragma unroll 4
    for (int b = ry; b < p.blocks[part]; b += 32) t += from[(size_t)b * p.dim];
  }
  s_t[ry][cx] = t;
  __syncthreads();
  t = s_t[cx][ry];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
  if (cx == 0 && blockIdx.x * 32 + ry < p.dim) p.out[part][blockIdx.x * 32 + ry] = t;
}

template <typename T, int U, bool kGrad>
void (*kernel_of(bool half))(const Args) {
  return half ? norm_rope_kernel<T, U, true, kGrad> : norm_rope_kernel<T, U, false, kGrad>;
}

template <typename T, bool kGrad>
void (*kernel_of(int units_a_lane, bool half))(const Args) {
  return units_a_lane == 1 ? kernel_of<T, 1, kGrad>(half)
                           : units_a_lane == 2 ? kernel_of<T, 2, kGrad>(half) : kernel_of<T, 4, kGrad>(half);
}

}  // namespace

size_t norm_rope_workspace(int dim) { return (size_t)(kGradBlocks + 2) * dim * sizeof(float); }

cudaError_t launch_norm_rope(const NormCall& c, cudaStream_t st) {
  const bool grad = c.grad;
  Args p;
  p.pos = c.pos;
  p.inv_freq = c.inv_freq;
  p.partial = (float*)c.workspace;
  p.rows = c.rows;
  p.eps = c.eps;
  p.inv_dim = 1.f / (float)c.dim;
  p.dim = c.dim;
  p.units = c.dim / 8;
  // lanes of a head: the next power of two of its units, a lane holding up to four
  const int U = p.units <= 32 ? 1 : p.units <= 64 ? 2 : 4;
  p.lg = 0;
  while ((U << p.lg) < p.units) ++p.lg;
  p.R = c.rope_dim;
  p.begin = c.rope_begin;
  const int half = p.R / 2;
  p.by_half.set((uint32_t)(half > 0 ? half : 1));
  const int groups = kThreads >> p.lg;
  const int es = c.dtype == V4_BF16 ? 2 : 4;
  // Heads of a tile: four rounds of loads, one while that would leave SMs without a
  // block; the gradient's blocks walk tiles of 16 rounds.
  int k = 8 / (U * es) / (grad ? 2 : 1);
  if (k < 1) k = 1;
  long long all = 0;
  for (int i = 0; i < 2; ++i) all += c.rows * (c.part[i].x ? c.part[i].heads : 0);
  int want = groups * k * (grad ? 16 : 4);
  while (want > groups && all / want < (grad ? kGradBlocks : 608)) want /= 2;
  if (want < groups) want = groups;
  long long first = 0, work[2] = {0, 0};
  for (int i = 0; i < 2; ++i) {
    Part& q = p.part[i];
    const NormPartCall& s = c.part[i];
    q.heads = s.x ? s.heads : 0;
    q.x = s.x;
    q.dy = s.dy;
    q.w = s.w;
    q.out = s.out;
    q.xr = s.x_row_stride;
    q.xh = s.x_head_stride;
    q.gr = s.dy_row_stride;
    q.gh = s.dy_head_stride;
    q.yr = s.out_row_stride;
    q.yh = s.out_head_stride;
    q.rb = q.hb = q.head_tiles = 1;
    q.tiles = q.blocks = 0;
    if (q.heads > 0) {
      q.hb = q.heads < want ? q.heads : want;
      long long rb = q.hb == q.heads ? want / q.heads : 1;
      if (half > 0 && rb > kMaxAngles / half) rb = kMaxAngles / half;
      if (rb < 1) rb = 1;
      if (rb > c.rows) rb = c.rows;
      q.rb = (int)rb;
      q.head_tiles = (q.heads + q.hb - 1) / q.hb;
      const long long tiles = ((c.rows + rb - 1) / rb) * q.head_tiles;
      if (tiles > 0x7FFFFFFF / 2) return cudaErrorInvalidValue;
      q.tiles = q.blocks = (int)tiles;
      work[i] = tiles;
    }
    q.by_tiles.set((uint32_t)q.head_tiles);
    q.by_hb.set((uint32_t)q.hb);
    first += q.blocks;
  }
  if (grad && work[0] + work[1] > kGradBlocks) {
    // blocks in proportion to the parts' tiles, one at least
    for (int i = 0; i < 2; ++i) {
      const long long n = work[i] * kGradBlocks / (work[0] + work[1]);
      p.part[i].blocks = work[i] == 0 ? 0 : n < 1 ? 1 : (int)n;
    }
  }
  const int blocks = p.part[0].blocks + p.part[1].blocks;
  void (*kern)(const Args);
  if (c.dtype == V4_BF16) kern = grad ? kernel_of<bf16, true>(U, c.half) : kernel_of<bf16, false>(U, c.half);
  else kern = grad ? kernel_of<float, true>(U, c.half) : kernel_of<float, false>(U, c.half);
  cudaError_t e = cudaSuccess;
  if (blocks > 0) {                              // else weight gradients of no rows: zeros
    e = launch_overlapped(kern, dim3((unsigned)blocks), dim3(kThreads), 0, st, p);
    if (e != cudaSuccess) return e;
    note_launch();
  }
  if (!grad) return cudaSuccess;
  SumArgs s;
  s.partial = p.partial;
  s.dim = c.dim;
  for (int i = 0; i < 2; ++i) {
    s.out[i] = c.part[i].dw;
    s.first[i] = i == 0 ? 0 : p.part[0].blocks;
    s.blocks[i] = p.part[i].blocks;
  }
  if (s.out[0] == nullptr && s.out[1] == nullptr) return cudaSuccess;
  e = launch_overlapped(norm_weight_kernel, dim3((unsigned)((c.dim + 31) / 32), 2), dim3(1024), 0, st, s);
  if (e == cudaSuccess) note_launch();
  return e;
}

}  // namespace v4
