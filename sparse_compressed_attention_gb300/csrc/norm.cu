// RMS norm of each query and key head with the position rotation in the same
// pass, and its gradients (v4_norm_rope_fwd, v4_norm_rope_bwd).
//
//   u = x r, r = 1 / sqrt(mean(x^2) + eps);   y = R(pos) (w u)
//   g = R(-pos) dy;   dw = sum g u;   dx = r (w g - x r^2 mean(w g x))
//
// Memory bound: x is read and y written once, the gradient reads x and dy and
// writes dx.  A head belongs to a group of 1 to 32 lanes that keeps it in
// registers, so the mean is a butterfly over the group and nothing is read
// twice.  A group takes a short run of consecutive heads, of queries or of keys,
// that arrive through a ring in shared memory (16-byte asynchronous copies, two or
// three heads a group in flight, which registers would not hold): the weight stays in
// registers and a row's angles are formed once in the run.  Weight gradients are
// summed in registers over the run, then over the block's warps; a second kernel
// adds the blocks' sums in a fixed order, so results repeat bit for bit.
//
// Times (device, in a replayed graph): 4096 rows of 64 + 1 heads of 512 in bf16 83 us
// (6.5 TB/s; a block for 16 heads with loads into registers 111), their gradients 132
// (6.2 TB/s; 310), gradients of 5003 rows of 32 + 8 heads of 128 in fp32, half layout, 58
// (5.3 TB/s, bound by instructions and shared memory; 101), 16 rows of 64 + 1 heads 2.4
// (launch).
#include <math.h>

#include "common.cuh"
#include "fastdiv.cuh"
#include "internal.h"
#include "turn.cuh"

namespace v4 {

namespace {

constexpr int kThreads = 128, kWarps = kThreads / 32;
constexpr int kMaxBlocks = 4864;                 // of the gradient: each leaves a row of sums

struct Part {
  const void* x;
  const void* dy;                                // gradient
  const float* w;                                // null: ones
  void* out;                                     // y or dx
  long long xr, xh, gr, gh, yr, yh;              // strides in elements
  long long items;                               // (row, head) pairs
  int heads, chunk, blocks;                      // chunk: items of a group
  FastDiv by_heads;
};

struct Args {
  Part part[2];
  const int32_t* pos;
  const float* inv_freq;
  float* partial;                                // [blocks of both parts][dim]
  float eps, inv_dim;
  int dim, units, lg;                            // units of eight, log2 of a group's lanes
  int R, begin;                                  // in elements
};

// What a kernel keeps in shared memory for each warp: a ring of raw heads (x, and dy
// for the gradient), the angles of each group's row, and for the forward half layout
// the values that partners exchange.
template <typename T, int U, bool kHalf, bool kGrad>
struct Lay {
  static constexpr int kTensors = kGrad ? 2 : 1;
  static constexpr int kHead = 256 * U * (int)sizeof(T);          // bytes of a warp's heads
  static constexpr int kWant = 256 / (kTensors * U * 8 * (int)sizeof(T));
  // (three stages at most: fp32 gradients of 128-wide heads 57.6 us, 59.6 with four, 57.3 with two, which cost
  // the bf16 gradients of 512-wide heads 138 instead of 131)
  static constexpr int kStages = kWant < 2 ? 2 : kWant > 3 ? 3 : kWant;
  static constexpr int kTable = kStages * kTensors * kHead;       // offset of the angles
  static constexpr int kStrip = kTable + 128 * U * (int)sizeof(float2);
  static constexpr int kWarp = kStrip + (kHalf && !kGrad ? 256 * U * (int)sizeof(float) : 0);
  // resident on an SM, without spills (but 8 bytes in the forward bf16 half layout of U = 2)
  static constexpr int kBlocks = kGrad ? (U == 1 ? 5 : U == 2 ? 4 : 2) : U > 2 ? 3 : 8;
};

__device__ __forceinline__ void copy_16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src)
               : "memory");
}

// Two fp32 operations in one instruction: the kernels are as near to the issue rate as
// to HBM's (the gradient of a head of 512: 309 instructions, 433 without).
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(reinterpret_cast<uint64_t&>(d))
      : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)), "l"(reinterpret_cast<uint64_t&>(c)));
  return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("mul.rn.f32x2 %0, %1, %2;"
      : "=l"(reinterpret_cast<uint64_t&>(d))
      : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)));
  return d;
}

// Eight elements as pairs.
__device__ __forceinline__ void load8(const bf16* p, float2* v) {
  const uint4 u = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
}
__device__ __forceinline__ void load8(const float* p, float2* v) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  v[0] = make_float2(a.x, a.y);
  v[1] = make_float2(a.z, a.w);
  v[2] = make_float2(b.x, b.y);
  v[3] = make_float2(b.z, b.w);
}
template <typename T>
__device__ __forceinline__ void store8(T* p, const float2* v) {
  const float f[8] = {v[0].x, v[0].y, v[1].x, v[1].y, v[2].x, v[2].y, v[3].x, v[3].y};
  v4::store8(p, f);
}

// U: units of a lane.  kHalf: pairs half a rotation apart.
template <typename T, int U, bool kHalf, bool kGrad>
__global__ void __launch_bounds__(kThreads, (Lay<T, U, kHalf, kGrad>::kBlocks)) norm_rope_kernel(const Args p) {
  using L = Lay<T, U, kHalf, kGrad>;
  constexpr int S = L::kStages, kWord = (int)sizeof(T) / 2;       // 16-byte words of a unit
  extern __shared__ __align__(16) uint8_t smem[];
  after_previous();
  const int warp = threadIdx.x >> 5;
  const int G = 1 << p.lg, lane = threadIdx.x & (G - 1), grp = (threadIdx.x & 31) >> p.lg;
  const bool second = blockIdx.x >= (unsigned)p.part[0].blocks;
  const Part& q = p.part[second];
  const int half = p.R >> 1;
  const int v0 = p.begin >> 3, nv = p.R >> 3;    // rotated units
  uint8_t* mine = smem + warp * L::kWarp;
  uint8_t* ring = mine + grp * (G * U * 8 * (int)sizeof(T));
  float2* cs = reinterpret_cast<float2*>(mine + L::kTable) + grp * (G * U * 4);
  float* strip = reinterpret_cast<float*>(mine + L::kStrip) + grp * (G * U * 8);

  float2 w[U][4], dw[kGrad ? U : 1][4];
  int rot[U];                                    // number of a rotated unit, -1: not rotated
  bool here[U];
#pragma unroll
  for (int s = 0; s < U; ++s) {
    const int u = lane + G * s;
    here[s] = u < p.units;
    rot[s] = u >= v0 && u < v0 + nv ? u - v0 : -1;
    if (q.w != nullptr && here[s]) {
      load8(q.w + 8 * u, w[s]);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) w[s][e] = make_float2(1.f, 1.f);
    }
    if (kGrad) {
#pragma unroll
      for (int e = 0; e < 4; ++e) dw[s][e] = make_float2(0.f, 0.f);
    }
  }
  // words of the ring behind a head's last stay zero
  for (int i = p.units * kWord + lane; i < G * U * kWord; i += G)
    for (int k = 0; k < S * L::kTensors; ++k) reinterpret_cast<uint4*>(ring + k * L::kHead)[i] = make_uint4(0, 0, 0, 0);

  // this group's items: consecutive heads, so that a row's angles are formed once
  const long long first =
      ((long long)((blockIdx.x - (second ? p.part[0].blocks : 0)) * kWarps + warp) * (32 >> p.lg) + grp) * q.chunk;
  const int n = (int)max(0ll, min((long long)q.chunk, q.items - first));
  int row = n > 0 ? (int)q.by_heads.div((uint32_t)first) : 0;
  int head = n > 0 ? (int)(first - (long long)row * q.heads) : 0;
  const T* x = reinterpret_cast<const T*>(q.x) + row * q.xr + head * q.xh + 8 / kWord * lane;
  const T* dy = kGrad ? reinterpret_cast<const T*>(q.dy) + row * q.gr + head * q.gh + 8 / kWord * lane : nullptr;
  T* out = reinterpret_cast<T*>(q.out) + row * q.yr + head * q.yh + 8 * lane;
  const long long xw = q.xr - (q.heads - 1) * q.xh, gw = q.gr - (q.heads - 1) * q.gh, yw = q.yr - (q.heads - 1) * q.yh;
  int ihead = head;                              // of the next item that is asked for
  auto ask = [&](int j) {
    if (j < n) {
      uint8_t* to = ring + (j % S) * (L::kTensors * L::kHead);
#pragma unroll
      for (int k = 0; k < U * kWord; ++k) {
        if (lane + G * k < p.units * kWord) {
          uint8_t* word = to + 16 * (lane + G * k);
          copy_16(word, x + 8 / kWord * G * k);
          if (kGrad) copy_16(word + L::kHead, dy + 8 / kWord * G * k);
        }
      }
      const bool wrap = ++ihead == q.heads;
      x += wrap ? xw : q.xh;
      if (kGrad) dy += wrap ? gw : q.gh;
      if (wrap) ihead = 0;
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int j = 0; j < S - 1; ++j) ask(j);
  int formed = -1;                               // row of the angles
  const int most = q.chunk;                      // the same for all lanes
  for (int j = 0; j < most; ++j) {
    ask(j + S - 1);
    asm volatile("cp.async.wait_group %0;" ::"n"(S - 1) : "memory");
    const bool live = j < n;
    if (live && half > 0 && row != formed) {
      formed = row;
      for (int c = lane; c < half; c += G) {
        float co, si;
        turn_cos_sin(p.pos[row], turn_fraction(p.inv_freq[c]), &co, &si);
        // two pairs to a word, words of a unit apart: neighbouring lanes read neighbouring words
        constexpr int kPairs = kHalf ? 8 : 4;
        const int unit = c / kPairs, e = c % kPairs;
        cs[((e >> 1) * (half / kPairs) + unit) * 2 + (e & 1)] = make_float2(co, kGrad ? -si : si);
      }
    }
    __syncwarp();
    const T* at = reinterpret_cast<const T*>(ring + (j % S) * (L::kTensors * L::kHead));
    const T* gat = reinterpret_cast<const T*>(reinterpret_cast<const uint8_t*>(at) + L::kHead);
    float2 v[U][4], g[kGrad ? U : 1][4];
    float2 sq = make_float2(0.f, 0.f), dot = make_float2(0.f, 0.f);
    // one unit of the tensor that is turned: y before its rotation, or dy.  o: its partners'.
    auto turn = [&](int s, float2* a, const float2* o) {
      if (kHalf) {
        const bool low = rot[s] < nv / 2;
        const float4* c = reinterpret_cast<const float4*>(cs) + (low ? rot[s] : rot[s] - nv / 2);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float4 t = c[e * (nv / 2)];
          a[e] = make_float2(fmaf(o[e].x, low ? -t.y : t.y, a[e].x * t.x),
                             fmaf(o[e].y, low ? -t.w : t.w, a[e].y * t.z));
        }
      } else {
        const float4* c = reinterpret_cast<const float4*>(cs) + rot[s];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float4 t = c[e * nv];
          rot_pair(a[2 * e].x, a[2 * e].y, t.x, t.y);
          rot_pair(a[2 * e + 1].x, a[2 * e + 1].y, t.z, t.w);
        }
      }
    };
    // the unit of the partners, kHalf alone
    auto partner = [&](int s) { return rot[s] < nv / 2 ? rot[s] + nv / 2 : rot[s] - nv / 2; };
#pragma unroll
    for (int s = 0; s < U; ++s) {
      const int u = lane + G * s;
      load8(at + 8 * u, v[s]);
      if (kGrad) {
        load8(gat + 8 * u, g[s]);
        if (rot[s] >= 0) {
          float2 o[4];
          if (kHalf) load8(gat + 8 * (v0 + partner(s)), o);
          turn(s, g[s], o);
        }
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        sq = fma2(v[s][e], v[s][e], sq);
        if (kGrad) dot = fma2(mul2(w[s][e], g[s][e]), v[s][e], dot);
      }
    }
    float t_sq = sq.x + sq.y, t_dot = dot.x + dot.y;
    for (int o = G >> 1; o > 0; o >>= 1) {
      t_sq += __shfl_xor_sync(0xffffffffu, t_sq, o);
      if (kGrad) t_dot += __shfl_xor_sync(0xffffffffu, t_dot, o);
    }
    const float r = rsqrtf(fmaf(t_sq, p.inv_dim, p.eps));
    const float2 r2 = make_float2(r, r);
    if (kGrad) {
      // r = 0: the sum of squares passed fp32's range and the head counts as zero, though t_dot may be infinite
      const float m = r == 0.f ? 0.f : -t_dot * p.inv_dim * (r * r) * r;
      const float2 m2 = make_float2(m, m);
      if (live) {                                // r of nothing may be infinite
#pragma unroll
        for (int s = 0; s < U; ++s)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            dw[s][e] = fma2(g[s][e], mul2(v[s][e], r2), dw[s][e]);
            v[s][e] = fma2(mul2(w[s][e], g[s][e]), r2, mul2(v[s][e], m2));
          }
      }
    } else {
#pragma unroll
      for (int s = 0; s < U; ++s)
#pragma unroll
        for (int e = 0; e < 4; ++e) v[s][e] = mul2(mul2(v[s][e], r2), w[s][e]);
      if (kHalf) {
#pragma unroll
        for (int s = 0; s < U; ++s)
          if (rot[s] >= 0) store8(strip + 8 * rot[s], v[s]);
        __syncwarp();
      }
#pragma unroll
      for (int s = 0; s < U; ++s) {
        if (rot[s] < 0) continue;
        float2 o[4];
        if (kHalf) load8(strip + 8 * partner(s), o);
        turn(s, v[s], o);
      }
    }
    if (live) {
#pragma unroll
      for (int s = 0; s < U; ++s)
        if (here[s]) store8(out + 8 * G * s, v[s]);
      const bool wrap = ++head == q.heads;
      out += wrap ? yw : q.yh;
      if (wrap) {
        head = 0;
        ++row;
      }
    }
    __syncwarp();                                // the slot, the angles and the strip are read
  }

  if (kGrad) {
    // a lane's sums over the groups of its warp, then over the warps
#pragma unroll
    for (int s = 0; s < U; ++s)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        for (int o = G; o < 32; o <<= 1) {
          dw[s][e].x += __shfl_xor_sync(0xffffffffu, dw[s][e].x, o);
          dw[s][e].y += __shfl_xor_sync(0xffffffffu, dw[s][e].y, o);
        }
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncthreads();                             // the rings are free
    float* sums = reinterpret_cast<float*>(smem);
    const int width = G * 8 * U;
    if (grp == 0) {
#pragma unroll
      for (int s = 0; s < U; ++s) store8(sums + warp * width + 8 * (lane + G * s), dw[s]);
    }
    __syncthreads();
    float* to = p.partial + (size_t)blockIdx.x * p.dim;
    for (int c = threadIdx.x; c < p.dim; c += kThreads) {
      float t = 0.f;
#pragma unroll
      for (int i = 0; i < kWarps; ++i) t += sums[i * width + c];
      to[c] = t;
    }
  }
}

// dw[c] = sum of the blocks' sums.  A cluster takes 32 columns, its blocks every eighth
// row of 1024-row steps, and adds up through distributed shared memory: always in the
// same order.
constexpr int kSumThreads = 1024, kSumCluster = 8, kSumRows = kSumThreads / 8;

struct SumArgs {
  const float* partial;
  float* out[2];
  int first[2], blocks[2];
  int dim;
};

__global__ void __launch_bounds__(kSumThreads) norm_weight_kernel(const SumArgs p) {
  __shared__ float4 s_t[kSumThreads / 32][8];
  __shared__ float s_sum[32];
  after_previous();
  const int part = blockIdx.z, rank = blockIdx.x;         // the cluster runs along x
  if (p.out[part] == nullptr) return;                     // the whole cluster
  const int c4 = threadIdx.x & 7, r0 = rank * kSumRows + (threadIdx.x >> 3), warp = threadIdx.x >> 5;
  const int col = blockIdx.y * 32 + 4 * c4;
  float4 t = make_float4(0.f, 0.f, 0.f, 0.f);
  if (col < p.dim) {
    const float* from = p.partial + (size_t)p.first[part] * p.dim + col;
#pragma unroll 4
    for (int b = r0; b < p.blocks[part]; b += kSumRows * kSumCluster) {
      const float4 v = *reinterpret_cast<const float4*>(from + (size_t)b * p.dim);
      t.x += v.x;
      t.y += v.y;
      t.z += v.z;
      t.w += v.w;
    }
  }
#pragma unroll
  for (int o = 8; o < 32; o <<= 1) {
    t.x += __shfl_xor_sync(0xffffffffu, t.x, o);
    t.y += __shfl_xor_sync(0xffffffffu, t.y, o);
    t.z += __shfl_xor_sync(0xffffffffu, t.z, o);
    t.w += __shfl_xor_sync(0xffffffffu, t.w, o);
  }
  if ((threadIdx.x & 31) < 8) s_t[warp][c4] = t;
  __syncthreads();
  // 32 columns x 32 warps' sums, one column a warp
  float v = reinterpret_cast<const float*>(s_t[threadIdx.x & 31])[warp];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if ((threadIdx.x & 31) == 0) s_sum[warp] = v;
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
  if (rank == 0 && threadIdx.x < 32 && blockIdx.y * 32 + threadIdx.x < p.dim) {
    float sum = 0.f;
    for (int k = 0; k < kSumCluster; ++k) {
      uint32_t at;
      float other;
      asm("mapa.shared::cluster.u32 %0, %1, %2;"
          : "=r"(at)
          : "r"((uint32_t)__cvta_generic_to_shared(&s_sum[threadIdx.x])), "r"(k));
      asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(other) : "r"(at) : "memory");
      sum += other;
    }
    p.out[part][blockIdx.y * 32 + threadIdx.x] = sum;
  }
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

struct Kernel {
  void (*run)(const Args);
  int smem, blocks;                              // of a block, resident on an SM
};

template <typename T, int U, bool kHalf, bool kGrad>
cudaError_t kernel_of(Kernel* k) {
  using L = Lay<T, U, kHalf, kGrad>;
  static_assert(L::kWarp >= 256 * U * (int)sizeof(float) || !kGrad, "the weight sums fit in the rings");
  k->run = norm_rope_kernel<T, U, kHalf, kGrad>;
  k->smem = kWarps * L::kWarp;
  k->blocks = L::kBlocks;
  while (k->blocks > 1 && k->blocks * (k->smem + 1024) > 227 * 1024) --k->blocks;
  static OncePerDevice once;
  return once.run([] {
    return cudaFuncSetAttribute(norm_rope_kernel<T, U, kHalf, kGrad>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                kWarps * Lay<T, U, kHalf, kGrad>::kWarp);
  });
}

template <typename T, bool kGrad>
cudaError_t kernel_of(int units_a_lane, bool half, Kernel* k) {
  if (units_a_lane == 1) return half ? kernel_of<T, 1, true, kGrad>(k) : kernel_of<T, 1, false, kGrad>(k);
  if (units_a_lane == 2) return half ? kernel_of<T, 2, true, kGrad>(k) : kernel_of<T, 2, false, kGrad>(k);
  return half ? kernel_of<T, 4, true, kGrad>(k) : kernel_of<T, 4, false, kGrad>(k);
}

}  // namespace

size_t norm_rope_workspace(int dim) { return (size_t)(kMaxBlocks + 2) * dim * sizeof(float); }

cudaError_t launch_norm_rope(const NormCall& c, cudaStream_t st) {
  const bool grad = c.grad;
  Args p;
  p.pos = c.pos;
  p.inv_freq = c.inv_freq;
  p.partial = (float*)c.workspace;
  p.eps = c.eps;
  p.inv_dim = 1.f / (float)c.dim;
  p.dim = c.dim;
  p.units = c.dim / 8;
  p.R = c.rope_dim;
  p.begin = c.rope_begin;
  // lanes of a head: the next power of two of its units, a lane holding up to four
  const int U = p.units <= 32 ? 1 : p.units <= 64 ? 2 : 4;
  p.lg = 0;
  while ((U << p.lg) < p.units) ++p.lg;
  const int groups = kThreads >> p.lg;
  Kernel k;
  cudaError_t e;
  if (c.dtype == V4_BF16) e = grad ? kernel_of<bf16, true>(U, c.half, &k) : kernel_of<bf16, false>(U, c.half, &k);
  else e = grad ? kernel_of<float, true>(U, c.half, &k) : kernel_of<float, false>(U, c.half, &k);
  if (e != cudaSuccess) return e;
  // A group takes a run of about `most` heads, such that the blocks fill whole waves, and
  // a shorter one while SMs would be left without blocks.  Runs as long as one wave allows
  // were slower, since SMs do not progress alike (4096 x 64 heads of 512: 120 against 84
  // us), and so were shorter ones in the gradient, whose blocks each leave sums (run 4: 220
  // us, 8 and 16: 131, 32: 141).
  const long long wave = 152ll * k.blocks * groups, most = grad ? 16 : 8;
  long long all = 0;
  for (int i = 0; i < 2; ++i) all += c.rows * (c.part[i].x ? c.part[i].heads : 0);
  long long waves = (all + most * wave / 2) / (most * wave);
  if (waves < 1) waves = 1;
  long long run = (all + waves * wave - 1) / (waves * wave);
  if (grad && all > run * groups * (kMaxBlocks - 2)) run = all / ((long long)groups * (kMaxBlocks - 2)) + 1;
  if (run < 1) run = 1;
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
    q.items = c.rows * q.heads;
    q.by_heads.set((uint32_t)(q.heads > 0 ? q.heads : 1));
    q.chunk = (int)run;
    q.blocks = (int)((q.items + run * groups - 1) / (run * groups));
  }
  const int blocks = p.part[0].blocks + p.part[1].blocks;
  if (blocks > 0) {                              // else weight gradients of no rows: zeros
    e = launch_overlapped(k.run, dim3((unsigned)blocks), dim3(kThreads), (size_t)k.smem, st, p);
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
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(kSumCluster, (unsigned)((c.dim + 31) / 32), 2);
  cfg.blockDim = dim3(kSumThreads);
  cfg.stream = st;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = kSumCluster;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  e = cudaLaunchKernelEx(&cfg, norm_weight_kernel, (const SumArgs)s);
  if (e == cudaSuccess) note_launch();
  return e;
}

}  // namespace v4
