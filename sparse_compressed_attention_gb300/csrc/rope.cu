// Rotary positions at given positions, and the paged cache write that rotates
// its rows (v4_rope, v4_cache_append).
//
// y = mscale * R(sign * pos * f) x on the rotated dims, a copy elsewhere; the
// gradient is the same map with the sign turned.  Memory bound: every element
// is read and written once.  A block takes a tile of rows x heads and streams
// it in units of eight elements: a thread's loads are all in flight, as raw
// bits (most units of a partly rotated head are copies and are never
// converted), while the block forms the tile's (row, pair) angles once in
// shared memory for all heads.
#include <math.h>

#include "common.cuh"
#include "internal.h"
#include "turn.cuh"

namespace v4 {

namespace {

// Small blocks: a block's first loads wait for nothing, its angles do, and the
// more blocks an SM holds the less of it stands still (256 threads against 128:
// 10.0 and 9.0 us for 16384 cache rows of 512, 82 and 83 us for 4096 x 64 heads).
constexpr int kRopeThreads = 128;
// Units that a thread has in flight.  A unit of the half layout in fp32 is 64
// bytes; four of them take 109 registers (5003 x 64 heads of 128: 56 us with
// four, 53 with two), while a bf16 unit is 16 (4096 x 64 heads of 512: 83 us with
// four, 90 with two).
template <typename T, bool kHalf>
constexpr int rope_units() {
  return sizeof(T) == 4 && kHalf ? 2 : 4;
}
constexpr int kMaxAngles = 1024;                 // (row, pair) angles of a tile

// Division by a run-time constant below 2^31: n / d for n < 2^31.
struct FastDiv {
  uint32_t mul, sh;
  void set(uint32_t v) {
    sh = 0;
    while ((1u << sh) < v) ++sh;                 // 2^sh >= v
    mul = (uint32_t)(((uint64_t)1 << 32) * (((uint64_t)1 << sh) - v) / v + 1);
  }
  __device__ __forceinline__ uint32_t div(uint32_t n) const {
    return (uint32_t)(((uint64_t)__umulhi(mul, n) + n) >> sh);
  }
};

struct RopeArgs {
  const void* x;
  void* out;
  const int32_t* pos;          // null: no rotation (cache write of finished rows)
  const float* inv_freq;
  const int32_t* slot;         // null: row t goes to row t
  long long n_slots, rows;
  long long xr, xh, yr, yh;    // strides in elements
  int* status;
  float mscale;
  int heads, R, begin, inverse;
  int rot_units, units;        // units of a (row, head): rotated ones first, then copied ones
  int rb, hb;                  // rows and heads of a tile
  FastDiv by_unit, by_head;
};

// Eight elements as raw 16-byte words: one for bf16, two for float.
template <typename T>
struct Raw {
  uint4 w[sizeof(T) / 2];
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < (int)(sizeof(T) / 2); ++i) w[i] = reinterpret_cast<const uint4*>(p)[i];
  }
  __device__ __forceinline__ void store(T* p) const {
#pragma unroll
    for (int i = 0; i < (int)(sizeof(T) / 2); ++i) reinterpret_cast<uint4*>(p)[i] = w[i];
  }
  __device__ __forceinline__ void floats(float* v) const { load8(reinterpret_cast<const T*>(w), v); }
};

// kHalf: pairs half a rotation apart.
template <typename T, bool kHalf>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const RopeArgs p) {
  __shared__ float2 s_cs[kMaxAngles];
  __shared__ uint64_t s_f[512];
  const long long row0 = (long long)blockIdx.x * p.rb;
  const int head0 = blockIdx.y * p.hb;
  const int nr = (int)min((long long)p.rb, p.rows - row0);
  const int nh = min(p.hb, p.heads - head0);
  const int n = nr * p.hb * p.units;
  const int half = p.R >> 1;
  constexpr int kUnits = rope_units<T, kHalf>();
  const T* x = reinterpret_cast<const T*>(p.x) + row0 * p.xr + (long long)head0 * p.xh;
  T* out = reinterpret_cast<T*>(p.out) + (long long)head0 * p.yh;

  bool angles = p.pos == nullptr;                 // formed once the first loads are in flight
  for (int base = 0; base < n; base += kRopeThreads * kUnits) {
    Raw<T> a[kUnits], b[kHalf ? kUnits : 1];
    int where[kUnits];                            // first angle of a rotated unit, -1: a copied one
    T* dst[kUnits];                               // null: nothing to do
#pragma unroll
    for (int k = 0; k < kUnits; ++k) {
      const int i = base + k * kRopeThreads + (int)threadIdx.x;
      dst[k] = nullptr;
      if (i >= n) continue;
      const int q = (int)p.by_unit.div((uint32_t)i);
      const int u = i - q * p.units;
      const int r = (int)p.by_head.div((uint32_t)q);
      const int h = q - r * p.hb;
      if (h >= nh) continue;
      // rotated units from `begin`, the others around the rotated part
      const bool rot = u < p.rot_units;
      const int c = 8 * (u - p.rot_units);
      const int dim = rot ? p.begin + 8 * u : (c < p.begin ? c : c + p.R);
      where[k] = rot ? r * half + (kHalf ? 8 : 4) * u : -1;
      const T* src = x + r * p.xr + (long long)h * p.xh + dim;
      a[k].load(src);
      if (kHalf && rot) b[kHalf ? k : 0].load(src + half);
      long long row = row0 + r;
      if (p.slot != nullptr) {
        const int s = p.slot[row];
        if (s < 0 || s >= p.n_slots) {
          if (s != -1) set_status(p.status, kStatusBadIndex);
          continue;
        }
        row = s;
      }
      dst[k] = out + row * p.yr + (long long)h * p.yh + dim;
    }
    if (!angles) {
      angles = true;
      for (int j = threadIdx.x; j < half; j += kRopeThreads) s_f[j] = turn_fraction(p.inv_freq[j]);
      __syncthreads();
      for (int j = threadIdx.x; j < nr * half; j += kRopeThreads) {
        const int r = j / half, c = j - r * half;
        float cs, sn;
        turn_cos_sin(p.pos[row0 + r], s_f[c], &cs, &sn);
        s_cs[j] = make_float2(cs * p.mscale, (p.inverse ? -sn : sn) * p.mscale);
      }
      __syncthreads();
    }
#pragma unroll
    for (int k = 0; k < kUnits; ++k) {
      if (dst[k] == nullptr) continue;
      if (where[k] >= 0) {
        const float2* cs = s_cs + where[k];
        float v[8];
        a[k].floats(v);
        if (kHalf) {
          float w[8];
          b[kHalf ? k : 0].floats(w);
#pragma unroll
          for (int e = 0; e < 8; ++e) rot_pair(v[e], w[e], cs[e].x, cs[e].y);
          store8(dst[k] + half, w);
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) rot_pair(v[2 * e], v[2 * e + 1], cs[e].x, cs[e].y);
        }
        store8(dst[k], v);
      } else {
        a[k].store(dst[k]);
      }
    }
  }
}

}  // namespace

cudaError_t launch_rope(const RopeCall& c, int* status, cudaStream_t st) {
  if (c.rows == 0) return cudaSuccess;
  RopeArgs p;
  p.x = c.x;
  p.out = c.out;
  p.pos = c.pos;
  p.inv_freq = c.inv_freq;
  p.slot = c.slot;
  p.n_slots = c.n_slots;
  p.rows = c.rows;
  p.xr = c.x_row_stride;
  p.xh = c.x_head_stride;
  p.yr = c.out_row_stride;
  p.yh = c.out_head_stride;
  p.status = status;
  p.mscale = c.mscale;
  p.heads = c.heads;
  p.R = c.pos != nullptr ? c.rope_dim : 0;
  p.begin = c.rope_begin;
  p.inverse = c.inverse;
  const bool by_half = c.layout == V4_ROPE_HALF;
  p.rot_units = p.R / (by_half ? 16 : 8);
  const bool in_place = c.x == c.out && c.slot == nullptr;
  p.units = p.rot_units + (in_place ? 0 : (c.dim - p.R) / 8);
  if (p.units == 0) return cudaSuccess;          // in place with nothing rotated
  // Tile: up to rope_units() units a thread, heads first (they share the
  // row's angles), then rows as far as the angle table reaches; fewer while
  // the tiles would not give every SM one.
  const long long all = c.rows * c.heads * p.units;
  int want = kRopeThreads * (c.dtype == V4_F32 && by_half ? rope_units<float, true>() : rope_units<bf16, false>());
  while (want > kRopeThreads && all / want < 304) want /= 2;
  const int per_row = c.heads * p.units;
  p.hb = per_row <= want ? c.heads : (want / p.units > 1 ? want / p.units : 1);
  long long rb = p.hb == c.heads ? want / per_row : 1;
  const int half = p.R / 2;
  if (half > 0 && rb > kMaxAngles / half) rb = kMaxAngles / half;
  if (rb < 1) rb = 1;
  if (rb > c.rows) rb = c.rows;
  p.rb = (int)rb;
  p.by_unit.set((uint32_t)p.units);
  p.by_head.set((uint32_t)p.hb);
  const long long gx = (c.rows + rb - 1) / rb;
  const dim3 grid((unsigned)gx, (unsigned)((c.heads + p.hb - 1) / p.hb));
  if (c.dtype == V4_BF16) {
    if (by_half) rope_kernel<bf16, true><<<grid, kRopeThreads, 0, st>>>(p);
    else rope_kernel<bf16, false><<<grid, kRopeThreads, 0, st>>>(p);
  } else {
    if (by_half) rope_kernel<float, true><<<grid, kRopeThreads, 0, st>>>(p);
    else rope_kernel<float, false><<<grid, kRopeThreads, 0, st>>>(p);
  }
  note_launch();
  return cudaGetLastError();
}

}  // namespace v4
