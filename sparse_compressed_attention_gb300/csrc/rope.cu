// Rotary positions at given positions, and the paged cache write that rotates
// its rows (v4_rope, v4_cache_append).
//
// y = mscale * R(sign * pos * f) x on the rotated dims, a copy elsewhere; the
// gradient is the same map with the sign turned.  Memory bound: every element
// is read and written once.  A block takes a tile of rows x heads, forms the
// tile's (row, pair) angles once in shared memory (they are shared by the
// heads), and streams the tile in 8-element units, all of a thread's loads in
// flight before the angles are formed.
#include <math.h>

#include "common.cuh"
#include "internal.h"
#include "turn.cuh"

namespace v4 {

namespace {

constexpr int kRopeThreads = 256;
constexpr int kUnitsPerThread = 4;
constexpr int kMaxAngles = 1024;                 // (row, pair) angles of a tile

// Division by a run-time constant below 2^31: n / d for n < 2^31.
struct FastDiv {
  uint32_t mul, sh, d;
  void set(uint32_t v) {
    d = v;
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
  int heads, R, begin, half, inverse;
  int rot_units, units;        // units of a (row, head): rotated ones first, then copied ones
  int rb, hb;                  // rows and heads of a tile
  FastDiv by_unit, by_head;
};

template <typename T>
struct Unit {
  float a[8], b[8];            // interleaved and copied units use a alone
};

// `kHalf`: pairs half a rotation apart.
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
  const T* x = reinterpret_cast<const T*>(p.x);
  T* out = reinterpret_cast<T*>(p.out);

  auto place = [&](int i, int& r, int& h, int& u) {
    const int q = (int)p.by_unit.div((uint32_t)i);
    u = i - q * p.units;
    r = (int)p.by_head.div((uint32_t)q);
    h = q - r * p.hb;
  };
  // first dim of a unit: rotated units from `begin`, the others around the
  // rotated part
  auto dim_of = [&](int u) {
    if (u < p.rot_units) return p.begin + 8 * u;
    const int c = 8 * (u - p.rot_units);
    return c < p.begin ? c : c + p.R;
  };
  bool angles = p.pos == nullptr;                 // formed after the first loads are in flight
  for (int i0 = threadIdx.x; i0 - (int)threadIdx.x < n; i0 += kRopeThreads * kUnitsPerThread) {
    Unit<T> v[kUnitsPerThread];
#pragma unroll
    for (int k = 0; k < kUnitsPerThread; ++k) {
      const int i = i0 + k * kRopeThreads;
      if (i < n) {
        int r, h, u;
        place(i, r, h, u);
        if (h < nh) {
          const T* src = x + (row0 + r) * p.xr + (long long)(head0 + h) * p.xh + dim_of(u);
          load8(src, v[k].a);
          if (kHalf && u < p.rot_units) load8(src + half, v[k].b);
        }
      }
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
    for (int k = 0; k < kUnitsPerThread; ++k) {
      const int i = i0 + k * kRopeThreads;
      if (i >= n) continue;
      int r, h, u;
      place(i, r, h, u);
      if (h >= nh) continue;
      long long row = row0 + r;
      if (p.slot != nullptr) {
        const int s = p.slot[row];
        if (s < 0 || s >= p.n_slots) {
          if (s != -1) set_status(p.status, kStatusBadIndex);
          continue;
        }
        row = s;
      }
      T* dst = out + row * p.yr + (long long)(head0 + h) * p.yh + dim_of(u);
      if (u < p.rot_units) {
        if (kHalf) {
          const float2* cs = s_cs + r * half + 8 * u;
#pragma unroll
          for (int e = 0; e < 8; ++e) rot_pair(v[k].a[e], v[k].b[e], cs[e].x, cs[e].y);
          store8(dst + half, v[k].b);
        } else {
          const float2* cs = s_cs + r * half + 4 * u;
#pragma unroll
          for (int e = 0; e < 4; ++e) rot_pair(v[k].a[2 * e], v[k].a[2 * e + 1], cs[e].x, cs[e].y);
        }
      }
      store8(dst, v[k].a);
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
  p.half = c.layout == V4_ROPE_HALF;
  p.inverse = c.inverse;
  p.rot_units = p.R / (p.half ? 16 : 8);
  const bool in_place = c.x == c.out && c.slot == nullptr;
  p.units = p.rot_units + (in_place ? 0 : (c.dim - p.R) / 8);
  if (p.units == 0) return cudaSuccess;          // in place with nothing rotated
  // Tile: about kUnitsPerThread units a thread, heads first (they share the
  // row's angles), then rows as far as the angle table reaches.
  const int want = kRopeThreads * kUnitsPerThread;
  const int per_row = c.heads * p.units;
  p.hb = per_row <= want ? c.heads : (want / p.units > 1 ? want / p.units : 1);
  if (p.hb > c.heads) p.hb = c.heads;
  long long rb = p.hb == c.heads ? want / per_row : 1;
  const int half = p.R / 2;
  if (half > 0 && rb > kMaxAngles / half) rb = kMaxAngles / half;
  if (rb < 1) rb = 1;
  if (rb > c.rows) rb = c.rows;
  p.rb = (int)rb;
  p.by_unit.set((uint32_t)p.units);
  p.by_head.set((uint32_t)p.hb);
  const long long gx = (c.rows + rb - 1) / rb;
  if (gx > 0x7FFFFFFFll) return cudaErrorInvalidValue;
  const dim3 grid((unsigned)gx, (unsigned)((c.heads + p.hb - 1) / p.hb));
  if (c.dtype == V4_BF16) {
    if (p.half) rope_kernel<bf16, true><<<grid, kRopeThreads, 0, st>>>(p);
    else rope_kernel<bf16, false><<<grid, kRopeThreads, 0, st>>>(p);
  } else {
    if (p.half) rope_kernel<float, true><<<grid, kRopeThreads, 0, st>>>(p);
    else rope_kernel<float, false><<<grid, kRopeThreads, 0, st>>>(p);
  }
  note_launch();
  return cudaGetLastError();
}

}  // namespace v4
