// Write into and read from the 4-bit cache (v4_cache_append_q4,
// v4_cache_read_q4).
//
//   scale = the 4-bit significand nearest to max|x| / 7 over 16 values (ties to
//   even), code = 8 + clamp(round_to_even(x / scale), -8, 7)
//
// Memory bound: a thread takes one group of 16 values, so its maximum needs no
// exchange, and a row's threads write neighbouring words.  16384 rows of 512 in bf16 are
// written and read back in 11.5 us (3.7 TB/s, of which 3 us are the two launches; 15.6
// with a division for each value), 64 rows in 2.8 (launches).
#include <math.h>

#include "common.cuh"
#include "fastdiv.cuh"
#include "internal.h"
#include "q4.cuh"

namespace v4 {

namespace {

constexpr int kThreads = 128;

struct Q4Args {
  const void* x;               // write: rows in; read: rows out
  void* out;
  uint8_t* cache;
  const int32_t* slot;
  long long n_slots, stride, groups;     // stride of the dense rows, groups of all rows
  int* status;
  int D, row_bytes;
  FastDiv by_groups;
};

// The byte of the scale nearest to amax / 7.  An IEEE quotient lies on the same side
// of every tie as the exact one (ties have at most five significant bits).
__device__ __forceinline__ uint32_t scale_byte(float amax) {
  const uint32_t f = __float_as_uint(__fdiv_rn(amax, 7.f));
  const int b = (int)((f + 0x7FFFFu + ((f >> 20) & 1u)) >> 20) - (107 << 3);
  return (uint32_t)min(max(b, 0), 255);
}

// Two words of codes of sixteen values.  x / scale is the correctly rounded quotient by
// Markstein's theorem: with inv the rounded reciprocal, q = x inv needs one step of its
// exact remainder.  Values outside [-8, 7] scales are cut before, exactly.  Adding 1.5
// 2^23 + 8 rounds to an integer, ties to even, and leaves the code in the low bits: the
// words are sums of those floats' bits, less what the constant adds.
__device__ __forceinline__ uint2 pack_codes(const float* v, float scale) {
  const float inv = __frcp_rn(scale), lo = -8.f * scale, hi = 7.f * scale;
  uint32_t w[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    w[k] = 0u - 0x4B400000u * 0x11111111u;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float x = fminf(fmaxf(v[8 * k + e], lo), hi);
      const float q0 = x * inv;
      const float q = fmaf(fmaf(-q0, scale, x), inv, q0);
      const int nib = (e & 1) * 4 + (e >> 1);
      w[k] += __float_as_uint(q + 12582920.f) << (4 * nib);
    }
  }
  return make_uint2(w[0], w[1]);
}

template <typename T, int K>
__global__ void __launch_bounds__(kThreads) q4_append_kernel(const Q4Args p) {
  after_previous();
  const int per = p.D / kQ4Group;
  const long long first = (long long)blockIdx.x * (kThreads * K) + threadIdx.x;
  Raw<T> a[K][2];
  int at[K], g[K];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const long long i = first + k * kThreads;
    at[k] = -1;
    if (i >= p.groups) continue;
    const int row = (int)p.by_groups.div((uint32_t)i);
    g[k] = (int)i - row * per;
    const T* x = reinterpret_cast<const T*>(p.x) + row * p.stride + kQ4Group * g[k];
    a[k][0].load(x);
    a[k][1].load(x + 8);
    const int s = p.slot[row];
    if (s < 0 || s >= p.n_slots) {
      if (s != -1) set_status(p.status, kStatusBadIndex);
      continue;
    }
    at[k] = s;
  }
#pragma unroll
  for (int k = 0; k < K; ++k) {
    if (at[k] < 0) continue;
    float v[16];
    a[k][0].floats(v);
    a[k][1].floats(v + 8);
    uint32_t top = 0;                              // bits of the largest magnitude: NaN lies above infinity
#pragma unroll
    for (int e = 0; e < 16; ++e) top = max(top, __float_as_uint(v[e]) & 0x7FFFFFFFu);
    if (top > 0x7F800000u) {                       // NaN counts as zero
      top = 0;
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        if (v[e] != v[e]) v[e] = 0.f;
        top = max(top, __float_as_uint(v[e]) & 0x7FFFFFFFu);
      }
    }
    const uint32_t b = scale_byte(fminf(__uint_as_float(top), 1e30f));
    uint8_t* row = p.cache + (size_t)at[k] * p.row_bytes;
    *reinterpret_cast<uint2*>(row + 8 * g[k]) = pack_codes(v, q4_scale(b));
    row[p.D / 2 + g[k]] = (uint8_t)b;
    if (g[k] == 0)
      for (int i = p.D / 2 + per; i < p.row_bytes; ++i) row[i] = 0;
  }
}

// Eight values, exact in bf16.
__device__ __forceinline__ void store_values(bf16* to, uint4 v) { *reinterpret_cast<uint4*>(to) = v; }
__device__ __forceinline__ void store_values(float* to, uint4 v) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  float f[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
  store8(to, f);
}

template <typename T, int K>
__global__ void __launch_bounds__(kThreads) q4_read_kernel(const Q4Args p) {
  after_previous();
  const int per = p.D / kQ4Group;
  const long long first = (long long)blockIdx.x * (kThreads * K) + threadIdx.x;
  uint2 w[K];
  uint32_t b[K];
  T* to[K];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const long long i = first + k * kThreads;
    to[k] = nullptr;
    if (i >= p.groups) continue;
    const int row = (int)p.by_groups.div((uint32_t)i);
    const int g = (int)i - row * per;
    to[k] = reinterpret_cast<T*>(p.out) + row * p.stride + kQ4Group * g;
    const int s = p.slot[row];
    if (s < 0 || s >= p.n_slots) {
      if (s != -1) set_status(p.status, kStatusBadIndex);
      w[k] = make_uint2(0x88888888u, 0x88888888u);       // zeros
      b[k] = 0;
      continue;
    }
    const uint8_t* from = p.cache + (size_t)s * p.row_bytes;
    w[k] = *reinterpret_cast<const uint2*>(from + 8 * g);
    b[k] = from[p.D / 2 + g];
  }
#pragma unroll
  for (int k = 0; k < K; ++k) {
    if (to[k] == nullptr) continue;
    store_values(to[k], q4_word_bf16(w[k].x, b[k]));
    store_values(to[k] + 8, q4_word_bf16(w[k].y, b[k]));
  }
}

}  // namespace

cudaError_t launch_q4_rows(const Q4Call& c, int* status, cudaStream_t st) {
  Q4Args p;
  p.x = c.x;
  p.out = c.out;
  p.cache = (uint8_t*)c.cache;
  p.slot = c.slot;
  p.n_slots = c.n_slots;
  p.stride = c.row_stride;
  p.groups = c.rows * (c.dim / kQ4Group);
  p.status = status;
  p.D = c.dim;
  p.row_bytes = q4_row_bytes(c.dim);
  p.by_groups.set((uint32_t)(c.dim / kQ4Group));
  const bool b16 = c.dtype == V4_BF16;
  // two groups a thread once every SM has eight blocks
  const bool two = p.groups >= (long long)152 * 8 * kThreads * 2;
  const int per = kThreads * (two ? 2 : 1);
  const dim3 grid((unsigned)((p.groups + per - 1) / per));
  auto kern = c.out == nullptr ? (b16 ? (two ? q4_append_kernel<bf16, 2> : q4_append_kernel<bf16, 1>)
                                      : (two ? q4_append_kernel<float, 2> : q4_append_kernel<float, 1>))
                               : (b16 ? (two ? q4_read_kernel<bf16, 2> : q4_read_kernel<bf16, 1>)
                                      : (two ? q4_read_kernel<float, 2> : q4_read_kernel<float, 1>));
  const cudaError_t e = launch_overlapped(kern, grid, dim3(kThreads), 0, st, p);
  if (e == cudaSuccess) note_launch();
  return e;
}

}  // namespace v4
