// Rotary positions at given positions, and the paged cache write that rotates
// its rows (v4_rope, v4_cache_append).
//
// y = mscale * R(sign * pos * f) x on the rotated dims, a copy elsewhere; the
// gradient is the same map with the sign turned.  Memory bound: every element
// is read and written once.  A block takes a tile of rows x heads and streams
// it in units of eight elements: a thread's loads are all in flight, as raw
// bits (most units of a partly rotated head are copies and are never
// converted), while the block forms the tile's (row, pair) angles once in
// shared memory for all heads.  4096 rows of 64 heads of 512 in bf16 take 81.6 us
// (6.6 TB/s), the gradient of 5003 rows of 64 heads of 128 in fp32 52.2 us
// (6.3 TB/s), 16384 cache rows 8.4 us (4.0 TB/s, nearly 2 us of it the launch),
// one decode step of 16 rows 1.8 us on the device (7 from one Python call to the next).
#include <math.h>

#include "common.cuh"
#include "fastdiv.cuh"
#include "internal.h"
#include "turn.cuh"

namespace v4 {

namespace {

// Small blocks: a block's first loads wait for nothing, its angles do, and the
// more blocks an SM holds the less of it stands still (256 threads against 128:
// 9.7 and 8.7 us for 16384 cache rows of 512, 86.6 and 82.7 us for 4096 x 64 heads
// of 512).  Bounds on registers for more of them spill: 93 us.
constexpr int kRopeThreads = 128;
// Units that a thread has in flight.  A unit of the half layout in fp32 is 64
// bytes (5003 x 64 heads of 128: 56 us with four, 53 with two), a bf16 unit 16
// (4096 x 64 heads of 512: 83 us with four, 90 with two, 85 with eight).
template <typename T, bool kHalf>
constexpr int rope_units() {
  return sizeof(T) == 4 && kHalf ? 2 : 4;
}
constexpr int kMaxAngles = 1024;                 // (row, pair) angles of a tile

struct RopeArgs {
  const void* x;
  void* out;
  const int32_t* pos;          // null: no rotation (cache write of finished rows)
  const float* inv_freq;
  const int32_t* slot;         // null: row t goes to row t
  long long n_slots, rows;
  long long xr, xh, yr, yh;    // strides in elements
  int txr, txh, tyr, tyh;      // the same within a tile, where offsets stay below 2^31
  int* status;
  float mscale;
  int heads, R, begin, inverse;
  int rot_units, units;        // units of a (row, head): rotated ones first, then copied ones
  int rb, hb;                  // rows and heads of a tile
  FastDiv by_unit, by_head, by_half;
};

// kHalf: pairs half a rotation apart.
template <typename T, bool kHalf>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const RopeArgs p) {
  __shared__ float2 s_cs[kMaxAngles];
  after_previous();
  const long long row0 = (long long)blockIdx.x * p.rb;
  const int head0 = blockIdx.y * p.hb;
  const int nr = (int)min((long long)p.rb, p.rows - row0);
  const int nh = min(p.hb, p.heads - head0);
  const int n = nr * p.hb * p.units;
  const int half = p.R >> 1;
  constexpr int kUnits = rope_units<T, kHalf>();
  const T* x = reinterpret_cast<const T*>(p.x) + row0 * p.xr + (long long)head0 * p.xh;
  T* out = reinterpret_cast<T*>(p.out) + (p.slot == nullptr ? row0 * p.yr : 0) + (long long)head0 * p.yh;

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
      const T* src = x + (r * p.txr + h * p.txh + dim);
      a[k].load(src);
      if (kHalf && rot) b[kHalf ? k : 0].load(src + half);
      if (p.slot != nullptr) {                     // one head
        const int s = p.slot[row0 + r];
        if (s < 0 || s >= p.n_slots) {
          if (s != -1) set_status(p.status, kStatusBadIndex);
          continue;
        }
        dst[k] = out + (long long)s * p.tyr + dim;
      } else {
        dst[k] = out + (r * p.tyr + h * p.tyh + dim);
      }
    }
    if (!angles) {
      angles = true;
      for (int j = threadIdx.x; j < nr * half; j += kRopeThreads) {
        const int r = (int)p.by_half.div((uint32_t)j), c = j - r * half;
        float cs, sn;
        turn_cos_sin(p.pos[row0 + r], turn_fraction(p.inv_freq[c]), &cs, &sn);
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
  while (want > kRopeThreads && all / want < 304) want /= 2;      // two for each of 152 SMs
  const int per_row = c.heads * p.units;
  p.hb = per_row <= want ? c.heads : (want / p.units > 1 ? want / p.units : 1);
  long long rb = p.hb == c.heads ? want / per_row : 1;
  const int half = p.R / 2;
  if (half > 0 && rb > kMaxAngles / half) rb = kMaxAngles / half;
  if (rb < 1) rb = 1;
  if (rb > c.rows) rb = c.rows;
  // offsets within a tile are 32 bits wide: strides that reach further get
  // tiles of one row, or of one row and head (whose strides are never used)
  const long long far = (long long)1 << 31;
  auto reach = [&](long long rs, long long hs) { return (rb - 1) * rs + (long long)(p.hb - 1) * hs + c.dim; };
  if (reach(p.xr, p.xh) >= far || reach(p.yr, p.yh) >= far) rb = 1;
  if (reach(p.xr, p.xh) >= far || reach(p.yr, p.yh) >= far) p.hb = 1;
  p.rb = (int)rb;
  p.txr = rb > 1 ? (int)p.xr : 0;
  p.txh = p.hb > 1 ? (int)p.xh : 0;
  p.tyr = rb > 1 || c.slot != nullptr ? (int)p.yr : 0;
  p.tyh = p.hb > 1 ? (int)p.yh : 0;
  p.by_unit.set((uint32_t)p.units);
  p.by_head.set((uint32_t)p.hb);
  p.by_half.set((uint32_t)(half > 0 ? half : 1));
  const long long gx = (c.rows + rb - 1) / rb;
  const dim3 grid((unsigned)gx, (unsigned)((c.heads + p.hb - 1) / p.hb));
  auto kern = c.dtype == V4_BF16 ? (by_half ? rope_kernel<bf16, true> : rope_kernel<bf16, false>)
                                 : (by_half ? rope_kernel<float, true> : rope_kernel<float, false>);
  const cudaError_t e = launch_overlapped(kern, grid, dim3(kRopeThreads), 0, st, p);
  if (e == cudaSuccess) note_launch();
  return e;
}

}  // namespace v4
