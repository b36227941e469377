// Rotation angles from a 64-bit fraction of a turn.
//
// The angle pos * f only matters modulo one turn, so the table entry f
// (radians per position) is first expressed as a fraction of a turn in
// 2^-64 units, F = f / (2 pi) mod 1, and the angle of a position is the
// 64-bit product pos * F, which wraps at whole turns by itself.  f = m * 2^e
// with a 24-bit m, so F = m * (2^66 / (2 pi)) * 2^(e-2) needs one 64 x 24
// bit product; the constant is rounded to 64 bits and F cut off behind its last,
// which leaves F within (1 + |f| / 8) 2^-64 and the angle within |pos| times that
// many turns: 2^-32 at the farthest positions for |f| <= 1.  The top 32 bits
// are split, still as integers, into quarter turns and a remainder of at most an
// eighth of a turn to either side, since fp32 holds 24 bits: sincospif gets the
// remainder to 2^-28 turns (the whole angle would come to 2^-26, the largest
// term in the error of an fp32 rotation), and the quarter turns only exchange and
// negate its results.  No fp64: this part's fp64 rate is low.
#pragma once

#include <stdint.h>

namespace v4 {

// f / (2 pi) modulo 1 in 2^-64 turns.  Meant for |f| < 2^16 (a rotation of
// more than 2^16 radians per position has no meaningful fp32 table entry).
__device__ __forceinline__ uint64_t turn_fraction(float f) {
  const uint64_t c = 11743562013128004906ull;      // round(2^66 / (2 pi))
  const uint32_t bits = __float_as_uint(f);
  const int ex = (int)((bits >> 23) & 255u);
  if (ex == 0 || ex == 255) return 0;               // zero, denormal or not finite
  const uint64_t m = (bits & 0x7FFFFFu) | 0x800000u;
  // m * c is an 88-bit number; F = (m * c) * 2^(ex - 150 - 2)
  const uint64_t lo = m * c, hi = __umul64hi(m, c);
  const int sh = 152 - ex;
  uint64_t r;
  if (sh <= 0) r = lo << (-sh > 63 ? 63 : -sh);
  else if (sh < 64) r = (lo >> sh) | (hi << (64 - sh));
  else r = sh < 128 ? hi >> (sh - 64) : 0;
  return (bits >> 31) ? (uint64_t)0 - r : r;
}

// cos and sin of pos * F turns.
__device__ __forceinline__ void turn_cos_sin(int pos, uint64_t F, float* c, float* s) {
  const uint32_t a = (uint32_t)(((uint64_t)(long long)pos * F) >> 32);
  const uint32_t quarters = (a + 0x20000000u) >> 30;        // modulo four
  const int rest = (int)(a - (quarters << 30));             // within 2^29 of zero
  float sr, cr;
  sincospif((float)rest * 4.656612873077393e-10f, &sr, &cr);      // 2^-31: half turns
  const bool swap = quarters & 1u;
  const float x = swap ? sr : cr, y = swap ? cr : sr;
  *c = (quarters + 1u) & 2u ? -x : x;
  *s = quarters & 2u ? -y : y;
}

}  // namespace v4
