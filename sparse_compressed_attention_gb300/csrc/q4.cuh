// Rows of the 4-bit cache.
//
// A row of D values is D / 2 bytes of codes, then D / 16 scale bytes, then zeros
// up to a multiple of 16 bytes.  Value i = (code - 8) * scale(byte i / 16);
// scale(8 e + m) = 2^(e - 20) (1 + m / 8).  Word i of the codes holds values 8 i ..
// 8 i + 7, from its lowest nibble in the order 0, 2, 4, 6, 1, 3, 5, 7: a shift and a
// mask then give two neighbours in the halves of a word.  A code has three
// significant bits and a scale four, so every value is exact in bf16.
#pragma once

#include "common.cuh"

namespace v4 {

struct Q4 {                                      // one byte of such a row
  uint8_t b;
};

constexpr int kQ4Group = 16;

__host__ __device__ __forceinline__ int q4_row_bytes(int D) { return (D / 2 + D / kQ4Group + 15) & ~15; }

__device__ __forceinline__ float q4_scale(uint32_t byte) { return __uint_as_float((byte << 20) + (107u << 23)); }

// Eight values of a word of codes.
__device__ __forceinline__ void q4_values(uint32_t word, float scale, float* v) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t two = word >> (4 * i);
    v[2 * i] = ((float)(int)(two & 15u) - 8.f) * scale;
    v[2 * i + 1] = ((float)(int)((two >> 16) & 15u) - 8.f) * scale;
  }
}

// Eight values of a word as bf16 pairs, value 0 lowest.  0x4300 | n is 128 + n in
// bf16; (128 + n) s - 136 s in one fused step is (n - 8) s, which bf16 holds, and so
// does 136 s = 17 (8 + m) 2^k, 17 * 15 being below 2^8.
__device__ __forceinline__ uint4 q4_word_bf16(uint32_t word, uint32_t byte) {
  const uint32_t s = byte * 0x00100010u + 0x35803580u;           // the scale in both halves
  const __nv_bfloat162 scale = *reinterpret_cast<const __nv_bfloat162*>(&s);
  const __nv_bfloat162 shift = __hmul2(scale, __float2bfloat162_rn(-136.f));
  uint32_t v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t two = ((word >> (4 * i)) & 0x000F000Fu) | 0x43004300u;
    const __nv_bfloat162 r = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&two), scale, shift);
    v[i] = *reinterpret_cast<const uint32_t*>(&r);
  }
  return make_uint4(v[0], v[1], v[2], v[3]);
}

}  // namespace v4
