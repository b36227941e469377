// Index division by run-time constants.
#pragma once

#include <stdint.h>

namespace v4 {

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

}  // namespace v4
