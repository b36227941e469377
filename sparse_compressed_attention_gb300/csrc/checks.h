// Argument checks that the entry points of the serving operators share.
#pragma once

#include <stdint.h>
#include <stdio.h>

#include "internal.h"

namespace v4 {

inline v4_status bad(const char* what) { return set_error(V4_ERR_INVALID_ARG, what); }

inline v4_status cuda_result(cudaError_t e, const char* what) {
  if (e == cudaSuccess) return V4_OK;
  char buf[256];
  snprintf(buf, sizeof(buf), "%s: %s", what, cudaGetErrorString(e));
  return set_error(V4_ERR_CUDA, buf);
}

inline v4_status check_ptr(const void* p, const char* name, bool required = true) {
  char buf[128];
  if (!p) {
    if (!required) return V4_OK;
    snprintf(buf, sizeof(buf), "%s is NULL", name);
    return bad(buf);
  }
  if ((uintptr_t)p & 15u) {
    snprintf(buf, sizeof(buf), "%s is not 16-byte aligned", name);
    return bad(buf);
  }
  return V4_OK;
}

#define TRY(expr)                     \
  do {                                \
    const v4_status s_ = (expr);      \
    if (s_ != V4_OK) return s_;       \
  } while (0)

inline v4_status check_rotation(int64_t rows, int32_t dim, int32_t rope_dim, int32_t rope_begin, int32_t layout,
                                int32_t dtype) {
  if (dtype != V4_F32 && dtype != V4_BF16) return bad("unknown dtype");
  if (layout != V4_ROPE_INTERLEAVED && layout != V4_ROPE_HALF) return bad("unknown rotation layout");
  if (rows < 0) return bad("rows must be >= 0");
  if (rows > 0x7FFFFFFF) return bad("rows above 2^31 - 1");
  if (dim < 8 || dim > 8192 || dim % 8) return bad("dim must be a multiple of 8 in [8, 8192]");
  if (rope_dim < 0 || rope_dim > 1024 || rope_dim % (layout == V4_ROPE_HALF ? 16 : 8))
    return bad("rope_dim must be a multiple of 8 (16 for the half layout) in [0, 1024]");
  if (rope_begin < 0 || rope_begin % 8 || rope_begin > dim - rope_dim)
    return bad("rope_begin must be a multiple of 8 with rope_begin + rope_dim <= dim");
  return V4_OK;
}

// Bytes from the first to behind the last element of a strided tensor.
inline int64_t extent(int64_t rows, int64_t heads, int64_t dim, int64_t rs, int64_t hs, int es) {
  return ((rows - 1) * rs + (heads - 1) * hs + dim) * es;
}

inline bool overlap(const void* a, int64_t na, const void* b, int64_t nb) {
  const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
  return x < y + (uintptr_t)nb && y < x + (uintptr_t)na;
}

// Whether a view of no x ni runs of dim elements (nested: the inner runs of one outer
// step end before the next) and the same view moved by `shift` elements have an
// element in common: some difference of outer and inner steps brings a run within
// dim of another.  The outer difference is one of the two around shift / so, since
// what is left is smaller than so, the inner one likewise.
inline bool views_meet(int64_t shift, int64_t no, int64_t so, int64_t ni, int64_t si, int64_t dim) {
  const int64_t moved = shift < 0 ? -shift : shift;                // the other way round it is the same
  const int64_t o0 = no > 1 ? moved / so : 0;
  for (int64_t o = o0; o <= o0 + 1 && o < no; ++o) {
    const int64_t rest = moved - o * so < 0 ? o * so - moved : moved - o * so;
    const int64_t i0 = ni > 1 ? rest / si : 0;
    for (int64_t i = i0; i <= i0 + 1 && i < ni; ++i)
      if (rest - i * si < dim && i * si - rest < dim) return true;
  }
  return false;
}

inline v4_status check_stride(int64_t s, int es, const char* name) {
  char buf[128];
  if (s < 0 || s > (int64_t)1 << 40 || (s * es) % 16) {
    snprintf(buf, sizeof(buf), "%s must be a multiple of 16 bytes in [0, 2^40]", name);
    return bad(buf);
  }
  return V4_OK;
}

}  // namespace v4
