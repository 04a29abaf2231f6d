// dit_checks.h -- the argument checks shared by the C entry points
// (dit_api.cu, dit_token_api.cu): sizes, spans, alignment.  Host code only.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "dit_elementwise.h"

namespace dit {

inline int elem_size(dit_dtype t) { return t == DIT_FP32 ? 4 : 2; }

inline bool valid_dtype(int t) { return t == DIT_BF16 || t == DIT_FP16 || t == DIT_FP32; }
inline bool valid_layout(int l) { return l == DIT_FULL || l == DIT_ROW_BCAST; }

// N = B * L * D elements; false on a negative size or overflow of the byte
// count of a tensor.
inline bool element_count(int64_t B, int64_t L, int64_t D, int es, int64_t* n) {
  if (B < 0 || L < 0 || D < 0) return false;
  int64_t bl, bld, bytes;
  if (__builtin_mul_overflow(B, L, &bl)) return false;
  if (__builtin_mul_overflow(bl, D, &bld)) return false;
  if (__builtin_mul_overflow(bld, (int64_t)es, &bytes)) return false;
  *n = bld;
  return true;
}

struct Span {
  uintptr_t lo, hi;  // [lo, hi) bytes
};
inline Span span(const void* p, int64_t bytes) {
  return Span{(uintptr_t)p, (uintptr_t)p + (uintptr_t)bytes};
}
inline bool overlaps(Span a, Span b) { return a.lo < b.hi && b.lo < a.hi; }

inline bool misaligned(const void* p, int es) {
  return ((uintptr_t)p & (uintptr_t)(es - 1)) != 0;
}

inline dit_status launch_status(cudaError_t e) { return e == cudaSuccess ? DIT_OK : DIT_ERR_LAUNCH; }

}  // namespace dit
