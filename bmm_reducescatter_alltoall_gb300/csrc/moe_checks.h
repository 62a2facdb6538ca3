// Checks of arguments that the host entry points of the ragged expert operators
// share.  Every rule is stated in include/bra_moe.h.
#pragma once

#include "moe_internal.h"

namespace bra {

// Rows of a call: a tile's last row index stays in 32 bits.
constexpr int64_t kMaxRows = (int64_t(1) << 31) - (int64_t(1) << 16);

inline bool off_by(const void* p, uintptr_t mask) { return (reinterpret_cast<uintptr_t>(p) & mask) != 0; }

inline bool overlap(const void* a, int64_t an, const void* b, int64_t bn) {
  if (!a || !b || an <= 0 || bn <= 0) return false;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + (uintptr_t)bn && y < x + (uintptr_t)an;
}

// Whether `rows` rows `pitch` elements apart (of at most 8 bytes) count in 64 bits.
inline bool counts_in_64_bits(int64_t rows, int64_t pitch) {
  return rows <= 0 || pitch <= (int64_t(1) << 59) / rows;
}

// Bytes of `rows` rows of n elements, ld apart (the last one without padding).
inline int64_t span(int64_t rows, int64_t ld, int64_t n, int64_t es) {
  return rows > 0 ? ((rows - 1) * ld + n) * es : 0;
}

inline int status_of(cudaError_t e) {
  return e == cudaSuccess ? BRA_OK : e == cudaErrorInvalidValue ? BRA_ERR_UNSUPPORTED
                                                                : BRA_ERR_CUDA;
}

inline int clear_status(int32_t* status, cudaStream_t st) {
  if (!status) return BRA_OK;
  return cudaMemsetAsync(status, 0, sizeof(int32_t), st) == cudaSuccess ? BRA_OK : BRA_ERR_CUDA;
}

// A range of memory of a call.
struct Span {
  const void* p;
  int64_t n;
};

// Whether an output overlaps an input or another output.
inline bool any_overlap(const Span* outs, int no, const Span* ins, int ni) {
  for (int i = 0; i < no; ++i) {
    for (int j = 0; j < ni; ++j)
      if (overlap(outs[i].p, outs[i].n, ins[j].p, ins[j].n)) return true;
    for (int j = 0; j < i; ++j)
      if (overlap(outs[i].p, outs[i].n, outs[j].p, outs[j].n)) return true;
  }
  return false;
}

inline int64_t element_size(int dtype) { return dtype == BRA_FP32 ? 4 : 2; }

inline bool row_dtype_ok(int dtype) {
  return dtype == BRA_FP16 || dtype == BRA_BF16 || dtype == BRA_FP32;
}

}  // namespace bra
