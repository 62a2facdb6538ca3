// A grid's warps dealt over (row, part of the row) units in order.
#pragma once

#include <stdint.h>

namespace bra {

// The units of one warp: row and part, the next one found by adding, not
// dividing (a 64-bit division costs as much as the few loads of a unit).
// Rows are below 2^31, so the row past the last never wraps.
struct Walk {
  uint32_t row, part, per_row, d_row, d_part;
  __device__ __forceinline__ explicit Walk(uint32_t parts) {
    per_row = parts;
    const uint32_t warps = gridDim.x * (blockDim.x / 32);
    const uint32_t w = blockIdx.x * (blockDim.x / 32) + threadIdx.x / 32;
    row = w / per_row;
    part = w - row * per_row;
    d_row = warps / per_row;
    d_part = warps - d_row * per_row;
  }
  __device__ __forceinline__ void next() {
    row += d_row;
    part += d_part;
    if (part >= per_row) {
      part -= per_row;
      ++row;
    }
  }
};

}  // namespace bra
