// The 8-bit block-scaled layout: codes of a byte, one fp32 scale to each 128
// elements of a row, or to each 128 x 128 of a weight.
//
// Codes: a row of K elements at a pitch of whole 16 bytes, which TMA can
// address; a K block of the products is 128 bytes of codes, one swizzle row,
// and one scale.  Scales of rows: row-major at a pitch of whole 16 bytes, so
// that a thread that follows a row takes four blocks' in one load.  Scales of
// weights: dense, as checkpoints hold them.
#pragma once

#include <stdint.h>

namespace bra {
namespace fp8 {

constexpr int kBlock = 128;

__host__ __device__ inline int64_t code_pitch(int64_t K) { return (K + 15) / 16 * 16; }
__host__ __device__ inline int64_t blocks(int64_t n) { return (n + kBlock - 1) / kBlock; }
// Floats between the scales of two rows.
__host__ __device__ inline int64_t scale_pitch(int64_t K) { return (blocks(K) + 3) / 4 * 4; }

}  // namespace fp8
}  // namespace bra
