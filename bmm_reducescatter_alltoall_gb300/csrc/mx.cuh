// The 4-bit microscaled layout: blocks of 32 elements along a row share one
// power-of-two scale.
//
// Codes: e2m1, two to a byte (the even element in the low half), a row of K
// elements padded with zeros to a multiple of 32: row pitch ceil(K/32) * 16
// bytes, which TMA can address.
//
// Scales: e8m0 bytes (255 = NaN) in the order the tensor core's copy from
// shared memory wants them, so that a product never rearranges them: per
// block of 128 rows and per 256 elements of K one 1 KiB unit, two atoms of
// 512 bytes (128 elements each): byte (r % 32) * 16 + (r / 32) * 4 + s for
// row r of the block and scale s of the atom.  Row blocks start anew at each
// row group, so that a group's row tile is a scale block whatever row the
// group starts at.  Bytes of rows that do not exist are not written.
#pragma once

#include <stdint.h>

namespace bra {
namespace mx {

constexpr int kBlock = 32;                 // elements to a scale
constexpr int kUnitK = 256;                // elements of K to a scale unit
constexpr int kUnitBytes = 1024;

__host__ __device__ inline int64_t code_pitch(int64_t K) { return (K + 31) / 32 * 16; }
__host__ __device__ inline int64_t units(int64_t K) { return (K + kUnitK - 1) / kUnitK; }
// Row blocks held for R rows in E groups: of `each` rows, or (0) of any sizes
// that add up to at most R: n rows take (n + 127) / 128 blocks, and at most
// min(R, E) groups have rows.  For one group the two are the same, as rows of
// one group may be quantized either way.
__host__ __device__ inline int64_t blocks_of(int64_t R, int64_t E, int64_t each) {
  return each > 0 ? E * ((each + 127) / 128) : (R + 127 * (R < E ? R : E)) / 128;
}
// Byte of scale s (of the whole row) in row r (0..127) of row block `blk`.
__host__ __device__ inline int64_t scale_at(int64_t blk, int r, int64_t s, int64_t k_units) {
  return blk * k_units * kUnitBytes + (s >> 2) * 512 + (r & 31) * 16 + (r >> 5) * 4 + (s & 3);
}

}  // namespace mx
}  // namespace bra
