// Quantisation to 4-bit microscaled values, and back.
//
// Of each 32 elements, a = max |x|; the scale is 2^s with
// s = max(floor(log2 a) - 2, -127), the largest power of two that puts a at or
// above 4 of the format's largest magnitude 6; the code is the nearest of
// +-{0, .5, 1, 1.5, 2, 3, 4, 6} to x / 2^s, ties to the even code, magnitudes
// past 6 to 6.  x / 2^s is exact (a product with a power of two), so the codes
// are a function of x alone.  A block with a NaN or an infinity has no scale:
// byte 255, every value NaN.
//
// 16 bits are read and 4.25 written to an element, but at those rates the
// instructions of a warp count as much as the bytes.  Quantising, a lane takes
// a whole block: no exchange for the maximum, one 16-byte store of codes, and
// the block's scale once (with 8 elements a lane, four lanes to a block, the
// same work took 112 instructions an 8 elements and 34 us for 64 Mi values
// where the bytes take 25).  Going back, a lane makes 8 elements, one 16-byte
// store.  A warp takes up to 1024 elements of a row with their loads issued
// together.  16384 x 4096: 28 us to codes (170 MB, 25 us at the copy rate), 30
// back.
#include <type_traits>

#include "grouped.cuh"
#include "mx.cuh"
#include "walk.cuh"

namespace bra {
namespace {

using namespace grp;

constexpr int kThreads = 256;
constexpr int kPieces = 4;                // 256-element pieces of a warp's unit

template <typename T>
__device__ __forceinline__ float2 pair_of(uint32_t w);
template <>
__device__ __forceinline__ float2 pair_of<__half>(uint32_t w) {
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}
template <>
__device__ __forceinline__ float2 pair_of<__nv_bfloat16>(uint32_t w) {
  return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w));
}

// Eight codes, the first in the lowest four bits.
__device__ __forceinline__ uint32_t code_word(const float (&f)[8]) {
  uint32_t r;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(r)
      : "f"(f[0]), "f"(f[1]), "f"(f[2]), "f"(f[3]), "f"(f[4]), "f"(f[5]), "f"(f[6]), "f"(f[7]));
  return r;
}
// Two codes (the low byte of w) as a pair of halves, which hold them exactly.
__device__ __forceinline__ float2 values_of(uint32_t w) {
  uint32_t h;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "mov.b32 {a, b, c, d}, %1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\t}"
      : "=r"(h)
      : "r"(w));
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// Row block and row within it of row r: groups of `each` rows, or of the
// table's counts.
__device__ __forceinline__ void locate(const GroupTable* gt, int E, int64_t each, int64_t r,
                                       int64_t* blk, int* in) {
  if (each > 0) {
    const uint32_t n = (uint32_t)each, g = (uint32_t)r / n, i = (uint32_t)r - g * n;
    *blk = (int64_t)g * ((n + 127) / 128) + (i >> 7);
    *in = (int)(i & 127);
    return;
  }
  int lo = 0, hi = E - 1;                 // the last group that starts at or before r
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (gt->off[mid] <= r) lo = mid;
    else hi = mid - 1;
  }
  const int i = (int)(r - gt->off[lo]);
  *blk = gt->tile[lo] + (i >> 7);
  *in = i & 127;
}

template <typename T>
__global__ void __launch_bounds__(kThreads)
    quantize_kernel(const T* x, int64_t ld, int64_t R, int64_t K, const int64_t* counts, int E,
                    int64_t each, uint8_t* codes, uint8_t* scales, int vec, int32_t* status) {
  __shared__ GroupTable gt;
  const int lane = threadIdx.x & 31;
  int64_t rows = R;
  grid_wait();
  grid_go();
  if (counts) {
    if (threadIdx.x < 32) build_table<128>(&gt, counts, E, R, lane);
    __syncthreads();
    if (gt.bad) {
      if (blockIdx.x == 0 && threadIdx.x == 0 && status)
        atomicExch(status, (int32_t)BRA_ERR_INVALID);
      return;
    }
    rows = gt.off[E];
  }
  const int64_t cpitch = mx::code_pitch(K), k_units = mx::units(K);
  const int nblocks = (int)((K + mx::kBlock - 1) / mx::kBlock), nscales = (int)k_units * 8;
  for (Walk at((uint32_t)((k_units + kPieces - 1) / kPieces)); at.row < rows; at.next()) {
    const int64_t r = at.row;
    const int b = (int)at.part * 32 + lane;         // this lane's block of the row
    const T* src = x + r * ld + (int64_t)b * mx::kBlock;
    uint32_t w[16];
    if (vec && (b + 1) * mx::kBlock <= K) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint4 q = reinterpret_cast<const uint4*>(src)[i];
        w[4 * i] = q.x, w[4 * i + 1] = q.y, w[4 * i + 2] = q.z, w[4 * i + 3] = q.w;
      }
    } else {
      const uint16_t* e = reinterpret_cast<const uint16_t*>(src);
      const int64_t left = K - (int64_t)b * mx::kBlock;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const uint32_t lo = 2 * i < left ? e[2 * i] : 0u;
        const uint32_t hi = 2 * i + 1 < left ? e[2 * i + 1] : 0u;
        w[i] = lo | hi << 16;
      }
    }
    int64_t blk;
    int in;
    locate(&gt, E, each, r, &blk, &in);
    // magnitudes ordered as 16-bit integers: NaN above infinity above all else
    uint32_t a = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) a = __vmaxu2(a, w[i] & 0x7fff7fffu);
    const float2 top = pair_of<T>(__vmaxu2(a, a >> 16));
    const uint32_t bits = __float_as_uint(top.x);
    const bool none = bits >= 0x7f800000u;
    const int field = (int)(bits >> 23);            // subnormals and zero: 0
    const uint32_t byte = none ? 255u : (uint32_t)max(field - 2, 0);
    const float inv = __uint_as_float((254u - (none ? 0u : byte)) << 23);   // 2^(127 - byte)
    if (b < nblocks) {
      uint32_t c[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float f[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 p = pair_of<T>(w[4 * i + j]);
          f[2 * j] = p.x * inv;
          f[2 * j + 1] = p.y * inv;
        }
        c[i] = none ? 0u : code_word(f);
      }
      *reinterpret_cast<uint4*>(codes + r * cpitch + (int64_t)b * 16) =
          make_uint4(c[0], c[1], c[2], c[3]);
    }
    // a 128-element atom's four scales as one word
    uint32_t s = byte << (8 * (lane & 3));
    s |= __shfl_xor_sync(0xffffffffu, s, 1);
    s |= __shfl_xor_sync(0xffffffffu, s, 2);
    if ((lane & 3) == 0 && b < nscales)
      *reinterpret_cast<uint32_t*>(scales + mx::scale_at(blk, in, b, k_units)) = s;
  }
}

template <typename T>
__device__ __forceinline__ T to(float v);
template <>
__device__ __forceinline__ __half to<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 to<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ float to<float>(float v) { return v; }

// value = code * 2^(byte - 127); a lane makes the 8 values of one code word.
template <typename T>
__global__ void __launch_bounds__(kThreads)
    dequantize_kernel(const uint8_t* codes, const uint8_t* scales, int64_t R, int64_t K,
                      const int64_t* counts, int E, int64_t each, T* y, int vec, int32_t* status) {
  __shared__ GroupTable gt;
  const int lane = threadIdx.x & 31;
  int64_t rows = R;
  grid_wait();
  grid_go();
  if (counts) {
    if (threadIdx.x < 32) build_table<128>(&gt, counts, E, R, lane);
    __syncthreads();
    if (gt.bad) {
      if (blockIdx.x == 0 && threadIdx.x == 0 && status)
        atomicExch(status, (int32_t)BRA_ERR_INVALID);
      return;
    }
    rows = gt.off[E];
  }
  const int64_t cpitch = mx::code_pitch(K), k_units = mx::units(K);
  for (Walk at((uint32_t)((k_units + kPieces - 1) / kPieces)); at.row < rows; at.next()) {
    const int64_t r = at.row;
    const int k0 = (int)at.part * (kPieces * mx::kUnitK) + lane * 8;
    int64_t blk;
    int in;
    locate(&gt, E, each, r, &blk, &in);
    const uint8_t* code = codes + r * cpitch + k0 / 2;
    const uint8_t* scale = scales + mx::scale_at(blk, in, k0 / mx::kBlock, k_units);
    T* dst = y + r * K + k0;
    uint32_t c[kPieces], b[kPieces];
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      c[i] = b[i] = 0u;
      if (k0 + i * mx::kUnitK < K) {
        c[i] = *reinterpret_cast<const uint32_t*>(code + i * (mx::kUnitK / 2));
        b[i] = scale[i * mx::kUnitBytes];     // a unit's scales are a unit's bytes on
      }
    }
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const int left = (int)K - (k0 + i * mx::kUnitK);
      if (left <= 0) break;
      // 2^(b - 127): b = 0 is the subnormal 2^-127, 255 is NaN
      const float s = __uint_as_float(b[i] == 255u ? 0x7fc00000u : b[i] ? b[i] << 23 : 1u << 22);
      T v[8];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 m = values_of(c[i] >> (8 * j));
        v[2 * j] = to<T>(m.x * s);
        v[2 * j + 1] = to<T>(m.y * s);
      }
      T* out = dst + i * mx::kUnitK;
      if (vec && left >= 8) {
#pragma unroll
        for (int j = 0; j < (int)sizeof(T) / 2; ++j)
          reinterpret_cast<uint4*>(out)[j] = reinterpret_cast<const uint4*>(v)[j];
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (j < left) out[j] = v[j];
      }
    }
  }
}

cudaError_t blocks_for(int64_t warps_wanted, unsigned* grid) {
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  const int64_t want = (warps_wanted + kThreads / 32 - 1) / (kThreads / 32), full = (int64_t)sms * 8;
  *grid = (unsigned)(want < 1 ? 1 : want < full ? want : full);
  return cudaSuccess;
}

int64_t warps_of(int64_t R, int64_t K) { return R * ((mx::units(K) + kPieces - 1) / kPieces); }

}  // namespace

cudaError_t launch_mx_quantize(const MxRows& q, const void* x, int64_t ld, int dtype,
                               cudaStream_t st) {
  unsigned grid = 0;
  cudaError_t e = blocks_for(warps_of(q.R, q.K), &grid);
  if (e != cudaSuccess) return e;
  const int vec = (reinterpret_cast<uintptr_t>(x) & 15u) == 0 && ld % 8 == 0;
  auto run = [&](auto* in) {
    using T = std::remove_pointer_t<decltype(in)>;
    return launch_overlapped(quantize_kernel<T>, grid, kThreads, 0, st, static_cast<const T*>(x),
                             ld, q.R, q.K, q.counts, q.E, q.each, q.codes, q.scales, vec, q.status);
  };
  return dtype == BRA_BF16 ? run((__nv_bfloat16*)nullptr) : run((__half*)nullptr);
}

cudaError_t launch_mx_dequantize(const MxRows& q, void* y, int dtype, cudaStream_t st) {
  unsigned grid = 0;
  cudaError_t e = blocks_for(warps_of(q.R, q.K), &grid);
  if (e != cudaSuccess) return e;
  const int64_t es = dtype == BRA_FP32 ? 4 : 2;
  const int vec = (reinterpret_cast<uintptr_t>(y) & 15u) == 0 && q.K * es % 16 == 0;
  auto run = [&](auto* out) {
    using T = std::remove_pointer_t<decltype(out)>;
    return launch_overlapped(dequantize_kernel<T>, grid, kThreads, 0, st, q.codes, q.scales, q.R,
                             q.K, q.counts, q.E, q.each, static_cast<T*>(y), vec, q.status);
  };
  if (dtype == BRA_BF16) return run((__nv_bfloat16*)nullptr);
  if (dtype == BRA_FP16) return run((__half*)nullptr);
  return run((float*)nullptr);
}

}  // namespace bra
