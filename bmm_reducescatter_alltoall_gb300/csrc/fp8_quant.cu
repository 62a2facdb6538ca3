// Quantisation to 8-bit block-scaled values, and back.
//
// Of each block (128 elements of a row, or 128 x 128 of a weight), a = max
// |x|; the scale is the smallest 2^s, s >= -126, with a <= 2^s * L, L = 1.75 *
// 2^8 (e4m3) or 1.75 * 2^15 (e5m2): s is a's exponent less 8 or 15, one more
// when a's significand passes 1.75.  The code is the nearest to x / 2^s, ties
// to even.  x / 2^s is a product with a power of two, exact but where it falls
// far below the smallest code, so that codes are a function of x alone.  A
// block with a NaN or an infinity gets the scale NaN and codes of zero.
//
// 16 bits are read and 8.25 written to an element, and HBM bounds it.  A lane
// takes 16 consecutive elements: 16 bytes of codes a store, eight lanes to a
// row's block, three exchanges for its maximum; a warp has the loads of 2048
// elements in flight.  A weight's block is a CTA's, held in registers
// between its maximum and its codes, so that it too is read once.  16384 x 4096
// bf16: rows 30 us (6.7 TB/s), weights 31, there and back 65 (92% of the copy
// rate).
#include <type_traits>

#include "fp8.cuh"
#include "grouped.cuh"
#include "walk.cuh"

namespace bra {
namespace {

using namespace grp;

constexpr int kThreads = 256;
constexpr int kPieces = 4;                // 512-element pieces of a warp's unit
constexpr int kUnit = kPieces * 512;

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

// 16 consecutive elements of a row as they are stored, read by 16-byte loads:
// ALIGNED rows as they lie, others from the aligned bytes around them, shifted
// (fp16, a weight of 12952 x 3365: 42 us by single elements, 28 by these).
template <typename T, bool ALIGNED>
struct Piece {
  static constexpr int W = 4 * (int)sizeof(T);          // words
  static constexpr int RAW = ALIGNED ? W : W + 4;       // words loaded
  uint32_t w[RAW];
  // `left` elements of the row are left from src on; zeros past it.  Memory
  // outside lo .. hi is not read.
  __device__ __forceinline__ void load(const T* src, int64_t left, uintptr_t lo, uintptr_t hi) {
    const uintptr_t at = reinterpret_cast<uintptr_t>(src) & ~(uintptr_t)15;
    if (left > 0 && at >= lo && at + RAW * 4 <= hi) {
#pragma unroll
      for (int i = 0; i < RAW / 4; ++i) {
        const uint4 q = reinterpret_cast<const uint4*>(at)[i];
        w[4 * i] = q.x, w[4 * i + 1] = q.y, w[4 * i + 2] = q.z, w[4 * i + 3] = q.w;
      }
      return;
    }
    // the ends of the matrix: to where the aligned bytes would be
    const int skip = ALIGNED ? 0 : (int)((reinterpret_cast<uintptr_t>(src) - at) / sizeof(T));
#pragma unroll
    for (int i = 0; i < RAW; ++i) w[i] = 0u;
    if constexpr (sizeof(T) == 4) {
      const uint32_t* e = reinterpret_cast<const uint32_t*>(src) - skip;
#pragma unroll
      for (int i = 0; i < RAW; ++i)
        if (i >= skip && i - skip < min(left, (int64_t)16)) w[i] = e[i];
    } else {
      const uint16_t* e = reinterpret_cast<const uint16_t*>(src) - skip;
#pragma unroll
      for (int i = 0; i < 2 * RAW; ++i)
        if (i >= skip && i - skip < min(left, (int64_t)16)) w[i / 2] |= (uint32_t)e[i] << (16 * (i & 1));
    }
  }
  // Brings the elements to the front, and zeros past the row's end.
  __device__ __forceinline__ void align(const T* src, int64_t left) {
    if constexpr (!ALIGNED) {
      const uint32_t d = (uint32_t)reinterpret_cast<uintptr_t>(src) & 15u;
#pragma unroll
      for (int i = 0; i < W + 2; ++i) w[i] = d & 8u ? w[i + 2] : w[i];
#pragma unroll
      for (int i = 0; i < W + 1; ++i) w[i] = d & 4u ? w[i + 1] : w[i];
      if constexpr (sizeof(T) == 2) {
#pragma unroll
        for (int i = 0; i < W; ++i) w[i] = d & 2u ? __funnelshift_r(w[i], w[i + 1], 16) : w[i];
      }
    }
    if (left < 16) {
      constexpr int PER = 4 / (int)sizeof(T);           // elements of a word
#pragma unroll
      for (int i = 0; i < W; ++i) {
        if (i * PER >= left) w[i] = 0u;
        else if (PER == 2 && i * PER + 1 >= left) w[i] &= 0xffffu;
      }
    }
  }
  // The largest magnitude as the bits of a float: NaN above infinity above all else.
  __device__ __forceinline__ uint32_t most() const {
    uint32_t a = 0;
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < 16; ++i) a = max(a, w[i] & 0x7fffffffu);
      return a;
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) a = __vmaxu2(a, w[i] & 0x7fff7fffu);
      return __float_as_uint(pair_of<T>(__vmaxu2(a, a >> 16)).x);
    }
  }
  __device__ __forceinline__ float2 pair(int i) const {
    if constexpr (sizeof(T) == 4)
      return make_float2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
    else
      return pair_of<T>(w[i]);
  }
};

// A block's scale as the exponent field of 2^s, 255 for none.
template <bool E5>
__device__ __forceinline__ uint32_t scale_field(uint32_t most) {
  if (most >= 0x7f800000u) return 255u;
  const int f = (int)(most >> 23) - (E5 ? 15 : 8) + ((most & 0x7fffffu) > 0x600000u ? 1 : 0);
  return (uint32_t)max(f, 1);
}
__device__ __forceinline__ float scale_of(uint32_t field) {
  return __uint_as_float(field == 255u ? 0x7fc00000u : field << 23);
}

template <bool E5>
__device__ __forceinline__ uint32_t code_pair(float lo, float hi) {
  uint16_t r;
  if constexpr (E5) asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  else asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// 16 codes under the scale of `field`.
template <bool E5, typename P>
__device__ __forceinline__ uint4 codes_of(const P& x, uint32_t field) {
  const float inv = __uint_as_float((254u - (field == 255u ? 0u : field)) << 23);   // 2^-s
  uint32_t c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 a = x.pair(2 * i), b = x.pair(2 * i + 1);
    c[i] = code_pair<E5>(a.x * inv, a.y * inv) | code_pair<E5>(b.x * inv, b.y * inv) << 16;
    if (field == 255u) c[i] = 0u;
  }
  return make_uint4(c[0], c[1], c[2], c[3]);
}

// Rows in use: R, or the counts' sum; -1 when the counts are refused.  Every thread.
__device__ __forceinline__ int64_t rows_used(GroupTable* gt, const int64_t* counts, int E, int64_t R,
                                             int32_t* status) {
  if (!counts) return R;
  if (threadIdx.x < 32) build_table<128>(gt, counts, E, R, threadIdx.x & 31);
  __syncthreads();
  if (!gt->bad) return gt->off[E];
  if (blockIdx.x == 0 && threadIdx.x == 0 && status) atomicExch(status, (int32_t)BRA_ERR_INVALID);
  return -1;
}

// NARROW: rows of fewer elements than a warp's unit.  The blocks of all rows are
// dealt out one after the other, four to a piece of a warp, so that no lane is
// without elements but in a row's last block (22630 rows of 128 bf16: 18 us with
// a warp to a row, 4 so).
template <typename T, bool E5, bool ALIGNED, bool NARROW>
__global__ void __launch_bounds__(kThreads)
    fp8_rows_kernel(const T* x, int64_t ld, int64_t R, int64_t K, const int64_t* counts, int E,
                    uint8_t* codes, float* scales, uint64_t per_block, int32_t* status) {
  __shared__ GroupTable gt;
  const int lane = threadIdx.x & 31;
  grid_wait();
  grid_go();
  const int64_t rows = rows_used(&gt, counts, E, R, status);
  const int64_t cpitch = fp8::code_pitch(K), spitch = fp8::scale_pitch(K);
  const uint32_t blocks = (uint32_t)fp8::blocks(K);
  const uintptr_t lo = reinterpret_cast<uintptr_t>(x);
  const uintptr_t hi = rows > 0 ? reinterpret_cast<uintptr_t>(x + (rows - 1) * ld + K) : lo;
  // four pieces: of row r[i] from element k[i] on, none where k[i] is K or more
  auto unit = [&](const uint32_t (&r)[kPieces], const uint32_t (&k)[kPieces]) {
    Piece<T, ALIGNED> p[kPieces];
#pragma unroll
    for (int i = 0; i < kPieces; ++i) p[i].load(x + r[i] * ld + k[i], K - k[i], lo, hi);
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      p[i].align(x + r[i] * ld + k[i], K - k[i]);
      uint32_t a = p[i].most();
      a = max(a, __shfl_xor_sync(0xffffffffu, a, 1));
      a = max(a, __shfl_xor_sync(0xffffffffu, a, 2));
      a = max(a, __shfl_xor_sync(0xffffffffu, a, 4));
      const uint32_t field = scale_field<E5>(a), b = k[i] / fp8::kBlock;
      if (k[i] < K)
        *reinterpret_cast<uint4*>(codes + r[i] * cpitch + k[i]) = codes_of<E5>(p[i], field);
      float* scale = scales + r[i] * spitch + b;
      if ((lane & 7) == 0 && b < blocks) *scale = scale_of(field);
      // zeros past the last block, by its other lanes
      if ((lane & 7) != 0 && b + 1 == blocks && b + (lane & 7) < spitch) scale[lane & 7] = 0.f;
    }
  };
  uint32_t r[kPieces], k[kPieces];
  if constexpr (NARROW) {
    const uint64_t total = rows > 0 ? (uint64_t)rows * blocks : 0;
    const uint64_t step = (uint64_t)gridDim.x * (kThreads / 32) * (4 * kPieces);
    uint64_t at = ((uint64_t)blockIdx.x * (kThreads / 32) + threadIdx.x / 32) * (4 * kPieces);
    for (; at < total; at += step) {
#pragma unroll
      for (int i = 0; i < kPieces; ++i) {
        const uint64_t item = at + i * 4 + (lane >> 3);
        const uint32_t row = (uint32_t)(per_block ? __umul64hi(item, per_block) : item);
        r[i] = item < total ? row : 0u;
        k[i] = (item < total ? (uint32_t)item - row * blocks : blocks) * fp8::kBlock + (lane & 7) * 16;
      }
      unit(r, k);
    }
  } else {
    for (Walk at((uint32_t)((K + kUnit - 1) / kUnit)); at.row < rows; at.next()) {
#pragma unroll
      for (int i = 0; i < kPieces; ++i) {
        r[i] = at.row;
        k[i] = at.part * kUnit + i * 512 + lane * 16;
      }
      unit(r, k);
    }
  }
}

// A CTA to a 128 x 128 block: eight lanes to a row, 32 rows at a time.
template <typename T, bool E5, bool ALIGNED>
__global__ void __launch_bounds__(kThreads)
    fp8_blocks_kernel(const T* x, int64_t R, int64_t K, int64_t N, int64_t total, uint8_t* codes,
                      float* scales) {
  __shared__ uint32_t warp_most[2][kThreads / 32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t cpitch = fp8::code_pitch(K);
  const uint32_t kb = (uint32_t)fp8::blocks(K), nb = (uint32_t)fp8::blocks(N);
  grid_wait();
  grid_go();
  const uintptr_t lo = reinterpret_cast<uintptr_t>(x), hi = reinterpret_cast<uintptr_t>(x + R * K);
  int turn = 0;
  for (int64_t at = blockIdx.x; at < total; at += gridDim.x, turn ^= 1) {
    const int64_t row_block = at / kb, g = row_block / nb;
    const int64_t n0 = (row_block - g * nb) * fp8::kBlock + (threadIdx.x >> 3);
    const int64_t k = (at - row_block * kb) * fp8::kBlock + (threadIdx.x & 7) * 16;
    Piece<T, ALIGNED> p[4];
    uint32_t a = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      p[i].load(x + (g * N + n0 + i * 32) * K + k, n0 + i * 32 < N ? K - k : 0, lo, hi);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      p[i].align(x + (g * N + n0 + i * 32) * K + k, n0 + i * 32 < N ? K - k : 0);
      a = max(a, p[i].most());
    }
    a = __reduce_max_sync(0xffffffffu, a);
    if (lane == 0) warp_most[turn][warp] = a;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) a = max(a, warp_most[turn][w]);
    const uint32_t field = scale_field<E5>(a);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (n0 + i * 32 < N && k < K)
        *reinterpret_cast<uint4*>(codes + (g * N + n0 + i * 32) * cpitch + k) =
            codes_of<E5>(p[i], field);
    if (threadIdx.x == 0) scales[at] = scale_of(field);
  }
}

template <typename T>
__device__ __forceinline__ uint32_t packed(float2 v);
template <>
__device__ __forceinline__ uint32_t packed<__half>(float2 v) {
  return Out<__half>::pack(v.x, v.y);
}
template <>
__device__ __forceinline__ uint32_t packed<__nv_bfloat16>(float2 v) {
  return Out<__nv_bfloat16>::pack(v.x, v.y);
}

// Two codes (the low half word of w): halves hold them exactly.
template <bool E5>
__device__ __forceinline__ float2 values_of(uint32_t w) {
  uint32_t h;
  if constexpr (E5) asm("cvt.rn.f16x2.e5m2x2 %0, %1;" : "=r"(h) : "h"((uint16_t)w));
  else asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)w));
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// The last `lead` bytes of the lane before (of `sent`, the first lane's before
// being the last one) and the first of `own`.
__device__ __forceinline__ uint4 led_by(const uint4& sent, const uint4& own, int lead, int lane) {
  const int from = (lane + 31) & 31;
  uint32_t z[8] = {__shfl_sync(0xffffffffu, sent.x, from), __shfl_sync(0xffffffffu, sent.y, from),
                   __shfl_sync(0xffffffffu, sent.z, from), __shfl_sync(0xffffffffu, sent.w, from),
                   own.x, own.y, own.z, own.w};
  // bytes 16 - lead .. 32 - lead of the eight words
  if (lead == 0) return own;
  const uint32_t d = 16u - (uint32_t)lead;
#pragma unroll
  for (int i = 0; i < 6; ++i) z[i] = d & 8u ? z[i + 2] : z[i];
#pragma unroll
  for (int i = 0; i < 5; ++i) z[i] = d & 4u ? z[i + 1] : z[i];
#pragma unroll
  for (int i = 0; i < 4; ++i) z[i] = d & 2u ? __funnelshift_r(z[i], z[i + 1], 16) : z[i];
  return make_uint4(z[0], z[1], z[2], z[3]);
}

// Elements k .. of a row's begin .. end, in one store where all of them are
// (off: the address's low bits).
template <typename T>
__device__ __forceinline__ void put_elements(T* row, const uint4& q, int64_t k, int64_t begin,
                                             int64_t end, uintptr_t off) {
  constexpr int OWN = 16 / (int)sizeof(T);
  if (off == 0 && k >= begin && k + OWN <= end) {
    *reinterpret_cast<uint4*>(row + k) = q;
    return;
  }
  const uint32_t z[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int j = 0; j < OWN; ++j)
    if (k + j >= begin && k + j < end) {
      if constexpr (sizeof(T) == 4)
        reinterpret_cast<uint32_t*>(row)[k + j] = z[j];
      else
        reinterpret_cast<uint16_t*>(row)[k + j] = (uint16_t)(z[j / 2] >> (16 * (j & 1)));
    }
}

// N: rows of a weight, or 0 for rows.  A lane takes the codes of 16 bytes of y,
// so that a warp's stores are whole lines (32 bytes a lane, in two stores, took
// 71 us in place of 26 for 16384 x 4096 bf16).  Rows of y that are not ALIGNED
// are stored by aligned 16 bytes too: each lane's first ones are the last of the
// lane before, single elements at a unit's ends (fp16, 12952 x 3365: 125 us by
// single elements, 28 by these).
template <typename T, bool E5, bool ALIGNED>
__global__ void __launch_bounds__(kThreads)
    fp8_back_kernel(const uint8_t* codes, const float* scales, int64_t R, int64_t K, uint32_t N,
                    const int64_t* counts, int E, T* y, int32_t* status) {
  constexpr int OWN = 16 / (int)sizeof(T), STEP = 32 * OWN, PIECES = kUnit / STEP;
  __shared__ GroupTable gt;
  const int lane = threadIdx.x & 31;
  grid_wait();
  grid_go();
  const int64_t rows = rows_used(&gt, counts, E, R, status);
  const int64_t cpitch = fp8::code_pitch(K), spitch = fp8::scale_pitch(K), blocks = fp8::blocks(K);
  for (Walk at((uint32_t)((K + kUnit - 1) / kUnit)); at.row < rows; at.next()) {
    const int64_t r = at.row, k0 = (int64_t)at.part * kUnit + lane * OWN;
    const float* scale = scales + r * spitch;
    if (N) {
      const uint32_t g = (uint32_t)r / N, n = (uint32_t)r - g * N;
      scale = scales + ((int64_t)g * fp8::blocks(N) + n / fp8::kBlock) * blocks;
    }
    uint32_t c[PIECES][OWN / 4];
    float s[PIECES];
#pragma unroll
    for (int i = 0; i < PIECES; ++i) {
      const int64_t k = k0 + i * STEP;                 // the pitch holds whole pieces
      const uint32_t* src = reinterpret_cast<const uint32_t*>(codes + r * cpitch + k);
      if constexpr (OWN == 8) {
        const uint2 q = k < K ? *reinterpret_cast<const uint2*>(src) : make_uint2(0, 0);
        c[i][0] = q.x, c[i][OWN / 4 - 1] = q.y;
      } else {
        c[i][0] = k < K ? *src : 0u;
      }
      s[i] = k < K ? scale[k / fp8::kBlock] : 0.f;
    }
    const int lead = ALIGNED ? 0 : (int)(reinterpret_cast<uintptr_t>(y + r * K) & 15u);   // bytes
    const int64_t begin = (int64_t)at.part * kUnit, end = min(begin + kUnit, K);
    uint4 last = make_uint4(0, 0, 0, 0);               // of the piece before
#pragma unroll
    for (int i = 0; i < PIECES; ++i) {
      int64_t k = k0 + i * STEP;
      if (begin + i * STEP - lead / (int)sizeof(T) >= end) break;      // the same for all lanes
      T* out = y + r * K;
      float v[OWN];
#pragma unroll
      for (int j = 0; j < OWN; j += 2) {
        const float2 a = values_of<E5>(c[i][j / 4] >> (8 * (j & 2)));
        v[j] = a.x * s[i], v[j + 1] = a.y * s[i];
      }
      uint4 q;
      if constexpr (sizeof(T) == 4)
        q = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                       __float_as_uint(v[3]));
      else
        q = make_uint4(packed<T>(make_float2(v[0], v[1])), packed<T>(make_float2(v[2], v[3])),
                       packed<T>(make_float2(v[OWN - 4], v[OWN - 3])),
                       packed<T>(make_float2(v[OWN - 2], v[OWN - 1])));
      if constexpr (!ALIGNED) {
        const uint4 own = q;
        q = led_by(lane == 31 ? last : own, own, lead, lane);
        last = own;
        k -= lead / (int)sizeof(T);
      }
      put_elements<T>(out, q, k, begin, end, reinterpret_cast<uintptr_t>(out + k) & 15u);
    }
    // the last of the unit's elements
    if constexpr (!ALIGNED) {
      const int64_t k = begin + kUnit - lead / (int)sizeof(T);
      if (lead && k < end) {
        const uint4 q = led_by(last, last, lead, lane);
        if (lane == 0) put_elements<T>(y + r * K, q, k, begin, end, 1u);
      }
    }
  }
}

cudaError_t grid_for(int64_t ctas_wanted, int per_sm, unsigned* grid) {
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  const int64_t full = (int64_t)sms * per_sm;
  *grid = (unsigned)(ctas_wanted < 1 ? 1 : ctas_wanted < full ? ctas_wanted : full);
  return cudaSuccess;
}

// CTAs of the kernels that give a warp a part of a row.
int64_t row_ctas(int64_t R, int64_t K) {
  return (R * ((K + kUnit - 1) / kUnit) + kThreads / 32 - 1) / (kThreads / 32);
}

// f for the element type, the format and whether rows are aligned.
template <typename F>
cudaError_t by_type(int dtype, int format, bool aligned, F&& f) {
  auto by_format = [&](auto* type) {
    auto by_alignment = [&](auto e5) {
      return aligned ? f(type, e5, std::true_type{}) : f(type, e5, std::false_type{});
    };
    return format == BRA_E5M2 ? by_alignment(std::true_type{}) : by_alignment(std::false_type{});
  };
  if (dtype == BRA_BF16) return by_format((__nv_bfloat16*)nullptr);
  if (dtype == BRA_FP16) return by_format((__half*)nullptr);
  return by_format((float*)nullptr);
}

}  // namespace

cudaError_t launch_fp8_quantize(const Fp8Data& q, const void* x, int64_t ld, int dtype,
                                cudaStream_t st) {
  const int64_t es = dtype == BRA_FP32 ? 4 : 2;
  const bool aligned = (reinterpret_cast<uintptr_t>(x) & 15u) == 0 && ld * es % 16 == 0;
  return by_type(dtype, q.format, aligned, [&](auto* in, auto e5, auto whole) {
    using T = std::remove_pointer_t<decltype(in)>;
    constexpr bool E5 = decltype(e5)::value, ALIGNED = decltype(whole)::value;
    unsigned grid = 0;
    if (q.each > 0) {
      const int64_t total = q.E * fp8::blocks(q.each) * fp8::blocks(q.K);
      const cudaError_t e = grid_for(total, 6, &grid);
      if (e != cudaSuccess) return e;
      return launch_clusters(fp8_blocks_kernel<T, E5, ALIGNED>, 1, grid, kThreads, 0, st,
                             static_cast<const T*>(x), q.R, q.K, q.each, total, q.codes, q.scales);
    }
    const bool narrow = q.K < kUnit;
    // 2^64 over the blocks of a row, rounded up (0 for one): the high half of its
    // product with a number below 2^36 is the quotient, as the error stays below
    // one block's share
    const uint64_t nb = (uint64_t)fp8::blocks(q.K), per_block = nb == 1 ? 0 : ~(uint64_t)0 / nb + 1;
    const int64_t warps = narrow ? (q.R * fp8::blocks(q.K) + 4 * kPieces - 1) / (4 * kPieces)
                                 : q.R * ((q.K + kUnit - 1) / kUnit);
    const cudaError_t e = grid_for((warps + kThreads / 32 - 1) / (kThreads / 32), 8, &grid);
    if (e != cudaSuccess) return e;
    return launch_clusters(narrow ? fp8_rows_kernel<T, E5, ALIGNED, true>
                                  : fp8_rows_kernel<T, E5, ALIGNED, false>,
                           1, grid, kThreads, 0, st, static_cast<const T*>(x), ld, q.R, q.K, q.counts,
                           q.E, q.codes, q.scales, per_block, q.status);
  });
}

cudaError_t launch_fp8_dequantize(const Fp8Data& q, void* y, int dtype, cudaStream_t st) {
  unsigned grid = 0;
  const cudaError_t e = grid_for(row_ctas(q.R, q.K), 8, &grid);
  if (e != cudaSuccess) return e;
  const int64_t es = dtype == BRA_FP32 ? 4 : 2;
  const bool aligned = (reinterpret_cast<uintptr_t>(y) & 15u) == 0 && q.K * es % 16 == 0;
  return by_type(dtype, q.format, aligned, [&](auto* out, auto e5, auto whole) {
    using T = std::remove_pointer_t<decltype(out)>;
    return launch_clusters(fp8_back_kernel<T, decltype(e5)::value, decltype(whole)::value>, 1, grid,
                           kThreads, 0, st, q.codes, q.scales, q.R, q.K, (uint32_t)q.each, q.counts,
                           q.E, static_cast<T*>(y), q.status);
  });
}

}  // namespace bra
