// What the routers share: logits as ordered integers, a chunk's experts as
// bits, and the places of its rows.  moe_route.cu describes the scheme.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "moe_internal.h"

namespace bra {

// Chunk, chunks and scanned of p, for its T; the launches after the choices.
struct RouteParams;
void route_chunks(RouteParams* p);
cudaError_t launch_route_places(const RouteParams& p, cudaStream_t st);

namespace route {

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kMostChunk = 1024;          // most tokens of a chunk
constexpr float kLargest = 3.402823466e+38f;

template <typename T>
__device__ __forceinline__ float logit(const T* p) {
  const float v = static_cast<float>(*p);
  // NaN stays NaN; +0 for -0, so that equal logits are equal as integers
  return (v > kLargest ? kLargest : v) + 0.0f;
}
// Order of floats as unsigned integers; 0 for -inf and NaN: not a choice.
__device__ __forceinline__ uint32_t key_of(float v) {
  const uint32_t u = __float_as_uint(v);
  return v >= -kLargest ? (u & 0x80000000u ? ~u : u | 0x80000000u) : 0u;
}
__device__ __forceinline__ float value_of(uint32_t key) {
  return __uint_as_float(key & 0x80000000u ? key & 0x7fffffffu : ~key);
}
}  // namespace route

struct RouteParams {
  const void* logits;
  int32_t* ids;        // [T][k]
  float* weights;      // [T][k]
  int64_t* counts;     // [E]
  int32_t* slots;      // [T][k]
  int32_t* tokens;     // [T*k]
  int32_t* hist;       // [chunks][E], unless there is one chunk
  int T, E, k, renorm;
  int chunk, chunks;   // tokens of a chunk (a multiple of 32)
  int vec;             // logits' rows are read four at a time
  int scanned;         // hist holds sums over the chunks up to each one
};

namespace route {

__device__ __forceinline__ float group_sum(float v, int L) {
  for (int d = L / 2; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  return v;
}

// Sorts eight (key, index) pairs, largest key first, equal keys by index:
// Batcher's odd-even merge sort, 19 exchanges.
__device__ __forceinline__ void sort_eight(uint32_t (&key)[8], int (&idx)[8]) {
  auto put = [&](int a, int b) {
    const bool swap = key[b] > key[a] || (key[b] == key[a] && idx[b] < idx[a]);
    const uint32_t ka = swap ? key[b] : key[a], kb = swap ? key[a] : key[b];
    const int ia = swap ? idx[b] : idx[a], ib = swap ? idx[a] : idx[b];
    key[a] = ka, key[b] = kb, idx[a] = ia, idx[b] = ib;
  };
  put(0, 1), put(2, 3), put(4, 5), put(6, 7);
  put(0, 2), put(1, 3), put(4, 6), put(5, 7);
  put(1, 2), put(5, 6);
  put(0, 4), put(1, 5), put(2, 6), put(3, 7);
  put(2, 4), put(3, 5);
  put(1, 2), put(3, 4), put(5, 6);
}

// Words from one expert's bits to the next: odd, so that the same word of
// different experts lies in different banks (1024 tokens a chunk, 32 words
// apart: 262144 tokens, 8 of 128, 257 us in place of 130).
__host__ __device__ constexpr int bit_stride(int chunk) { return (chunk / 32) | 1; }

// The chunk's experts as bits: chunk / 32 words to an expert.
__device__ __forceinline__ void clear_bits(uint32_t* bits, int n) {
  for (int i = threadIdx.x; i < n; i += kThreads) bits[i] = 0u;
}

// Rows before each expert's in this chunk: base[e], from the counts of the
// chunks before (before[e]) and of all chunks (total[e]).  Every thread; ends
// with a barrier.
__device__ __forceinline__ void scan_experts(const RouteParams& p, const int* total,
                                             const int* before, int* base, int* used) {
  __shared__ int sums[kMaxGroups / 32];
  const int e = threadIdx.x, lane = e & 31;
  int n = 0, inc = 0;
  if (e < kMaxGroups) {
    n = e < p.E ? total[e] : 0;
    inc = n;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int a = __shfl_up_sync(0xffffffffu, inc, d);
      if (lane >= d) inc += a;
    }
    if (lane == 31) sums[e >> 5] = inc;
  }
  __syncthreads();
  if (e < kMaxGroups) {
    int at = inc - n;
    for (int w = 0; w < (e >> 5); ++w) at += sums[w];
    if (e < p.E) base[e] = at + before[e];
    if (e == kMaxGroups - 1) *used = at + n;
  }
  __syncthreads();
}

// This chunk's share of the rows that no pair has.
__device__ __forceinline__ void mark_unused(const RouteParams& p, int c, int used) {
  const int64_t R = (int64_t)p.T * p.k;
  for (int64_t r = used + (int64_t)c * kThreads + threadIdx.x; r < R;
       r += (int64_t)p.chunks * kThreads)
    p.tokens[r] = -1;
}

// Choices of one chunk, by `choose` (token, lane, bits' stride, word and bit:
// whole warps), and each pair's place among the chunk's rows of its expert in
// `slots`; with a single chunk, everything.  L lanes take a token; the bits are
// clear.
template <int L, typename Choose>
__device__ __forceinline__ void route_chunk_of(const RouteParams& p, uint32_t* bits,
                                               Choose&& choose) {
  __shared__ int total[kMaxGroups], base[kMaxGroups], zero[kMaxGroups];
  __shared__ int used;
  const int words = p.chunk / 32, stride = bit_stride(p.chunk), c = blockIdx.x, t0 = c * p.chunk;
  const int n = min(p.chunk, p.T - t0);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int G = 32 / L;                             // tokens of a warp
  for (int i0 = warp * G; i0 < n; i0 += kWarps * G) {
    const int i = i0 + lane / L;
    choose(i < n ? t0 + i : -1, lane, stride, i >> 5, 1u << (i & 31));
  }
  __syncthreads();
  for (int e = threadIdx.x; e < p.E; e += kThreads) {
    int s = 0;
    for (int w = 0; w < words; ++w) s += __popc(bits[e * stride + w]);
    if (p.chunks > 1) {
      p.hist[(int64_t)c * p.E + e] = s;
    } else {
      total[e] = s;
      zero[e] = 0;
      p.counts[e] = s;
    }
  }
  if (p.chunks == 1) {
    __syncthreads();
    scan_experts(p, total, zero, base, &used);
    mark_unused(p, 0, used);
  }
  for (int i = threadIdx.x; i < n * p.k; i += kThreads) {
    const int local = i / p.k;
    const int64_t at = (int64_t)t0 * p.k + i;
    const int e = p.ids[at];
    int slot = -1;
    if (e >= 0) {
      const uint32_t* b = bits + e * stride;
      slot = __popc(b[local >> 5] & ((1u << (local & 31)) - 1u));
      for (int w = 0; w < (local >> 5); ++w) slot += __popc(b[w]);
      if (p.chunks == 1) {
        slot += base[e];
        p.tokens[slot] = local;
      }
    }
    p.slots[at] = slot;
  }
}

// Whether rows of E elements can be read four at a time.
inline int rows_vec(const void* p, int E, int dtype) {
  return E % 4 == 0 && (reinterpret_cast<uintptr_t>(p) & (dtype == BRA_FP32 ? 15u : 7u)) == 0;
}

}  // namespace route
}  // namespace bra
