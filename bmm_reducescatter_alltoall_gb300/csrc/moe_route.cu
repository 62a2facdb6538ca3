// The router: each token's k experts, their weights, and the order that
// sorts the (token, choice) pairs by expert.
//
//   valid_i = l_i > -inf (NaN counts as -inf, +inf as the largest float)
//   ids     = the k largest valid logits, largest first, ties to the lowest i
//   w_j     = exp(l_j - m) / sum over the valid (or, renormalised, over the
//             chosen) of exp(l - m), m the largest logit
//   row of (t, j) = rows of lower experts + earlier tokens with this expert
//
// One warp takes a token: lane l holds logits l, l + 32, ...  A choice is two
// warp reductions, of the logit as an ordered integer and of the lowest index
// that has it.  Tokens are dealt to CTAs in chunks.  In a chunk each expert
// has a bit per token, set by whoever chose it: a population count below a
// token's bit is its place among the chunk's rows of that expert, in token
// order and without any order of the setting.  The chunks' counts go to a
// small matrix; a second kernel sums the chunks before its own and the lower
// experts and writes the rows.  A single chunk does both in one launch.
// Bound by reading the logits once (4 bytes x E a token) and, for few tokens,
// by latency.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "moe_internal.h"

namespace bra {
namespace {

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
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
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  return v;
}

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
};

// One token's choice: lane j < k gets the j-th expert (-1: none) and weight.
template <typename T, int V>
__device__ __forceinline__ void choose(const RouteParams& p, int t, int lane, int* id, float* w) {
  const T* row = static_cast<const T*>(p.logits) + (int64_t)t * p.E;
  float v[V];
  uint32_t key[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const bool in = lane + 32 * i < p.E;
    v[i] = in ? logit(row + lane + 32 * i) : 0.f;
    key[i] = in ? key_of(v[i]) : 0u;
  }
  int my_id = -1;
  uint32_t my_key = 0u, top = 0u;
  for (int j = 0; j < p.k; ++j) {
    uint32_t best = key[0];
#pragma unroll
    for (int i = 1; i < V; ++i) best = max(best, key[i]);
    const uint32_t most = __reduce_max_sync(0xffffffffu, best);
    if (most == 0u) break;                       // no valid expert is left
    if (j == 0) top = most;
    uint32_t at = 0xffffffffu;
#pragma unroll
    for (int i = V - 1; i >= 0; --i)
      if (key[i] == most) at = lane + 32 * i;
    at = __reduce_min_sync(0xffffffffu, at);
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (at == (uint32_t)(lane + 32 * i)) key[i] = 0u;
    if (lane == j) {
      my_id = (int)at;
      my_key = most;
    }
  }
  const float m = value_of(top);
  const float e = my_id >= 0 ? expf(value_of(my_key) - m) : 0.f;
  float s;
  if (p.renorm) {
    s = warp_sum(e);
  } else {
    // all valid logits: those still marked, and the chosen ones
    s = e;
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (key[i]) s += expf(v[i] - m);
    s = warp_sum(s);
  }
  *id = my_id;
  *w = my_id >= 0 ? e / s : 0.f;
}

// The chunk's experts as bits: words (chunk / 32) to an expert.
__device__ __forceinline__ void clear_bits(uint32_t* bits, int n) {
  for (int i = threadIdx.x; i < n; i += kThreads) bits[i] = 0u;
}

// Rows before each expert's in this chunk: base[e], from the counts of the
// chunks before (before[e]) and of all chunks (total[e]).  Every thread.
__device__ __forceinline__ void scan_experts(const RouteParams& p, const int* total,
                                             const int* before, int* base, int* used) {
  // one warp: 16 experts a lane at most, in order
  if (threadIdx.x < 32) {
    const int lane = threadIdx.x, per = (p.E + 31) / 32;
    int s = 0;
    for (int i = 0; i < per; ++i) {
      const int e = lane * per + i;
      if (e < p.E) s += total[e];
    }
    int inc = s;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int a = __shfl_up_sync(0xffffffffu, inc, d);
      if (lane >= d) inc += a;
    }
    int at = inc - s;
    for (int i = 0; i < per; ++i) {
      const int e = lane * per + i;
      if (e < p.E) {
        base[e] = at + before[e];
        at += total[e];
      }
    }
    if (lane == 31) *used = inc;
  }
}

// Slots and tokens of the chunk's pairs, whose bits and bases are known, and
// this chunk's share of the rows that no pair has.
__device__ __forceinline__ void place(const RouteParams& p, int c, const uint32_t* bits,
                                      const int* base, int used) {
  const int words = p.chunk / 32, t0 = c * p.chunk, n = min(p.chunk, p.T - t0);
  for (int i = threadIdx.x; i < n * p.k; i += kThreads) {
    const int local = i / p.k;
    const int64_t at = (int64_t)t0 * p.k + i;
    const int e = p.ids[at];
    int slot = -1;
    if (e >= 0) {
      const uint32_t* b = bits + e * words;
      int rank = __popc(b[local >> 5] & ((1u << (local & 31)) - 1u));
      for (int w = 0; w < (local >> 5); ++w) rank += __popc(b[w]);
      slot = base[e] + rank;
      p.tokens[slot] = t0 + local;
    }
    p.slots[at] = slot;
  }
  const int64_t R = (int64_t)p.T * p.k;
  for (int64_t r = used + (int64_t)c * kThreads + threadIdx.x; r < R;
       r += (int64_t)p.chunks * kThreads)
    p.tokens[r] = -1;
}

// Choices of one chunk; with a single chunk, everything.
template <typename T, int V>
__global__ void __launch_bounds__(kThreads) route_choose_kernel(const RouteParams p) {
  extern __shared__ uint32_t bits[];                    // [E][chunk / 32]
  __shared__ int total[kMaxGroups], base[kMaxGroups], zero[kMaxGroups];
  __shared__ int used;
  const int words = p.chunk / 32, c = blockIdx.x, t0 = c * p.chunk;
  const int n = min(p.chunk, p.T - t0);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  clear_bits(bits, p.E * words);
  __syncthreads();
  for (int i = warp; i < n; i += kWarps) {
    int id;
    float w;
    choose<T, V>(p, t0 + i, lane, &id, &w);
    if (lane < p.k) {
      const int64_t at = (int64_t)(t0 + i) * p.k + lane;
      p.ids[at] = id;
      p.weights[at] = w;
      if (id >= 0) atomicOr(&bits[id * words + (i >> 5)], 1u << (i & 31));
    }
  }
  __syncthreads();
  for (int e = threadIdx.x; e < p.E; e += kThreads) {
    int s = 0;
    for (int w = 0; w < words; ++w) s += __popc(bits[e * words + w]);
    if (p.chunks > 1) {
      p.hist[(int64_t)c * p.E + e] = s;
    } else {
      total[e] = s;
      zero[e] = 0;
      p.counts[e] = s;
    }
  }
  if (p.chunks > 1) return;
  __syncthreads();
  scan_experts(p, total, zero, base, &used);
  __syncthreads();
  place(p, 0, bits, base, used);
}

// Rows of one chunk, from the counts of all of them.
__global__ void __launch_bounds__(kThreads) route_place_kernel(const RouteParams p) {
  extern __shared__ uint32_t bits[];
  __shared__ int total[kMaxGroups], before[kMaxGroups], base[kMaxGroups];
  __shared__ int used;
  const int words = p.chunk / 32, c = blockIdx.x, t0 = c * p.chunk;
  const int n = min(p.chunk, p.T - t0);
  clear_bits(bits, p.E * words);
  for (int e = threadIdx.x; e < p.E; e += kThreads) total[e] = before[e] = 0;
  __syncthreads();
  // threads of a row of the matrix side by side, rows dealt over the rest
  const int width = (p.E + 31) / 32 * 32, rows = kThreads / width;
  const int e = threadIdx.x % width, r0 = threadIdx.x / width;
  if (e < p.E && r0 < rows) {
    int all = 0, old = 0;
#pragma unroll 4
    for (int r = r0; r < p.chunks; r += rows) {
      const int h = p.hist[(int64_t)r * p.E + e];
      all += h;
      old += r < c ? h : 0;
    }
    atomicAdd(&total[e], all);
    atomicAdd(&before[e], old);
  }
  for (int i = threadIdx.x; i < n * p.k; i += kThreads) {
    const int id = p.ids[(int64_t)t0 * p.k + i], local = i / p.k;
    if (id >= 0) atomicOr(&bits[id * words + (local >> 5)], 1u << (local & 31));
  }
  __syncthreads();
  scan_experts(p, total, before, base, &used);
  if (c == 0)
    for (int i = threadIdx.x; i < p.E; i += kThreads) p.counts[i] = total[i];
  __syncthreads();
  place(p, c, bits, base, used);
}

// --------------------------------------------------------------------------
// Gradient of the logits: with g the gradient of the weights and s = sum w g,
//   renormalised:  dl_i = w_j (g_j - s) for the chosen i = id_j, else 0
//   otherwise:     dl_i = p_i ([i = id_j] g_j - s), p the softmax
// --------------------------------------------------------------------------
struct RouteGradParams {
  const float* dweights;
  const void* logits;
  const int32_t* ids;
  const float* weights;
  void* dlogits;
  int T, E, k, renorm;
};

template <typename T>
__device__ __forceinline__ T rounded(float v) {
  return static_cast<T>(v);
}

template <typename T, int V>
__global__ void __launch_bounds__(256) route_grad_kernel(const RouteGradParams p) {
  const int lane = threadIdx.x & 31;
  const int warps = gridDim.x * 8;
  for (int t = blockIdx.x * 8 + (threadIdx.x >> 5); t < p.T; t += warps) {
    int id = -1;
    float w = 0.f, g = 0.f;
    if (lane < p.k) {
      const int64_t at = (int64_t)t * p.k + lane;
      id = p.ids[at];
      if (id >= 0) {
        w = p.weights[at];
        g = p.dweights[at];
      }
    }
    const float s = warp_sum(w * g);
    float d[V];
#pragma unroll
    for (int i = 0; i < V; ++i) d[i] = 0.f;
    if (p.renorm) {
      const float mine = w * (g - s);
      for (int j = 0; j < p.k; ++j) {
        const int at = __shfl_sync(0xffffffffu, id, j);
        const float dj = __shfl_sync(0xffffffffu, mine, j);
#pragma unroll
        for (int i = 0; i < V; ++i)
          if (at == lane + 32 * i) d[i] = dj;
      }
    } else {
      const T* row = static_cast<const T*>(p.logits) + (int64_t)t * p.E;
      float v[V];
      uint32_t best = 0u;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        v[i] = lane + 32 * i < p.E ? logit(row + lane + 32 * i) : -INFINITY;
        best = max(best, key_of(v[i]));
      }
      const uint32_t top = __reduce_max_sync(0xffffffffu, best);
      const float m = value_of(top);
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        v[i] = key_of(v[i]) ? expf(v[i] - m) : 0.f;
        sum += v[i];
      }
      sum = warp_sum(sum);
      const float inv = sum > 0.f ? 1.f / sum : 0.f;
#pragma unroll
      for (int i = 0; i < V; ++i) d[i] = -s;
      for (int j = 0; j < p.k; ++j) {
        const int at = __shfl_sync(0xffffffffu, id, j);
        const float gj = __shfl_sync(0xffffffffu, g, j);
#pragma unroll
        for (int i = 0; i < V; ++i)
          if (at == lane + 32 * i) d[i] = gj - s;
      }
#pragma unroll
      for (int i = 0; i < V; ++i) d[i] *= v[i] * inv;
    }
    T* out = static_cast<T*>(p.dlogits) + (int64_t)t * p.E;
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (lane + 32 * i < p.E) out[lane + 32 * i] = rounded<T>(d[i]);
  }
}

// Calls f.template operator()<T, V>() for the logits' type and E.
template <typename F>
cudaError_t by_type(int dtype, int E, F&& f) {
  auto by_width = [&](auto* type) {
    if (E <= 32) return f(type, std::integral_constant<int, 1>{});
    if (E <= 64) return f(type, std::integral_constant<int, 2>{});
    if (E <= 128) return f(type, std::integral_constant<int, 4>{});
    if (E <= 256) return f(type, std::integral_constant<int, 8>{});
    return f(type, std::integral_constant<int, 16>{});
  };
  if (dtype == BRA_FP32) return by_width((float*)nullptr);
  if (dtype == BRA_BF16) return by_width((__nv_bfloat16*)nullptr);
  return by_width((__half*)nullptr);
}

}  // namespace

// Tokens of a chunk: one chunk up to 64 tokens (one launch); else about 128
// chunks, of at most 1024 tokens.
int route_chunk(int64_t T) {
  if (T <= 64) return 64;
  const int64_t c = ((T + 127) / 128 + 31) / 32 * 32;
  return (int)(c > 1024 ? 1024 : c);
}

cudaError_t launch_route(const RouteCall& r, cudaStream_t st) {
  RouteParams p = {r.logits, r.ids,   r.weights, r.counts, r.slots, r.tokens, r.hist, (int)r.T,
                   r.E,      r.k,     r.renorm,  route_chunk(r.T), 0};
  p.chunks = (int)((r.T + p.chunk - 1) / p.chunk);
  const int smem = r.E * (p.chunk / 32) * 4;
  const cudaError_t e = by_type(r.dtype, r.E, [&](auto* type, auto v) {
    using T = std::remove_pointer_t<decltype(type)>;
    if (smem > 32768) {
      const cudaError_t a =
          cudaFuncSetAttribute(route_choose_kernel<T, decltype(v)::value>,
                               cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
      if (a != cudaSuccess) return a;
    }
    route_choose_kernel<T, decltype(v)::value><<<p.chunks, kThreads, smem, st>>>(p);
    return cudaGetLastError();
  });
  if (e != cudaSuccess || p.chunks == 1) return e;
  if (smem > 32768) {
    const cudaError_t a = cudaFuncSetAttribute(
        route_place_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (a != cudaSuccess) return a;
  }
  route_place_kernel<<<p.chunks, kThreads, smem, st>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_route_grad(const RouteGradCall& r, cudaStream_t st) {
  const RouteGradParams p = {r.dweights, r.logits, r.ids, r.weights, r.dlogits,
                             (int)r.T,   r.E,      r.k,   r.renorm};
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  const int64_t want = (r.T + 7) / 8, full = (int64_t)sms * 8;
  const unsigned grid = (unsigned)(want < full ? want : full);
  return by_type(r.dtype, r.E, [&](auto* type, auto v) {
    using T = std::remove_pointer_t<decltype(type)>;
    route_grad_kernel<T, decltype(v)::value><<<grid, 256, 0, st>>>(p);
    return cudaGetLastError();
  });
}

}  // namespace bra
