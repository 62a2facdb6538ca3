// Moving token rows to their experts and back, with the gradients.
//
//   dispatch       xs[r] = x[tokens[r]]                     (0 for -1)
//   combine        y[t]  = sum_j w[t,j] ys[slots[t,j]]      (-1: nothing)
//   dispatch grad  dx[t] = sum_j dxs[slots[t,j]]            combine with w = 1
//   combine grad   dys[slots[t,j]] = w[t,j] dy[t], dw[t,j] = <dy[t], ys[slots[t,j]]>
//
// All bound by memory: every row is read and written once.  (dispatch by
// gathering reads a token's row once for each of its experts, from L2 where it
// still is; when the tokens are too many for that, the rows of each token are
// listed first and its row is read once.)  Sums are in fp32, in the order of j
// and of a fixed tree, so results do not change from run to run; nothing is
// added atomically.
// 16384 tokens x 8 rows of 4096 bf16 values (1.2 GB a move, 2.3 the combine's
// gradient): dispatch 195 us, combine 178, their gradients 177 and 350; 6.5
// TB/s in all, 96% of a copy's rate.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "moe_internal.h"
#include "walk.cuh"

namespace bra {
namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxK = BRA_MAX_CHOICES;

// Eight elements of a row held by a lane: consecutive ones with 16-byte
// accesses (VEC), else 32 apart so that a warp's accesses stay together.
// `load` only issues the loads; `get` converts what has come.
template <typename T, bool VEC>
struct Eight {
  static constexpr int N = (int)sizeof(T) / 2;      // 16-byte accesses
  uint4 raw[N];
  __device__ __forceinline__ void load(const T* row, int base, int lane, int H) {
    if constexpr (VEC) {
      const bool in = base + lane * 8 < H;
#pragma unroll
      for (int i = 0; i < N; ++i)
        raw[i] = in ? reinterpret_cast<const uint4*>(row + base + lane * 8)[i]
                    : make_uint4(0, 0, 0, 0);
    } else {
      T* e = reinterpret_cast<T*>(raw);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int c = base + lane + 32 * i;
        e[i] = c < H ? row[c] : T(0.f);
      }
    }
  }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    const T* e = reinterpret_cast<const T*>(raw);
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = static_cast<float>(e[i]);
  }
  static __device__ __forceinline__ void store(T* row, int base, int lane, int H,
                                               const float (&f)[8]) {
    if constexpr (VEC) {
      if (base + lane * 8 >= H) return;
      uint4 w[N];
      T* e = reinterpret_cast<T*>(w);
#pragma unroll
      for (int i = 0; i < 8; ++i) e[i] = static_cast<T>(f[i]);
#pragma unroll
      for (int i = 0; i < N; ++i) reinterpret_cast<uint4*>(row + base + lane * 8)[i] = w[i];
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int c = base + lane + 32 * i;
        if (c < H) row[c] = static_cast<T>(f[i]);
      }
    }
  }
};

// Rows as `units` of sizeof(W) bytes; a warp copies 8 of its lanes' units at
// once.  The next rows' tokens are fetched meanwhile.
template <typename W>
__global__ void __launch_bounds__(kThreads)
    dispatch_kernel(const W* x, const int32_t* tokens, W* xs, uint32_t R, int64_t T, int units) {
  constexpr int U = 8;
  const int lane = threadIdx.x & 31;
  Walk at((uint32_t)(units + 32 * U - 1) / (32 * U));
  grid_wait();
  grid_go();
  int t = at.row < R ? tokens[at.row] : -1;
  while (at.row < R) {
    const uint32_t r = at.row;
    const int c0 = (int)at.part * (32 * U) + lane;
    const bool have = t >= 0 && t < T;
    const W* src = x + (int64_t)(have ? t : 0) * units;
    W v[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      v[i] = W{};
      if (have && c0 + 32 * i < units) v[i] = src[c0 + 32 * i];
    }
    at.next();
    t = at.row < R ? tokens[at.row] : -1;
    W* dst = xs + (int64_t)r * units;
#pragma unroll
    for (int i = 0; i < U; ++i)
      if (c0 + 32 * i < units) __stcs(dst + c0 + 32 * i, v[i]);
  }
}

// The rows of each token: list[t][0 .. min(count[t], kMaxK)), in any order (the
// copies they lead to are the same).  Rows of a token past kMaxK of them, and
// rows without a token, are written here, a warp to a row.
template <typename W>
__global__ void __launch_bounds__(kThreads)
    list_rows_kernel(const W* x, const int32_t* tokens, W* xs, int64_t R, int64_t T, int units,
                     int32_t* count, int32_t* list) {
  grid_wait();
  grid_go();
  const int lane = threadIdx.x & 31;
  const int64_t step = (int64_t)gridDim.x * kThreads;
  for (int64_t r0 = (int64_t)blockIdx.x * kThreads + (threadIdx.x & ~31); r0 < R; r0 += step) {
    const int64_t r = r0 + lane;
    int t = -1;
    bool rest = false;
    if (r < R) {
      t = tokens[r];
      if (t >= 0 && t < T) {
        const int at = atomicAdd(count + t, 1);
        if (at < kMaxK) list[(int64_t)t * kMaxK + at] = (int32_t)r;
        else rest = true;
      } else {
        t = -1;
        rest = true;
      }
    }
    for (uint32_t m = __ballot_sync(0xffffffffu, rest); m; m &= m - 1) {
      const int from = __ffs(m) - 1, tr = __shfl_sync(0xffffffffu, t, from);
      W* dst = xs + (r0 + from) * units;
      const W* src = x + (int64_t)(tr < 0 ? 0 : tr) * units;
      for (int c = lane; c < units; c += 32) dst[c] = tr < 0 ? W{} : src[c];
    }
  }
}

// Each token's row to the rows on its list; the next list is fetched meanwhile.
template <typename W>
__global__ void __launch_bounds__(kThreads)
    spread_kernel(const W* x, W* xs, uint32_t T, int units, const int32_t* count,
                  const int32_t* list) {
  constexpr int U = 8;
  const int lane = threadIdx.x & 31;
  Walk at((uint32_t)(units + 32 * U - 1) / (32 * U));
  grid_wait();
  grid_go();
  int n = 0, row = 0;
  auto fetch = [&] {
    n = 0;
    if (at.row >= T) return;
    n = min(count[at.row], kMaxK);
    if (lane < kMaxK) row = list[(int64_t)at.row * kMaxK + lane];   // lanes past n: unused
  };
  fetch();
  while (at.row < T) {
    const W* src = x + (int64_t)at.row * units;
    const int c0 = (int)at.part * (32 * U) + lane, my_n = n, my_row = row;
    W v[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      v[i] = W{};
      if (my_n > 0 && c0 + 32 * i < units) v[i] = src[c0 + 32 * i];
    }
    at.next();
    fetch();
    for (int j = 0; j < my_n; ++j) {
      W* dst = xs + (int64_t)__shfl_sync(0xffffffffu, my_row, j) * units;
#pragma unroll
      for (int i = 0; i < U; ++i)
        if (c0 + 32 * i < units) __stcs(dst + c0 + 32 * i, v[i]);
    }
  }
}

// y[t] = sum_j w[t,j] rows[slots[t,j]]; w NULL: ones.  A warp takes 256
// elements of a token; the rows' loads are issued eight (fp32: four) at a
// time, and the next token's slots before this one's sums.  Eight blocks to an
// SM: with a few registers more there are seven, and 16384 tokens x 8 rows of
// 4096 bf16 values take 303 us in place of 178.
template <typename T, bool VEC>
__global__ void __launch_bounds__(kThreads, VEC ? 8 : 4)
    combine_kernel(const T* rows, const int32_t* slots, const float* w, T* y, uint32_t tokens,
                   int64_t R, int k, int H) {
  constexpr int U = sizeof(T) == 4 ? 4 : 8;
  const int lane = threadIdx.x & 31;
  Walk at((uint32_t)(H + 255) / 256);
  grid_wait();
  grid_go();
  int slot = -1;
  float wt = 0.f;
  auto fetch = [&] {
    slot = -1;
    wt = 0.f;
    if (at.row < tokens && lane < k) {
      const int64_t i = (int64_t)at.row * k + lane;
      slot = slots[i];
      wt = w ? w[i] : 1.f;
    }
  };
  fetch();
  while (at.row < tokens) {
    const int64_t t = at.row;
    const int base = (int)at.part * 256;
    const int my_slot = slot >= 0 && slot < R ? slot : -1;
    const float my_w = wt;
    at.next();
    fetch();
    float s[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    for (int j0 = 0; j0 < k; j0 += U) {
      Eight<T, VEC> e[U];
      int sj[U];
#pragma unroll
      for (int j = 0; j < U; ++j) {
        sj[j] = j0 + j < k ? __shfl_sync(0xffffffffu, my_slot, (j0 + j) & 31) : -1;
        if (sj[j] >= 0) e[j].load(rows + (int64_t)sj[j] * H, base, lane, H);
      }
#pragma unroll
      for (int j = 0; j < U; ++j) {
        const float wj = __shfl_sync(0xffffffffu, my_w, (j0 + j) & 31);
        if (sj[j] >= 0) {
          float f[8];
          e[j].get(f);
#pragma unroll
          for (int i = 0; i < 8; ++i) s[i] = fmaf(wj, f[i], s[i]);
        }
      }
    }
    Eight<T, VEC>::store(y + t * H, base, lane, H, s);
  }
}

// One token to WPT warps: dys rows and the k dot products.  The block also
// zeroes its share of the rows that no token has.  Eight blocks to an SM, as
// above (488 us in place of 350 for the same rows).
template <typename T, bool VEC, int WPT>
__global__ void __launch_bounds__(kThreads, VEC && sizeof(T) == 2 ? 8 : 5)
    combine_grad_kernel(const T* dy, const T* ys, const int32_t* slots, const float* w,
                        const int32_t* row_tokens, T* dys, float* dw, int64_t tokens, int64_t R,
                        int k, int H) {
  __shared__ float part[kWarps][kMaxK];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  constexpr int TPB = kWarps / WPT;              // tokens of a block
  constexpr int U = 4;                           // rows in flight
  const int sub = warp % WPT;
  grid_wait();
  grid_go();
  for (int64_t t0 = (int64_t)blockIdx.x * TPB; t0 < tokens; t0 += (int64_t)gridDim.x * TPB) {
    const int64_t t = t0 + warp / WPT;
    if (t < tokens) {
      int slot = -1;
      float wt = 0.f;
      if (lane < k) {
        slot = slots[t * k + lane];
        if (slot < 0 || slot >= R) slot = -1;
        wt = w[t * k + lane];
      }
#pragma unroll 1
      for (int j0 = 0; j0 < k; j0 += U) {
        float dot[U] = {0.f, 0.f, 0.f, 0.f}, wj[U];
        int sj[U];
#pragma unroll
        for (int j = 0; j < U; ++j) {
          sj[j] = j0 + j < k ? __shfl_sync(0xffffffffu, slot, (j0 + j) & 31) : -1;
          wj[j] = __shfl_sync(0xffffffffu, wt, (j0 + j) & 31);
        }
        for (int base = sub * 256; base < H; base += WPT * 256) {
          Eight<T, VEC> d, e[U];
          d.load(dy + t * H, base, lane, H);       // again for the next four, from L1 or L2
#pragma unroll
          for (int j = 0; j < U; ++j)
            if (sj[j] >= 0) e[j].load(ys + (int64_t)sj[j] * H, base, lane, H);
          float dv[8];
          d.get(dv);
#pragma unroll
          for (int j = 0; j < U; ++j)
            if (sj[j] >= 0) {
              float f[8], o[8], a = 0.f;
              e[j].get(f);
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                a = fmaf(dv[i], f[i], a);
                o[i] = wj[j] * dv[i];
              }
              dot[j] += a;
              Eight<T, VEC>::store(dys + (int64_t)sj[j] * H, base, lane, H, o);
            }
        }
#pragma unroll
        for (int j = 0; j < U; ++j) {
#pragma unroll
          for (int m = 16; m > 0; m >>= 1) dot[j] += __shfl_xor_sync(0xffffffffu, dot[j], m);
          if (lane == 0 && j0 + j < k) part[warp][j0 + j] = dot[j];
        }
      }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < TPB * k; i += kThreads) {
      const int tok = i / k, j = i - tok * k;
      if (t0 + tok < tokens) {
        float a = 0.f;
#pragma unroll
        for (int q = 0; q < WPT; ++q) a += part[tok * WPT + q][j];
        dw[(t0 + tok) * k + j] = a;
      }
    }
    __syncthreads();
  }
  if (row_tokens) {
    // rows without a token (none in [0, tokens)): a warp looks at 32 rows at once
    const int64_t warps = (int64_t)gridDim.x * kWarps;
    const float z[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    for (int64_t r0 = ((int64_t)blockIdx.x * kWarps + warp) * 32; r0 < R; r0 += warps * 32) {
      const int t = r0 + lane < R ? row_tokens[r0 + lane] : 0;
      uint32_t idle = __ballot_sync(0xffffffffu, r0 + lane < R && (t < 0 || t >= tokens));
      for (; idle; idle &= idle - 1) {
        T* row = dys + (r0 + __ffs(idle) - 1) * H;
        for (int base = 0; base < H; base += 256) Eight<T, VEC>::store(row, base, lane, H, z);
      }
    }
  }
}

cudaError_t grid_of(int64_t blocks, int per_sm, unsigned* grid) {
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  const int64_t full = (int64_t)sms * per_sm;
  *grid = (unsigned)(blocks < 1 ? 1 : blocks < full ? blocks : full);
  return cudaSuccess;
}

bool aligned(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

template <typename F>
cudaError_t by_type(int dtype, bool vec, F&& f) {
  auto go = [&](auto* type) {
    return vec ? f(type, std::true_type{}) : f(type, std::false_type{});
  };
  if (dtype == BRA_FP32) return go((float*)nullptr);
  if (dtype == BRA_BF16) return go((__nv_bfloat16*)nullptr);
  return go((__half*)nullptr);
}

}  // namespace

// Whether a token's rows are listed first: there are several on average, rows
// are long enough for the lists to be little beside them, and the token rows
// do not stay in L2 between the experts' passes over them.  16384 tokens x 8,
// 8 KiB rows: 287 us gathering, 190 with lists; with 4096 tokens (32 MiB)
// gathering reads each row from memory once and is faster.
bool dispatch_lists(int64_t T, int64_t R, int64_t row_bytes) {
  return R >= 2 * T && row_bytes >= 512 && T * row_bytes >= (int64_t(48) << 20);
}

cudaError_t launch_dispatch(const PermuteCall& c, void* workspace, cudaStream_t st) {
  const int64_t bytes = (int64_t)c.H * (c.dtype == BRA_FP32 ? 4 : 2);
  auto run = [&](auto* type) {
    using W = std::remove_pointer_t<decltype(type)>;
    const int64_t units = bytes / (int64_t)sizeof(W);
    unsigned grid = 0;
    if (dispatch_lists(c.T, c.R, bytes)) {
      int32_t* list = static_cast<int32_t*>(workspace);
      int32_t* count = list + c.T * kMaxK;
      cudaError_t e = cudaMemsetAsync(count, 0, (size_t)c.T * 4, st);
      if (e == cudaSuccess) e = grid_of((c.R + kThreads - 1) / kThreads, 16, &grid);
      if (e == cudaSuccess)
        e = launch_overlapped(list_rows_kernel<W>, grid, kThreads, 0, st,
                              static_cast<const W*>(c.in), c.row_tokens, static_cast<W*>(c.out),
                              c.R, c.T, (int)units, count, list);
      if (e == cudaSuccess) e = grid_of((c.T * ((units + 255) / 256) + kWarps - 1) / kWarps, 16, &grid);
      if (e != cudaSuccess) return e;
      return launch_overlapped(spread_kernel<W>, grid, kThreads, 0, st,
                               static_cast<const W*>(c.in), static_cast<W*>(c.out), (uint32_t)c.T,
                               (int)units, count, list);
    }
    const int64_t warps = c.R * ((units + 255) / 256);
    cudaError_t e = grid_of((warps + kWarps - 1) / kWarps, 16, &grid);
    if (e != cudaSuccess) return e;
    return launch_overlapped(dispatch_kernel<W>, grid, kThreads, 0, st,
                             static_cast<const W*>(c.in), c.row_tokens, static_cast<W*>(c.out),
                             (uint32_t)c.R, c.T, (int)units);
  };
  auto fits = [&](uintptr_t n) {
    return bytes % (int64_t)n == 0 && (reinterpret_cast<uintptr_t>(c.in) & (n - 1)) == 0 &&
           (reinterpret_cast<uintptr_t>(c.out) & (n - 1)) == 0;
  };
  if (fits(16)) return run((uint4*)nullptr);
  if (fits(4)) return run((uint32_t*)nullptr);
  return run((unsigned short*)nullptr);
}

cudaError_t launch_combine(const PermuteCall& c, cudaStream_t st) {
  const bool vec = c.H % 8 == 0 && aligned(c.in) && aligned(c.out);
  unsigned grid = 0;
  const int64_t warps = c.T * ((c.H + 255) / 256);
  cudaError_t e = grid_of((warps + kWarps - 1) / kWarps, 16, &grid);
  if (e != cudaSuccess) return e;
  return by_type(c.dtype, vec, [&](auto* type, auto v) {
    using T = std::remove_pointer_t<decltype(type)>;
    return launch_overlapped(combine_kernel<T, decltype(v)::value>, grid, kThreads, 0, st,
                             static_cast<const T*>(c.in), c.slots, c.weights,
                             static_cast<T*>(c.out), (uint32_t)c.T, c.R, c.k, c.H);
  });
}

cudaError_t launch_combine_grad(const PermuteCall& c, const void* ys, float* dw, cudaStream_t st) {
  const bool vec = c.H % 8 == 0 && aligned(c.in) && aligned(c.out) && aligned(ys);
  return by_type(c.dtype, vec, [&](auto* type, auto v) {
    using T = std::remove_pointer_t<decltype(type)>;
    constexpr bool V = decltype(v)::value;
    auto run = [&](auto kernel, int tpb) {
      unsigned grid = 0;
      cudaError_t e = grid_of((c.T + tpb - 1) / tpb, 16, &grid);
      if (e != cudaSuccess) return e;
      return launch_overlapped(kernel, grid, kThreads, 0, st, static_cast<const T*>(c.in),
                               static_cast<const T*>(ys), c.slots, c.weights, c.row_tokens,
                               static_cast<T*>(c.out), dw, c.T, c.R, c.k, c.H);
    };
    return c.H >= 1024 ? run(combine_grad_kernel<T, V, 4>, 1) : run(combine_grad_kernel<T, V, 1>, 4);
  });
}

}  // namespace bra
