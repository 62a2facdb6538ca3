// Memory-bound companions of the grouped products: the bias gradient and the
// copy of operands whose rows TMA cannot describe.
#include "grouped.cuh"

namespace bra {
namespace {

using namespace grp;

// --------------------------------------------------------------------------
// dbias: column sums of each group's rows.  A cluster of 8 CTAs takes 64
// columns of one group and splits its rows; a thread sums 8 columns of every
// 32nd row in fp32, the CTA adds its 32 partial rows and the cluster's first
// CTA the 8 CTAs' sums, always in the same order: no atomics.
// --------------------------------------------------------------------------
constexpr int kBgThreads = 256;
constexpr int kBgSplit = 8;

template <typename T>
__device__ __forceinline__ float elt(const T* p) {
  return static_cast<float>(*p);
}

template <typename T, typename B>
__global__ void __cluster_dims__(kBgSplit, 1, 1) __launch_bounds__(kBgThreads)
    bias_grad_kernel(const T* dy, B* db, const int64_t* counts, int32_t* status, int64_t R,
                     int64_t ld, int E, int N, int vec) {
  __shared__ GroupTable gt;
  __shared__ float part[32][64];
  __shared__ float sum[64];
  const int tid = threadIdx.x;
  if (tid < 32) build_table<1>(&gt, counts, E, R, tid);
  __syncthreads();
  const uint32_t rank = cluster_rank();
  if (gt.bad) {   // the same for every CTA
    if (tid == 0 && blockIdx.x == 0 && status) atomicExch(status, (int32_t)BRA_ERR_INVALID);
    return;
  }
  const int col_tiles = (N + 63) / 64;
  const int unit = blockIdx.x / kBgSplit;
  const int e = unit / col_tiles, n0 = (unit - e * col_tiles) * 64;
  const int r0 = gt.off[e], r1 = gt.off[e + 1];
  const int64_t rows = r1 - r0;
  const int64_t a = r0 + rows * rank / kBgSplit, b = r0 + rows * (rank + 1) / kBgSplit;
  const int c = (tid & 7) * 8, rl = tid >> 3;
  float s[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  const int n = min(8, N - n0 - c);
  if (vec && n == 8) {
#pragma unroll 4
    for (int64_t r = a + rl; r < b; r += 32) {
      const uint4 w = __ldg(reinterpret_cast<const uint4*>(dy + r * ld + n0 + c));
      const T* h = reinterpret_cast<const T*>(&w);
#pragma unroll
      for (int i = 0; i < 8; ++i) s[i] += elt(h + i);
    }
  } else {
    for (int64_t r = a + rl; r < b; r += 32)
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < n) s[i] += elt(dy + r * ld + n0 + c + i);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) part[rl][c + i] = s[i];
  __syncthreads();
  if (tid < 64) {
    float t = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) t += part[i][tid];
    sum[tid] = t;
  }
  cluster_sync();
  if (rank == 0 && tid < 64 && n0 + tid < N) {
    float t = 0.f;
#pragma unroll
    for (int k = 0; k < kBgSplit; ++k) {
      float v;
      asm volatile("ld.shared::cluster.f32 %0, [%1];"
                   : "=f"(v)
                   : "r"(map_to_rank(smem_u32(&sum[tid]), (uint32_t)k))
                   : "memory");
      t += v;
    }
    db[(int64_t)e * N + n0 + tid] = static_cast<B>(t);
  }
  cluster_sync();   // the peers' sums have been read
}

// --------------------------------------------------------------------------
// Row copy: a thread makes one 16-byte chunk of the destination from the
// 32-bit words of the source that hold its elements (a funnel shift joins
// them when the row starts in a word's upper half).  Words outside the row's
// elements are not read.
// --------------------------------------------------------------------------
__global__ void __launch_bounds__(256)
    pack_rows_kernel(const uint16_t* src, int64_t ld, uint4* dst, int64_t chunks, int64_t rows,
                     int64_t len) {
  const int64_t total = rows * chunks, step = (int64_t)gridDim.x * 256;
  for (int64_t u = (int64_t)blockIdx.x * 256 + threadIdx.x; u < total; u += step) {
    const int64_t r = u / chunks, c = u - r * chunks;
    const uint16_t* s = src + r * ld + c * 8;
    const int n = (int)min((int64_t)8, len - c * 8);
    uint32_t w[4] = {0, 0, 0, 0};
    const uintptr_t at = reinterpret_cast<uintptr_t>(s);
    if (n == 8 && (at & 15) == 0) {
      const uint4 q = __ldg(reinterpret_cast<const uint4*>(s));
      w[0] = q.x, w[1] = q.y, w[2] = q.z, w[3] = q.w;
    } else if (n == 8 && (at & 3) == 0) {
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = __ldg(reinterpret_cast<const uint32_t*>(s) + i);
    } else if (n == 8) {
      uint32_t v[5];
      v[0] = (uint32_t)__ldg(s) << 16;
#pragma unroll
      for (int i = 0; i < 3; ++i) v[i + 1] = __ldg(reinterpret_cast<const uint32_t*>(s + 1) + i);
      v[4] = __ldg(s + 7);
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = __funnelshift_r(v[i], v[i + 1], 16);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < n) w[i >> 1] |= (uint32_t)__ldg(s + i) << ((i & 1) * 16);
    }
    dst[u] = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

}  // namespace

cudaError_t launch_bias_grad(const BiasGradProblem& g, cudaStream_t st) {
  const int64_t units = (int64_t)g.E * ((g.N + 63) / 64);
  if (units * kBgSplit >= (int64_t(1) << 31)) return cudaErrorInvalidValue;
  const unsigned grid = (unsigned)(units * kBgSplit);
  const int vec = (reinterpret_cast<uintptr_t>(g.dy) & 15u) == 0 && g.ld % 8 == 0;
  if (g.dtype == BRA_BF16)
    bias_grad_kernel<__nv_bfloat16, float><<<grid, kBgThreads, 0, st>>>(
        static_cast<const __nv_bfloat16*>(g.dy), static_cast<float*>(g.db), g.counts, g.status,
        g.R, g.ld, g.E, g.N, vec);
  else
    bias_grad_kernel<__half, __half><<<grid, kBgThreads, 0, st>>>(
        static_cast<const __half*>(g.dy), static_cast<__half*>(g.db), g.counts, g.status, g.R,
        g.ld, g.E, g.N, vec);
  return cudaGetLastError();
}

cudaError_t launch_pack_rows(const void* src, int64_t ld, void* dst, int64_t pitch, int64_t rows,
                             int64_t len, cudaStream_t st) {
  const int64_t chunks = pitch / 8, total = rows * chunks;
  if (total == 0) return cudaSuccess;
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  const int64_t want = (total + 255) / 256, full = (int64_t)sms * 8;
  pack_rows_kernel<<<(unsigned)(want < full ? want : full), 256, 0, st>>>(
      static_cast<const uint16_t*>(src), ld, static_cast<uint4*>(dst), chunks, rows, len);
  return cudaGetLastError();
}

}  // namespace bra
