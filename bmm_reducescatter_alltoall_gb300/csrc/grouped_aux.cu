// Memory-bound companions of the grouped products: the bias gradient and the
// copy of operands whose rows TMA cannot describe.
#include <type_traits>

#include "grouped.cuh"

namespace bra {
namespace {

using namespace grp;

// --------------------------------------------------------------------------
// dbias: column sums of each group's rows.  A unit is 64 columns of one
// group; a thread sums 8 columns of every 64th row (rows without 16-byte
// alignment: one column of every 8th) in fp32 and the CTA adds its partial
// rows, always in the same order: no atomics.  With few units a
// cluster of 8 CTAs splits a unit's rows and its first CTA adds their sums.
// Memory bound: dy is read once (16384 x 4096, 8 groups: 27 us, 4.9 TB/s).
// --------------------------------------------------------------------------
constexpr int kBgThreads = 512;
constexpr int kBgRows = kBgThreads / 8;

template <typename T, typename B, int SPLIT>
__global__ void __cluster_dims__(SPLIT, 1, 1) __launch_bounds__(kBgThreads)
    bias_grad_kernel(const T* dy, B* db, const int64_t* counts, int32_t* status, int64_t R,
                     int64_t ld, int E, int N, int vec, int late) {
  __shared__ int32_t first, past, bad;           // the group's rows
  __shared__ float part[kBgRows][64];
  __shared__ float sum[64];
  const int tid = threadIdx.x;
  if (!late) grid_wait();
  grid_go();
  const int col_tiles = (N + 63) / 64;
  const int unit = blockIdx.x / SPLIT;
  const int e = unit / col_tiles, n0 = (unit - e * col_tiles) * 64;
  if (tid < 32) {
    // one group's offset needs no table
    int64_t before = 0, mine = 0, total = 0;
    bool wrong = false;
#pragma unroll
    for (int i = 0; i < kMaxGroups / 32; ++i) {
      const int g = i * 32 + tid;
      const int64_t n = g < E ? __ldcg(reinterpret_cast<const long long*>(counts) + g) : 0;
      wrong = wrong || n < 0 || n > R;
      total += n;
      before += g < e ? n : 0;
      mine += g == e ? n : 0;
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
      before += __shfl_xor_sync(0xffffffffu, before, d);
      mine += __shfl_xor_sync(0xffffffffu, mine, d);
      total += __shfl_xor_sync(0xffffffffu, total, d);
    }
    wrong = __any_sync(0xffffffffu, wrong) || total > R;
    if (tid == 0) {
      bad = wrong ? 1 : 0;
      first = wrong ? 0 : (int32_t)before;
      past = wrong ? 0 : (int32_t)(before + mine);
    }
  }
  __syncthreads();
  const uint32_t rank = SPLIT > 1 ? cluster_rank() : 0u;
  if (bad) {   // the same for every CTA
    if (tid == 0 && blockIdx.x == 0 && status) atomicExch(status, (int32_t)BRA_ERR_INVALID);
    if (late) grid_wait();
    return;
  }
  const int r0 = first, r1 = past;
  const int64_t rows = r1 - r0;
  const int64_t a = r0 + rows * rank / SPLIT, b = r0 + rows * (rank + 1) / SPLIT;
  const int c = (tid & 7) * 8, rl = tid >> 3;
  if (vec && n0 + 64 <= N) {
    constexpr int U = 8;                       // rows in flight
    float s[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    const T* p = dy + n0 + c;
    int64_t r = a + rl;
    for (; r + (U - 1) * kBgRows < b; r += U * kBgRows) {
      uint4 w[U];
#pragma unroll
      for (int u = 0; u < U; ++u)
        w[u] = __ldcg(reinterpret_cast<const uint4*>(p + (r + u * kBgRows) * ld));
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const T* h = reinterpret_cast<const T*>(&w[u]);
#pragma unroll
        for (int i = 0; i < 8; ++i) s[i] += static_cast<float>(h[i]);
      }
    }
    for (; r < b; r += kBgRows) {
      const uint4 w = __ldcg(reinterpret_cast<const uint4*>(p + r * ld));
      const T* h = reinterpret_cast<const T*>(&w);
#pragma unroll
      for (int i = 0; i < 8; ++i) s[i] += static_cast<float>(h[i]);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) part[rl][c + i] = s[i];
    __syncthreads();
    // eight threads to a column, then their sums
    const int col = tid & 63, q = tid >> 6;
    float t = 0.f;
#pragma unroll
    for (int i = 0; i < kBgRows / 8; ++i) t += part[q * (kBgRows / 8) + i][col];
    __syncthreads();
    part[q][col] = t;
  } else {
    // rows of any alignment, or the last columns: a column to a thread
    const int col = tid & 63, q = tid >> 6;
    float t = 0.f;
    if (n0 + col < N) {
      const unsigned short* p = reinterpret_cast<const unsigned short*>(dy) + n0 + col;
#pragma unroll 16
      for (int64_t r = a + q; r < b; r += 8) {
        const unsigned short h = __ldcg(p + r * ld);
        t += static_cast<float>(*reinterpret_cast<const T*>(&h));
      }
    }
    part[q][col] = t;
  }
  __syncthreads();
  if (tid < 64) {
    float t = 0.f;
#pragma unroll
    for (int q = 0; q < 8; ++q) t += part[q][tid];
    if (SPLIT > 1) sum[tid] = t;
    else if (n0 + tid < N) db[(int64_t)e * N + n0 + tid] = static_cast<B>(t);
  }
  if (SPLIT == 1) {
    if (late) grid_wait();
    return;
  }
  __syncwarp();
  cluster_sync();
  if (rank == 0 && tid < 64 && n0 + tid < N) {
    float t = 0.f;
#pragma unroll
    for (int k = 0; k < SPLIT; ++k) {
      float v;
      asm volatile("ld.shared::cluster.f32 %0, [%1];"
                   : "=f"(v)
                   : "r"(map_to_rank(smem_u32(&sum[tid]), (uint32_t)k))
                   : "memory");
      t += v;
    }
    db[(int64_t)e * N + n0 + tid] = static_cast<B>(t);
  }
  __syncwarp();     // columns past N were left out
  cluster_sync();   // the peers' sums have been read
  if (late) grid_wait();
}

// --------------------------------------------------------------------------
// Row copy: a thread makes one 16-byte chunk of the destination from the
// 32-bit words of the source that hold its elements (a funnel shift joins
// them when the row starts in a word's upper half).  Words outside the row's
// elements are not read.
// --------------------------------------------------------------------------
__global__ void __launch_bounds__(256) pack_rows_kernel(const __grid_constant__ PackJobs jobs) {
  grid_wait();
  grid_go();
  const int64_t step = (int64_t)gridDim.x * 256;
  int64_t u = (int64_t)blockIdx.x * 256 + threadIdx.x;
  for (int j = 0; j < jobs.n; ++j) {
    const PackJob& job = jobs.job[j];
    const uint16_t* src = static_cast<const uint16_t*>(job.src);
    uint4* dst = static_cast<uint4*>(job.dst);
    const int64_t chunks = job.pitch / 8, len = job.len, ld = job.ld, total = job.rows * chunks;
    for (; u < total; u += step) {
      int64_t r;
      if (total <= 0xffffffffll) r = (uint32_t)u / (uint32_t)chunks;
      else r = u / chunks;
      const int64_t c = u - r * chunks;
      if (job.per_group > 0 && jobs.counts[r / job.per_group] == 0) continue;
      const uint16_t* s = src + r * ld + c * 8;
      const int n = (int)min((int64_t)8, len - c * 8);
      uint32_t w[4] = {0, 0, 0, 0};
      const uintptr_t at = reinterpret_cast<uintptr_t>(s);
      if (n == 8 && (at & 15) == 0) {
        const uint4 q = *reinterpret_cast<const uint4*>(s);
        w[0] = q.x, w[1] = q.y, w[2] = q.z, w[3] = q.w;
      } else if (n == 8 && (at & 3) == 0) {
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = reinterpret_cast<const uint32_t*>(s)[i];
      } else if (n == 8) {
        uint32_t v[5];
        v[0] = (uint32_t)*s << 16;
#pragma unroll
        for (int i = 0; i < 3; ++i) v[i + 1] = reinterpret_cast<const uint32_t*>(s + 1)[i];
        v[4] = s[7];
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = __funnelshift_r(v[i], v[i + 1], 16);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (i < n) w[i >> 1] |= (uint32_t)s[i] << ((i & 1) * 16);
    }
      dst[u] = make_uint4(w[0], w[1], w[2], w[3]);
    }
    u -= total;          // this thread's first chunk of the next job
  }
}

}  // namespace

cudaError_t launch_bias_grad(const BiasGradProblem& g, cudaStream_t st) {
  const int64_t units = (int64_t)g.E * ((g.N + 63) / 64);
  // Under one unit to an SM the rows are split as well; with more, the
  // clusters' barriers cost more than the balance gives (12 groups, 3063 rows,
  // N = 775, 156 units: 22 us split; 8 groups x 2048 rows x 4096, 512 units:
  // 50 split, 27 unsplit).
  const int split = units < 152 ? 8 : 1;
  if (units * split >= (int64_t(1) << 31)) return cudaErrorInvalidValue;
  const unsigned grid = (unsigned)(units * split);
  const int vec = (reinterpret_cast<uintptr_t>(g.dy) & 15u) == 0 && g.ld % 8 == 0;
  auto run = [&](auto kernel, auto* dy, auto* db) {
    using T = std::remove_pointer_t<decltype(dy)>;
    using B = std::remove_pointer_t<decltype(db)>;
    return launch_overlapped(kernel, grid, kBgThreads, 0, st, static_cast<const T*>(g.dy),
                             static_cast<B*>(g.db), g.counts, g.status, g.R, g.ld, g.E, g.N, vec,
                             g.late);
  };
  __nv_bfloat16* b = nullptr;
  __half* h = nullptr;
  float* f = nullptr;
  if (g.dtype == BRA_BF16)
    return split == 1 ? run(bias_grad_kernel<__nv_bfloat16, float, 1>, b, f)
                      : run(bias_grad_kernel<__nv_bfloat16, float, 8>, b, f);
  return split == 1 ? run(bias_grad_kernel<__half, __half, 1>, h, h)
                    : run(bias_grad_kernel<__half, __half, 8>, h, h);
}

cudaError_t launch_pack_rows(const PackJobs& jobs, cudaStream_t st) {
  int64_t total = 0;
  for (int j = 0; j < jobs.n; ++j) total += jobs.job[j].rows * (jobs.job[j].pitch / 8);
  if (total == 0) return cudaSuccess;
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  const int64_t want = (total + 255) / 256, full = (int64_t)sms * 8;
  return launch_overlapped(pack_rows_kernel, (unsigned)(want < full ? want : full), 256, 0, st, jobs);
}

}  // namespace bra
