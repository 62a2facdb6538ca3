// Grouped products with few output tiles and a long contraction (sm_103a):
// forward with narrow outputs, weight gradients of small matrices over many
// rows.  The formulas, tiles and tail handling are grouped_tc.cu's; here a
// cluster of S = 2, 4 or 8 CTAs takes one 128 x 128 tile and splits its K
// blocks, so that a handful of tiles still occupies the SMs.  Each CTA
// accumulates its share in tensor memory and drains it to its shared memory as
// fp32; after a cluster barrier each CTA adds up 128/S rows of all S shares,
// read through the cluster's shared memory in rank order (so results do not
// change from run to run), adds the bias and rounds once.  No workspace, one
// launch.  (4 experts of 5630 rows, K = 101, N = 64: the weight gradient's four
// tiles take 14 us, 30 unsplit.)
// Bound by latency: the first loads, K blocks / S, the exchange.
#include <cstring>
#include <mutex>

#include "grouped.cuh"

namespace bra {

__device__ int32_t g_bra_fault_word_split = 0;

namespace {

using namespace tc;
using namespace grp;

constexpr int BM = 128, BN = 128, BK = 64;
constexpr int THREADS = 256;
constexpr int STAGES = 4;
constexpr int A_BYTES = BM * BK * 2, B_BYTES = BN * BK * 2;
constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
constexpr int PART_LD = BN + 4;                         // floats between rows of a share
constexpr int PART_BYTES = BM * PART_LD * 4;
constexpr int BAR_BYTES = 256;
constexpr int SMEM_BYTES =
    STAGES * STAGE_BYTES + PART_BYTES + BAR_BYTES + (int)sizeof(GroupTable) + 1024;

struct SplitParams {
  CUtensorMap ta, ta32, tb;
  const void* bias;
  void* y;
  const int64_t* counts;
  int32_t* status;
  int64_t R, ldy;
  int E, K, N;
  int m_tiles, n_tiles, k_blocks;
  int b_kmajor, aligned, late, split;
  uint32_t idesc;
};

template <typename T, bool WG>
__global__ void __launch_bounds__(THREADS, 1)
    grouped_split_kernel(const __grid_constant__ SplitParams p) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t raw_addr = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + (((raw_addr + 1023u) & ~1023u) - raw_addr);
  const uint32_t smem_base = smem_u32(smem);
  float* part = reinterpret_cast<float*>(smem + STAGES * STAGE_BYTES);
  uint8_t* bars = smem + STAGES * STAGE_BYTES + PART_BYTES;
  const uint32_t bar_base = smem_u32(bars);
  auto full_bar = [&](int s) { return bar_base + 8u * s; };
  auto empty_bar = [&](int s) { return bar_base + 8u * (STAGES + s); };
  const uint32_t tail_bar = bar_base + 8u * (2 * STAGES);
  const uint32_t tfull_bar = bar_base + 8u * (2 * STAGES + 1);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + BAR_BYTES - 16);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(bars + BAR_BYTES - 8);
  GroupTable* gt = reinterpret_cast<GroupTable*>(bars + BAR_BYTES);
  int32_t* fault = &g_bra_fault_word_split;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = (int)cluster_rank();
  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
    }
    mbar_init(tail_bar, 1);
    mbar_init(tfull_bar, 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    tma_prefetch_desc(&p.ta);
    if (!WG) tma_prefetch_desc(&p.ta32);
    tma_prefetch_desc(&p.tb);
  }
  if (warp == 2) {
    tmem_alloc<1>(smem_u32(tmem_slot), BN);
    tmem_relinquish<1>();
  }
  if (!p.late) grid_wait();
  grid_go();
  if (warp == 3) build_table<BM>(gt, p.counts, p.E, p.R, lane);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;

  // this cluster's tile, and this CTA's K blocks of it
  const int t = blockIdx.x / p.split;
  const int total = gt->bad ? 0 : (WG ? p.E * p.m_tiles : gt->tile[p.E]) * p.n_tiles;
  const bool live = t < total;
  int e = 0, mt = 0, nt = 0;
  if (live) {
    if (WG) {
      e = t / (p.m_tiles * p.n_tiles);
      mt = t / p.n_tiles % p.m_tiles;
    } else {
      while (gt->tile[e + 1] * p.n_tiles <= t) ++e;
      mt = t / p.n_tiles - gt->tile[e];
    }
    nt = t % p.n_tiles;
  }
  const int r0 = live ? gt->off[e] : 0, r1 = live ? gt->off[e + 1] : 0;
  const int rows = r1 - r0;
  const int blocks = !live ? 0 : WG ? (rows + BK - 1) / BK : p.k_blocks;
  const int kb0 = (int)((int64_t)blocks * rank / p.split);
  const int kb1 = (int)((int64_t)blocks * (rank + 1) / p.split);
  // rows of the last block, when it is this CTA's and not full
  const int tail = WG && kb1 == blocks && kb1 > kb0 ? rows % BK : 0;

  if ((warp == 0 || warp == 2) && lane == 0) {
    // ---------------- TMA producers: warp 0 for A, warp 2 for B ----------------
    const bool is_a = warp == 0;
    int stage = 0;
    uint32_t phase = 0;
    bool ok = true;
    const int row = r0 + mt * BM;                             // forward
    const int valid = r1 - row, boxes = valid <= 64 ? (max(valid, 0) + 31) / 32 : 4;
    for (int kb = kb0; kb < kb1; ++kb) {
      if (!mbar_wait(empty_bar(stage), phase ^ 1u, abort_flag, fault)) {
        ok = false;
        break;
      }
      const uint32_t a_dst = smem_base + stage * STAGE_BYTES, b_dst = a_dst + A_BYTES;
      if (WG) {
        const uint32_t bar = tail && kb + 1 == kb1 ? tail_bar : full_bar(stage);
        const CUtensorMap* m = is_a ? &p.ta : &p.tb;
        const int col = is_a ? mt * BM : nt * BN;
        if (is_a) mbar_expect_tx(bar, STAGE_BYTES);
#pragma unroll
        for (int i = 0; i < 2; ++i)
          tma_load_3d((is_a ? a_dst : b_dst) + i * 8192, m, bar, col + i * 64, r0 + kb * BK, 0);
      } else if (is_a) {
        mbar_expect_tx(full_bar(stage), boxes * (A_BYTES / 4) + B_BYTES);
        if (boxes == 4) tma_load_3d(a_dst, &p.ta, full_bar(stage), kb * BK, row, 0);
        else
          for (int i = 0; i < boxes; ++i)
            tma_load_3d(a_dst + i * (A_BYTES / 4), &p.ta32, full_bar(stage), kb * BK, row + i * 32,
                        0);
      } else if (p.b_kmajor) {
        tma_load_3d(b_dst, &p.tb, full_bar(stage), kb * BK, nt * BN, e);
      } else {
#pragma unroll
        for (int i = 0; i < 2; ++i)
          tma_load_3d(b_dst + i * 8192, &p.tb, full_bar(stage), nt * BN + i * 64, kb * BK, e);
      }
      if (++stage == STAGES) {
        stage = 0;
        phase ^= 1u;
      }
    }
    if (!ok) spin_ns(2000000ull);   // let copies already issued land
  } else if (warp == 1 && lane == 0) {
    // ---------------- MMA issuer ----------------
    const uint64_t a0 = WG ? smem_desc_sw128(smem_base, 8192, 1024)
                           : smem_desc_sw128(smem_base, 16, 1024);
    const bool bk = !WG && p.b_kmajor;
    const uint64_t b0 = bk ? smem_desc_sw128(smem_base + A_BYTES, 16, 1024)
                           : smem_desc_sw128(smem_base + A_BYTES, 8192, 1024);
    const uint32_t a_step = WG ? 128u : 2u, b_step = bk ? 2u : 128u;
    int stage = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int kb = kb0; kb < kb1; ++kb) {
      if (!mbar_wait(full_bar(stage), phase, abort_flag, fault)) {
        ok = false;
        break;
      }
      tc_fence_after();
      const uint64_t so = (uint64_t)((stage * STAGE_BYTES) >> 4);
      const int steps = tail && kb + 1 == kb1 ? (tail + 15) / 16 : BK / 16;
      for (int k = 0; k < steps; ++k)
        tc_mma<1>(tmem_base, a0 + so + a_step * k, b0 + so + b_step * k, p.idesc,
                  (kb > kb0 || k > 0) ? 1u : 0u);
      tc_commit(empty_bar(stage));
      if (++stage == STAGES) {
        stage = 0;
        phase ^= 1u;
      }
    }
    if (ok) tc_commit(tfull_bar);
    else spin_ns(2000000ull);       // let MMAs already issued complete
  } else if (WG && warp == 3 && tail) {
    // ---------------- tail rows of the group's last block ----------------
    const int s = (kb1 - 1 - kb0) % STAGES;
    const bool got = mbar_wait_sum(tail_bar, 0, abort_flag, fault, kb1 - kb0);
    if (__all_sync(0xffffffffu, got)) {
      const int stop = (tail + 15) & ~15;
      const uint32_t base = smem_base + s * STAGE_BYTES;
      for (int i = tail * 8 + lane; i < stop * 8; i += 32)
#pragma unroll
        for (int b = 0; b < 4; ++b) sts128(base + b * 8192 + i * 16, make_uint4(0, 0, 0, 0));
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) mbar_arrive(full_bar(s));
    }
  } else if (warp >= 4 && live) {
    // ---------------- this CTA's share to shared memory ----------------
    const int q = warp & 3;
    const bool none = kb1 == kb0;
    const bool waited = mbar_wait_sum(tfull_bar, 0, abort_flag, fault, kb1 - kb0);
    if (__all_sync(0xffffffffu, waited)) {
      tc_fence_after();
      float* mine = part + (q * 32 + lane) * PART_LD;
#pragma unroll 1
      for (int c = 0; c < BN; c += 32) {
        uint32_t v[32];
        tmem_ld32(tmem_base + (uint32_t)c + ((uint32_t)(q * 32) << 16), v);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 8; ++i)
          *reinterpret_cast<uint4*>(mine + c + 4 * i) =
              none ? make_uint4(0, 0, 0, 0)
                   : make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
      }
      tc_fence_before();
    }
  }

  __syncwarp();
  __syncthreads();
  cluster_sync();                   // every share is written
  if (live) {
    const int each = BM / p.split, first = rank * each;
    const int valid = min(BM, (WG ? p.K : rows) - mt * BM);
    const int64_t row = WG ? (int64_t)e * p.K + mt * BM : (int64_t)r0 + mt * BM;
    const int c = lane * 4, n = nt * BN + c;
    float bias[4] = {0.f, 0.f, 0.f, 0.f};
    if (!WG && p.bias)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (n + i < p.N) bias[i] = Num<T>::bias(p.bias, (int64_t)e * p.N + n + i);
    for (int r = first + warp; r < min(first + each, valid); r += THREADS / 32) {
      float s[4] = {0.f, 0.f, 0.f, 0.f};
      const uint32_t at = smem_u32(part + r * PART_LD + c);
      for (int k = 0; k < p.split; ++k) {
        float4 v;
        asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                     : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                     : "r"(map_to_rank(at, (uint32_t)k))
                     : "memory");
        s[0] += v.x, s[1] += v.y, s[2] += v.z, s[3] += v.w;
      }
      T* dst = static_cast<T*>(p.y) + (row + r) * p.ldy + n;
      const uint32_t lo = Out<T>::pack(s[0] + bias[0], s[1] + bias[1]);
      const uint32_t hi = Out<T>::pack(s[2] + bias[2], s[3] + bias[3]);
      if (p.aligned && n < p.N) {
        *reinterpret_cast<uint2*>(dst) = make_uint2(lo, hi);
      } else {
        uint16_t* d = reinterpret_cast<uint16_t*>(dst);
        const uint16_t w[4] = {(uint16_t)lo, (uint16_t)(lo >> 16), (uint16_t)hi,
                               (uint16_t)(hi >> 16)};
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (n + i < p.N) d[i] = w[i];
      }
    }
  }
  __syncwarp();                     // lanes past the matrix stored nothing, or element by element
  cluster_sync();                   // the peers have read this CTA's share
  if (threadIdx.x == 0 && p.status) {
    if (gt->bad) atomicExch(p.status, (int32_t)BRA_ERR_INVALID);
    else if (*abort_flag) atomicExch(p.status, (int32_t)BRA_ERR_TIMEOUT);
  }
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc<1>(tmem_base, BN);
  }
  if (p.late) grid_wait();
}

template <typename T, bool WG>
cudaError_t launch(const GroupedProblem& g, int split, int64_t tiles, cudaStream_t st) {
  static std::mutex mu;
  static bool ready[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  {
    std::lock_guard<std::mutex> lk(mu);
    if (!ready[dev & 63]) {
      e = cudaFuncSetAttribute(grouped_split_kernel<T, WG>,
                               cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_BYTES);
      if (e != cudaSuccess) return e;
      ready[dev & 63] = true;
    }
  }
  SplitParams p;
  std::memset(&p, 0, sizeof(p));
  const CUtensorMapDataType dt =
      g.dtype == BRA_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  const uint64_t K = g.K, N = g.N, R = g.R, E = g.E;
  bool ok;
  if (WG) {
    ok = encode_3d(&p.ta, dt, g.x, K, R, 1, 64, BK, g.ldx) &&
         encode_3d(&p.tb, dt, g.w, N, R, 1, 64, BK, g.ldw);
  } else {
    ok = encode_3d(&p.ta, dt, g.x, K, R, 1, BK, 128, g.ldx) &&
         encode_3d(&p.ta32, dt, g.x, K, R, 1, BK, 32, g.ldx) &&
         (g.wt ? encode_3d(&p.tb, dt, g.w, K, N, E, BK, BN, g.ldw)
               : encode_3d(&p.tb, dt, g.w, N, K, E, 64, BK, g.ldw));
  }
  if (!ok) return cudaErrorInvalidValue;
  p.bias = g.bias;
  p.y = g.y;
  p.counts = g.counts;
  p.status = g.status;
  p.R = g.R;
  p.ldy = g.ldy;
  p.E = g.E;
  p.K = g.K;
  p.N = g.N;
  p.m_tiles = (g.K + BM - 1) / BM;
  p.n_tiles = (g.N + BN - 1) / BN;
  p.k_blocks = (g.K + BK - 1) / BK;
  p.b_kmajor = g.wt;
  p.late = g.late;
  p.split = split;
  p.aligned = (reinterpret_cast<uintptr_t>(g.y) & 7u) == 0 && g.ldy % 4 == 0 && g.N % 4 == 0;
  p.idesc = make_idesc(g.dtype == BRA_BF16, BM, BN, !WG && g.wt) | (WG ? 1u << 15 : 0u);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(tiles * split), 1, 1);
  cfg.blockDim = dim3(THREADS, 1, 1);
  cfg.dynamicSmemBytes = SMEM_BYTES;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)split;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, grouped_split_kernel<T, WG>, p);
}

}  // namespace

int grouped_split(const GroupedProblem& g, bool wgrad, int64_t* tiles) {
  const int64_t groups = g.R < g.E ? g.R : g.E, nt = (g.N + BN - 1) / BN;
  *tiles = (wgrad ? (int64_t)g.E * ((g.K + BM - 1) / BM) : g.R / BM + groups) * nt;
  const int64_t blocks = (wgrad ? g.R / g.E : g.K) / BK;       // of a tile, on average
  // From 16 blocks on, at least four to a CTA: with 8 (1024 rows, 512 x 512,
  // by two) the exchange cost more than it saved, 8.4 against 6.6 us forward;
  // with 32 (2 rows, 2048 x 4096) 9.8 against 13.0, with 64 (4096 x 512, by
  // eight) 9.6 against 21.5.
  int split = 1;
  while (split < 8 && blocks >= 16 && *tiles * split * 2 <= 152 && blocks >= 4 * split * 2) split *= 2;
  return split;
}

cudaError_t launch_grouped_split(const GroupedProblem& g, bool wgrad, int split, int64_t tiles,
                                 cudaStream_t st) {
  if (wgrad)
    return g.dtype == BRA_BF16 ? launch<__nv_bfloat16, true>(g, split, tiles, st)
                               : launch<__half, true>(g, split, tiles, st);
  return g.dtype == BRA_BF16 ? launch<__nv_bfloat16, false>(g, split, tiles, st)
                             : launch<__half, false>(g, split, tiles, st);
}

cudaError_t read_split_fault_word(int32_t* code, int clear) {
  cudaError_t e = cudaMemcpyFromSymbol(code, g_bra_fault_word_split, sizeof(int32_t));
  if (e != cudaSuccess) return e;
  if (clear) {
    const int32_t z = 0;
    e = cudaMemcpyToSymbol(g_bra_fault_word_split, &z, sizeof(int32_t));
  }
  return e;
}

}  // namespace bra
