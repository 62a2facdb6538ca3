// Products grouped by expert with ragged row groups, on tcgen05 (sm_103a).
//
//   forward  y[r,:]  = x[r,:] W_e + b_e     for the rows r of group e
//   wgrad    dW_e    = x_e^T dy_e           (zero for an empty group)
//
// (the gradient of x is the forward form with the weight read the other way).
// The group sizes are on the device.  Every CTA builds the table of group
// offsets and row tiles in shared memory (grouped.cuh) and walks the same
// static tile list, so one launch covers all groups with no host sync.
//
// Tiles are 128*CG rows x BN columns with a K loop of 64, one CTA (CG = 1) or
// a CTA pair (CG = 2, tcgen05.mma.cta_group::2) per tile; roles as in
// fused_tc2.cu: a TMA producer, an MMA issuer, four epilogue warps on
// alternating accumulators.  What is ragged:
//   forward: a tile's rows start at any row (a TMA row coordinate has no
//     alignment rule).  Rows past the group belong to the next group: they
//     are computed and not stored, as an accumulator row depends on its own
//     operand row alone.  At most 64 valid rows are fetched as 32-row boxes,
//     so that a decoding batch's tiles move little beside the weights; operand
//     rows that were not fetched hold whatever the stage held before.
//   wgrad: the K loop runs over the group's rows, 64 at a time; both operands
//     are read transposed (M- and N-major boxes of 64 columns x 64 rows).  In
//     a group's last block the rows past its end must add nothing, and zero
//     times another group's infinity would: warp 3 zeroes them in both
//     operands (a box row is 128 bytes of shared memory, whatever the
//     swizzle), up to the next multiple of 16, where the block's MMAs stop.
//     Its tiles cost as many blocks as the group has rows, so the groups are
//     walked largest first: a long tile begun last would be waited for alone
//     (32 experts of 1300 to 13000 rows, K = N = 1024: 134 us in the groups'
//     own order, 92 for equal ones).
// With many rows the tensor cores bound it: bf16, 8 x 2048 rows, K = 2048, N =
// 4096, 151 us forward and for the weight gradient (1820 TFLOP/s; cuBLAS's
// batched product of equal groups 1945).  With few, the weights' bytes: 128
// rows over 64 experts, 140 us for 949 MB, the rate of a copy.
// Every wait is bounded (about 4 s, those for a whole group's sum by its size
// as well) and reports through the fault word.
#include <cstring>
#include <mutex>

#include "grouped.cuh"

namespace bra {

__device__ int32_t g_bra_fault_word_grouped = 0;

namespace {

using namespace tc;
using namespace grp;

constexpr int BK = 64;
constexpr int kGroupM = 8;                  // raster: row tiles of a super-row
constexpr int THREADS = 256;                // 4 role warps, 4 epilogue warps
constexpr int EPI_WARP0 = 4;
constexpr int BAR_BYTES = 512;

struct GroupedParams {
  CUtensorMap ta;      // forward: x, boxes of 128 rows; wgrad: x, 64 x 64 boxes
  CUtensorMap ta32;    // forward: x, boxes of 32 rows
  CUtensorMap tb;      // forward: weights; wgrad: dy, 64 x 64 boxes
  const void* bias;
  void* y;
  const int64_t* counts;
  int32_t* status;
  int64_t R, ldy;
  int E, K, N;
  int m_tiles, n_tiles, k_blocks;   // wgrad: row tiles of K; forward: K blocks
  int b_kmajor, aligned, late;
  uint32_t idesc;
};

template <int CG, int BN>
struct GShape {
  static constexpr int A_BYTES = 128 * BK * 2;
  static constexpr int B_COLS = BN / CG;                 // columns held by one CTA
  static constexpr int B_BYTES = B_COLS * BK * 2;
  static constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
  static constexpr int EPI_BYTES = 4 * (kSegBytes + BN * 4);
  static constexpr int FIXED =
      BAR_BYTES + EPI_BYTES + (int)sizeof(GroupTable) + kMaxGroups * 2 + 16 + 1024;
  static constexpr int FIT = (232448 - FIXED) / STAGE_BYTES;
  static constexpr int STAGES = FIT > 8 ? 8 : FIT;
  static constexpr int SMEM_BYTES = STAGES * STAGE_BYTES + FIXED;
  static constexpr uint32_t TMEM_COLS = 2 * BN;
  static_assert(STAGES >= 4, "ring");
};

// One tile of the walk.
struct Tile {
  int e, mt, nt;
};

template <bool WG>
__device__ __forceinline__ Tile find_tile(const GroupedParams& p, const GroupTable* gt,
                                          const uint16_t* order, int t, int& e_hint) {
  Tile r;
  if (WG) {
    const TileCoord c = tile_coord(t, p.m_tiles, p.n_tiles, kGroupM);
    r.e = order[c.g];
    r.mt = c.mt;
    r.nt = c.nt;
  } else {
    // t only grows along a CTA's walk: go on from the last group
    int e = e_hint;
    while (gt->tile[e + 1] * p.n_tiles <= t) ++e;
    e_hint = e;
    const int first = gt->tile[e];
    const TileCoord c =
        tile_coord(t - first * p.n_tiles, gt->tile[e + 1] - first, p.n_tiles, kGroupM);
    r.e = e;
    r.mt = c.mt;
    r.nt = c.nt;
  }
  return r;
}

template <typename T, int CG, int BN, bool WG>
__global__ void __cluster_dims__(CG, 1, 1) __launch_bounds__(THREADS, 1)
    grouped_kernel(const __grid_constant__ GroupedParams p) {
  using S = GShape<CG, BN>;
  constexpr int STAGES = S::STAGES, STAGE_BYTES = S::STAGE_BYTES, A_BYTES = S::A_BYTES;
  constexpr int BM = 128 * CG;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t raw_addr = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + (((raw_addr + 1023u) & ~1023u) - raw_addr);
  const uint32_t smem_base = smem_u32(smem);
  uint8_t* bars = smem + STAGES * STAGE_BYTES;
  const uint32_t bar_base = smem_u32(bars);
  // barriers (8 bytes each): full, empty, tail and ptail (wgrad) per stage; tfull[2], tempty[2]
  auto full_bar = [&](int s) { return bar_base + 8u * s; };
  auto empty_bar = [&](int s) { return bar_base + 8u * (STAGES + s); };
  auto tail_bar = [&](int s) { return bar_base + 8u * (2 * STAGES + s); };
  auto ptail_bar = [&](int s) { return bar_base + 8u * (3 * STAGES + s); };
  auto tfull_bar = [&](int a) { return bar_base + 8u * (4 * STAGES + a); };
  auto tempty_bar = [&](int a) { return bar_base + 8u * (4 * STAGES + 2 + a); };
  static_assert(8 * (4 * STAGES + 4) + 16 <= BAR_BYTES, "barrier area");
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + BAR_BYTES - 16);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(bars + BAR_BYTES - 8);
  GroupTable* gt = reinterpret_cast<GroupTable*>(bars + BAR_BYTES);
  uint16_t* order = reinterpret_cast<uint16_t*>(gt + 1);       // wgrad: groups, largest first
  uint8_t* epi = bars + BAR_BYTES + ((sizeof(GroupTable) + kMaxGroups * 2 + 15) & ~15);
  int32_t* fault = &g_bra_fault_word_grouped;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = CG == 2 ? cluster_rank() : 0u;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(full_bar(s), 1);     // leader: its expect_tx; the bytes of both CTAs
      mbar_init(empty_bar(s), 1);
      mbar_init(tail_bar(s), 1);     // this CTA's copies of a tail block
      mbar_init(ptail_bar(s), 1);    // leader: the peer's tail block is ready
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(tfull_bar(a), 1);
      mbar_init(tempty_bar(a), 4 * CG);
    }
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    tma_prefetch_desc(&p.ta);
    if (!WG) tma_prefetch_desc(&p.ta32);
    tma_prefetch_desc(&p.tb);
  }
  if (warp == 2) {
    tmem_alloc<CG>(smem_u32(tmem_slot), S::TMEM_COLS);
    tmem_relinquish<CG>();
  }
  if (!p.late) grid_wait();
  grid_go();
  if (warp == 3) build_table<BM>(gt, p.counts, p.E, p.R, lane);
  tc_fence_before();
  __syncthreads();
  if (WG) {
    for (int e = threadIdx.x; e < p.E; e += THREADS) {
      const int n = gt->off[e + 1] - gt->off[e];
      int at = 0;
      for (int i = 0; i < p.E; ++i) {
        const int m = gt->off[i + 1] - gt->off[i];
        at += m > n || (m == n && i < e);
      }
      order[at] = (uint16_t)e;
    }
    __syncthreads();
  }
  if (CG == 2) cluster_sync();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const int total = gt->bad ? 0 : (WG ? p.E * p.m_tiles : gt->tile[p.E]) * p.n_tiles;
  // This cluster's tile of each round over the clusters.  wgrad: largest first,
  // every second round backwards, so that who began with a long tile goes on
  // with a short one.
  const int walk0 = blockIdx.x / CG, step = gridDim.x / CG;
  const int rounds = (total + step - 1) / step;
  auto tile_at = [&](int round) {
    return round * step + (WG && (round & 1) ? step - 1 - walk0 : walk0);
  };

  if ((warp == 0 || warp == 2) && lane == 0) {
    // ---------------- TMA producers (every CTA): warp 0 for A, warp 2 for B ----------------
    // One thread issuing a block's four boxes was the bound of the weight
    // gradient (1345 against 1650 TFLOP/s with fewer instructions a box).
    const bool is_a = warp == 0;
    const uint32_t leader_full0 = CG == 2 ? map_to_rank(full_bar(0), 0) : full_bar(0);
    const uint32_t own_tail0 = CG == 2 ? map_to_rank(tail_bar(0), rank) : tail_bar(0);
    int stage = 0, hint = 0;
    uint32_t phase = 0;
    bool ok = true;
    auto next = [&] {
      if (++stage == STAGES) {
        stage = 0;
        phase ^= 1u;
      }
    };
    auto load = [&](uint32_t dst, const CUtensorMap* m, uint32_t bar, int c0, int c1, int c2) {
      if (CG == 2) tma_load_3d_pair(dst, m, bar, c0, c1, c2);
      else tma_load_3d(dst, m, bar, c0, c1, c2);
    };
    for (int round = 0; ok && round < rounds; ++round) {
      const int t = tile_at(round);
      if (t >= total) break;
      const Tile c = find_tile<WG>(p, gt, order, t, hint);
      const int r0 = gt->off[c.e], r1 = gt->off[c.e + 1];
      const int a_row = c.mt * BM + (int)rank * 128;            // of the output
      const int b_col = c.nt * BN + (int)rank * S::B_COLS;
      if (WG) {
        for (int row = r0; row < r1; row += BK) {
          if (!mbar_wait(empty_bar(stage), phase ^ 1u, abort_flag, fault)) {
            ok = false;
            break;
          }
          const uint32_t a_dst = smem_base + stage * STAGE_BYTES, b_dst = a_dst + A_BYTES;
          const bool tail = r1 - row < BK;     // this CTA's own barrier: warp 3 passes it on
          const uint32_t bar = (tail ? own_tail0 : leader_full0) + 8u * stage;
          if (is_a) {
            // only the leader arrives on a full barrier: a remote arrive of the peer for
            // each block (release at cluster scope) held the pair to 790 TFLOP/s
            if (tail) mbar_expect_tx(tail_bar(stage), STAGE_BYTES);
            else if (rank == 0) mbar_expect_tx(full_bar(stage), CG * STAGE_BYTES);
#pragma unroll
            for (int i = 0; i < 2; ++i)
              load(a_dst + i * 8192, &p.ta, bar, a_row + i * 64, row, 0);
          } else {
#pragma unroll
            for (int i = 0; i < S::B_COLS / 64; ++i)
              load(b_dst + i * 8192, &p.tb, bar, b_col + i * 64, row, 0);
          }
          next();
        }
      } else {
        const int row = r0 + a_row;
        // 32-row boxes of A to fetch (none past the group), or one of 128 rows
        auto boxes = [&](int valid) { return valid <= 64 ? (max(valid, 0) + 31) / 32 : 4; };
        const int mine = boxes(r1 - row);
        uint32_t bytes = CG * S::B_BYTES + mine * (A_BYTES / 4);
        if (CG == 2) bytes += boxes(r1 - row - 128) * (A_BYTES / 4);   // used by the leader
        for (int kb = 0; kb < p.k_blocks; ++kb) {
          if (!mbar_wait(empty_bar(stage), phase ^ 1u, abort_flag, fault)) {
            ok = false;
            break;
          }
          const uint32_t fb = leader_full0 + 8u * stage;
          const uint32_t a_dst = smem_base + stage * STAGE_BYTES, b_dst = a_dst + A_BYTES;
          if (is_a) {
            if (rank == 0) mbar_expect_tx(full_bar(stage), bytes);
            if (mine == 4) load(a_dst, &p.ta, fb, kb * BK, row, 0);
            else
              for (int i = 0; i < mine; ++i)
                load(a_dst + i * (A_BYTES / 4), &p.ta32, fb, kb * BK, row + i * 32, 0);
          } else if (p.b_kmajor) {
            load(b_dst, &p.tb, fb, kb * BK, b_col, c.e);
          } else {
#pragma unroll
            for (int i = 0; i < S::B_COLS / 64; ++i)
              load(b_dst + i * 8192, &p.tb, fb, b_col + i * 64, kb * BK, c.e);
          }
          next();
        }
      }
    }
    if (!ok) spin_ns(2000000ull);   // let copies already issued land
  } else if (warp == 1 && lane == 0 && rank == 0) {
    // ---------------- MMA issuer (leader only) ----------------
    // K-major operands step 32 bytes per K = 16, transposed ones 16 box rows
    const uint64_t a0 = WG ? smem_desc_sw128(smem_base, 8192, 1024)
                           : smem_desc_sw128(smem_base, 16, 1024);
    const bool bk = !WG && p.b_kmajor;
    const uint64_t b0 = bk ? smem_desc_sw128(smem_base + A_BYTES, 16, 1024)
                           : smem_desc_sw128(smem_base + A_BYTES, 8192, 1024);
    const uint32_t a_step = WG ? 128u : 2u, b_step = bk ? 2u : 128u;
    int stage = 0, acc = 0, hint = 0;
    uint32_t phase = 0, acc_phase = 0, pused = 0;
    bool ok = true;
    auto next = [&] {
      if (CG == 2) tc_commit_pair(empty_bar(stage), 0x3);
      else tc_commit(empty_bar(stage));
      if (++stage == STAGES) {
        stage = 0;
        phase ^= 1u;
      }
    };
    for (int round = 0; ok && round < rounds; ++round) {
      const int t = tile_at(round);
      if (t >= total) break;
      int full = p.k_blocks, tail = 0;     // whole blocks, rows of a last one
      if (WG) {
        const Tile c = find_tile<WG>(p, gt, order, t, hint);
        const int n = gt->off[c.e + 1] - gt->off[c.e];
        full = n / BK;
        tail = n % BK;
      }
      if (!mbar_wait(tempty_bar(acc), acc_phase ^ 1u, abort_flag, fault)) break;
      tc_fence_after();
      const uint32_t d_tmem = tmem_base + (uint32_t)(acc * BN);
      // the last block's wait and shorter MMA run are outside this loop: with
      // them inside, the issuing thread fell behind (1650 against 1730 TFLOP/s)
      for (int kb = 0; kb < full; ++kb) {
        if (!mbar_wait(full_bar(stage), phase, abort_flag, fault)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint64_t so = (uint64_t)((stage * STAGE_BYTES) >> 4);
#pragma unroll
        for (int k = 0; k < BK / 16; ++k)
          tc_mma<CG>(d_tmem, a0 + so + a_step * k, b0 + so + b_step * k, p.idesc,
                     (kb > 0 || k > 0) ? 1u : 0u);
        next();
      }
      if (WG && ok && tail) {
        ok = mbar_wait(full_bar(stage), phase, abort_flag, fault);
        if (CG == 2 && ok) {
          ok = mbar_wait_acq(ptail_bar(stage), (pused >> stage) & 1u, abort_flag, fault);
          pused ^= 1u << stage;
        }
        if (ok) {
          tc_fence_after();
          const uint64_t so = (uint64_t)((stage * STAGE_BYTES) >> 4);
          for (int k = 0; k * 16 < tail; ++k)
            tc_mma<CG>(d_tmem, a0 + so + a_step * k, b0 + so + b_step * k, p.idesc,
                       (full > 0 || k > 0) ? 1u : 0u);
          next();
        }
      }
      if (!ok) break;
      if (CG == 2) tc_commit_pair(tfull_bar(acc), 0x3);
      else tc_commit(tfull_bar(acc));
      if (++acc == 2) {
        acc = 0;
        acc_phase ^= 1u;
      }
    }
    if (!ok) spin_ns(2000000ull);   // let MMAs already issued complete
  } else if (WG && warp == 3) {
    // ---------------- tail rows of a group's last block (every CTA) ----------------
    const uint32_t leader_ptail0 = CG == 2 ? map_to_rank(ptail_bar(0), 0) : 0u;
    int stage = 0, hint = 0;
    uint32_t used = 0;              // parity of each stage's tail barrier
    for (int round = 0; round < rounds; ++round) {
      const int t = tile_at(round);
      if (t >= total) break;
      const Tile c = find_tile<WG>(p, gt, order, t, hint);
      const int n = gt->off[c.e + 1] - gt->off[c.e];
      const int blocks = (n + BK - 1) / BK, valid = n % BK;
      if (blocks == 0) continue;
      const int s = (stage + blocks - 1) % STAGES;
      stage = (stage + blocks) % STAGES;
      if (valid == 0) continue;
      const bool got = mbar_wait_sum(tail_bar(s), (used >> s) & 1u, abort_flag, fault, blocks);
      if (!__all_sync(0xffffffffu, got)) break;
      used ^= 1u << s;
      const int stop = (valid + 15) & ~15;
      const uint32_t base = smem_base + s * STAGE_BYTES;
      for (int i = valid * 8 + lane; i < stop * 8; i += 32)
#pragma unroll
        for (int b = 0; b < 2 + S::B_COLS / 64; ++b)
          sts128(base + b * 8192 + i * 16, make_uint4(0, 0, 0, 0));
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) {
        if (rank == 0) mbar_arrive(full_bar(s));
        else mbar_arrive_cluster(leader_ptail0 + 8u * s);
      }
    }
  } else if (warp >= EPI_WARP0) {
    // ---------------- epilogue (every CTA, its own 128 rows) ----------------
    const int q = warp & 3;
    uint8_t* mine = epi + q * (kSegBytes + BN * 4);
    const uint32_t seg = smem_u32(mine), bias_s = seg + kSegBytes;
    const uint32_t leader_tempty0 = CG == 2 ? map_to_rank(tempty_bar(0), 0) : tempty_bar(0);
    int acc = 0, hint = 0;
    uint32_t acc_phase = 0;
    for (int round = 0; round < rounds; ++round) {
      const int t = tile_at(round);
      if (t >= total) break;
      const Tile c = find_tile<WG>(p, gt, order, t, hint);
      const int r0 = gt->off[c.e], r1 = gt->off[c.e + 1];
      const int tile_row = c.mt * BM + (int)rank * 128 + q * 32;
      const int n0 = c.nt * BN;
      const int valid = min(32, (WG ? p.K : r1 - r0) - tile_row);
      const int64_t row = WG ? (int64_t)c.e * p.K + tile_row : (int64_t)r0 + tile_row;
      if (!WG && p.bias) {   // while the accumulator is being computed
        for (int i = lane; i < BN; i += 32) {
          const float b = n0 + i < p.N ? Num<T>::bias(p.bias, (int64_t)c.e * p.N + n0 + i) : 0.f;
          asm volatile("st.shared.f32 [%0], %1;" ::"r"(bias_s + i * 4), "f"(b) : "memory");
        }
        __syncwarp();
      }
      const bool waited =
          WG ? mbar_wait_sum(tfull_bar(acc), acc_phase, abort_flag, fault, (r1 - r0 + BK - 1) / BK)
             : mbar_wait(tfull_bar(acc), acc_phase, abort_flag, fault);
      if (!__all_sync(0xffffffffu, waited)) break;
      tc_fence_after();
      auto release = [&] {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          // tensor memory alone is handed back; a release would wait for the
          // stores of the segments before
          if (CG == 2 && rank != 0) arrive_relaxed(leader_tempty0 + 8u * acc);
          else mbar_arrive(tempty_bar(acc));
        }
      };
      if (valid > 0)
        store_rows<T, BN>(tmem_base + (uint32_t)(acc * BN) + ((uint32_t)(q * 32) << 16),
                          static_cast<T*>(p.y) + row * p.ldy, p.ldy, valid, n0, p.N, seg,
                          !WG && p.bias ? bias_s : 0u, WG && r1 == r0, p.aligned != 0, lane,
                          release);
      else
        release();
      if (++acc == 2) {
        acc = 0;
        acc_phase ^= 1u;
      }
    }
  }

  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (CG == 2) cluster_sync();   // no remote arrive or MMA of the pair still pending
  if (threadIdx.x == 0 && p.status) {
    if (gt->bad) atomicExch(p.status, (int32_t)BRA_ERR_INVALID);
    else if (*abort_flag) atomicExch(p.status, (int32_t)BRA_ERR_TIMEOUT);
  }
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc<CG>(tmem_base, S::TMEM_COLS);
  }
  if (p.late) grid_wait();
}

// Clusters of the kernel that are resident at once, found on first use.
template <typename T, int CG, int BN, bool WG>
cudaError_t resident(int* clusters) {
  static std::mutex mu;
  static int known[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  std::lock_guard<std::mutex> lk(mu);
  int& n = known[dev & 63];
  if (n == 0) {
    constexpr int smem = GShape<CG, BN>::SMEM_BYTES;
    e = cudaFuncSetAttribute(grouped_kernel<T, CG, BN, WG>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(CG, 1, 1);
    cfg.blockDim = dim3(THREADS, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = CG;
    attr.val.clusterDim.y = 1;
    attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    int m = 0;
    e = cudaOccupancyMaxActiveClusters(&m, grouped_kernel<T, CG, BN, WG>, &cfg);
    if (e != cudaSuccess) return e;
    n = m < 1 ? 1 : m;
  }
  *clusters = n;
  return cudaSuccess;
}

template <typename T, int CG, int BN, bool WG>
cudaError_t launch(const GroupedProblem& g, cudaStream_t st) {
  using S = GShape<CG, BN>;
  int clusters = 0;
  cudaError_t e = resident<T, CG, BN, WG>(&clusters);
  if (e != cudaSuccess) return e;
  GroupedParams p;
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
         (g.wt ? encode_3d(&p.tb, dt, g.w, K, N, E, BK, S::B_COLS, g.ldw)
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
  p.b_kmajor = g.wt;
  p.late = g.late;
  p.aligned = (reinterpret_cast<uintptr_t>(g.y) & 15u) == 0 && g.ldy % 8 == 0 && g.N % 8 == 0;
  p.idesc = make_idesc(g.dtype == BRA_BF16, 128 * CG, BN, !WG && g.wt) | (WG ? 1u << 15 : 0u);
  constexpr int BM = 128 * CG;
  p.m_tiles = (g.K + BM - 1) / BM;
  p.n_tiles = (g.N + BN - 1) / BN;
  p.k_blocks = (g.K + BK - 1) / BK;
  const int64_t groups = g.R < g.E ? g.R : g.E;
  int64_t tiles = WG ? (int64_t)g.E * p.m_tiles : g.R / BM + groups;   // at most
  tiles *= p.n_tiles;
  if (tiles >= (int64_t(1) << 31)) return cudaErrorInvalidValue;
  const int nc = (int)(tiles < clusters ? tiles : clusters);
  return launch_overlapped(grouped_kernel<T, CG, BN, WG>, CG * nc, THREADS, S::SMEM_BYTES, st, p);
}

template <int CG, int BN, bool WG>
cudaError_t launch_t(const GroupedProblem& g, cudaStream_t st) {
  return g.dtype == BRA_BF16 ? launch<__nv_bfloat16, CG, BN, WG>(g, st)
                             : launch<__half, CG, BN, WG>(g, st);
}

}  // namespace

// Tile shape, forward.  What feeds a tile's K block from L2 bounds it, about
// 58 bytes a clock and SM: 560 cycles for a pair's 256 x 256 tile (32 KiB a
// CTA), 850 for one CTA's 128 x 256 (48 KiB), 565 for its 128 x 128; the pair
// starts some 4 us later.  The waves of tiles over the SMs then decide.
// Measured, bf16, pair / 256 / 128 columns, us (rows an expert x experts, K, N):
//   128 x  8, 1024, 1024   11 /  10 /  9      512 x  8, 2048, 4096   59 /  59 /  -
//   256 x  8, 2048, 4096   38 /  36 / 43      128 x 64, 2048, 4096  159 / 171 / 189
//  2048 x  4,  256,  512    8 /   7 /  7     1024 x 32, 1024, 1024   61 /  71 /  -
//   620 x 17, 3176,  296    - /  61 / 44     2048 x  8, 2048, 4096  163 / 177 /  -
//
// The weight gradient's K loop is the rows; with few the stores of its large
// output bound it, and twice as many CTAs store more at once.  Pair / one CTA:
//   128 x 64, 2048, 4096  310 / 222          1024 x 64, 2048, 4096  832 / 839
//   512 x 64, 2048, 4096  586 / 547          2048 x 64, 2048, 4096 1407 / 1511
// It takes the pair from 1024 rows an expert on.
GroupedTile grouped_fwd_tile(const GroupedProblem& g) {
  int64_t tiles = 0;
  const int split = grouped_split(g, false, &tiles);
  if (split > 1) return {128, 128, split, tiles};
  // rows to an expert on average, and the most experts that can have rows
  const int64_t avg = g.R / g.E, groups = g.R < g.E ? g.R : g.E;
  if (avg < 16) {
    // the weights' bytes bound the call: the widest tiles that still occupy
    // the SMs (a token's two experts, 2048 x 4096: 64 columns, 128 tiles)
    const int64_t mt = g.R / 128 + groups;
    if (mt * ((g.N + 255) / 256) >= 100) return {128, 256, 1, 0};
    if (mt * ((g.N + 127) / 128) >= 152) return {128, 128, 1, 0};
    return {128, 64, 1, 0};
  }
  const int64_t kb = (g.K + BK - 1) / BK;
  auto cycles = [&](int64_t bm, int64_t bn, int64_t slots, int64_t block, int64_t start) {
    const int64_t n = (2 * (g.R / bm) + groups) * ((g.N + bn - 1) / bn) / 2;   // half filled ends
    return (n + slots - 1) / slots * kb * block + start;
  };
  const int64_t pair = cycles(256, 256, 76, 560, 10000), wide = cycles(128, 256, 152, 850, 3000),
                narrow = cycles(128, 128, 152, 565, 3000);
  if (pair <= wide && pair <= narrow) return {256, 256, 1, 0};
  return {128, wide <= narrow ? 256 : 128, 1, 0};
}

GroupedTile grouped_wgrad_tile(const GroupedProblem& g) {
  int64_t tiles = 0;
  const int split = grouped_split(g, true, &tiles);
  if (split > 1) return {128, 128, split, tiles};
  if (g.R / g.E >= 1024 && g.K > 128 && g.N > 128) return {256, 256, 1, 0};
  return {128, g.N > 128 ? 256 : 128, 1, 0};
}

cudaError_t launch_grouped_fwd(const GroupedProblem& g, cudaStream_t st) {
  const GroupedTile t = grouped_fwd_tile(g);
  if (t.split > 1) return launch_grouped_split(g, false, t.split, t.tiles, st);
  if (t.rows == 256) return launch_t<2, 256, false>(g, st);
  return t.cols == 256   ? launch_t<1, 256, false>(g, st)
         : t.cols == 128 ? launch_t<1, 128, false>(g, st)
                         : launch_t<1, 64, false>(g, st);
}

cudaError_t launch_grouped_wgrad(const GroupedProblem& g, cudaStream_t st) {
  const GroupedTile t = grouped_wgrad_tile(g);
  if (t.split > 1) return launch_grouped_split(g, true, t.split, t.tiles, st);
  if (t.rows == 256) return launch_t<2, 256, true>(g, st);
  return t.cols == 256 ? launch_t<1, 256, true>(g, st) : launch_t<1, 128, true>(g, st);
}

cudaError_t read_grouped_fault_word(int32_t* code, int clear) {
  cudaError_t e = cudaMemcpyFromSymbol(code, g_bra_fault_word_grouped, sizeof(int32_t));
  if (e != cudaSuccess) return e;
  if (clear) {
    const int32_t z = 0;
    e = cudaMemcpyToSymbol(g_bra_fault_word_grouped, &z, sizeof(int32_t));
  }
  return e;
}

}  // namespace bra
