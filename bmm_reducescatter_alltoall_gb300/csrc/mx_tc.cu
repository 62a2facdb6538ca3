// Products of 4-bit microscaled rows and weights, grouped by expert, on
// tcgen05 kind::mxf4 (sm_103a): y[r, n] = sum over blocks of 32 of
// 2^(sx + sw) * sum qx qw, both sums on the tensor core in fp32.
//
// The walk over ragged row groups is grouped_tc.cu's.  A K block is 256
// elements (128 bytes of codes to a row, one 128-byte swizzle row) and four
// MMAs of K = 64; their scales, one byte to 32 elements of each row and
// weight column, have to be in tensor memory, the same in all four lane
// quarters.  They are stored in memory in atoms (mx.cuh) in which a lane's
// four words are 16 bytes, so one TMA box brings a unit to shared memory and
// each of four writer warps, one to a lane quarter, passes it on with a few
// 16-byte loads and tcgen05.st.  An MMA picks its two bytes of a column by the
// scale ids of its instruction descriptor.
//   Writers and not tcgen05.cp: a copy takes its 55 cycles of the tensor pipe
//   itself, and a 256 x 256 pair tile needs six to a K block, next to 512
//   cycles of MMAs; 8 x 2048 rows, K = 16384, N = 4096 took 442 us with
//   copies and 346 with stores beside the MMAs.
//   The writers' word to the MMA issuer carries no memory of theirs, only
//   that their tcgen05.st have completed (tcgen05.wait::st, and the tcgen05
//   fences on both sides of the barrier): the arrival is relaxed.  With a
//   release at cluster scope the remote one took 1400 cycles a K block.  It
//   goes to the barrier that the codes complete: a second barrier to wait for
//   cost the issuer 70 cycles a K block (344 us in place of 314).
//   CG = 2, BN = 256: 256 x 256 tile of a CTA pair, 297 us (7400 TFLOP/s) on
//     the sizes above, 91 us at K = 4096.  The MMAs and a commit a K block
//     alone, without codes, scales or their waits, take 274 and 83 us: 512
//     cycles and some 55 of the commit.  Codes without scales: 285 and 90.
//     With one accumulator the epilogue first drains it into registers (eight
//     warps, 128 columns each, rounded and packed), hands it back, and stores
//     while the next tile is computed.  256 x 192 tiles, whose two
//     accumulators fit beside the scales, took a third longer; two
//     accumulators of 256 columns that share 128 of them, 6%.
//   CG = 1, BN = 128: 128 x 128 tile, two accumulators, for few rows to an
//     expert (the weights' bytes bound the call).
// Every wait is bounded (about 4 s) and reports through the fault word.
#include <cstring>
#include <mutex>
#include <type_traits>

#include "grouped.cuh"
#include "mx.cuh"

namespace bra {

__device__ int32_t g_bra_fault_word_mx = 0;

namespace {

using namespace tc;
using namespace grp;

constexpr int BKB = 128;                    // bytes of codes of a K block (256 elements)
constexpr int kGroupM = 8;
constexpr int WRITE_WARP0 = 4;
constexpr int EPI_WARP0 = 8;
constexpr int BAR_BYTES = 512;

struct MxParams {
  CUtensorMap ta, ta32;                     // row codes, boxes of 128 and 32 rows
  CUtensorMap tb;                           // weight codes
  CUtensorMap tsa, tsb;                     // scale units of the rows, of the weights
  const void* bias;
  void* y;
  const int64_t* counts;
  int32_t* status;
  int64_t R, ldy;
  int E, N, n_tiles, k_blocks, nb;          // nb: scale blocks of one expert's weight
  int bias_fp16, aligned;
  uint32_t idesc;
};

template <int CG, int BN>
struct MShape {
  static constexpr int A_BYTES = 128 * BKB;
  static constexpr int B_ROWS = BN / CG;                  // weight rows held by one CTA
  static constexpr int B_BYTES = B_ROWS * BKB;
  static constexpr int NSB = BN / 128;                    // weight scale blocks of a tile
  static constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
  // The scales' way to tensor memory has a ring of its own, so that it runs
  // ahead of the codes.
  static constexpr int SF_BYTES = (1 + NSB) * mx::kUnitBytes;
  static constexpr int SF_STAGES = 4;
  static constexpr int EPI_WARPS = BN / 32;               // 128 columns each
  static constexpr int THREADS = (EPI_WARP0 + EPI_WARPS) * 32;   // 4 role and 4 writer warps
  static constexpr int NACC = BN == 128 ? 2 : 1;
  static constexpr int EPI_BYTES = EPI_WARPS * (kSegBytes + 512);
  static constexpr int FIXED = BAR_BYTES + EPI_BYTES + 2 * (int)sizeof(GroupTable) + 16 + 1024 +
                               SF_STAGES * SF_BYTES;
  static constexpr int FIT = (232448 - FIXED) / STAGE_BYTES;
  static constexpr int STAGES = FIT > 6 ? 6 : FIT;
  static constexpr int SMEM_BYTES = STAGES * STAGE_BYTES + FIXED;
  // scale columns of a K block: 8 of the rows, 8 for each half's weights
  static constexpr int SF_COLS = 24;
  static constexpr uint32_t SF0 = NACC * BN;
  static_assert(STAGES >= 4 && SF0 + STAGES * SF_COLS <= 512, "ring, tensor memory");
  static_assert(STAGE_BYTES % 1024 == 0, "swizzle atoms");
};

// D (TMEM) [+]= A (smem) x B (smem) with block scales in TMEM, e2m1 x e2m1.
template <int CG>
__device__ __forceinline__ void mx_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                       uint32_t sa, uint32_t sb, uint32_t accumulate) {
  if constexpr (CG == 1)
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.block32 [%0], %1, %2, %3, [%5], [%6], p;"
        "\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(sa), "r"(sb)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.block32 [%0], %1, %2, %3, [%5], [%6], p;"
        "\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(sa), "r"(sb)
        : "memory");
}
// N words a lane to N columns of this warp's lane quarter.
__device__ __forceinline__ void tmem_st8(uint32_t t, const uint32_t (&v)[8]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(t),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
// The four writer warps meet; whether `ok` holds for every thread of theirs.
__device__ __forceinline__ bool join_writers(bool ok) {
  uint32_t all;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.and.pred q, 1, 128, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(all)
      : "r"((uint32_t)ok)
      : "memory");
  return all != 0;
}

template <typename T, int CG, int BN>
__global__ void __cluster_dims__(CG, 1, 1) __launch_bounds__(MShape<CG, BN>::THREADS, 1)
    mx_grouped_kernel(const __grid_constant__ MxParams p) {
  using S = MShape<CG, BN>;
  constexpr int STAGES = S::STAGES, STAGE_BYTES = S::STAGE_BYTES, BM = 128 * CG;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t raw_addr = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + (((raw_addr + 1023u) & ~1023u) - raw_addr);
  const uint32_t smem_base = smem_u32(smem);
  const uint32_t sf_base = smem_base + STAGES * STAGE_BYTES;
  uint8_t* bars = smem + STAGES * STAGE_BYTES + S::SF_STAGES * S::SF_BYTES;
  const uint32_t bar_base = smem_u32(bars);
  // barriers (8 bytes each): per stage full (leader: both CTAs' codes have
  // come, and their scales are in tensor memory), empty; per scale stage sfull
  // (this CTA's scales have come) and sempty (they have been passed on);
  // tfull[2], tempty[2]
  auto full_bar = [&](int s) { return bar_base + 8u * s; };
  auto empty_bar = [&](int s) { return bar_base + 8u * (STAGES + s); };
  constexpr int SFS = S::SF_STAGES;
  auto sfull_bar = [&](int s) { return bar_base + 8u * (2 * STAGES + s); };
  auto sempty_bar = [&](int s) { return bar_base + 8u * (2 * STAGES + SFS + s); };
  auto tfull_bar = [&](int a) { return bar_base + 8u * (2 * STAGES + 2 * SFS + a); };
  auto tempty_bar = [&](int a) { return tfull_bar(2 + a); };
  static_assert(8 * (2 * STAGES + 2 * SFS + 4) + 16 <= BAR_BYTES, "barrier area");
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + BAR_BYTES - 16);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(bars + BAR_BYTES - 8);
  GroupTable* gt = reinterpret_cast<GroupTable*>(bars + BAR_BYTES);      // row tiles
  GroupTable* gb = gt + 1;                                               // scale blocks
  uint8_t* epi = bars + BAR_BYTES + ((2 * sizeof(GroupTable) + 15) & ~15);
  int32_t* fault = &g_bra_fault_word_mx;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = CG == 2 ? cluster_rank() : 0u;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      // leader: its expect_tx, the bytes of both CTAs, their scale writers
      mbar_init(full_bar(s), 1 + CG);
      mbar_init(empty_bar(s), 1);
    }
    for (int s = 0; s < SFS; ++s) {
      mbar_init(sfull_bar(s), 1);
      mbar_init(sempty_bar(s), 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(tfull_bar(a), 1);
      mbar_init(tempty_bar(a), S::EPI_WARPS * CG);
    }
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    tma_prefetch_desc(&p.ta);
    tma_prefetch_desc(&p.ta32);
    tma_prefetch_desc(&p.tb);
    tma_prefetch_desc(&p.tsa);
    tma_prefetch_desc(&p.tsb);
  }
  if (warp == 2) {
    tmem_alloc<CG>(smem_u32(tmem_slot), 512);
    tmem_relinquish<CG>();
  }
  grid_wait();
  grid_go();
  if (warp == 3) build_table<BM>(gt, p.counts, p.E, p.R, lane);
  if (warp == 1) build_table<128>(gb, p.counts, p.E, p.R, lane);
  tc_fence_before();
  __syncthreads();
  if (CG == 2) cluster_sync();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const int total = gt->bad ? 0 : gt->tile[p.E] * p.n_tiles;
  const int walk0 = blockIdx.x / CG, step = gridDim.x / CG;
  int e_at = 0;                      // group of this role's current tile
  auto find = [&](int t) {
    while (gt->tile[e_at + 1] * p.n_tiles <= t) ++e_at;
    const int first = gt->tile[e_at];
    TileCoord c = tile_coord(t - first * p.n_tiles, gt->tile[e_at + 1] - first, p.n_tiles, kGroupM);
    c.g = e_at;
    return c;
  };

  if ((warp == 0 || warp == 2) && lane == 0) {
    // ---------------- producers (every CTA): warp 0 for A, warp 2 for B ----------------
    const bool is_a = warp == 0;
    const uint32_t leader_full0 = CG == 2 ? map_to_rank(full_bar(0), 0) : full_bar(0);
    int stage = 0;
    uint32_t phase = 0;
    bool ok = true;
    auto load = [&](uint32_t dst, const CUtensorMap* m, uint32_t bar, int c0, int c1, int c2) {
      if (CG == 2) tma_load_3d_pair(dst, m, bar, c0, c1, c2);
      else tma_load_3d(dst, m, bar, c0, c1, c2);
    };
    for (int t = walk0; ok && t < total; t += step) {
      const TileCoord c = find(t);
      const int r0 = gt->off[c.g], r1 = gt->off[c.g + 1];
      const int row = r0 + c.mt * BM + (int)rank * 128;
      auto boxes = [&](int valid) { return valid <= 64 ? (max(valid, 0) + 31) / 32 : 4; };
      const int mine = boxes(r1 - row);
      uint32_t bytes = CG * S::B_BYTES + mine * (S::A_BYTES / 4);
      if (CG == 2) bytes += boxes(r1 - row - 128) * (S::A_BYTES / 4);   // used by the leader
      const int b_row = c.nt * BN + (int)rank * S::B_ROWS;
      for (int kb = 0; kb < p.k_blocks; ++kb) {
        if (!mbar_wait(empty_bar(stage), phase ^ 1u, abort_flag, fault)) {
          ok = false;
          break;
        }
        const uint32_t fb = leader_full0 + 8u * stage;
        const uint32_t a_dst = smem_base + stage * STAGE_BYTES, b_dst = a_dst + S::A_BYTES;
        if (is_a) {
          if (rank == 0) mbar_expect_tx(full_bar(stage), bytes);
          if (mine == 4) load(a_dst, &p.ta, fb, kb * BKB, row, 0);
          else
            for (int i = 0; i < mine; ++i)
              load(a_dst + i * (S::A_BYTES / 4), &p.ta32, fb, kb * BKB, row + i * 32, 0);
        } else {
          load(b_dst, &p.tb, fb, kb * BKB, b_row, c.g);
        }
        if (++stage == STAGES) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    if (!ok) spin_ns(2000000ull);   // let copies already issued land
  } else if (warp == 3 && lane == 0) {
    // ---------------- scale loads (every CTA, onto its own barriers) ----------------
    int stage = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int t = walk0; ok && t < total; t += step) {
      const TileCoord c = find(t);
      // scale blocks; those past the group's or the weight's last belong to
      // rows and columns that are not stored
      const int ablk = gb->tile[c.g] + c.mt * CG + (int)rank;
      const int bblk = c.g * p.nb + c.nt * BN / 128;
      for (int kb = 0; kb < p.k_blocks; ++kb) {
        if (!mbar_wait(sempty_bar(stage), phase ^ 1u, abort_flag, fault)) {
          ok = false;
          break;
        }
        const uint32_t dst = sf_base + stage * S::SF_BYTES;
        mbar_expect_tx(sfull_bar(stage), S::SF_BYTES);
        tma_load_3d(dst, &p.tsa, sfull_bar(stage), 0, kb, ablk);
        tma_load_3d(dst + mx::kUnitBytes, &p.tsb, sfull_bar(stage), 0, kb, bblk);
        if (++stage == SFS) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    if (!ok) spin_ns(2000000ull);   // let copies already issued land
  } else if (warp == 1 && rank == 0) {
    // ---------------- MMA issuer (leader only) ----------------
    // the whole warp walks and waits, so that addresses stay warp-uniform; one
    // lane issues (one lane for everything: 60 us in place of 58 at K = 2048)
    const uint64_t a0 = smem_desc_sw128(smem_base, 16, 1024);
    const uint64_t b0 = smem_desc_sw128(smem_base + S::A_BYTES, 16, 1024);
    int stage = 0, acc = 0;
    uint32_t phase = 0, acc_phase = 0;
    bool ok = true;
    for (int t = walk0; ok && t < total; t += step) {
      const bool drained = mbar_wait(tempty_bar(acc), acc_phase ^ 1u, abort_flag, fault);
      ok = __all_sync(0xffffffffu, drained);
      if (!ok) break;
      tc_fence_after();
      const uint32_t d = tmem_base + (uint32_t)(acc * BN);
      int kb = 0;
      // One K block; whether the walk goes on.  The stage is a constant, so
      // that a block's addresses are too: computed for each block they held
      // the issuer up (8 x 2048 rows, K = 16384: 313 against 297 us).
      auto block = [&](auto at) -> bool {
        constexpr int s = decltype(at)::value;
        if constexpr (s < STAGES) {
          const bool here = mbar_wait(full_bar(s), phase, abort_flag, fault);
          ok = __all_sync(0xffffffffu, here);
          if (!ok) return false;
          tc_fence_after();
          constexpr uint64_t so = (uint64_t)((s * STAGE_BYTES) >> 4);
          // half h (128 elements): rows' columns 4h, weights' 8 + 8h
          const uint32_t sf = tmem_base + S::SF0 + (uint32_t)(s * S::SF_COLS);
          if (lane == 0) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
              mx_mma<CG>(d, a0 + so + 2 * k, b0 + so + 2 * k,
                         p.idesc | ((k & 1) ? (2u << 4 | 2u << 29) : 0u), sf + 4 * (k >> 1),
                         sf + 8 + 8 * (k >> 1), (kb > 0 || k > 0) ? 1u : 0u);
            if (CG == 2) tc_commit_pair(empty_bar(s), 0x3);
            else tc_commit(empty_bar(s));
          }
          __syncwarp();
          if (++kb < p.k_blocks) return true;
          stage = s + 1;
          return false;
        }
        return true;
      };
      static_assert(STAGES <= 6, "stages below");
      for (bool more = true; more;) {
        switch (stage) {
          case 0: more = block(std::integral_constant<int, 0>{}); if (!more) break; [[fallthrough]];
          case 1: more = block(std::integral_constant<int, 1>{}); if (!more) break; [[fallthrough]];
          case 2: more = block(std::integral_constant<int, 2>{}); if (!more) break; [[fallthrough]];
          case 3: more = block(std::integral_constant<int, 3>{}); if (!more) break; [[fallthrough]];
          case 4: more = block(std::integral_constant<int, 4>{}); if (!more) break; [[fallthrough]];
          default: more = block(std::integral_constant<int, 5>{});
        }
        if (more || stage == STAGES) {
          stage = 0;
          phase ^= 1u;
        }
      }
      if (!ok) break;
      if (lane == 0) {
        if (CG == 2) tc_commit_pair(tfull_bar(acc), 0x3);
        else tc_commit(tfull_bar(acc));
      }
      __syncwarp();
      if (++acc == S::NACC) {
        acc = 0;
        acc_phase ^= 1u;
      }
    }
    if (!ok) spin_ns(2000000ull);   // let MMAs already issued complete
  } else if (warp >= WRITE_WARP0 && warp < EPI_WARP0) {
    // ---------------- scale writers: lane quarter q, every CTA ----------------
    const int q = warp & 3;
    const uint32_t leader_full0 = CG == 2 ? map_to_rank(full_bar(0), 0) : full_bar(0);
    int from = 0, stage = 0;             // in the scales' ring, in the codes'
    uint32_t from_phase = 0, phase = 0;
    bool ok = true;
    auto step_ring = [](int& at, uint32_t& ph, int size) {
      if (++at == size) {
        at = 0;
        ph ^= 1u;
      }
    };
    // One K block, or two at once: a block's waits, loads and stores are a
    // chain of some 700 cycles, longer than its MMAs.  The four warps join
    // before one of them arrives (eight arrivals a K block, half of them
    // remote, in place of two: 39 against 36 us at 8 x 2048 rows, K = 512,
    // N = 4096), and leave together when a wait of any has run out.
    auto pass_on = [&](auto count) -> bool {
      constexpr int C = decltype(count)::value;
      int at_from = from, to[C];
      uint32_t at_phase = from_phase;
      uint32_t va[C][8], vb[C][2][8];
      bool got = true;
#pragma unroll
      for (int n = 0; n < C; ++n) {
        got = got && mbar_wait(sfull_bar(at_from), at_phase, abort_flag, fault);
        const uint32_t at = sf_base + at_from * S::SF_BYTES + (uint32_t)lane * 16;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint4 x = lds128e(at + h * 512);
          va[n][4 * h] = x.x, va[n][4 * h + 1] = x.y, va[n][4 * h + 2] = x.z, va[n][4 * h + 3] = x.w;
          uint32_t* w = vb[n][h];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint4 y = i < S::NSB ? lds128e(at + (1 + i) * mx::kUnitBytes + h * 512)
                                       : make_uint4(0, 0, 0, 0);
            w[4 * i] = y.x, w[4 * i + 1] = y.y, w[4 * i + 2] = y.z, w[4 * i + 3] = y.w;
          }
        }
        step_ring(at_from, at_phase, SFS);
        // the MMAs that read this stage's columns have completed
        got = got && mbar_wait(empty_bar(stage), phase ^ 1u, abort_flag, fault);
        to[n] = stage;
        step_ring(stage, phase, STAGES);
      }
      if (__all_sync(0xffffffffu, got)) {
        tc_fence_after();
#pragma unroll
        for (int n = 0; n < C; ++n) {
          const uint32_t sf =
              tmem_base + S::SF0 + (uint32_t)(to[n] * S::SF_COLS) + ((uint32_t)(q * 32) << 16);
          tmem_st8(sf, va[n]);
          tmem_st8(sf + 8, vb[n][0]);
          tmem_st8(sf + 16, vb[n][1]);
        }
        tmem_st_wait();
        tc_fence_before();
      }
      if (!join_writers(got)) return false;
#pragma unroll
      for (int n = 0; n < C; ++n) {
        if (warp == WRITE_WARP0 && lane == 0) {
          if (rank == 0) mbar_arrive(full_bar(to[n]));
          else arrive_relaxed(leader_full0 + 8u * to[n]);
          mbar_arrive(sempty_bar(from));
        }
        step_ring(from, from_phase, SFS);
      }
      return true;
    };
    for (int t = walk0; ok && t < total; t += step) {
      int kb = 0;
      for (; ok && kb + 2 <= p.k_blocks; kb += 2) ok = pass_on(std::integral_constant<int, 2>{});
      if (ok && kb < p.k_blocks) ok = pass_on(std::integral_constant<int, 1>{});
    }
  } else if (warp >= EPI_WARP0) {
    // ---------------- epilogue: lane quarter q, columns h*128 .. +128 ----------------
    const int q = warp & 3, h = (warp - EPI_WARP0) >> 2;
    uint8_t* mine = epi + (warp - EPI_WARP0) * (kSegBytes + 512);
    const uint32_t seg = smem_u32(mine), bias_s = seg + kSegBytes;
    const uint32_t leader_tempty0 = CG == 2 ? map_to_rank(tempty_bar(0), 0) : tempty_bar(0);
    int acc = 0;
    uint32_t acc_phase = 0;
    for (int t = walk0; t < total; t += step) {
      const TileCoord c = find(t);
      const int r0 = gt->off[c.g], r1 = gt->off[c.g + 1];
      const int tile_row = c.mt * BM + (int)rank * 128 + q * 32;
      const int n0 = c.nt * BN + h * 128;
      const int valid = min(32, r1 - r0 - tile_row);
      if (p.bias) {   // while the accumulator is being computed
        for (int i = lane; i < 128; i += 32) {
          const int64_t at = (int64_t)c.g * p.N + n0 + i;
          const float b = n0 + i >= p.N  ? 0.f
                          : p.bias_fp16 ? Num<__half>::bias(p.bias, at)
                                        : static_cast<const float*>(p.bias)[at];
          asm volatile("st.shared.f32 [%0], %1;" ::"r"(bias_s + i * 4), "f"(b) : "memory");
        }
        __syncwarp();
      }
      const bool waited = mbar_wait(tfull_bar(acc), acc_phase, abort_flag, fault);
      if (!__all_sync(0xffffffffu, waited)) break;
      tc_fence_after();
      const uint32_t t_base =
          tmem_base + (uint32_t)(acc * BN + h * 128) + ((uint32_t)(q * 32) << 16);
      const bool any = valid > 0 && n0 < p.N;
      uint32_t o[2][32];
      if (any) {
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          uint32_t v[64];
          tmem_ld32(t_base + half * 64, *reinterpret_cast<uint32_t(*)[32]>(&v[0]));
          tmem_ld32(t_base + half * 64 + 32, *reinterpret_cast<uint32_t(*)[32]>(&v[32]));
          tmem_ld_wait();
          pack_segment<T>(v, o[half], p.bias ? bias_s + half * 256 : 0u, false);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        // tensor memory alone is handed back: no memory of this thread to order
        if (CG == 2 && rank != 0) arrive_relaxed(leader_tempty0 + 8u * acc);
        else mbar_arrive(tempty_bar(acc));
      }
      if (any) {
        T* y0 = static_cast<T*>(p.y) + ((int64_t)r0 + tile_row) * p.ldy;
        const int segs = min(2, (p.N - n0 + 63) / 64);
        Carry carry;
#pragma unroll
        for (int ch = 0; ch < 2; ++ch)
          if (ch < segs)
            put_segment<T>(o[ch], carry, ch == 0, ch + 1 == segs, y0, p.ldy, valid, n0 + ch * 64,
                           p.N, seg, p.aligned != 0, lane, [] {});
      }
      if (++acc == S::NACC) {
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
    tmem_dealloc<CG>(tmem_base, 512);
  }
}

// Clusters of the kernel that are resident at once, found on first use.
template <typename T, int CG, int BN>
cudaError_t resident(int* clusters) {
  static std::mutex mu;
  static int known[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  std::lock_guard<std::mutex> lk(mu);
  int& n = known[dev & 63];
  if (n == 0) {
    using S = MShape<CG, BN>;
    e = cudaFuncSetAttribute(mx_grouped_kernel<T, CG, BN>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize, S::SMEM_BYTES);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(CG, 1, 1);
    cfg.blockDim = dim3(S::THREADS, 1, 1);
    cfg.dynamicSmemBytes = S::SMEM_BYTES;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = CG;
    attr.val.clusterDim.y = 1;
    attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    int m = 0;
    e = cudaOccupancyMaxActiveClusters(&m, mx_grouped_kernel<T, CG, BN>, &cfg);
    if (e != cudaSuccess) return e;
    n = m < 1 ? 1 : m;
  }
  *clusters = n;
  return cudaSuccess;
}

// Codes {row bytes, rows, groups}, box {128 bytes, b1, 1}, 128-byte swizzle.
bool encode_codes(CUtensorMap* m, const void* base, uint64_t pitch, uint64_t rows, uint64_t groups,
                  uint32_t b1) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[3] = {pitch, rows, groups};
  const cuuint64_t strides[2] = {pitch, pitch * rows};
  const cuuint32_t box[3] = {BKB, b1, 1};
  const cuuint32_t estr[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Scale units as 256 words: {256, K units, row blocks}, box of nb blocks.
bool encode_scales(CUtensorMap* m, const void* base, uint64_t k_units, uint64_t blocks,
                   uint32_t nb) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[3] = {256, k_units, blocks};
  const cuuint64_t strides[2] = {mx::kUnitBytes, mx::kUnitBytes * k_units};
  const cuuint32_t box[3] = {256, 1, nb};
  const cuuint32_t estr[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT32, 3, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename T, int CG, int BN>
cudaError_t launch(const MxProblem& g, cudaStream_t st) {
  using S = MShape<CG, BN>;
  int clusters = 0;
  cudaError_t e = resident<T, CG, BN>(&clusters);
  if (e != cudaSuccess) return e;
  MxParams p;
  std::memset(&p, 0, sizeof(p));
  const uint64_t pitch = (uint64_t)mx::code_pitch(g.K);
  if (!encode_codes(&p.ta, g.xc, pitch, g.R, 1, 128) ||
      !encode_codes(&p.ta32, g.xc, pitch, g.R, 1, 32) ||
      !encode_codes(&p.tb, g.wc, pitch, g.N, g.E, S::B_ROWS) ||
      !encode_scales(&p.tsa, g.xs, mx::units(g.K), mx::blocks_of(g.R, g.E, 0), 1) ||
      !encode_scales(&p.tsb, g.ws, mx::units(g.K), mx::blocks_of(g.E * (int64_t)g.N, g.E, g.N),
                     S::NSB))
    return cudaErrorInvalidValue;
  p.bias = g.bias;
  p.y = g.y;
  p.counts = g.counts;
  p.status = g.status;
  p.R = g.R;
  p.ldy = g.ldy;
  p.E = g.E;
  p.N = g.N;
  p.n_tiles = (g.N + BN - 1) / BN;
  p.k_blocks = (int)mx::units(g.K);
  p.nb = (g.N + 127) / 128;
  p.bias_fp16 = g.dtype == BRA_FP16;
  p.aligned = (reinterpret_cast<uintptr_t>(g.y) & 15u) == 0 && g.ldy % 8 == 0 && g.N % 8 == 0;
  // kind::mxf4: A and B e2m1 (bits 7, 10), N >> 3 at 17, e8m0 scales (bit 23),
  // M >> 7 at 27; scale ids (bits 4 and 29) per MMA
  p.idesc = 1u << 7 | 1u << 10 | (uint32_t)(BN >> 3) << 17 | 1u << 23 | (uint32_t)CG << 27;
  const int64_t groups = g.R < g.E ? g.R : g.E;
  const int64_t tiles = (g.R / (128 * CG) + groups) * p.n_tiles;         // at most
  if (tiles >= (int64_t(1) << 31)) return cudaErrorInvalidValue;
  const int nc = (int)(tiles < clusters ? tiles : clusters);
  return launch_overlapped(mx_grouped_kernel<T, CG, BN>, CG * nc, S::THREADS, S::SMEM_BYTES, st, p);
}

}  // namespace

// The pair from 128 rows an expert on, with a tile for each pair of SMs.
// bf16, one CTA against pair, us (rows an expert x experts, K, N):
//   equal groups                           groups drawn at random
//    96 x  8, 2048, 4096   10 / 13         112 x  8, 2048, 4096   10 / 13
//   160 x  8, 2048, 4096   17 / 13         128 x  8, 2048, 4096   13 / 13
//   128 x 64, 2048, 4096   60 / 66         120 x 64, 2048, 4096   65 / 66
//   160 x 64, 2048, 4096   91 / 69         128 x 64, 2048, 4096   71 / 67
//   512 x 16, 2048, 4096   47 / 36         140 x 64, 2048, 4096   84 / 68
//  1024 x 16, 2048, 4096   82 / 59
//   256 x  8, 4096, 1024   10 / 12 (96 tiles)   512 x 8, 4096, 1024   15 / 13 (160)
bool mx_pair(const MxProblem& g) {
  const int64_t groups = g.R < g.E ? g.R : g.E;
  return g.R / g.E >= 128 && (2 * (g.R / 256) + groups) * ((g.N + 255) / 256) >= 2 * 76;
}

cudaError_t launch_mx_grouped(const MxProblem& g, cudaStream_t st) {
  const bool bf16 = g.dtype == BRA_BF16;
  if (mx_pair(g))
    return bf16 ? launch<__nv_bfloat16, 2, 256>(g, st) : launch<__half, 2, 256>(g, st);
  return bf16 ? launch<__nv_bfloat16, 1, 128>(g, st) : launch<__half, 1, 128>(g, st);
}

cudaError_t read_mx_fault_word(int32_t* code, int clear) {
  cudaError_t e = cudaMemcpyFromSymbol(code, g_bra_fault_word_mx, sizeof(int32_t));
  if (e != cudaSuccess) return e;
  if (clear) {
    const int32_t z = 0;
    e = cudaMemcpyToSymbol(g_bra_fault_word_mx, &z, sizeof(int32_t));
  }
  return e;
}

}  // namespace bra
