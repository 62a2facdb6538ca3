// Products of 8-bit block-scaled rows and weights, grouped by expert, on
// tcgen05 kind::f8f6f4 (sm_103a):
//   y[r, n]  = sum over blocks b of sx[r, b] sw[n / 128, b] * (x_b . w_b) + bias
//   dx[r, k] = sum over blocks b of sd[r, b] sw[b, k / 128] * (dy_b . w_b)
// with fp32 scales of any value, a block being 128 elements of the contraction.
//
// A block's sum of code products is the tensor core's, in fp32 and in an
// accumulator of its own; the scales are applied as it is added to the running
// sum, which the epilogue warps hold in registers: acc += (sx sw) * block, a
// lane to a row, 64 or 128 columns a lane, one factor a row and block (an
// output tile's columns share a weight block by 128).  Tensor memory holds two
// or four block accumulators, so that one is drained while the next are
// computed.  The walk over ragged row groups is grouped_tc.cu's.  The gradient
// reads the same weight boxes the other way: 128 contraction rows of 128
// columns, N-major.
//
// What bounds it: with 256 x 256 tiles the two block accumulators' round trip
// (65536 rows, 4096 x 4096: 905 us, 2430 TFLOP/s).  A block's MMAs take some
// 380 ns, but an accumulator is free only after its commit, the loads of its
// sums and the pair's hand-back, so that a block takes 520 ns: at 935 us, the
// same product took 860 without the additions, 820 without the loads too, and
// 655 with one hand-back a tile, as a plain 8-bit product has.  Smaller
// accumulators do not help: a pair's MMA of 128 columns takes as long as one of
// 256 (tiles of 256 x 128: 1420 us; accumulators in two halves: 1157).
// Storing a tile is next: whole boxes of 32 rows and 64 columns go by TMA, as
// the epilogue warps are then free for the next tile's blocks (87108 rows, 384 x
// 1304: 113 us by the warps' own stores, 99 so, 73 without stores); rows
// without a 16-byte pitch and a group's last rows by the warps.
// With few rows HBM does (below), and with few tiles the blocks of a tile, one
// after the other: then a cluster of 2, 4 or 8 CTAs shares a tile's blocks, each
// leaves its sums in its shared memory, and each adds up a part of the rows of
// all of them, in their order.
// Every wait is bounded (about 4 s) and reports through the fault word.
#include <cstring>
#include <mutex>

#include "fp8.cuh"
#include "grouped.cuh"

namespace bra {

__device__ int32_t g_bra_fault_word_fp8 = 0;

namespace {

using namespace tc;
using namespace grp;

constexpr int BKB = 128;                    // bytes (elements) of a K block
constexpr int kGroupM = 8;
// Rows an expert, on average, up to which a tile is 32 rows by 128 columns of
// the weight (below).  2048 x 4096, us, by 32 x 128 / by 128 x 128 tiles: 64
// experts of 32 rows 92 / 118, of 33 (two tiles of rows) 167 / 118; 8 experts
// of 32 rows 18.5 / 20.9, of 33 28.8 / 20.9.
constexpr int64_t kFewRows = 32;
constexpr int EPI_WARP0 = 4;
constexpr int BAR_BYTES = 512;

struct Fp8Params {
  CUtensorMap ta, ta32;                     // row codes, boxes of 128 and 32 rows
  CUtensorMap tb;                           // weight codes
  CUtensorMap ty;                           // y, boxes of 64 columns and 32 rows, if y_boxes
  const float* xs;
  const float* ws;
  const void* bias;
  void* y;
  const int64_t* counts;
  int32_t* status;
  int64_t R, ldy, xs_pitch;
  int64_t ws_group, ws_out, ws_block;       // weight scales: from expert to expert, from output
                                            // block to output block, from K block to K block
  int E, N, n_tiles, k_blocks;              // N: columns of the output
  int bias_fp16, aligned, y_boxes;
  int split;                                // CTAs that share a tile's K blocks (one tile each)
  uint32_t idesc;
};

template <int CG, int BN>
struct FShape {
  static constexpr int A_BYTES = 128 * BKB;
  static constexpr int B_COLS = BN / CG;                  // output columns held by one CTA
  static constexpr int B_BYTES = B_COLS * BKB;
  static constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
  static constexpr int EPI_WARPS = 8;
  static constexpr int WC = BN / (EPI_WARPS / 4);         // columns of an epilogue warp
  static constexpr int THREADS = (EPI_WARP0 + EPI_WARPS) * 32;
  static constexpr int NBUF = BN == 256 ? 2 : 4;          // block accumulators
  static constexpr uint32_t TMEM_COLS = NBUF * BN;
  // each epilogue warp's segment (also a box of 32 swizzled rows of 128 bytes)
  static constexpr int SEG_BYTES = 5120;
  static_assert(SEG_BYTES >= kSegBytes && SEG_BYTES % 1024 == 0, "segments");
  static constexpr int EPI_BYTES = EPI_WARPS * (SEG_BYTES + WC * 4);
  static constexpr int FIXED = BAR_BYTES + EPI_BYTES + (int)sizeof(GroupTable) + 16 + 1024;
  static constexpr int FIT = (232448 - FIXED) / STAGE_BYTES;
  static constexpr int STAGES = FIT > 8 ? 8 : FIT;
  static constexpr int SMEM_BYTES = STAGES * STAGE_BYTES + FIXED;
  // Eight epilogue warps with narrow tiles too: two to a scheduler (2538 rows, 23
  // experts, gradient of 2665 x 128: 17.8 us with four, 13.9).
  // Registers of a thread: 168 at a launch of 384 threads, then 40 for the four
  // role warps and 232 for the eight epilogue warps (the same sum).
  static constexpr int LAUNCH_REGS = 168, ROLE_REGS = 40, EPI_REGS = 232;
  static_assert(128 * ROLE_REGS + 256 * EPI_REGS <= 384 * LAUNCH_REGS, "registers");
  static_assert(STAGES >= 4 && TMEM_COLS <= 512, "ring, tensor memory");
  static_assert(STAGE_BYTES % 1024 == 0, "swizzle atoms");
};

// D (TMEM) [+]= A (smem) x B (smem), 8-bit codes, fp32 sums.
template <int CG>
__device__ __forceinline__ void fp8_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                        uint32_t accumulate) {
  if constexpr (CG == 1)
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Waits for this warp's tensor memory loads; v's uses stay behind it.
__device__ __forceinline__ void tmem_ld_wait_for(uint32_t (&v)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]),
                 "+r"(v[6]), "+r"(v[7]), "+r"(v[8]), "+r"(v[9]), "+r"(v[10]), "+r"(v[11]),
                 "+r"(v[12]), "+r"(v[13]), "+r"(v[14]), "+r"(v[15]), "+r"(v[16]), "+r"(v[17]),
                 "+r"(v[18]), "+r"(v[19]), "+r"(v[20]), "+r"(v[21]), "+r"(v[22]), "+r"(v[23]),
                 "+r"(v[24]), "+r"(v[25]), "+r"(v[26]), "+r"(v[27]), "+r"(v[28]), "+r"(v[29]),
                 "+r"(v[30]), "+r"(v[31])::"memory");
}
__device__ __forceinline__ uint64_t pair64(uint32_t lo, uint32_t hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(lo), "r"(hi));
  return r;
}
// acc[i] += f * v[i], two at a time.
__device__ __forceinline__ void add_scaled(uint64_t* acc, const uint32_t (&v)[32], uint64_t ff) {
#pragma unroll
  for (int i = 0; i < 16; ++i)
    asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(acc[i]) : "l"(pair64(v[2 * i], v[2 * i + 1])), "l"(ff));
}

// The product of two scales within the floats; NaN stays.
__device__ __forceinline__ float within(float f) {
  constexpr float most = 3.402823466e+38f;
  return f > most ? most : f < -most ? -most : f;
}

// mbar_wait without a call: a kernel that splits its registers cannot have one.
__device__ __forceinline__ bool wait_here(uint32_t bar, uint32_t parity, volatile int* abort_flag,
                                          int32_t* fault) {
  if (mbar_try(bar, parity)) return true;
  const unsigned long long t0 = global_ns();
  for (;;) {
#pragma unroll 1
    for (int k = 0; k < 64; ++k)
      if (mbar_try(bar, parity)) return true;
    if (*abort_flag) return false;
    if (global_ns() - t0 > kWaitTimeoutNs) {
      *abort_flag = 1;
      atomicExch(fault, (int32_t)BRA_ERR_TIMEOUT);
      return false;
    }
  }
}

template <int N>
__device__ __forceinline__ void regs_to(bool up) {
  if (up) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
  else asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// A box of y from shared memory, behind this thread's next wait.
__device__ __forceinline__ void put_box(const CUtensorMap* m, uint32_t src, int col, int row) {
  asm volatile(
      "cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%2, %3, %4}], [%1];\n\t"
      "cp.async.bulk.commit_group;" ::"l"(m),
      "r"(src), "r"(col), "r"(row), "r"(0)
      : "memory");
}

// The K blocks of one CTA of those that share a tile: whole groups of four, as
// scales are read.
__device__ __forceinline__ int share_begin(int k_blocks, int share, int split) {
  const int fours = (k_blocks + 3) / 4;
  return min(4 * (fours * share / split), k_blocks);
}
__device__ __forceinline__ float4 peer_load4(uint32_t at, uint32_t rank) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(map_to_rank(at, rank))
               : "memory");
  return v;
}

// GRAD: the weight's rows are the contraction.
template <typename T, int CG, int BN, bool GRAD>
__global__ void __launch_bounds__(FShape<CG, BN>::THREADS, 1)
    fp8_grouped_kernel(const __grid_constant__ Fp8Params p) {
  using S = FShape<CG, BN>;
  constexpr int STAGES = S::STAGES, STAGE_BYTES = S::STAGE_BYTES, BM = 128 * CG, WC = S::WC;
  constexpr int PART_LD = BN + 4;             // floats between rows of a share's sums
  static_assert(CG == 2 || 128 * PART_LD * 4 <= STAGES * STAGE_BYTES, "a share's sums");
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t raw_addr = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + (((raw_addr + 1023u) & ~1023u) - raw_addr);
  const uint32_t smem_base = smem_u32(smem);
  uint8_t* segs = smem + STAGES * STAGE_BYTES;
  uint8_t* bars = segs + S::EPI_WARPS * S::SEG_BYTES;
  const uint32_t bar_base = smem_u32(bars);
  // barriers (8 bytes each): per stage full (leader: both CTAs' bytes) and
  // empty; per block accumulator tfull and tempty (leader: both CTAs' warps)
  auto full_bar = [&](int s) { return bar_base + 8u * s; };
  auto empty_bar = [&](int s) { return bar_base + 8u * (STAGES + s); };
  auto tfull_bar = [&](int a) { return bar_base + 8u * (2 * STAGES + a); };
  auto tempty_bar = [&](int a) { return bar_base + 8u * (2 * STAGES + S::NBUF + a); };
  static_assert(8 * (2 * STAGES + 2 * S::NBUF) + 16 <= BAR_BYTES, "barrier area");
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + BAR_BYTES - 16);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(bars + BAR_BYTES - 8);
  GroupTable* gt = reinterpret_cast<GroupTable*>(bars + BAR_BYTES);
  uint8_t* bias_rows = bars + BAR_BYTES + ((sizeof(GroupTable) + 15) & ~15);
  int32_t* fault = &g_bra_fault_word_fp8;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = CG == 2 ? cluster_rank() : 0u;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(full_bar(s), 1);     // leader: its expect_tx; the bytes of both CTAs
      mbar_init(empty_bar(s), 1);
    }
    for (int a = 0; a < S::NBUF; ++a) {
      mbar_init(tfull_bar(a), 1);
      mbar_init(tempty_bar(a), S::EPI_WARPS * CG);
    }
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    tma_prefetch_desc(&p.ta);
    tma_prefetch_desc(&p.ta32);
    tma_prefetch_desc(&p.tb);
  }
  if (warp == 2) {
    tmem_alloc<CG>(smem_u32(tmem_slot), S::TMEM_COLS);
    tmem_relinquish<CG>();
  }
  grid_wait();
  grid_go();
  if (warp == 3) build_table<BM>(gt, p.counts, p.E, p.R, lane);
  tc_fence_before();
  __syncthreads();
  if (CG == 2) cluster_sync();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const int total = gt->bad ? 0 : gt->tile[p.E] * p.n_tiles;
  const int split = CG == 1 ? p.split : 1, share = split > 1 ? (int)cluster_rank() : 0;
  const int kb0 = CG == 1 ? share_begin(p.k_blocks, share, split) : 0;
  const int kb1 = CG == 1 ? share_begin(p.k_blocks, share + 1, split) : p.k_blocks;
  const int walk0 = blockIdx.x / (CG * split), step = gridDim.x / (CG * split);
  int e_at = 0;                      // group of this role's current tile
  auto find = [&](int t) {
    while (gt->tile[e_at + 1] * p.n_tiles <= t) ++e_at;
    const int first = gt->tile[e_at];
    TileCoord c = tile_coord(t - first * p.n_tiles, gt->tile[e_at + 1] - first, p.n_tiles, kGroupM);
    c.g = e_at;
    return c;
  };

  if (warp < EPI_WARP0) {
    regs_to<S::ROLE_REGS>(false);
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
        // 32-row boxes of A to fetch (none past the group), or one of 128 rows
        auto boxes = [&](int valid) { return valid <= 64 ? (max(valid, 0) + 31) / 32 : 4; };
        const int mine = boxes(r1 - row);
        uint32_t bytes = CG * S::B_BYTES + mine * (S::A_BYTES / 4);
        if (CG == 2) bytes += boxes(r1 - row - 128) * (S::A_BYTES / 4);   // used by the leader
        const int b_col = c.nt * BN + (int)rank * S::B_COLS;
        for (int kb = kb0; kb < kb1; ++kb) {
          if (!wait_here(empty_bar(stage), phase ^ 1u, abort_flag, fault)) {
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
          } else if (!GRAD) {
            load(b_dst, &p.tb, fb, kb * BKB, b_col, c.g);
          } else {
#pragma unroll
            for (int i = 0; i < S::B_COLS / 128; ++i)
              load(b_dst + i * 16384, &p.tb, fb, b_col + i * 128, kb * BKB, c.g);
          }
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      if (!ok) spin_ns(2000000ull);   // let copies already issued land
    } else if (warp == 1 && lane == 0 && rank == 0) {
      // ---------------- MMA issuer (leader only) ----------------
      // K-major operands step 32 bytes per K = 32, the N-major one 32 box rows
      const uint64_t a0 = smem_desc_sw128(smem_base, 16, 1024);
      const uint64_t b0 = GRAD ? smem_desc_sw128(smem_base + S::A_BYTES, 16384, 1024)
                               : smem_desc_sw128(smem_base + S::A_BYTES, 16, 1024);
      constexpr uint32_t b_step = GRAD ? 256u : 2u;
      int stage = 0, buf = 0;
      uint32_t phase = 0, buf_phase = 0;
      bool ok = true;
      for (int t = walk0; ok && t < total; t += step) {
        for (int kb = kb0; kb < kb1; ++kb) {
          ok = wait_here(tempty_bar(buf), buf_phase ^ 1u, abort_flag, fault) &&
               wait_here(full_bar(stage), phase, abort_flag, fault);
          if (!ok) break;
          tc_fence_after();
          const uint32_t d = tmem_base + (uint32_t)(buf * BN);
          const uint64_t so = (uint64_t)((stage * STAGE_BYTES) >> 4);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            fp8_mma<CG>(d, a0 + so + 2 * k, b0 + so + b_step * k, p.idesc, k > 0 ? 1u : 0u);
          if (CG == 2) {
            tc_commit_pair(tfull_bar(buf), 0x3);
            tc_commit_pair(empty_bar(stage), 0x3);
          } else {
            tc_commit(tfull_bar(buf));
            tc_commit(empty_bar(stage));
          }
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1u;
          }
          if (++buf == S::NBUF) {
            buf = 0;
            buf_phase ^= 1u;
          }
        }
      }
      if (!ok) spin_ns(2000000ull);   // let MMAs already issued complete
    }
    if (CG == 1 && split > 1) {
      __syncwarp();
      cluster_sync();
      __syncwarp();
      cluster_sync();
    }
  } else {
    regs_to<S::EPI_REGS>(true);
    // ---------------- epilogue: lane quarter q, columns h*WC .. +WC ----------------
    const int q = warp & 3, h = (warp - EPI_WARP0) >> 2;
    const uint32_t seg = smem_u32(segs + (warp - EPI_WARP0) * S::SEG_BYTES);
    const uint32_t bias_s = smem_u32(bias_rows + (warp - EPI_WARP0) * WC * 4);
    const uint32_t leader_tempty0 = CG == 2 ? map_to_rank(tempty_bar(0), 0) : tempty_bar(0);
    int buf = 0;
    uint32_t buf_phase = 0;
    bool ok = true;
    auto next_buf = [&] {
      if (++buf == S::NBUF) {
        buf = 0;
        buf_phase ^= 1u;
      }
    };
    // tensor memory alone is handed back: no memory of this thread to order
    auto hand_back = [&] {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (CG == 2 && rank != 0) arrive_relaxed(leader_tempty0 + 8u * buf);
        else mbar_arrive(tempty_bar(buf));
      }
    };
    // What a tile needs besides its blocks, fetched while the tile before is
    // being stored: scales (four blocks of this lane's row in a load, 32 blocks
    // of the weight over the lanes, each ahead of its use) and the bias.
    struct Tile {
      int g, row, n0, valid;
    };
    Tile c;
    const float *sx = nullptr, *sw = nullptr;
    float4 x_at, x_next;
    float w_at = 0.f, w_next = 0.f, bias[WC / 32];
    auto fetch_x = [&](int kb) {
      return kb < p.k_blocks ? *reinterpret_cast<const float4*>(sx + kb) : make_float4(0, 0, 0, 0);
    };
    auto fetch_w = [&](int kb) {
      return kb + lane < p.k_blocks ? sw[(int64_t)(kb + lane) * p.ws_block] : 0.f;
    };
    auto begin = [&](int t) {
      const TileCoord at = find(t);
      const int tile_row = at.mt * BM + (int)rank * 128 + q * 32;
      c.g = at.g;
      c.row = gt->off[at.g] + tile_row;
      c.n0 = at.nt * BN + h * WC;
      c.valid = c.n0 < p.N ? min(32, gt->off[at.g + 1] - c.row) : 0;
      if (c.valid <= 0) return;
      sx = p.xs + ((int64_t)c.row + min(lane, c.valid - 1)) * p.xs_pitch;
      sw = p.ws + c.g * p.ws_group + (c.n0 / fp8::kBlock) * p.ws_out;
      x_at = fetch_x(kb0), x_next = fetch_x(kb0 + 4);
      w_at = fetch_w(kb0), w_next = fetch_w(kb0 + 32);
      if (p.bias)
#pragma unroll
        for (int i = 0; i < WC / 32; ++i) {
          const int n = c.n0 + i * 32 + lane;
          const int64_t b = (int64_t)c.g * p.N + n;
          bias[i] = n >= p.N      ? 0.f
                    : p.bias_fp16 ? Num<__half>::bias(p.bias, b)
                                  : static_cast<const float*>(p.bias)[b];
        }
    };
    uint32_t o[WC / 64][32];          // the tile before, rounded
    T* y0 = nullptr;
    int row = 0, n0 = 0, valid = 0;
    auto segment_free = [&] {         // the box before has been read
      if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
      __syncwarp();
    };
    for (int t = walk0; ok; t += step) {
      if (t < total) begin(t);
      if (valid > 0) {
        const int parts = min(WC / 64, (p.N - n0 + 63) / 64);
        segment_free();
        if (p.y_boxes && valid == 32) {
#pragma unroll
          for (int ch = 0; ch < WC / 64; ++ch)
            if (ch < parts) {
              if (ch > 0) segment_free();
#pragma unroll
              for (int i = 0; i < 8; ++i)
                sts128(seg + lane * 128 + ((i ^ (lane & 7)) << 4),
                       make_uint4(o[ch][4 * i], o[ch][4 * i + 1], o[ch][4 * i + 2], o[ch][4 * i + 3]));
              asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
              __syncwarp();
              if (lane == 0) put_box(&p.ty, seg, n0 + ch * 64, row);
            }
        } else {
          Carry carry;
#pragma unroll
          for (int ch = 0; ch < WC / 64; ++ch)
            if (ch < parts)
              put_segment<T>(o[ch], carry, ch == 0, ch + 1 == parts, y0, p.ldy, valid, n0 + ch * 64,
                             p.N, seg, p.aligned != 0, lane, [] {});
        }
      }
      if (t >= total) break;
      row = c.row, n0 = c.n0, valid = c.valid;
      if (valid <= 0) {
        for (int kb = kb0; kb < kb1; ++kb) {
          const bool got = wait_here(tfull_bar(buf), buf_phase, abort_flag, fault);
          if (!__all_sync(0xffffffffu, got)) {
            ok = false;
            break;
          }
          hand_back();
          next_buf();
        }
        continue;
      }
      y0 = static_cast<T*>(p.y) + (int64_t)c.row * p.ldy;
      if (p.bias) {
#pragma unroll
        for (int i = 0; i < WC / 32; ++i)
          asm volatile("st.shared.f32 [%0], %1;" ::"r"(bias_s + (i * 32 + lane) * 4), "f"(bias[i])
                       : "memory");
        __syncwarp();
      }
      uint64_t acc[WC / 2];
#pragma unroll
      for (int i = 0; i < WC / 2; ++i) acc[i] = 0ull;
#pragma unroll 1
      for (int kb = kb0; kb < kb1; ++kb) {
        const float f = within(x_at.x * __shfl_sync(0xffffffffu, w_at, (kb - kb0) & 31));
        const uint64_t ff = pair64(__float_as_uint(f), __float_as_uint(f));
        if ((kb & 3) == 3) {
          x_at = x_next;
          x_next = fetch_x(kb + 5);
          if (((kb - kb0) & 31) == 31) {
            w_at = w_next;
            w_next = fetch_w(kb + 33);
          }
        } else {
          x_at = make_float4(x_at.y, x_at.z, x_at.w, 0.f);
        }
        const bool got = wait_here(tfull_bar(buf), buf_phase, abort_flag, fault);
        if (!__all_sync(0xffffffffu, got)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t t_base =
            tmem_base + (uint32_t)(buf * BN + h * WC) + ((uint32_t)(q * 32) << 16);
        uint32_t v0[32], v1[32];
        tmem_ld32(t_base, v0);
        tmem_ld32(t_base + 32, v1);
        tmem_ld_wait_for(v0);
        tmem_ld_wait_for(v1);
        if constexpr (WC == 128) {
          add_scaled(acc, v0, ff);
          tmem_ld32(t_base + 64, v0);
          add_scaled(acc + 16, v1, ff);
          tmem_ld32(t_base + 96, v1);
          tmem_ld_wait_for(v0);
          tmem_ld_wait_for(v1);
          hand_back();
          add_scaled(acc + 32, v0, ff);
          add_scaled(acc + 48, v1, ff);
        } else {
          hand_back();
          add_scaled(acc, v0, ff);
          add_scaled(acc + 16, v1, ff);
        }
        next_buf();
      }
      if (!ok) break;
      if (CG == 1 && split > 1) {      // the stages are read: this CTA's sums take their place
        const uint32_t at = smem_base + (uint32_t)((q * 32 + lane) * PART_LD + h * WC) * 4;
#pragma unroll
        for (int i = 0; i < WC / 4; ++i)
          asm volatile("st.shared.v2.b64 [%0], {%1, %2};" ::"r"(at + i * 16), "l"(acc[2 * i]),
                       "l"(acc[2 * i + 1])
                       : "memory");
        valid = 0;
        continue;
      }
#pragma unroll
      for (int ch = 0; ch < WC / 64; ++ch) {
        uint32_t v[64];
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          v[2 * i] = (uint32_t)acc[ch * 32 + i];
          v[2 * i + 1] = (uint32_t)(acc[ch * 32 + i] >> 32);
        }
        pack_segment<T>(v, o[ch], p.bias ? bias_s + ch * 256 : 0u, false);
      }
    }
    if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    if (CG == 1 && split > 1) {        // 128 / split rows of all shares, added in their order
      __syncwarp();
      cluster_sync();
      if (walk0 < total) {
        const int each = BM / split, row0 = c.row - q * 32, n = c.n0 - h * WC + lane * 4;
        const int rows = min(min(BM, gt->off[c.g + 1] - row0), (share + 1) * each);
        float b[4] = {0.f, 0.f, 0.f, 0.f};
        if (p.bias)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (n + i < p.N)
              b[i] = p.bias_fp16 ? Num<__half>::bias(p.bias, (int64_t)c.g * p.N + n + i)
                                 : static_cast<const float*>(p.bias)[(int64_t)c.g * p.N + n + i];
        for (int r = share * each + warp - EPI_WARP0; r < rows; r += S::EPI_WARPS) {
          float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
          for (int k = 0; k < split; ++k) {
            const float4 v = peer_load4(smem_base + (uint32_t)(r * PART_LD + lane * 4) * 4, k);
            sum.x += v.x, sum.y += v.y, sum.z += v.z, sum.w += v.w;
          }
          T* dst = static_cast<T*>(p.y) + (int64_t)(row0 + r) * p.ldy + n;
          const uint32_t lo = Out<T>::pack(sum.x + b[0], sum.y + b[1]);
          const uint32_t hi = Out<T>::pack(sum.z + b[2], sum.w + b[3]);
          if (p.aligned && n < p.N) {
            *reinterpret_cast<uint2*>(dst) = make_uint2(lo, hi);
          } else {
            const uint16_t w[4] = {(uint16_t)lo, (uint16_t)(lo >> 16), (uint16_t)hi,
                                   (uint16_t)(hi >> 16)};
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (n + i < p.N) reinterpret_cast<uint16_t*>(dst)[i] = w[i];
          }
        }
      }
      __syncwarp();
      cluster_sync();                  // the peers have read this CTA's share
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
}

// --------------------------------------------------------------------------
// Few rows an expert: the operands change places.  A tile is 128 columns of the
// output (rows of the weight: the M side, a lane each) by up to 32 rows (the N
// side), so that a block's sum is 32 columns of tensor memory in place of 128
// that hold few rows.  The factors then go with the columns: a warp lays those
// of 16 blocks out in shared memory while the 16 before are being added, and
// reads them as pairs.  HBM bounds it: ten stages of 16 KB of weights in flight
// an SM (64 experts x 2 rows, 2048 x 4096: 537 MB in 89 us, 6.0 TB/s; by 128 x
// 128 tiles 120).
// --------------------------------------------------------------------------
struct FewShape {
  static constexpr int ROWS = 32, CHUNK = 16;             // rows of a tile; blocks of factors
  static constexpr int A_BYTES = 128 * BKB, B_BYTES = ROWS * BKB;
  static constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
  static constexpr int THREADS = (EPI_WARP0 + 4) * 32;
  static constexpr int NBUF = 8;
  static constexpr uint32_t TMEM_COLS = NBUF * ROWS;
  static constexpr int FACTORS = CHUNK * ROWS * 4;        // bytes of a warp
  static constexpr int STAGES = 10;
  static constexpr int SMEM_BYTES =
      STAGES * STAGE_BYTES + BAR_BYTES + 4 * FACTORS + (int)sizeof(GroupTable) + 16 + 1024;
  static_assert(SMEM_BYTES <= 232448 && STAGE_BYTES % 1024 == 0, "shared memory");
  static_assert(8 * (2 * STAGES + 2 * NBUF) + 16 <= BAR_BYTES, "barrier area");
};

template <typename T, bool GRAD>
__global__ void __launch_bounds__(FewShape::THREADS, 1)
    fp8_few_kernel(const __grid_constant__ Fp8Params p) {
  using S = FewShape;
  constexpr int STAGES = S::STAGES, STAGE_BYTES = S::STAGE_BYTES, ROWS = S::ROWS;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t raw_addr = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + (((raw_addr + 1023u) & ~1023u) - raw_addr);
  const uint32_t smem_base = smem_u32(smem);
  uint8_t* bars = smem + STAGES * STAGE_BYTES;
  const uint32_t bar_base = smem_u32(bars);
  auto full_bar = [&](int s) { return bar_base + 8u * s; };
  auto empty_bar = [&](int s) { return bar_base + 8u * (STAGES + s); };
  auto tfull_bar = [&](int a) { return bar_base + 8u * (2 * STAGES + a); };
  auto tempty_bar = [&](int a) { return bar_base + 8u * (2 * STAGES + S::NBUF + a); };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + BAR_BYTES - 16);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(bars + BAR_BYTES - 8);
  uint8_t* factors = bars + BAR_BYTES;
  GroupTable* gt = reinterpret_cast<GroupTable*>(factors + 4 * S::FACTORS);
  int32_t* fault = &g_bra_fault_word_fp8;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
    }
    for (int a = 0; a < S::NBUF; ++a) {
      mbar_init(tfull_bar(a), 1);
      mbar_init(tempty_bar(a), 4);
    }
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    tma_prefetch_desc(&p.ta32);
    tma_prefetch_desc(&p.tb);
  }
  if (warp == 2) {
    tmem_alloc<1>(smem_u32(tmem_slot), S::TMEM_COLS);
    tmem_relinquish<1>();
  }
  grid_wait();
  grid_go();
  if (warp == 3) build_table<ROWS>(gt, p.counts, p.E, p.R, lane);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const int total = gt->bad ? 0 : gt->tile[p.E] * p.n_tiles;
  const int split = p.split, share = split > 1 ? (int)cluster_rank() : 0;
  const int first = share_begin(p.k_blocks, share, split);
  const int past = share_begin(p.k_blocks, share + 1, split);
  const int walk0 = blockIdx.x / split, step = gridDim.x / split;
  int e_at = 0;                      // group of this role's current tile
  auto find = [&](int t) {
    while (gt->tile[e_at + 1] * p.n_tiles <= t) ++e_at;
    const int first = gt->tile[e_at];
    TileCoord c = tile_coord(t - first * p.n_tiles, gt->tile[e_at + 1] - first, p.n_tiles, kGroupM);
    c.g = e_at;
    return c;
  };

  if (warp == 0 && lane == 0) {
    // ---------------- producer ----------------
    int stage = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int t = walk0; ok && t < total; t += step) {
      const TileCoord c = find(t);
      const int row = gt->off[c.g] + c.mt * ROWS, n0 = c.nt * 128;
      for (int kb = first; kb < past; ++kb) {
        if (!wait_here(empty_bar(stage), phase ^ 1u, abort_flag, fault)) {
          ok = false;
          break;
        }
        const uint32_t a_dst = smem_base + stage * STAGE_BYTES;
        mbar_expect_tx(full_bar(stage), STAGE_BYTES);
        if (GRAD) tma_load_3d(a_dst, &p.tb, full_bar(stage), n0, kb * BKB, c.g);
        else tma_load_3d(a_dst, &p.tb, full_bar(stage), kb * BKB, n0, c.g);
        tma_load_3d(a_dst + S::A_BYTES, &p.ta32, full_bar(stage), kb * BKB, row, 0);
        if (++stage == STAGES) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    if (!ok) spin_ns(2000000ull);   // let copies already issued land
  } else if (warp == 1 && lane == 0) {
    // ---------------- MMA issuer ----------------
    const uint64_t a0 = GRAD ? smem_desc_sw128(smem_base, 16384, 1024)
                             : smem_desc_sw128(smem_base, 16, 1024);
    const uint64_t b0 = smem_desc_sw128(smem_base + S::A_BYTES, 16, 1024);
    constexpr uint32_t a_step = GRAD ? 256u : 2u;
    int stage = 0, buf = 0;
    uint32_t phase = 0, buf_phase = 0;
    bool ok = true;
    for (int t = walk0; ok && t < total; t += step) {
      for (int kb = first; kb < past; ++kb) {
        ok = wait_here(tempty_bar(buf), buf_phase ^ 1u, abort_flag, fault) &&
             wait_here(full_bar(stage), phase, abort_flag, fault);
        if (!ok) break;
        tc_fence_after();
        const uint64_t so = (uint64_t)((stage * STAGE_BYTES) >> 4);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          fp8_mma<1>(tmem_base + (uint32_t)(buf * ROWS), a0 + so + a_step * k, b0 + so + 2 * k,
                     p.idesc, k > 0 ? 1u : 0u);
        tc_commit(tfull_bar(buf));
        tc_commit(empty_bar(stage));
        if (++stage == STAGES) {
          stage = 0;
          phase ^= 1u;
        }
        if (++buf == S::NBUF) {
          buf = 0;
          buf_phase ^= 1u;
        }
      }
    }
    if (!ok) spin_ns(2000000ull);   // let MMAs already issued complete
  } else if (warp >= EPI_WARP0) {
    // ---------------- epilogue: output column n0 + q * 32 + lane ----------------
    const int q = warp & 3;
    const uint32_t fac = smem_u32(factors) + (warp - EPI_WARP0) * S::FACTORS;
    int buf = 0;
    uint32_t buf_phase = 0;
    bool ok = true;
    struct Tile {
      int g, row, n0, valid;
    };
    auto tile_of = [&](int t) {
      const TileCoord c = find(t);
      const int row = gt->off[c.g] + c.mt * ROWS;
      return Tile{c.g, row, c.nt * 128, min(ROWS, gt->off[c.g + 1] - row)};
    };
    // the factors of 16 blocks: this lane's row's scales, and (lanes 0 to 15)
    // the weight's
    float4 fx[S::CHUNK / 4];
    float fw = 0.f;
    auto fetch = [&](const Tile& c, int kb0) {
      const float* sx = p.xs + ((int64_t)c.row + min(lane, c.valid - 1)) * p.xs_pitch + kb0;
      const float* sw = p.ws + c.g * p.ws_group + (c.n0 / fp8::kBlock) * p.ws_out;
#pragma unroll
      for (int i = 0; i < S::CHUNK / 4; ++i)
        fx[i] = kb0 + 4 * i < p.k_blocks ? *reinterpret_cast<const float4*>(sx + 4 * i)
                                         : make_float4(0.f, 0.f, 0.f, 0.f);
      fw = lane < S::CHUNK && kb0 + lane < p.k_blocks ? sw[(int64_t)(kb0 + lane) * p.ws_block] : 0.f;
    };
    Tile next = {0, 0, 0, 1};
    if (walk0 < total) {
      next = tile_of(walk0);
      fetch(next, first);
    }
    for (int t = walk0; ok && t < total; t += step) {
      const Tile c = next;
      const int n = c.n0 + q * 32 + lane;
      float bias = 0.f;
      if (p.bias && n < p.N) {
        const int64_t at = (int64_t)c.g * p.N + n;
        bias = p.bias_fp16 ? Num<__half>::bias(p.bias, at) : static_cast<const float*>(p.bias)[at];
      }
      uint64_t acc[ROWS / 2];
#pragma unroll
      for (int i = 0; i < ROWS / 2; ++i) acc[i] = 0ull;
      for (int kb0 = first; ok && kb0 < past; kb0 += S::CHUNK) {
        __syncwarp();                       // the factors before have been read
#pragma unroll
        for (int i = 0; i < S::CHUNK; ++i) {
          const float4 x = fx[i / 4];
          const float f =
              within((i % 4 == 0 ? x.x : i % 4 == 1 ? x.y : i % 4 == 2 ? x.z : x.w) *
                     __shfl_sync(0xffffffffu, fw, i));
          asm volatile("st.shared.f32 [%0], %1;" ::"r"(fac + (i * ROWS + lane) * 4), "f"(f) : "memory");
        }
        __syncwarp();
        if (kb0 + S::CHUNK < past) {
          fetch(c, kb0 + S::CHUNK);
        } else if (t + step < total) {
          next = tile_of(t + step);
          fetch(next, first);
        }
        const int blocks = min(S::CHUNK, past - kb0);
#pragma unroll 1
        for (int b = 0; b < blocks; ++b) {
          const bool got = wait_here(tfull_bar(buf), buf_phase, abort_flag, fault);
          if (!__all_sync(0xffffffffu, got)) {
            ok = false;
            break;
          }
          tc_fence_after();
          uint32_t v[32];
          tmem_ld32(tmem_base + (uint32_t)(buf * ROWS) + ((uint32_t)(q * 32) << 16), v);
          tmem_ld_wait_for(v);
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(tempty_bar(buf));
#pragma unroll
          for (int i = 0; i < ROWS / 4; ++i) {
            uint64_t f0, f1;
            asm volatile("ld.shared.v2.u64 {%0, %1}, [%2];"
                         : "=l"(f0), "=l"(f1)
                         : "r"(fac + (b * ROWS + 4 * i) * 4)
                         : "memory");
            asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(acc[2 * i]) : "l"(pair64(v[4 * i], v[4 * i + 1])), "l"(f0));
            asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(acc[2 * i + 1]) : "l"(pair64(v[4 * i + 2], v[4 * i + 3])), "l"(f1));
          }
          if (++buf == S::NBUF) {
            buf = 0;
            buf_phase ^= 1u;
          }
        }
      }
      if (!ok) break;
      T* y0 = static_cast<T*>(p.y) + (int64_t)c.row * p.ldy + n;
      if (split > 1) {        // the stages are read: this CTA's sums take their place
        const uint32_t at = smem_base + (uint32_t)(q * 32 + lane) * 4;
#pragma unroll
        for (int j = 0; j < ROWS; ++j)
          if (j < c.valid)
            asm volatile("st.shared.b32 [%0], %1;" ::"r"(at + j * 512),
                         "r"((uint32_t)(acc[j / 2] >> (32 * (j & 1))))
                         : "memory");
      } else if (n < p.N) {
#pragma unroll
        for (int j = 0; j < ROWS; ++j)
          if (j < c.valid)
            y0[j * p.ldy] = static_cast<T>(
                __uint_as_float((uint32_t)(acc[j / 2] >> (32 * (j & 1)))) + bias);
      }
    }
  }

  __syncwarp();
  if (split > 1) {               // every split-th row of all shares, added in their order
    __syncwarp();
    cluster_sync();
    const int n = walk0 < total ? find(walk0).nt * 128 + (warp & 3) * 32 + lane : p.N;
    if (warp >= EPI_WARP0 && n < p.N) {
      const TileCoord c = find(walk0);
      const int row = gt->off[c.g] + c.mt * ROWS, valid = min(ROWS, gt->off[c.g + 1] - row);
      const uint32_t at = smem_base + (uint32_t)((warp & 3) * 32 + lane) * 4;
      float bias = 0.f;
      if (p.bias) {
        const int64_t b = (int64_t)c.g * p.N + n;
        bias = p.bias_fp16 ? Num<__half>::bias(p.bias, b) : static_cast<const float*>(p.bias)[b];
      }
      for (int r = share; r < valid; r += split) {
        float sum = 0.f;
        for (int k = 0; k < split; ++k) {
          float v;
          asm volatile("ld.shared::cluster.f32 %0, [%1];"
                       : "=f"(v)
                       : "r"(map_to_rank(at + r * 512, (uint32_t)k))
                       : "memory");
          sum += v;
        }
        static_cast<T*>(p.y)[(int64_t)(row + r) * p.ldy + n] = static_cast<T>(sum + bias);
      }
    }
    __syncwarp();
    cluster_sync();              // the peers have read this CTA's share
  }
  tc_fence_before();
  __syncthreads();
  if (threadIdx.x == 0 && p.status) {
    if (gt->bad) atomicExch(p.status, (int32_t)BRA_ERR_INVALID);
    else if (*abort_flag) atomicExch(p.status, (int32_t)BRA_ERR_TIMEOUT);
  }
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc<1>(tmem_base, S::TMEM_COLS);
  }
}

// Clusters of the kernel that are resident at once, found on first use.
template <typename T, int CG, int BN, bool GRAD>
cudaError_t resident(int* clusters) {
  static std::mutex mu;
  static int known[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  std::lock_guard<std::mutex> lk(mu);
  int& n = known[dev & 63];
  if (n == 0) {
    using S = FShape<CG, BN>;
    const auto kernel = fp8_grouped_kernel<T, CG, BN, GRAD>;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, S::SMEM_BYTES);
    if (e != cudaSuccess) return e;
    // the register split waits for ever unless the launch brings its sum
    cudaFuncAttributes at;
    e = cudaFuncGetAttributes(&at, kernel);
    if (e != cudaSuccess) return e;
    if (at.numRegs < S::LAUNCH_REGS) return cudaErrorLaunchOutOfResources;
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
    e = cudaOccupancyMaxActiveClusters(&m, kernel, &cfg);
    if (e != cudaSuccess) return e;
    n = m < 1 ? 1 : m;
  }
  *clusters = n;
  return cudaSuccess;
}

// Codes {K bytes, rows, groups} at a pitch of whole 16 bytes, box {128 bytes, b1, 1},
// 128-byte swizzle, zeros outside.
bool encode_codes(CUtensorMap* m, const void* base, uint64_t K, uint64_t rows, uint64_t groups,
                  uint32_t b1) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  const uint64_t pitch = (uint64_t)fp8::code_pitch((int64_t)K);
  const cuuint64_t dims[3] = {K, rows, groups};
  const cuuint64_t strides[2] = {pitch, pitch * rows};
  const cuuint32_t box[3] = {BKB, b1, 1};
  const cuuint32_t estr[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Parameters of a launch with tiles of `rows` rows and `cols` columns, the
// weight read in boxes of `box` rows; the instruction is the caller's.
bool fill(Fp8Params* out, const Fp8Problem& g, const GroupedTile& t, uint32_t box) {
  Fp8Params& p = *out;
  std::memset(&p, 0, sizeof(p));
  const int K = g.grad ? g.out : g.in, N = g.grad ? g.in : g.out;      // contraction, columns
  if (!encode_codes(&p.ta, g.xc, K, g.R, 1, 128) || !encode_codes(&p.ta32, g.xc, K, g.R, 1, 32) ||
      !encode_codes(&p.tb, g.wc, g.in, g.out, g.E, box))
    return false;
  p.xs = g.xs;
  p.ws = g.ws;
  p.bias = g.bias;
  p.y = g.y;
  p.counts = g.counts;
  p.status = g.status;
  p.R = g.R;
  p.ldy = g.ldy;
  p.xs_pitch = fp8::scale_pitch(K);
  const int64_t in_blocks = fp8::blocks(g.in);
  p.ws_group = fp8::blocks(g.out) * in_blocks;
  p.ws_out = g.grad ? 1 : in_blocks;
  p.ws_block = g.grad ? in_blocks : 1;
  p.E = g.E;
  p.N = N;
  p.n_tiles = (N + t.cols - 1) / t.cols;
  p.k_blocks = (int)fp8::blocks(K);
  p.bias_fp16 = g.dtype == BRA_FP16;
  p.aligned = (reinterpret_cast<uintptr_t>(g.y) & 15u) == 0 && g.ldy % 8 == 0 && N % 8 == 0;
  p.split = t.split;
  // whole boxes of rows go by TMA: rows of whole 16 bytes (it writes the last
  // ones whole, also past the row's end) at such a pitch, strides below 2^40
  const CUtensorMapDataType dt =
      g.dtype == BRA_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  p.y_boxes = t.rows >= 128 && p.aligned && g.ldy <= (int64_t(1) << 38) / g.R &&
              encode_3d(&p.ty, dt, g.y, N, g.R, 1, 64, 32, g.ldy);
  return t.tiles < (int64_t(1) << 31);
}

template <typename T, int CG, int BN, bool GRAD>
cudaError_t launch(const Fp8Problem& g, const GroupedTile& t, cudaStream_t st) {
  using S = FShape<CG, BN>;
  int clusters = 0;
  cudaError_t e = resident<T, CG, BN, GRAD>(&clusters);
  if (e != cudaSuccess) return e;
  Fp8Params p;
  if (!fill(&p, g, t, GRAD ? 128 : S::B_COLS)) return cudaErrorInvalidValue;
  // D fp32 (bit 4), the codes' formats (bits 7, 10: 0 e4m3, 1 e5m2), B N-major
  // (bit 16), N >> 3 at 17, M >> 4 at 24
  p.idesc = 1u << 4 | (uint32_t)g.xf << 7 | (uint32_t)g.wf << 10 | (GRAD ? 1u << 16 : 0u) |
            (uint32_t)(BN >> 3) << 17 | (uint32_t)(8 * CG) << 24;
  const int nc = (int)(t.tiles < clusters ? t.tiles : clusters), each = CG * t.split;
  return launch_clusters(fp8_grouped_kernel<T, CG, BN, GRAD>, each, each * nc, S::THREADS,
                         S::SMEM_BYTES, st, p);
}

template <typename T, bool GRAD>
cudaError_t launch_few(const Fp8Problem& g, const GroupedTile& t, cudaStream_t st) {
  using S = FewShape;
  static std::mutex mu;
  static int known[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  int sms = 0;
  {
    std::lock_guard<std::mutex> lk(mu);
    int& n = known[dev & 63];
    if (n == 0) {
      e = cudaFuncSetAttribute(fp8_few_kernel<T, GRAD>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               S::SMEM_BYTES);
      if (e != cudaSuccess) return e;
      e = cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
      if (e != cudaSuccess) return e;
    }
    sms = n;
  }
  Fp8Params p;
  if (!fill(&p, g, t, 128)) return cudaErrorInvalidValue;
  // as above, with the weight as A (M-major, bit 15, in the gradient)
  p.idesc = 1u << 4 | (uint32_t)g.wf << 7 | (uint32_t)g.xf << 10 | (GRAD ? 1u << 15 : 0u) |
            (uint32_t)(S::ROWS >> 3) << 17 | 8u << 24;
  return launch_clusters(fp8_few_kernel<T, GRAD>, t.split,
                         (unsigned)(t.tiles < sms ? t.tiles : sms) * t.split, S::THREADS,
                         S::SMEM_BYTES, st, p);
}

template <int CG, int BN, bool GRAD>
cudaError_t launch_t(const Fp8Problem& g, const GroupedTile& t, cudaStream_t st) {
  return g.dtype == BRA_BF16 ? launch<__nv_bfloat16, CG, BN, GRAD>(g, t, st)
                             : launch<__half, CG, BN, GRAD>(g, t, st);
}

template <bool GRAD>
cudaError_t launch_few_t(const Fp8Problem& g, const GroupedTile& t, cudaStream_t st) {
  return g.dtype == BRA_BF16 ? launch_few<__nv_bfloat16, GRAD>(g, t, st)
                             : launch_few<__half, GRAD>(g, t, st);
}

// CTAs to a tile, where there are few tiles: as long as all of them have an SM
// and each at least four blocks (6 rows, 5 experts, 3823 x 128: 13.3 us alone,
// 9.7 with eight blocks each, 7.4 with four; 4230 rows, 3 experts, 3520 x 88,
// 33 tiles: 15.9, 14.4, 10.9; 3 rows, 1728 x 192: 8.7, 8.7, 8.2).
int split_of(int64_t tiles, int k_blocks) {
  int split = 1;
  while (split < 8 && tiles * split * 2 <= 152 && k_blocks >= 4 * split * 2) split *= 2;
  return split;
}

}  // namespace

// The tiles that a model of their waves finds faster: nanoseconds of a tile as
// fitted to 30 sizes (256 x 256 by a pair: 2400 and 540 a block, 128 x 128: 1200
// and 410), half a tile of rows lost to each expert.  us by pairs / by 128 x 128:
// 12 experts, 3063 rows, 1026 x 775 11.9 / 15.0; 39, 60000, 2755 x 682 141 / 206;
// 39, 60000, 1043 x 126 29.6 / 25.5; 31, 7677, 448 x 1569 29.9 / 26.2; 58, 24444,
// 192 x 896 26.2 / 23.2.
GroupedTile fp8_tile(const Fp8Problem& g) {
  const int64_t N = g.grad ? g.in : g.out, groups = g.R < g.E ? g.R : g.E;
  const int64_t blocks = fp8::blocks(g.grad ? g.out : g.in);
  auto waves = [&](int64_t side, int64_t slots) {
    const int64_t tiles = (2 * (g.R / side) + groups) * ((N + side - 1) / side);   // twice
    return (tiles + 2 * slots - 1) / (2 * slots);
  };
  GroupedTile t = {128, 128, 1, 0};
  if (g.R <= kFewRows * g.E) t.rows = FewShape::ROWS;
  else if (waves(256, 76) * (2400 + 540 * blocks) < waves(128, 152) * (1200 + 410 * blocks))
    t.rows = t.cols = 256;
  t.tiles = (g.R / t.rows + groups) * ((N + t.cols - 1) / t.cols);                 // at most
  if (t.rows < 256) t.split = split_of(t.tiles, (int)blocks);
  return t;
}

cudaError_t launch_fp8_grouped(const Fp8Problem& g, cudaStream_t st) {
  const GroupedTile t = fp8_tile(g);
  if (t.rows == FewShape::ROWS)
    return g.grad ? launch_few_t<true>(g, t, st) : launch_few_t<false>(g, t, st);
  if (t.rows == 256)
    return g.grad ? launch_t<2, 256, true>(g, t, st) : launch_t<2, 256, false>(g, t, st);
  return g.grad ? launch_t<1, 128, true>(g, t, st) : launch_t<1, 128, false>(g, t, st);
}

cudaError_t read_fp8_fault_word(int32_t* code, int clear) {
  cudaError_t e = cudaMemcpyFromSymbol(code, g_bra_fault_word_fp8, sizeof(int32_t));
  if (e != cudaSuccess) return e;
  if (clear) {
    const int32_t z = 0;
    e = cudaMemcpyToSymbol(g_bra_fault_word_fp8, &z, sizeof(int32_t));
  }
  return e;
}

}  // namespace bra
