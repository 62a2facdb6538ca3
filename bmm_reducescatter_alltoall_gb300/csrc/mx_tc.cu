// Products of 4-bit microscaled rows and weights, grouped by expert, on
// tcgen05 kind::mxf4 (sm_103a): y[r, n] = sum over blocks of 32 of
// 2^(sx + sw) * sum qx qw, both sums on the tensor core in fp32.
//
// The walk over ragged row groups is grouped_tc.cu's.  A K block is 256
// elements (128 bytes of codes to a row, one 128-byte swizzle row) and four
// MMAs of K = 64; their scales, one byte to 32 elements of each row and
// weight column, have to be in tensor memory.  They are stored in memory in
// the order tcgen05.cp wants (mx.cuh), so one TMA box of 1 KiB (2 KiB for two
// weight blocks) brings the scales of 128 rows and 256 elements to shared
// memory (a tensor copy, which in a pair may complete on the leader's barrier,
// as an untiled one may not) and two tcgen05.cp
// (32 lanes x 128 bits, broadcast to the four lane quarters) to 8 columns of
// tensor memory; an MMA picks its two bytes of a column by the scale ids of
// its instruction descriptor.  Each ring stage has its own scale columns, so
// a stage's commit also frees them.
//   CG = 2, BN = 256: 256 x 256 tile of a CTA pair.  Accumulator (256
//     columns) and scales (5 x 24) fit tensor memory once, so the epilogue
//     first drains the accumulator into registers (eight warps, 128 columns
//     each, rounded and packed), hands it back, and stores while the next
//     tile is computed.
//   CG = 1, BN = 128: 128 x 128 tile, two accumulators, for few rows to an
//     expert (the weights' bytes bound the call).
// Every wait is bounded (about 4 s) and reports through the fault word.
#include <cstring>
#include <mutex>

#include "grouped.cuh"
#include "mx.cuh"

namespace bra {

__device__ int32_t g_bra_fault_word_mx = 0;

namespace {

using namespace tc;
using namespace grp;

constexpr int BKB = 128;                    // bytes of codes of a K block (256 elements)
constexpr int kGroupM = 8;
constexpr int EPI_WARP0 = 4;
constexpr int BAR_BYTES = 256;

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
  static constexpr int SF_BYTES = (1 + NSB) * mx::kUnitBytes;
  static constexpr int STAGE_BYTES = A_BYTES + B_BYTES + SF_BYTES;
  static constexpr int EPI_WARPS = BN / 32;               // 128 columns each
  static constexpr int THREADS = (EPI_WARP0 + EPI_WARPS) * 32;
  static constexpr int NACC = BN == 128 ? 2 : 1;
  static constexpr int EPI_BYTES = EPI_WARPS * (kSegBytes + 512);
  static constexpr int FIXED = BAR_BYTES + EPI_BYTES + 2 * (int)sizeof(GroupTable) + 64 + 1024;
  static constexpr int FIT = (232448 - FIXED) / STAGE_BYTES;
  static constexpr int STAGES = FIT > 6 ? 6 : FIT;
  static constexpr int SMEM_BYTES = STAGES * STAGE_BYTES + FIXED;
  static constexpr int SF_COLS = 8 + 8 * NSB;             // scale columns of a stage
  static constexpr uint32_t SF0 = NACC * BN;
  static_assert(SF0 + STAGES * SF_COLS <= 512 && STAGES >= 4, "tensor memory, ring");
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
// 32 lanes x 16 bytes (512 contiguous bytes) to four columns, repeated in the
// four lane quarters; with CG == 2 in both CTAs, each from its own memory.
template <int CG>
__device__ __forceinline__ void scale_copy(uint32_t taddr, uint64_t desc) {
  if constexpr (CG == 1)
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc)
                 : "memory");
  else
    asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc)
                 : "memory");
}
// Descriptor of a scale atom: no swizzle, groups of 8 rows 128 bytes apart.
__device__ __forceinline__ uint64_t scale_desc(uint32_t saddr) {
  return (uint64_t)((saddr & 0x3FFFFu) >> 4) | (uint64_t)(128 >> 4) << 16 |
         (uint64_t)(128 >> 4) << 32 | (uint64_t)1 << 46;
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
  uint8_t* bars = smem + STAGES * STAGE_BYTES;
  const uint32_t bar_base = smem_u32(bars);
  // barriers (8 bytes each): full, empty per stage; tfull[2], tempty[2]
  auto full_bar = [&](int s) { return bar_base + 8u * s; };
  auto empty_bar = [&](int s) { return bar_base + 8u * (STAGES + s); };
  auto tfull_bar = [&](int a) { return bar_base + 8u * (2 * STAGES + a); };
  auto tempty_bar = [&](int a) { return bar_base + 8u * (2 * STAGES + 2 + a); };
  static_assert(8 * (2 * STAGES + 4) + 16 <= BAR_BYTES, "barrier area");
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
      mbar_init(full_bar(s), 1);     // leader: its expect_tx; the bytes of both CTAs
      mbar_init(empty_bar(s), 1);
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
      uint32_t bytes = CG * (S::B_BYTES + S::SF_BYTES) + mine * (S::A_BYTES / 4);
      if (CG == 2) bytes += boxes(r1 - row - 128) * (S::A_BYTES / 4);   // used by the leader
      // scale blocks; those past the group's or the weight's last belong to
      // rows and columns that are not stored
      const int ablk = gb->tile[c.g] + c.mt * CG + (int)rank;
      const int bblk = c.g * p.nb + c.nt * S::NSB;
      const int b_row = c.nt * BN + (int)rank * S::B_ROWS;
      for (int kb = 0; kb < p.k_blocks; ++kb) {
        if (!mbar_wait(empty_bar(stage), phase ^ 1u, abort_flag, fault)) {
          ok = false;
          break;
        }
        const uint32_t fb = leader_full0 + 8u * stage;
        const uint32_t a_dst = smem_base + stage * STAGE_BYTES, b_dst = a_dst + S::A_BYTES;
        const uint32_t s_dst = b_dst + S::B_BYTES;
        if (is_a) {
          if (rank == 0) mbar_expect_tx(full_bar(stage), bytes);
          load(s_dst, &p.tsa, fb, 0, kb, ablk);
          if (mine == 4) load(a_dst, &p.ta, fb, kb * BKB, row, 0);
          else
            for (int i = 0; i < mine; ++i)
              load(a_dst + i * (S::A_BYTES / 4), &p.ta32, fb, kb * BKB, row + i * 32, 0);
        } else {
          load(b_dst, &p.tb, fb, kb * BKB, b_row, c.g);
          load(s_dst + mx::kUnitBytes, &p.tsb, fb, 0, kb, bblk);
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
    const uint64_t a0 = smem_desc_sw128(smem_base, 16, 1024);
    const uint64_t b0 = smem_desc_sw128(smem_base + S::A_BYTES, 16, 1024);
    const uint64_t s0 = scale_desc(smem_base + S::A_BYTES + S::B_BYTES);
    int stage = 0, acc = 0;
    uint32_t phase = 0, acc_phase = 0;
    bool ok = true;
    for (int t = walk0; ok && t < total; t += step) {
      if (!mbar_wait(tempty_bar(acc), acc_phase ^ 1u, abort_flag, fault)) break;
      tc_fence_after();
      const uint32_t d = tmem_base + (uint32_t)(acc * BN);
      for (int kb = 0; kb < p.k_blocks; ++kb) {
        if (!mbar_wait(full_bar(stage), phase, abort_flag, fault)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint64_t so = (uint64_t)((stage * STAGE_BYTES) >> 4);
        const uint32_t sfa = tmem_base + S::SF0 + (uint32_t)(stage * S::SF_COLS), sfb = sfa + 8;
        // atom h (128 elements) of the rows to columns 4h, of weight block i
        // to columns 4 (NSB h + i)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          scale_copy<CG>(sfa + 4 * h, s0 + so + 32 * h);
#pragma unroll
          for (int i = 0; i < S::NSB; ++i)
            scale_copy<CG>(sfb + 4 * (S::NSB * h + i), s0 + so + 64 * (1 + i) + 32 * h);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k)
          mx_mma<CG>(d, a0 + so + 2 * k, b0 + so + 2 * k,
                     p.idesc | ((k & 1) ? (2u << 4 | 2u << 29) : 0u), sfa + 4 * (k >> 1),
                     sfb + 4 * S::NSB * (k >> 1), (kb > 0 || k > 0) ? 1u : 0u);
        if (CG == 2) tc_commit_pair(empty_bar(stage), 0x3);
        else tc_commit(empty_bar(stage));
        if (++stage == STAGES) {
          stage = 0;
          phase ^= 1u;
        }
      }
      if (!ok) break;
      if (CG == 2) tc_commit_pair(tfull_bar(acc), 0x3);
      else tc_commit(tfull_bar(acc));
      if (++acc == S::NACC) {
        acc = 0;
        acc_phase ^= 1u;
      }
    }
    if (!ok) spin_ns(2000000ull);   // let MMAs already issued complete
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
        for (int ch = 0; ch < 2; ++ch) {
          uint32_t v[64];
          tmem_ld32(t_base + ch * 64, *reinterpret_cast<uint32_t(*)[32]>(&v[0]));
          tmem_ld32(t_base + ch * 64 + 32, *reinterpret_cast<uint32_t(*)[32]>(&v[32]));
          tmem_ld_wait();
          pack_segment<T>(v, o[ch], p.bias ? bias_s + ch * 256 : 0u, false);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (CG == 2 && rank != 0) mbar_arrive_cluster(leader_tempty0 + 8u * acc);
        else mbar_arrive(tempty_bar(acc));
      }
      if (any) {
        T* y0 = static_cast<T*>(p.y) + ((int64_t)r0 + tile_row) * p.ldy;
#pragma unroll
        for (int ch = 0; ch < 2; ++ch)
          put_segment<T>(o[ch], y0, p.ldy, valid, n0 + ch * 64, p.N, seg, p.aligned != 0, lane,
                         [] {});
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

cudaError_t launch_mx_grouped(const MxProblem& g, cudaStream_t st) {
  const bool bf16 = g.dtype == BRA_BF16;
  if (g.R / g.E >= 128)
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
