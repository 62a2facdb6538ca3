// What the kernels over ragged row groups share: the table of group offsets
// and row tiles each CTA builds from the device counts, and the epilogue that
// turns one accumulator quarter into masked row stores of any alignment.
#pragma once

#include "moe_internal.h"
#include "tc_ptx.cuh"

namespace bra {
namespace grp {

using namespace tc;

// Offsets of the groups' rows and of their row tiles, in shared memory.
struct GroupTable {
  int32_t off[kMaxGroups + 1];    // first row of each group; off[E] = rows used
  int32_t tile[kMaxGroups + 1];   // first row tile of each group; tile[E] = row tiles
  int32_t bad;                    // a count is negative or the counts pass R
};

// Built by one warp.  The counts are loaded together (one latency), scanned in
// 64 bits: counts may hold anything, and a table is only used when it is good.
template <int BM>
__device__ __forceinline__ void build_table(GroupTable* t, const int64_t* counts, int E, int64_t R,
                                            int lane) {
  int64_t c[kMaxGroups / 32];
#pragma unroll
  for (int i = 0; i < kMaxGroups / 32; ++i)
    c[i] = i * 32 + lane < E ? __ldcg(reinterpret_cast<const long long*>(counts) + i * 32 + lane) : 0;
  int64_t rows = 0;
  int32_t tiles = 0;
  bool bad = false;
#pragma unroll
  for (int i = 0; i < kMaxGroups / 32; ++i) {
    if (i * 32 >= E) break;
    bad = bad || c[i] < 0 || c[i] > R;
    int64_t n = bad ? 0 : c[i];
    int32_t m = (int32_t)((n + BM - 1) / BM);
    const int64_t n0 = n;
    const int32_t m0 = m;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int64_t a = __shfl_up_sync(0xffffffffu, n, d);
      const int32_t b = __shfl_up_sync(0xffffffffu, m, d);
      if (lane >= d) {
        n += a;
        m += b;
      }
    }
    if (i * 32 + lane < E) {
      t->off[i * 32 + lane] = (int32_t)(rows + n - n0);
      t->tile[i * 32 + lane] = tiles + m - m0;
    }
    rows += __shfl_sync(0xffffffffu, n, 31);
    tiles += __shfl_sync(0xffffffffu, m, 31);
  }
  bad = __any_sync(0xffffffffu, bad) || rows > R;
  if (lane == 0) {
    t->off[E] = (int32_t)rows;
    t->tile[E] = tiles;
    t->bad = bad ? 1 : 0;
  }
}

// Wait on a barrier that CTAs of the cluster arrive on (acquire at cluster
// scope); bounded as mbar_wait.
__device__ __forceinline__ bool mbar_try_acq(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
static __device__ __noinline__ bool mbar_wait_acq_slow(uint32_t bar, uint32_t parity,
                                                       volatile int* abort_flag, int32_t* fault) {
  const unsigned long long t0 = global_ns();
  for (;;) {
#pragma unroll 1
    for (int k = 0; k < 64; ++k)
      if (mbar_try_acq(bar, parity)) return true;
    if (*abort_flag) return false;
    if (global_ns() - t0 > kWaitTimeoutNs) {
      *abort_flag = 1;
      atomicExch(fault, (int32_t)BRA_ERR_TIMEOUT);
      return false;
    }
  }
}
__device__ __forceinline__ bool mbar_wait_acq(uint32_t bar, uint32_t parity,
                                              volatile int* abort_flag, int32_t* fault) {
  return mbar_try_acq(bar, parity) || mbar_wait_acq_slow(bar, parity, abort_flag, fault);
}

// Wait for the end of a sum over `blocks` blocks of 64 rows, or for its last
// block's operands: as mbar_wait, with a limit that grows with the blocks.  A
// block takes 0.27 us (64 x 128 columns of zeros, one tile a CTA), so that a
// group of 2^30 rows alone passes the limit of the other waits, which are each
// for one block.
static __device__ __noinline__ bool mbar_wait_sum_slow(uint32_t bar, uint32_t parity,
                                                       volatile int* abort_flag, int32_t* fault,
                                                       int blocks) {
  const unsigned long long t0 = global_ns(), limit = kWaitTimeoutNs + blocks * 4000ull;
  for (;;) {
#pragma unroll 1
    for (int k = 0; k < 64; ++k)
      if (mbar_try(bar, parity)) return true;
    if (*abort_flag) return false;
    if (global_ns() - t0 > limit) {
      *abort_flag = 1;
      atomicExch(fault, (int32_t)BRA_ERR_TIMEOUT);
      return false;
    }
  }
}
__device__ __forceinline__ bool mbar_wait_sum(uint32_t bar, uint32_t parity,
                                              volatile int* abort_flag, int32_t* fault,
                                              int blocks) {
  return mbar_try(bar, parity) || mbar_wait_sum_slow(bar, parity, abort_flag, fault, blocks);
}

// Arrive on a barrier of another CTA of the cluster without ordering this
// thread's memory accesses.
__device__ __forceinline__ void arrive_relaxed(uint32_t cluster_bar) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_bar)
               : "memory");
}

// 16-bit element access of the two output types, and their bias type.
template <typename T>
struct Num;
template <>
struct Num<__half> {
  static __device__ __forceinline__ float bias(const void* p, int64_t i) {
    return __half2float(static_cast<const __half*>(p)[i]);
  }
};
template <>
struct Num<__nv_bfloat16> {
  static __device__ __forceinline__ float bias(const void* p, int64_t i) {
    return static_cast<const float*>(p)[i];
  }
};

// Staging of one epilogue warp: 32 row segments of 64 outputs (128 bytes, and
// up to 14 bytes of shift), 144 bytes apart: 16-byte writes of consecutive
// lanes' rows and 16-byte reads along a row are both free of bank conflicts.
constexpr int kSegStride = 144;
constexpr int kSegBytes = 32 * kSegStride;

// 64 accumulator columns (fp32 bits) plus their bias (64 floats in shared
// memory at bias_s, or 0), rounded once to packed pairs of T; zeros for an
// empty sum.
template <typename T>
__device__ __forceinline__ void pack_segment(uint32_t (&v)[64], uint32_t (&o)[32], uint32_t bias_s,
                                             bool zero) {
  if (bias_s) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      uint4 b[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) b[i] = lds128e(bias_s + (uint32_t)(q * 16 + i * 4) * 4);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t* w = &v[q * 16 + i * 4];
        w[0] = __float_as_uint(__uint_as_float(w[0]) + __uint_as_float(b[i].x));
        w[1] = __float_as_uint(__uint_as_float(w[1]) + __uint_as_float(b[i].y));
        w[2] = __float_as_uint(__uint_as_float(w[2]) + __uint_as_float(b[i].z));
        w[3] = __float_as_uint(__uint_as_float(w[3]) + __uint_as_float(b[i].w));
      }
    }
  }
#pragma unroll
  for (int k = 0; k < 32; ++k)
    o[k] = zero ? 0u : Out<T>::pack(__uint_as_float(v[2 * k]), __uint_as_float(v[2 * k + 1]));
}

// What a lane keeps between the segments of its row when rows are not 16-byte
// aligned: the last elements, which share a 16-byte chunk with the next ones.
struct Carry {
  uint32_t w[4] = {0u, 0u, 0u, 0u};
};

// One warp writes a 64-column segment of its 32 rows (lane = row, packed
// pairs in o) to rows y0, y0 + ldy, ... of which `valid` (1 .. 32) exist, at
// columns nc .. below N (nc < N).  `aligned`: every row starts on a 16-byte
// boundary and N % 8 == 0.  Otherwise a row's segments go out in order, from
// the one marked `first` to the one marked `last`: each lane shifts its
// segment to the row's place in 16-byte chunks, whole chunks are stored as
// vectors, and the elements past the last whole one are carried to the next
// segment, so that only a run's two ends are stored in smaller pieces.  (With
// both ends of every segment stored so, a 128 x 256 tile of odd rows took 5 us
// to store: 4000 rows x 2257 gradient, 161 us.)  between() runs after the
// segment is staged.
template <typename T, typename Between>
__device__ __forceinline__ void put_segment(const uint32_t (&o)[32], Carry& carry, bool first,
                                            bool last, T* y0, int64_t ldy, int valid, int nc, int N,
                                            uint32_t seg, bool aligned, int lane,
                                            Between&& between) {
  const uint32_t my = seg + (uint32_t)lane * kSegStride;
  const int cols = min(64, N - nc);
  if (aligned) {
#pragma unroll
    for (int g = 0; g < 8; ++g)
      sts128(my + g * 16, make_uint4(o[4 * g], o[4 * g + 1], o[4 * g + 2], o[4 * g + 3]));
  } else {
    // element shift d = 4 b2 + 2 b1 + b0: by one half word, one word, two words
    const uint32_t d = (uint32_t)(reinterpret_cast<uintptr_t>(y0 + lane * ldy + nc) & 15u) >> 1;
    uint32_t z[36];
#pragma unroll
    for (int k = 0; k < 32; ++k)
      z[k] = (d & 1) ? __funnelshift_l(k ? o[k - 1] : 0u, o[k], 16) : o[k];
    z[32] = (d & 1) ? o[31] >> 16 : 0u;
    z[33] = z[34] = z[35] = 0u;
#pragma unroll
    for (int k = 33; k >= 0; --k) z[k] = (d & 2) ? (k >= 1 ? z[k - 1] : 0u) : z[k];
#pragma unroll
    for (int k = 35; k >= 0; --k) z[k] = (d & 4) ? (k >= 2 ? z[k - 2] : 0u) : z[k];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      z[k] |= carry.w[k];
      carry.w[k] = z[32 + k];
    }
#pragma unroll
    for (int g = 0; g < 9; ++g)
      sts128(my + g * 16, make_uint4(z[4 * g], z[4 * g + 1], z[4 * g + 2], z[4 * g + 3]));
  }
  between();
  __syncwarp();
  // 8 lanes to a row's 128 bytes, 4 rows an instruction
  const int c8 = (lane & 7) * 8, r0 = lane >> 3;
  if (aligned) {
    if (c8 < cols) {
      uint4 w[8];
#pragma unroll
      for (int q = 0; q < 8; ++q) w[q] = lds128e(seg + (uint32_t)(4 * q + r0) * kSegStride + c8 * 2);
#pragma unroll
      for (int q = 0; q < 8; ++q)
        if (4 * q + r0 < valid)
          *reinterpret_cast<uint4*>(y0 + (4 * q + r0) * ldy + nc + c8) = w[q];
    }
  } else {
    // the run lies at [d, d + cols) of the segment, after d carried elements
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const int r = 4 * q + r0;
      T* dst = y0 + r * ldy + nc;
      const int d = (int)((reinterpret_cast<uintptr_t>(dst) & 15u) >> 1);
      if (r < valid && c8 + 8 <= d + cols && (c8 >= d || !first))
        *reinterpret_cast<uint4*>(dst + (c8 - d)) = lds128e(seg + (uint32_t)r * kSegStride + c8 * 2);
    }
    if ((first || last) && lane < valid) {
      T* dst = y0 + lane * ldy + nc;
      const int d = (int)((reinterpret_cast<uintptr_t>(dst) & 15u) >> 1), end = d + cols;
      uint16_t* out = reinterpret_cast<uint16_t*>(dst) - d;        // by place in the segment
      auto put2 = [&](int i) {
        uint16_t w;
        asm volatile("ld.shared.u16 %0, [%1];" : "=h"(w) : "r"(my + i * 2) : "memory");
        out[i] = w;
      };
      auto put4 = [&](int i) {
        uint32_t w;
        asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w) : "r"(my + i * 2) : "memory");
        *reinterpret_cast<uint32_t*>(out + i) = w;
      };
      auto put8 = [&](int i) {
        uint2 w;
        asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];"
                     : "=r"(w.x), "=r"(w.y)
                     : "r"(my + i * 2)
                     : "memory");
        *reinterpret_cast<uint2*>(out + i) = w;
      };
      if (first && d > 0) {
        const int stop = min(8, end);
        int i = d;
        if ((i & 1) && i < stop) put2(i++);
        if ((i & 2) && i + 2 <= stop) put4(i), i += 2;
        if ((i & 4) && i + 4 <= stop) put8(i), i += 4;
        for (; i < stop; ++i) put2(i);                             // a run within one chunk
      }
      const int from = end & ~7;
      if (last && (end & 7) && (from > 0 || !first || d == 0)) {
        int i = from;
        if (end & 4) put8(i), i += 4;
        if (end & 2) put4(i), i += 2;
        if (end & 1) put2(i);
      }
    }
  }
  __syncwarp();
}

// One warp's 32 accumulator rows (TMEM address t_base, this warp's lane
// quarter), columns n0 .. n0+BN-1, 64 at a time: the next segment's TMEM
// loads are issued while the staged one goes out.  bias_s: BN floats in
// shared memory, or 0.  tmem_done() runs after the last TMEM load.
template <typename T, int BN, typename Done>
__device__ __forceinline__ void store_rows(uint32_t t_base, T* y0, int64_t ldy, int valid, int n0,
                                           int N, uint32_t seg, uint32_t bias_s, bool zero,
                                           bool aligned, int lane, Done&& tmem_done) {
  uint32_t v[64];
  tmem_ld32(t_base, *reinterpret_cast<uint32_t(*)[32]>(&v[0]));
  tmem_ld32(t_base + 32, *reinterpret_cast<uint32_t(*)[32]>(&v[32]));
  const int segs = min(BN / 64, (N - n0 + 63) / 64);        // the others lie past the matrix
  Carry carry;
#pragma unroll 1
  for (int ch = 0; ch < segs; ++ch) {
    tmem_ld_wait();
    if (ch + 1 == segs) tmem_done();
    uint32_t o[32];
    pack_segment<T>(v, o, bias_s ? bias_s + ch * 256 : 0u, zero);
    put_segment<T>(o, carry, ch == 0, ch + 1 == segs, y0, ldy, valid, n0 + ch * 64, N, seg, aligned,
                   lane, [&] {
      if (ch + 1 < segs) {
        tmem_ld32(t_base + (ch + 1) * 64, *reinterpret_cast<uint32_t(*)[32]>(&v[0]));
        tmem_ld32(t_base + (ch + 1) * 64 + 32, *reinterpret_cast<uint32_t(*)[32]>(&v[32]));
      }
    });
  }
}

}  // namespace grp
}  // namespace bra
