// Internal declarations of the ragged expert operators: the grouped products,
// the 4-bit microscaled formats, the router and the row permutation.
// Not installed; the public ABI is include/bra_moe.h.
#pragma once

#include "bra_internal.h"
#include "bra_moe.h"
#include "launch.cuh"

namespace bra {

// Groups of one call: the table of group offsets lives in shared memory.
constexpr int kMaxGroups = BRA_MAX_GROUPS;

// y = x W_e (+ bias) over row groups, or dW_e = x_e^T dy_e.
struct GroupedProblem {
  const void* x;         // [R][ldx], K used
  const void* w;         // forward: weights; wgrad: dy [R][ldw], N used
  const void* bias;      // forward: [E][N] or nullptr
  void* y;               // forward: [R][ldy]; wgrad: [E][K][N]
  const int64_t* counts; // device [E]
  int32_t* status;       // device, optional
  int64_t R, ldx, ldw, ldy;
  int E, K, N;
  int dtype;             // BRA_FP16 | BRA_BF16
  int wt;                // forward: weights stored (E, N, K)
  int late;              // needs nothing of the kernel launched before it
};
// Operands must be TMA-ready: pointers 16-byte aligned, row pitches a
// multiple of 8 elements.  cudaErrorInvalidValue if a map cannot be encoded.
cudaError_t launch_grouped_fwd(const GroupedProblem& g, cudaStream_t st);
cudaError_t launch_grouped_wgrad(const GroupedProblem& g, cudaStream_t st);
// The output tile they take (256 rows: a CTA pair's), by how many CTAs its
// contraction is split, and then the most tiles there can be.
struct GroupedTile {
  int rows, cols, split;
  int64_t tiles;
};
GroupedTile grouped_fwd_tile(const GroupedProblem& g);
GroupedTile grouped_wgrad_tile(const GroupedProblem& g);
// The same with each output tile's contraction split over a cluster: by how
// much (1: not at all), the most tiles there can be, and the launch.
int grouped_split(const GroupedProblem& g, bool wgrad, int64_t* tiles);
cudaError_t launch_grouped_split(const GroupedProblem& g, bool wgrad, int split, int64_t tiles,
                                 cudaStream_t st);
cudaError_t read_split_fault_word(int32_t* code, int clear);
// db_e = the sum of the rows of dy_e, in fp16 (FP16) or fp32 (BF16).
struct BiasGradProblem {
  const void* dy;
  void* db;
  const int64_t* counts;
  int32_t* status;
  int64_t R, ld;
  int E, N, dtype;
  int late;              // as above
};
cudaError_t launch_bias_grad(const BiasGradProblem& g, cudaStream_t st);
// Copies rows of `len` 16-bit elements, ld apart, to rows `pitch` apart (a
// multiple of 8) at a 16-byte aligned dst; a call's copies in one launch.
struct PackJob {
  const void* src;
  void* dst;
  int64_t ld, pitch, rows, len;
  int64_t per_group;       // 0, or: rows of a group, left out where its count is 0
};
struct PackJobs {
  PackJob job[3];
  const int64_t* counts;
  int n;
};
cudaError_t launch_pack_rows(const PackJobs& jobs, cudaStream_t st);
// Rows in the 4-bit microscaled layout (mx.cuh): row groups of `each` rows,
// or of counts[E] rows when each is 0.
struct MxRows {
  uint8_t* codes;
  uint8_t* scales;
  const int64_t* counts;
  int32_t* status;
  int64_t R, K, each;
  int E;
};
cudaError_t launch_mx_quantize(const MxRows& q, const void* x, int64_t ld, int dtype,
                               cudaStream_t st);
cudaError_t launch_mx_dequantize(const MxRows& q, void* y, int dtype, cudaStream_t st);
struct MxProblem {
  const uint8_t* xc;     // rows: codes and scales, grouped by counts
  const uint8_t* xs;
  const uint8_t* wc;     // weights: E groups of N rows
  const uint8_t* ws;
  const void* bias;
  void* y;
  const int64_t* counts;
  int32_t* status;
  int64_t R, ldy;
  int E, K, N, dtype;
};
cudaError_t launch_mx_grouped(const MxProblem& g, cudaStream_t st);
// Whether it takes the CTA pair's 256 x 256 tiles, or 128 x 128.
bool mx_pair(const MxProblem& g);
cudaError_t read_mx_fault_word(int32_t* code, int clear);

// The router.  hist: workspace of chunks x E int32 when there are several.
struct RouteCall {
  const void* logits;
  int32_t* ids;
  float* weights;
  int64_t* counts;
  int32_t* slots;
  int32_t* tokens;
  int32_t* hist;
  int64_t T;
  int E, k, renorm, dtype;
};
int route_chunk(int64_t T);                     // tokens of a chunk
cudaError_t launch_route(const RouteCall& r, cudaStream_t st);
struct RouteGradCall {
  const float* dweights;
  const void* logits;
  const int32_t* ids;
  const float* weights;
  void* dlogits;
  int64_t T;
  int E, k, renorm, dtype;
};
cudaError_t launch_route_grad(const RouteGradCall& r, cudaStream_t st);
// Row permutation; in and out are token rows (T) or expert rows (R).
struct PermuteCall {
  const void* in;
  void* out;
  const int32_t* row_tokens;   // [R], or nullptr
  const int32_t* slots;        // [T][k], or nullptr
  const float* weights;        // [T][k], or nullptr: ones
  int64_t T, R;
  int k, H, dtype;
};
// With dispatch_lists, `workspace` holds T * (BRA_MAX_CHOICES + 1) int32.
bool dispatch_lists(int64_t T, int64_t R, int64_t row_bytes);
cudaError_t launch_dispatch(const PermuteCall& c, void* workspace, cudaStream_t st);
cudaError_t launch_combine(const PermuteCall& c, cudaStream_t st);
// in: dy, out: dys
cudaError_t launch_combine_grad(const PermuteCall& c, const void* ys, float* dw, cudaStream_t st);
cudaError_t read_grouped_fault_word(int32_t* code, int clear);

}  // namespace bra
