/*
 * bra_moe.h -- ragged expert operators of libbmmrsa2a.so: matrix products
 * grouped by expert with row groups of any size, and their gradients; the
 * same products on 4-bit microscaled weights and rows; the router that makes
 * the groups, and the moves of token rows to their experts and back.
 *
 * They work on one matrix of rows sorted by expert, and the number of rows of
 * each expert in device memory (int64).  all_to_all_v counts elements, not
 * rows, and delivers by source rank: what a rank of one expert receives is
 * such a matrix as it stands, what one of several receives is in (source,
 * expert) order and is sorted by moe_dispatch, given the order of its rows.
 * The conventions of
 * bmm_rs_a2a.h hold: device pointers, row-major tensors, work enqueued on
 * `stream`, status codes, no device memory allocated, thread-safe, no state
 * from one call to the next.
 */
#ifndef BRA_MOE_H
#define BRA_MOE_H

#include "bmm_rs_a2a.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Most row groups (experts) of one call, and most experts of one token. */
#define BRA_MAX_GROUPS 512
#define BRA_MAX_CHOICES 16

/* ------------------------------------------------------------------------ */
/* Products grouped by expert                                                */
/* ------------------------------------------------------------------------ */

/* Sizes and options of a grouped product.  Zero-initialise. */
typedef struct {
  int64_t rows;        /* R: rows of x, y and dy, at most 2^31 - 2^16         */
  int64_t groups;      /* E: 1 .. BRA_MAX_GROUPS                              */
  int64_t in;          /* K: 1 .. 2^24                                        */
  int64_t out;         /* N: 1 .. 2^24                                        */
  int32_t dtype;       /* BRA_FP16 or BRA_BF16: x, weight, y and gradients    */
  int32_t transpose_weight;  /* non-zero: weight (and dweight) is (E, N, K)   */
  int64_t x_pitch;     /* elements between rows of x; 0 = K.  A pitch is at   */
                       /* most 2^36, and rows times it 2^59                   */
  int64_t y_pitch;     /* elements between rows of y (forward) or dy (grad); 0 = N */
  void* workspace;     /* 256-byte aligned, or NULL                           */
  int64_t workspace_bytes;
  int32_t* status;     /* device int32 of this call, or NULL (see below)      */
} bra_grouped_args;

/*
 * grouped_matmul -- y[r, :] = x[r, :] W_e + bias[e, :] for the rows r of each
 * expert e: rows off_e .. off_e + counts[e] - 1, off_e = sum of the counts
 * before e.  Sums in fp32, the bias added in fp32, one rounding to dtype.
 *
 *   x       device (R, K), row pitch x_pitch, rows sorted by expert.
 *   weight  device (E, K, N), or (E, N, K) with transpose_weight; dense.
 *   bias    NULL, or device (E, N): fp16 for FP16, fp32 for BF16.
 *   counts  device int64 (E).  Their sum R' may be below R: rows R' .. R-1 of
 *           x are not read into any result and those of y not written.
 *   y       device (R, N), row pitch y_pitch.
 * A count of 0 is an expert without rows.  Counts are checked on the device:
 * when one is negative or their sum passes R, nothing is written and
 * *status becomes BRA_ERR_INVALID.
 * status: set to BRA_OK on the stream before the kernels; BRA_ERR_TIMEOUT if
 * a bounded wait of this call gave up.
 *
 * The kernels read operands by TMA.  An operand whose rows lack a 16-byte
 * pitch or whose pointer is not 16-byte aligned is first copied to the
 * workspace (grouped_matmul_workspace_size; 0 when none is).  y may have any
 * element-aligned pointer and pitch.
 *
 * Errors (nothing launched):
 *   BRA_ERR_NULLPTR      args, x, weight, counts or y is NULL (x and y may be
 *                        NULL when rows is 0).
 *   BRA_ERR_INVALID      a size outside the ranges above, another dtype, a
 *                        pitch below the row length, a pointer that is not
 *                        element-aligned (counts: 8 bytes, status: 4), a
 *                        workspace not 256-byte aligned or smaller than
 *                        needed, y overlapping an input or the workspace,
 *                        the part of the workspace in use an input.
 *   BRA_ERR_UNSUPPORTED  a copy is needed and there is no workspace; more
 *                        than 2^31 - 1 output tiles.
 *   BRA_ERR_CUDA         the launch failed.
 */
BRA_API int grouped_matmul(const void* x, const void* weight, const void* bias,
                           const int64_t* counts, void* y, const bra_grouped_args* args,
                           bra_stream_t stream);

/*
 * grouped_matmul_grad -- the gradients of grouped_matmul for the output's
 * gradient dy; each output may be NULL (not wanted):
 *   dx[r, :]   = dy[r, :] W_e^T           (R, K) dense; rows R' .. R-1 not written
 *   dweight[e] = x_e^T dy_e               the weight's shape and layout; zero
 *                                         for an expert without rows
 *   dbias[e]   = sum of the rows of dy_e  (E, N), the bias's type
 * Sums in fp32, one rounding; results do not change from run to run.  x is
 * read for dweight only, weight for dx only (NULL otherwise allowed).
 * y_pitch is dy's.  Errors, counts, status and workspace as grouped_matmul
 * (grouped_matmul_grad_workspace_size); BRA_ERR_NULLPTR when all three
 * outputs are NULL.
 */
BRA_API int grouped_matmul_grad(const void* dy, const void* x, const void* weight,
                                const int64_t* counts, void* dx, void* dweight, void* dbias,
                                const bra_grouped_args* args, bra_stream_t stream);

/* Workspace bytes of the two calls for these pointers and sizes: 0 when every
 * operand can be read in place.  Pointers are only inspected for alignment;
 * the workspace fields are ignored.  A negative bra_status when the call
 * would be rejected.  Pure host. */
BRA_API int64_t grouped_matmul_workspace_size(const void* x, const void* weight,
                                              const bra_grouped_args* args);
BRA_API int64_t grouped_matmul_grad_workspace_size(const void* dy, const void* x,
                                                   const void* weight, int want_dx,
                                                   int want_dweight,
                                                   const bra_grouped_args* args);

/* ------------------------------------------------------------------------ */
/* 4-bit microscaled floating point (MXFP4)                                  */
/* ------------------------------------------------------------------------ */

/*
 * Rows of e2m1 codes with one power-of-two scale to 32 elements.  For a block
 * with largest magnitude a, s = max(floor(log2 a) - 2, -127) (a = 0: -127),
 * the scale byte is s + 127 and an element's code the nearest of
 * +-{0, .5, 1, 1.5, 2, 3, 4, 6} to x / 2^s, ties to the even code, magnitudes
 * past 6 to 6.  A block with a NaN or an infinity gets byte 255: every value
 * of it is NaN.
 *
 * codes: mxfp4_code_bytes: rows of ceil(K/32) * 16 bytes, two codes to a byte
 * (the even element in the low half), zeros past K.  scales:
 * mxfp4_scale_bytes: in the tensor core's order, per 128 rows and 256
 * elements a unit of 1024 bytes (byte (s/4)*512 + (r%32)*16 + (r/32)*4 + s%4
 * for row r and scale s of the unit); a unit's bytes of rows that do not
 * exist are not written.  The 128-row blocks start anew at each row group, so
 * scales belong to the grouping they were made with.
 */
typedef struct {
  int64_t rows;            /* R: 0 .. 2^31 - 2^16                              */
  int64_t k;               /* K: elements of a row, 1 .. 2^24                  */
  int64_t groups;          /* E: 1 .. BRA_MAX_GROUPS                           */
  int64_t rows_per_group;  /* groups of this many rows (R = E * that); 0: of   */
                           /* counts[E] rows, device int64, sum at most R      */
  int64_t x_pitch;         /* quantize: elements between rows of x; 0 = K; at  */
                           /* most 2^36, and rows times it 2^59                */
  int32_t dtype;           /* x: FP16 or BF16; dequantized y: FP16, BF16, FP32 */
  int32_t reserved;        /* 0                                                */
  int32_t* status;         /* device int32 of this call, or NULL               */
} bra_mx_args;

/* Bytes of the two buffers (or a negative bra_status).  Pure host. */
BRA_API int64_t mxfp4_code_bytes(const bra_mx_args* args);
BRA_API int64_t mxfp4_scale_bytes(const bra_mx_args* args);

/*
 * mxfp4_quantize -- x (R, K) to codes and scales; mxfp4_dequantize -- back to
 * y (R, K), dense, each value exact before its rounding to dtype.  With
 * counts, rows past their sum are neither read nor written, and counts are
 * checked on the device as in grouped_matmul.
 * Errors: BRA_ERR_NULLPTR for a NULL args, or data with R > 0 (counts when
 * rows_per_group is 0); BRA_ERR_INVALID for sizes outside the ranges, rows
 * other than groups * rows_per_group, another dtype, a pitch below K, codes
 * or scales not 16-byte aligned, x or y not element-aligned, an output
 * overlapping an input or the other output; BRA_ERR_CUDA.
 */
BRA_API int mxfp4_quantize(const void* x, const int64_t* counts, uint8_t* codes, uint8_t* scales,
                           const bra_mx_args* args, bra_stream_t stream);
BRA_API int mxfp4_dequantize(const uint8_t* codes, const uint8_t* scales, const int64_t* counts,
                             void* y, const bra_mx_args* args, bra_stream_t stream);

/*
 * mxfp4_grouped_matmul -- grouped_matmul on 4-bit operands: rows quantized
 * with the same counts (with one group also as a group of R rows), weights
 * (E, N, K) quantized as E groups of N rows.
 * y[r, n] = sum of the dequantized products in fp32 + bias[e, n], one
 * rounding to args->dtype (FP16 or BF16; the bias is fp16 or fp32 as there).
 * Of bra_grouped_args, x_pitch and transpose_weight must be 0 and no
 * workspace is used.  Errors, counts and status as grouped_matmul; codes and
 * scales have to be 16-byte aligned (BRA_ERR_INVALID).
 */
BRA_API int mxfp4_grouped_matmul(const uint8_t* x_codes, const uint8_t* x_scales,
                                 const uint8_t* w_codes, const uint8_t* w_scales,
                                 const void* bias, const int64_t* counts, void* y,
                                 const bra_grouped_args* args, bra_stream_t stream);

/* ------------------------------------------------------------------------ */
/* Router                                                                    */
/* ------------------------------------------------------------------------ */

typedef struct {
  int64_t tokens;      /* T: 0 .. 2^31 - 1, T * k below 2^31                  */
  int64_t experts;     /* E: 1 .. BRA_MAX_GROUPS                              */
  int64_t choices;     /* k: 1 .. min(E, BRA_MAX_CHOICES)                     */
  int32_t dtype;       /* logits: BRA_FP16, BRA_BF16 or BRA_FP32              */
  int32_t renormalize; /* non-zero: weights add up to 1 over the chosen       */
} bra_route_args;

/*
 * moe_route -- each token's k experts from its logits (T, E), and the order
 * that sorts the (token, choice) pairs by expert.
 *   A logit of -inf or NaN closes an expert to a token; +inf counts as the
 *   largest float.  The k largest open logits are chosen, largest first, ties
 *   to the lowest expert.  With fewer than k open ones the choices left have
 *   id -1, weight 0 and slot -1.
 *   ids     (T, k) int32.
 *   weights (T, k) fp32: the softmax over the token's open experts at the
 *           chosen ones; with renormalize divided by their sum.
 *   counts  (E) int64: pairs (rows) of each expert: grouped_matmul's counts.
 *           Added up over a rank's experts, times the elements of a row, they
 *           are a row of all_to_all_v's send_counts.
 *   slots   (T, k) int32: the pair's row among the R = T * k rows sorted by
 *           expert, within an expert by token.
 *   tokens  (R) int32: the token of each row; -1 for the rows past the last
 *           pair.
 * workspace: moe_route_workspace_size bytes (0 for a few tokens), 256-byte
 * aligned.
 * Errors: BRA_ERR_NULLPTR (args or counts; with tokens > 0 any pointer, or a
 * workspace where one is needed); BRA_ERR_INVALID: sizes outside the ranges,
 * another dtype, pointers not element-aligned, a workspace too small or
 * misaligned, an output overlapping the logits or another output;
 * BRA_ERR_CUDA.
 */
BRA_API int moe_route(const void* logits, int32_t* ids, float* weights, int64_t* counts,
                      int32_t* slots, int32_t* tokens, void* workspace, int64_t workspace_bytes,
                      const bra_route_args* args, bra_stream_t stream);
BRA_API int64_t moe_route_workspace_size(const bra_route_args* args);

/*
 * moe_route_grad -- the gradient of the logits (T, E, their type) for the
 * gradient dweights (T, k) fp32 of moe_route's weights, with its ids and
 * weights: the softmax's, closed experts and missing choices get 0.  logits
 * are read without renormalize only (NULL otherwise allowed).  ids outside
 * [0, E) count as missing.  Errors as moe_route.
 */
BRA_API int moe_route_grad(const float* dweights, const void* logits, const int32_t* ids,
                           const float* weights, void* dlogits, const bra_route_args* args,
                           bra_stream_t stream);

/* ------------------------------------------------------------------------ */
/* Token rows to their experts and back                                      */
/* ------------------------------------------------------------------------ */

typedef struct {
  int64_t tokens;      /* T: 0 .. 2^31 - 1                                    */
  int64_t rows;        /* R: 0 .. 2^31 - 1                                    */
  int64_t choices;     /* k: 1 .. BRA_MAX_CHOICES                             */
  int64_t width;       /* H: elements of a row, 1 .. 2^24                     */
  int32_t dtype;       /* rows: BRA_FP16, BRA_BF16 or BRA_FP32                */
  int32_t reserved;    /* 0                                                   */
} bra_permute_args;

/*
 * Token rows are (T, H), expert rows (R, H), dense; tokens (R) and slots
 * (T, k) int32 as moe_route writes them, weights (T, k) fp32.  Sums in fp32
 * in the order of the choices, one rounding; results do not change from run
 * to run.  Entries outside their range count as -1 and are never followed.
 *   moe_dispatch       xs[r] = x[tokens[r]]; zeros for -1.  (choices unused)
 *                      tokens may be in any order.  workspace: 256-byte
 *                      aligned, moe_dispatch_workspace_size bytes (0 unless
 *                      there are many long token rows with several rows each).
 *   moe_dispatch_grad  dx[t] = sum of dxs[slots[t, j]] over j, -1 left out.
 *   moe_combine        y[t] = sum of weights[t, j] * ys[slots[t, j]].
 *   moe_combine_grad   dys[slots[t, j]] = weights[t, j] * dy[t];
 *                      dweights[t, j] = <dy[t], ys[slots[t, j]]>, 0 for -1.
 *                      Rows whose token is -1 get zeros (tokens NULL: they
 *                      are not written).  No two slots may be the same.
 * Errors: BRA_ERR_NULLPTR for a NULL args, or pointer to data there is;
 * BRA_ERR_INVALID: sizes outside the ranges, another dtype, pointers not
 * element-aligned, an output overlapping an input or the other output;
 * BRA_ERR_CUDA.
 */
BRA_API int moe_dispatch(const void* x, const int32_t* tokens, void* xs, void* workspace,
                         int64_t workspace_bytes, const bra_permute_args* args,
                         bra_stream_t stream);
BRA_API int64_t moe_dispatch_workspace_size(const bra_permute_args* args);
BRA_API int moe_dispatch_grad(const void* dxs, const int32_t* slots, void* dx,
                              const bra_permute_args* args, bra_stream_t stream);
BRA_API int moe_combine(const void* ys, const int32_t* slots, const float* weights, void* y,
                        const bra_permute_args* args, bra_stream_t stream);
BRA_API int moe_combine_grad(const void* dy, const void* ys, const int32_t* slots,
                             const float* weights, const int32_t* tokens, void* dys,
                             float* dweights, const bra_permute_args* args, bra_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* BRA_MOE_H */
