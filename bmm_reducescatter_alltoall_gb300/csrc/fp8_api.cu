// Host entry points of the 8-bit block-scaled operators: argument checks and
// launches.  Every rule cited here is stated in include/bra_moe.h.
#include <cstdio>

#include "fp8.cuh"
#include "moe_checks.h"

namespace {

using namespace bra;

constexpr int64_t kWide = int64_t(1) << 24;

bool format_ok(int format) { return format == BRA_E4M3 || format == BRA_E5M2; }

int check_fp8(const bra_fp8_args* a) {
  if (!a) return BRA_ERR_NULLPTR;
  if (a->rows < 0 || a->rows > kMaxRows || a->k < 1 || a->k > kWide || a->groups < 1 ||
      a->groups > BRA_MAX_GROUPS || a->rows_per_group < 0 || a->rows_per_group > kMaxRows)
    return BRA_ERR_INVALID;
  if (a->rows_per_group > 0 && a->rows != a->groups * a->rows_per_group) return BRA_ERR_INVALID;
  if (a->x_pitch != 0 && (a->x_pitch < a->k || a->x_pitch > (int64_t(1) << 36) ||
                          !counts_in_64_bits(a->rows, a->x_pitch)))
    return BRA_ERR_INVALID;
  if (!row_dtype_ok(a->dtype) || !format_ok(a->format) || off_by(a->status, 3u))
    return BRA_ERR_INVALID;
  return BRA_OK;
}

// The parts of the two conversions that are the same.  `data` is x or y, `ld` its pitch.
int check_call(const void* data, int64_t ld, const int64_t* counts, const uint8_t* codes,
               const float* scales, const bra_fp8_args* a, bool quantize) {
  if (a->rows > 0 && (!data || !codes || !scales)) return BRA_ERR_NULLPTR;
  const int64_t es = element_size(a->dtype);
  if (counts && a->rows_per_group > 0) return BRA_ERR_INVALID;
  if (off_by(data, es - 1) || off_by(codes, 15u) || off_by(scales, 15u) || off_by(counts, 7u))
    return BRA_ERR_INVALID;
  const Span d = {data, span(a->rows, ld, a->k, es)}, c = {codes, fp8_code_bytes(a)},
             s = {scales, fp8_scale_bytes(a)}, n = {counts, a->groups * 8};
  if (quantize) {
    const Span outs[2] = {c, s}, ins[2] = {d, n};
    return any_overlap(outs, 2, ins, 2) ? BRA_ERR_INVALID : BRA_OK;
  }
  const Span ins[3] = {c, s, n};
  return any_overlap(&d, 1, ins, 3) ? BRA_ERR_INVALID : BRA_OK;
}

Fp8Data data_of(const uint8_t* codes, const float* scales, const int64_t* counts,
                const bra_fp8_args* a) {
  return {const_cast<uint8_t*>(codes),
          const_cast<float*>(scales),
          counts,
          a->status,
          a->rows,
          a->k,
          a->rows_per_group,
          (int)a->groups,
          a->format};
}

int run_product(const uint8_t* xc, const float* xs, const uint8_t* wc, const float* ws,
                const void* bias, const int64_t* counts, void* y, const bra_fp8_product_args* a,
                bool grad, cudaStream_t st) {
  if (!a) return BRA_ERR_NULLPTR;
  if (a->rows < 0 || a->rows > kMaxRows || a->groups < 1 || a->groups > BRA_MAX_GROUPS ||
      a->in < 1 || a->in > kWide || a->out < 1 || a->out > kWide ||
      (a->dtype != BRA_FP16 && a->dtype != BRA_BF16) || !format_ok(a->x_format) ||
      !format_ok(a->w_format) || a->reserved != 0 || off_by(a->status, 3u))
    return BRA_ERR_INVALID;
  const int64_t R = a->rows, E = a->groups, K = grad ? a->out : a->in, N = grad ? a->in : a->out;
  const int64_t ld = a->y_pitch ? a->y_pitch : N;
  if (ld < N || ld > (int64_t(1) << 36) || !counts_in_64_bits(R, ld)) return BRA_ERR_INVALID;
  if (!wc || !ws || !counts || (R > 0 && (!xc || !xs || !y))) return BRA_ERR_NULLPTR;
  const int64_t bes = a->dtype == BRA_BF16 ? 4 : 2;
  if (off_by(xc, 15u) || off_by(xs, 15u) || off_by(wc, 15u) || off_by(ws, 3u) || off_by(y, 1u) ||
      off_by(bias, bes - 1) || off_by(counts, 7u))
    return BRA_ERR_INVALID;
  const Span out = {y, span(R, ld, N, 2)};
  const Span ins[6] = {{xc, R * fp8::code_pitch(K)},
                       {xs, R * fp8::scale_pitch(K) * 4},
                       {wc, E * a->out * fp8::code_pitch(a->in)},
                       {ws, E * fp8::blocks(a->out) * fp8::blocks(a->in) * 4},
                       {bias, E * N * bes},
                       {counts, E * 8}};
  if (any_overlap(&out, 1, ins, 6)) return BRA_ERR_INVALID;
  const int rc = clear_status(a->status, st);
  if (rc != BRA_OK || R == 0) return rc;
  const Fp8Problem g = {xc,     xs,          wc,          ws,           bias,         y,
                        counts, a->status,   R,           ld,           (int)E,       (int)a->in,
                        (int)a->out, grad ? 1 : 0, a->dtype, a->x_format, a->w_format};
  if (log_enabled()) {
    const GroupedTile t = fp8_tile(g);
    char how[32] = "";
    if (t.rows == 256) std::snprintf(how, sizeof(how), " by CTA pairs");
    else if (t.split > 1) std::snprintf(how, sizeof(how), ", sums over %d CTAs", t.split);
    std::fprintf(stderr, "[bra] fp8_grouped_matmul%s rows=%lld experts=%d K=%d N=%d -> %dx%d tiles%s\n",
                 grad ? "_grad" : "", (long long)R, g.E, (int)K, (int)N, t.rows, t.cols, how);
  }
  return status_of(launch_fp8_grouped(g, st));
}

}  // namespace

extern "C" {

int64_t fp8_code_bytes(const bra_fp8_args* args) {
  const int rc = check_fp8(args);
  return rc != BRA_OK ? -rc : args->rows * fp8::code_pitch(args->k);
}

int64_t fp8_scale_bytes(const bra_fp8_args* args) {
  const int rc = check_fp8(args);
  if (rc != BRA_OK) return -rc;
  if (args->rows_per_group == 0) return args->rows * fp8::scale_pitch(args->k) * 4;
  return args->groups * fp8::blocks(args->rows_per_group) * fp8::blocks(args->k) * 4;
}

int fp8_quantize(const void* x, const int64_t* counts, uint8_t* codes, float* scales,
                 const bra_fp8_args* args, bra_stream_t stream) {
  int rc = check_fp8(args);
  if (rc != BRA_OK) return rc;
  const int64_t ld = args->x_pitch ? args->x_pitch : args->k;
  if ((rc = check_call(x, ld, counts, codes, scales, args, true)) != BRA_OK) return rc;
  const cudaStream_t st = (cudaStream_t)stream;
  if ((rc = clear_status(args->status, st)) != BRA_OK || args->rows == 0) return rc;
  return status_of(launch_fp8_quantize(data_of(codes, scales, counts, args), x, ld, args->dtype, st));
}

int fp8_dequantize(const uint8_t* codes, const float* scales, const int64_t* counts, void* y,
                   const bra_fp8_args* args, bra_stream_t stream) {
  int rc = check_fp8(args);
  if (rc != BRA_OK) return rc;
  if (args->x_pitch != 0) return BRA_ERR_INVALID;
  if ((rc = check_call(y, args->k, counts, codes, scales, args, false)) != BRA_OK) return rc;
  const cudaStream_t st = (cudaStream_t)stream;
  if ((rc = clear_status(args->status, st)) != BRA_OK || args->rows == 0) return rc;
  return status_of(launch_fp8_dequantize(data_of(codes, scales, counts, args), y, args->dtype, st));
}

int fp8_grouped_matmul(const uint8_t* x_codes, const float* x_scales, const uint8_t* w_codes,
                       const float* w_scales, const void* bias, const int64_t* counts, void* y,
                       const bra_fp8_product_args* args, bra_stream_t stream) {
  return run_product(x_codes, x_scales, w_codes, w_scales, bias, counts, y, args, false,
                     (cudaStream_t)stream);
}

int fp8_grouped_matmul_grad(const uint8_t* dy_codes, const float* dy_scales, const uint8_t* w_codes,
                            const float* w_scales, const int64_t* counts, void* dx,
                            const bra_fp8_product_args* args, bra_stream_t stream) {
  return run_product(dy_codes, dy_scales, w_codes, w_scales, nullptr, counts, dx, args, true,
                     (cudaStream_t)stream);
}

}  // extern "C"
