// Host entry points of the ragged expert operators: argument checks and
// launches.  Every rule cited here is stated in include/bra_moe.h.
#include <cstdio>
#include <cstring>

#include "moe_internal.h"
#include "mx.cuh"

namespace {

using namespace bra;

// Rows of a call: a tile's last row index stays in 32 bits.
constexpr int64_t kMaxRows = (int64_t(1) << 31) - (int64_t(1) << 16);

bool off_by(const void* p, uintptr_t mask) { return (reinterpret_cast<uintptr_t>(p) & mask) != 0; }

bool overlap(const void* a, int64_t an, const void* b, int64_t bn) {
  if (!a || !b || an <= 0 || bn <= 0) return false;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + (uintptr_t)bn && y < x + (uintptr_t)an;
}

// Whether `rows` rows `pitch` elements apart (of at most 8 bytes) count in 64 bits.
bool counts_in_64_bits(int64_t rows, int64_t pitch) {
  return rows <= 0 || pitch <= (int64_t(1) << 59) / rows;
}

// Bytes of `rows` rows of n elements, ld apart (the last one without padding).
int64_t span(int64_t rows, int64_t ld, int64_t n, int64_t es) {
  return rows > 0 ? ((rows - 1) * ld + n) * es : 0;
}

struct GroupedSizes {
  int64_t R, E, K, N, xp, yp;
};

int check_sizes(const bra_grouped_args* a, GroupedSizes* s) {
  if (!a) return BRA_ERR_NULLPTR;
  constexpr int64_t kWide = int64_t(1) << 24;
  if (a->rows < 0 || a->rows > kMaxRows || a->groups < 1 ||
      a->groups > BRA_MAX_GROUPS || a->in < 1 || a->in > kWide || a->out < 1 || a->out > kWide)
    return BRA_ERR_INVALID;
  if (a->dtype != BRA_FP16 && a->dtype != BRA_BF16) return BRA_ERR_INVALID;
  *s = {a->rows, a->groups, a->in, a->out, a->x_pitch ? a->x_pitch : a->in,
        a->y_pitch ? a->y_pitch : a->out};
  if (s->xp < s->K || s->yp < s->N || s->xp > (int64_t(1) << 36) || s->yp > (int64_t(1) << 36) ||
      !counts_in_64_bits(s->R, s->xp) || !counts_in_64_bits(s->R, s->yp))
    return BRA_ERR_INVALID;
  if (off_by(a->status, 3u) || off_by(a->workspace, 255u) || a->workspace_bytes < 0 ||
      (!a->workspace && a->workspace_bytes != 0))
    return BRA_ERR_INVALID;
  return BRA_OK;
}

// An operand's copy: rows of n elements at a pitch of whole 128-byte lines.
struct Copy {
  bool need = false;
  int64_t rows = 0, n = 0, ld = 0, pitch = 0, bytes = 0;
};

Copy copy_of(const void* p, int64_t rows, int64_t n, int64_t ld) {
  Copy c;
  c.rows = rows;
  c.n = n;
  c.ld = ld;
  c.pitch = ld;
  // TMA: 16-byte aligned base and pitch, pitch below 2^40 bytes
  c.need = rows > 0 && (off_by(p, 15u) || ld % 8 != 0);
  if (c.need) {
    c.pitch = (n + 63) / 64 * 64;
    c.bytes = (rows * c.pitch * 2 + 255) / 256 * 256;
  }
  return c;
}

// Hands out workspace; copy() enqueues what was taken, before the products.
// A weight's copy leaves out the experts without rows.
struct Workspace {
  uint8_t* at;
  PackJobs jobs = {};
  const void* take(const void* src, const Copy& c, int64_t per_group = 0) {
    if (!c.need) return src;
    void* dst = at;
    at += c.bytes;
    jobs.job[jobs.n++] = {src, dst, c.ld, c.pitch, c.rows, c.n, per_group};
    return dst;
  }
  int copy(const int64_t* counts, cudaStream_t st) {
    jobs.counts = counts;
    return launch_pack_rows(jobs, st) == cudaSuccess ? BRA_OK : BRA_ERR_CUDA;
  }
};

// What the copies need, against what the caller gave.
int check_workspace(const bra_grouped_args* a, int64_t need) {
  if (need == 0) return BRA_OK;
  if (!a->workspace) return BRA_ERR_UNSUPPORTED;
  return a->workspace_bytes >= need ? BRA_OK : BRA_ERR_INVALID;
}

int status_of(cudaError_t e) {
  return e == cudaSuccess ? BRA_OK : e == cudaErrorInvalidValue ? BRA_ERR_UNSUPPORTED
                                                                : BRA_ERR_CUDA;
}

int clear_status(int32_t* status, cudaStream_t st) {
  if (!status) return BRA_OK;
  return cudaMemsetAsync(status, 0, sizeof(int32_t), st) == cudaSuccess ? BRA_OK : BRA_ERR_CUDA;
}

// Says which kernel a grouped product takes.
void log_tile(const char* what, const GroupedProblem& g, const GroupedTile& t) {
  if (!log_enabled()) return;
  char how[48] = "";
  if (t.rows == 256) std::snprintf(how, sizeof(how), " by CTA pairs");
  else if (t.split > 1) std::snprintf(how, sizeof(how), ", sums over %d CTAs", t.split);
  std::fprintf(stderr, "[bra] %s rows=%lld experts=%d K=%d N=%d -> %dx%d tiles%s\n", what,
               (long long)g.R, g.E, g.K, g.N, t.rows, t.cols, how);
}

// The weight as rows: (E*K) rows of N, or (E*N) rows of K when transposed.
Copy weight_copy(const void* w, const bra_grouped_args* a, const GroupedSizes& s) {
  const int64_t n = a->transpose_weight ? s.K : s.N, rows = a->transpose_weight ? s.N : s.K;
  return copy_of(w, s.E * rows, n, n);
}

int check_mx(const bra_mx_args* a) {
  if (!a) return BRA_ERR_NULLPTR;
  if (a->rows < 0 || a->rows > kMaxRows || a->k < 1 || a->k > (int64_t(1) << 24) ||
      a->groups < 1 || a->groups > BRA_MAX_GROUPS || a->rows_per_group < 0 ||
      a->rows_per_group > kMaxRows || a->reserved != 0)
    return BRA_ERR_INVALID;
  if (a->rows_per_group > 0 && a->rows != a->groups * a->rows_per_group) return BRA_ERR_INVALID;
  if (a->x_pitch != 0 && (a->x_pitch < a->k || a->x_pitch > (int64_t(1) << 36) ||
                          !counts_in_64_bits(a->rows, a->x_pitch)))
    return BRA_ERR_INVALID;
  if (off_by(a->status, 3u)) return BRA_ERR_INVALID;
  return BRA_OK;
}

// The parts of the two conversions that are the same: pointers and sizes.
// `data` is x or y, `ld` its pitch.
int check_mx_call(const void* data, int64_t ld, int64_t es, const int64_t* counts,
                  const uint8_t* codes, const uint8_t* scales, const bra_mx_args* a, bool quantize) {
  if (a->rows > 0 && (!data || !codes || !scales)) return BRA_ERR_NULLPTR;
  if (a->rows > 0 && a->rows_per_group == 0 && !counts) return BRA_ERR_NULLPTR;
  if (off_by(data, es - 1) || off_by(codes, 15u) || off_by(scales, 15u) || off_by(counts, 7u))
    return BRA_ERR_INVALID;
  const int64_t db = span(a->rows, ld, a->k, es), cb = mxfp4_code_bytes(a),
                sb = mxfp4_scale_bytes(a), nb = a->rows_per_group == 0 ? a->groups * 8 : 0;
  if (overlap(data, db, codes, cb) || overlap(data, db, scales, sb)) return BRA_ERR_INVALID;
  if (quantize && (overlap(codes, cb, scales, sb) || overlap(counts, nb, codes, cb) ||
                   overlap(counts, nb, scales, sb)))
    return BRA_ERR_INVALID;
  if (!quantize && overlap(counts, nb, data, db)) return BRA_ERR_INVALID;
  return BRA_OK;
}

MxRows mx_rows(const uint8_t* codes, const uint8_t* scales, const int64_t* counts,
               const bra_mx_args* a) {
  return {const_cast<uint8_t*>(codes),
          const_cast<uint8_t*>(scales),
          a->rows_per_group == 0 ? counts : nullptr,
          a->status,
          a->rows,
          a->k,
          a->rows_per_group,
          (int)a->groups};
}

// A range of memory of a call.
struct Span {
  const void* p;
  int64_t n;
};

// Whether an output overlaps an input or another output.
bool any_overlap(const Span* outs, int no, const Span* ins, int ni) {
  for (int i = 0; i < no; ++i) {
    for (int j = 0; j < ni; ++j)
      if (overlap(outs[i].p, outs[i].n, ins[j].p, ins[j].n)) return true;
    for (int j = 0; j < i; ++j)
      if (overlap(outs[i].p, outs[i].n, outs[j].p, outs[j].n)) return true;
  }
  return false;
}

int64_t element_size(int dtype) { return dtype == BRA_FP32 ? 4 : 2; }

bool row_dtype_ok(int dtype) {
  return dtype == BRA_FP16 || dtype == BRA_BF16 || dtype == BRA_FP32;
}

int check_route(const bra_route_args* a) {
  if (!a) return BRA_ERR_NULLPTR;
  if (a->tokens < 0 || a->experts < 1 || a->experts > BRA_MAX_GROUPS || a->choices < 1 ||
      a->choices > BRA_MAX_CHOICES || a->choices > a->experts ||
      a->tokens >= (int64_t(1) << 31) || a->tokens * a->choices >= (int64_t(1) << 31) ||
      !row_dtype_ok(a->dtype))
    return BRA_ERR_INVALID;
  return BRA_OK;
}

int check_permute(const bra_permute_args* a) {
  if (!a) return BRA_ERR_NULLPTR;
  if (a->tokens < 0 || a->tokens >= (int64_t(1) << 31) || a->rows < 0 ||
      a->rows >= (int64_t(1) << 31) || a->choices < 1 || a->choices > BRA_MAX_CHOICES ||
      a->width < 1 || a->width > (int64_t(1) << 24) || !row_dtype_ok(a->dtype) || a->reserved != 0)
    return BRA_ERR_INVALID;
  return BRA_OK;
}

PermuteCall permute_call(const void* in, void* out, const int32_t* row_tokens, const int32_t* slots,
                         const float* weights, const bra_permute_args* a) {
  return {in,      out,     row_tokens,      slots,         weights,  a->tokens,
          a->rows, (int)a->choices, (int)a->width, a->dtype};
}

// dispatch_grad (weights NULL and unused) and combine.
int run_combine(const void* rows, const int32_t* slots, const float* weights, bool weighted, void* y,
                const bra_permute_args* args, cudaStream_t st) {
  const int rc = check_permute(args);
  if (rc != BRA_OK) return rc;
  if (args->tokens == 0) return BRA_OK;
  if (!slots || !y || (weighted && !weights) || (args->rows > 0 && !rows)) return BRA_ERR_NULLPTR;
  const int64_t es = element_size(args->dtype), n = args->tokens * args->choices * 4;
  if (off_by(rows, es - 1) || off_by(y, es - 1) || off_by(slots, 3u) || off_by(weights, 3u))
    return BRA_ERR_INVALID;
  const Span outs[1] = {{y, args->tokens * args->width * es}};
  const Span ins[3] = {{rows, args->rows * args->width * es}, {slots, n}, {weights, n}};
  if (any_overlap(outs, 1, ins, 3)) return BRA_ERR_INVALID;
  return status_of(launch_combine(permute_call(rows, y, nullptr, slots, weights, args), st));
}

}  // namespace

extern "C" {

int64_t moe_route_workspace_size(const bra_route_args* args) {
  const int rc = check_route(args);
  if (rc != BRA_OK) return -rc;
  const int64_t chunk = route_chunk(args->tokens);
  const int64_t chunks = (args->tokens + chunk - 1) / chunk;
  return chunks > 1 ? (chunks * args->experts * 4 + 255) / 256 * 256 : 0;
}

int moe_route(const void* logits, int32_t* ids, float* weights, int64_t* counts, int32_t* slots,
              int32_t* tokens, void* workspace, int64_t workspace_bytes,
              const bra_route_args* args, bra_stream_t stream) {
  const int64_t need = moe_route_workspace_size(args);
  if (need < 0) return (int)-need;
  const bool some = args->tokens > 0;
  if (!counts || (some && (!logits || !ids || !weights || !slots || !tokens)) ||
      (need > 0 && !workspace))
    return BRA_ERR_NULLPTR;
  const int64_t es = element_size(args->dtype), n = args->tokens * args->choices * 4;
  if (off_by(logits, es - 1) || off_by(ids, 3u) || off_by(weights, 3u) || off_by(counts, 7u) ||
      off_by(slots, 3u) || off_by(tokens, 3u) || off_by(workspace, 255u) || workspace_bytes < need)
    return BRA_ERR_INVALID;
  const Span outs[6] = {{ids, n},   {weights, n}, {counts, args->experts * 8},
                        {slots, n}, {tokens, n},  {workspace, need}};
  const Span ins[1] = {{logits, args->tokens * args->experts * es}};
  if (any_overlap(outs, 6, ins, 1)) return BRA_ERR_INVALID;
  const cudaStream_t st = (cudaStream_t)stream;
  if (!some)
    return cudaMemsetAsync(counts, 0, (size_t)args->experts * 8, st) == cudaSuccess ? BRA_OK
                                                                                    : BRA_ERR_CUDA;
  const RouteCall r = {logits,       ids,
                       weights,      counts,
                       slots,        tokens,
                       static_cast<int32_t*>(workspace),
                       args->tokens, (int)args->experts,
                       (int)args->choices, args->renormalize ? 1 : 0,
                       args->dtype};
  return status_of(launch_route(r, st));
}

int moe_route_grad(const float* dweights, const void* logits, const int32_t* ids,
                   const float* weights, void* dlogits, const bra_route_args* args,
                   bra_stream_t stream) {
  const int rc = check_route(args);
  if (rc != BRA_OK) return rc;
  if (args->tokens == 0) return BRA_OK;
  if (!dweights || !ids || !weights || !dlogits || (!args->renormalize && !logits))
    return BRA_ERR_NULLPTR;
  const int64_t es = element_size(args->dtype), n = args->tokens * args->choices * 4,
                lb = args->tokens * args->experts * es;
  if (off_by(logits, es - 1) || off_by(dlogits, es - 1) || off_by(dweights, 3u) || off_by(ids, 3u) ||
      off_by(weights, 3u))
    return BRA_ERR_INVALID;
  const Span outs[1] = {{dlogits, lb}};
  const Span ins[4] = {{dweights, n}, {ids, n}, {weights, n}, {logits, lb}};
  if (any_overlap(outs, 1, ins, 4)) return BRA_ERR_INVALID;
  const RouteGradCall r = {dweights,     logits,
                           ids,          weights,
                           dlogits,      args->tokens,
                           (int)args->experts, (int)args->choices,
                           args->renormalize ? 1 : 0, args->dtype};
  return status_of(launch_route_grad(r, (cudaStream_t)stream));
}

int64_t moe_dispatch_workspace_size(const bra_permute_args* args) {
  const int rc = check_permute(args);
  if (rc != BRA_OK) return -rc;
  if (!dispatch_lists(args->tokens, args->rows, args->width * element_size(args->dtype))) return 0;
  return (args->tokens * (BRA_MAX_CHOICES + 1) * 4 + 255) / 256 * 256;
}

int moe_dispatch(const void* x, const int32_t* tokens, void* xs, void* workspace,
                 int64_t workspace_bytes, const bra_permute_args* args, bra_stream_t stream) {
  const int64_t need = moe_dispatch_workspace_size(args);
  if (need < 0) return (int)-need;
  if (args->rows == 0) return BRA_OK;
  if (!tokens || !xs || (args->tokens > 0 && !x) || (need > 0 && !workspace))
    return BRA_ERR_NULLPTR;
  const int64_t es = element_size(args->dtype);
  if (off_by(x, es - 1) || off_by(xs, es - 1) || off_by(tokens, 3u) || off_by(workspace, 255u) ||
      workspace_bytes < need)
    return BRA_ERR_INVALID;
  const Span outs[2] = {{xs, args->rows * args->width * es}, {workspace, need}};
  const Span ins[2] = {{x, args->tokens * args->width * es}, {tokens, args->rows * 4}};
  if (any_overlap(outs, 2, ins, 2)) return BRA_ERR_INVALID;
  return status_of(launch_dispatch(permute_call(x, xs, tokens, nullptr, nullptr, args), workspace,
                                   (cudaStream_t)stream));
}

int moe_dispatch_grad(const void* dxs, const int32_t* slots, void* dx, const bra_permute_args* args,
                      bra_stream_t stream) {
  return run_combine(dxs, slots, nullptr, false, dx, args, (cudaStream_t)stream);
}

int moe_combine(const void* ys, const int32_t* slots, const float* weights, void* y,
                const bra_permute_args* args, bra_stream_t stream) {
  return run_combine(ys, slots, weights, true, y, args, (cudaStream_t)stream);
}

int moe_combine_grad(const void* dy, const void* ys, const int32_t* slots, const float* weights,
                     const int32_t* tokens, void* dys, float* dweights,
                     const bra_permute_args* args, bra_stream_t stream) {
  const int rc = check_permute(args);
  if (rc != BRA_OK) return rc;
  if (args->tokens == 0 && args->rows == 0) return BRA_OK;
  if ((args->tokens > 0 && (!dy || !slots || !weights || !dweights)) ||
      (args->rows > 0 && (!ys || !dys)))
    return BRA_ERR_NULLPTR;
  const int64_t es = element_size(args->dtype), n = args->tokens * args->choices * 4,
                rb = args->rows * args->width * es;
  if (off_by(dy, es - 1) || off_by(ys, es - 1) || off_by(dys, es - 1) || off_by(slots, 3u) ||
      off_by(weights, 3u) || off_by(tokens, 3u) || off_by(dweights, 3u))
    return BRA_ERR_INVALID;
  const Span outs[2] = {{dys, rb}, {dweights, n}};
  const Span ins[5] = {{dy, args->tokens * args->width * es}, {ys, rb}, {slots, n}, {weights, n},
                       {tokens, tokens ? args->rows * 4 : 0}};
  if (any_overlap(outs, 2, ins, 5)) return BRA_ERR_INVALID;
  return status_of(launch_combine_grad(permute_call(dy, dys, tokens, slots, weights, args), ys,
                                       dweights, (cudaStream_t)stream));
}

int64_t mxfp4_code_bytes(const bra_mx_args* args) {
  const int rc = check_mx(args);
  return rc != BRA_OK ? -rc : args->rows * mx::code_pitch(args->k);
}

int64_t mxfp4_scale_bytes(const bra_mx_args* args) {
  const int rc = check_mx(args);
  if (rc != BRA_OK) return -rc;
  return mx::blocks_of(args->rows, args->groups, args->rows_per_group) * mx::units(args->k) *
         mx::kUnitBytes;
}

int mxfp4_quantize(const void* x, const int64_t* counts, uint8_t* codes, uint8_t* scales,
                   const bra_mx_args* args, bra_stream_t stream) {
  int rc = check_mx(args);
  if (rc != BRA_OK) return rc;
  if (args->dtype != BRA_FP16 && args->dtype != BRA_BF16) return BRA_ERR_INVALID;
  const int64_t ld = args->x_pitch ? args->x_pitch : args->k;
  if ((rc = check_mx_call(x, ld, 2, counts, codes, scales, args, true)) != BRA_OK) return rc;
  const cudaStream_t st = (cudaStream_t)stream;
  if ((rc = clear_status(args->status, st)) != BRA_OK || args->rows == 0) return rc;
  return status_of(launch_mx_quantize(mx_rows(codes, scales, counts, args), x, ld, args->dtype, st));
}

int mxfp4_dequantize(const uint8_t* codes, const uint8_t* scales, const int64_t* counts, void* y,
                     const bra_mx_args* args, bra_stream_t stream) {
  int rc = check_mx(args);
  if (rc != BRA_OK) return rc;
  if ((args->dtype != BRA_FP16 && args->dtype != BRA_BF16 && args->dtype != BRA_FP32) ||
      args->x_pitch != 0)
    return BRA_ERR_INVALID;
  const int64_t es = args->dtype == BRA_FP32 ? 4 : 2;
  if ((rc = check_mx_call(y, args->k, es, counts, codes, scales, args, false)) != BRA_OK) return rc;
  const cudaStream_t st = (cudaStream_t)stream;
  if ((rc = clear_status(args->status, st)) != BRA_OK || args->rows == 0) return rc;
  return status_of(launch_mx_dequantize(mx_rows(codes, scales, counts, args), y, args->dtype, st));
}

int mxfp4_grouped_matmul(const uint8_t* x_codes, const uint8_t* x_scales, const uint8_t* w_codes,
                         const uint8_t* w_scales, const void* bias, const int64_t* counts, void* y,
                         const bra_grouped_args* args, bra_stream_t stream) {
  GroupedSizes s;
  int rc = check_sizes(args, &s);
  if (rc != BRA_OK) return rc;
  if (args->x_pitch != 0 || args->transpose_weight != 0) return BRA_ERR_INVALID;
  if (!w_codes || !w_scales || !counts || (s.R > 0 && (!x_codes || !x_scales || !y)))
    return BRA_ERR_NULLPTR;
  const int64_t bes = args->dtype == BRA_BF16 ? 4 : 2;
  if (off_by(x_codes, 15u) || off_by(x_scales, 15u) || off_by(w_codes, 15u) ||
      off_by(w_scales, 15u) || off_by(y, 1u) || off_by(bias, bes - 1) || off_by(counts, 7u))
    return BRA_ERR_INVALID;
  const int64_t cp = mx::code_pitch(s.K), unit = mx::units(s.K) * mx::kUnitBytes;
  const int64_t yb = span(s.R, s.yp, s.N, 2);
  if (overlap(y, yb, x_codes, s.R * cp) ||
      overlap(y, yb, x_scales, mx::blocks_of(s.R, s.E, 0) * unit) ||
      overlap(y, yb, w_codes, s.E * s.N * cp) ||
      overlap(y, yb, w_scales, mx::blocks_of(s.E * s.N, s.E, s.N) * unit) ||
      overlap(y, yb, bias, s.E * s.N * bes) || overlap(y, yb, counts, s.E * 8))
    return BRA_ERR_INVALID;
  const cudaStream_t st = (cudaStream_t)stream;
  if ((rc = clear_status(args->status, st)) != BRA_OK || s.R == 0) return rc;
  const MxProblem g = {x_codes, x_scales, w_codes,      w_scales, bias,
                       y,       counts,   args->status, s.R,      s.yp,
                       (int)s.E, (int)s.K, (int)s.N,     args->dtype};
  if (log_enabled())
    std::fprintf(stderr, "[bra] mxfp4_grouped_matmul rows=%lld experts=%d K=%d N=%d -> %s\n",
                 (long long)g.R, g.E, g.K, g.N,
                 mx_pair(g) ? "256x256 tiles by CTA pairs" : "128x128 tiles");
  return status_of(launch_mx_grouped(g, st));
}

int64_t grouped_matmul_workspace_size(const void* x, const void* weight,
                                      const bra_grouped_args* args) {
  GroupedSizes s;
  const int rc = check_sizes(args, &s);
  if (rc != BRA_OK) return -rc;
  if (s.R == 0) return 0;
  return copy_of(x, s.R, s.K, s.xp).bytes + weight_copy(weight, args, s).bytes;
}

int64_t grouped_matmul_grad_workspace_size(const void* dy, const void* x, const void* weight,
                                           int want_dx, int want_dweight,
                                           const bra_grouped_args* args) {
  GroupedSizes s;
  const int rc = check_sizes(args, &s);
  if (rc != BRA_OK) return -rc;
  if (s.R == 0) return 0;
  int64_t n = 0;
  if (want_dx || want_dweight) n += copy_of(dy, s.R, s.N, s.yp).bytes;
  if (want_dx) n += weight_copy(weight, args, s).bytes;
  if (want_dweight) n += copy_of(x, s.R, s.K, s.xp).bytes;
  return n;
}

int grouped_matmul(const void* x, const void* weight, const void* bias, const int64_t* counts,
                   void* y, const bra_grouped_args* args, bra_stream_t stream) {
  GroupedSizes s;
  int rc = check_sizes(args, &s);
  if (rc != BRA_OK) return rc;
  if (!weight || !counts || (s.R > 0 && (!x || !y))) return BRA_ERR_NULLPTR;
  const int64_t bes = args->dtype == BRA_BF16 ? 4 : 2;
  if (off_by(x, 1u) || off_by(weight, 1u) || off_by(y, 1u) || off_by(bias, bes - 1) ||
      off_by(counts, 7u))
    return BRA_ERR_INVALID;
  const Copy cx = copy_of(x, s.R, s.K, s.xp), cw = weight_copy(weight, args, s);
  const int64_t yb = span(s.R, s.yp, s.N, 2);
  if (overlap(y, yb, x, span(s.R, s.xp, s.K, 2)) || overlap(y, yb, weight, s.E * s.K * s.N * 2) ||
      overlap(y, yb, bias, s.E * s.N * bes) || overlap(y, yb, counts, s.E * 8) ||
      overlap(y, yb, args->workspace, args->workspace_bytes))
    return BRA_ERR_INVALID;
  const cudaStream_t st = (cudaStream_t)stream;
  if (s.R == 0) return clear_status(args->status, st);
  const int64_t need = cx.bytes + cw.bytes;
  if ((rc = check_workspace(args, need)) != BRA_OK) return rc;
  const Span ins[4] = {{x, span(s.R, s.xp, s.K, 2)},
                       {weight, s.E * s.K * s.N * 2},
                       {bias, s.E * s.N * bes},
                       {counts, s.E * 8}};
  const Span ws_used[1] = {{args->workspace, need}};
  if (any_overlap(ws_used, 1, ins, 4)) return BRA_ERR_INVALID;
  if ((rc = clear_status(args->status, st)) != BRA_OK) return rc;
  Workspace ws{static_cast<uint8_t*>(args->workspace)};
  GroupedProblem g;
  std::memset(&g, 0, sizeof(g));
  g.x = ws.take(x, cx);
  g.w = ws.take(weight, cw, cw.rows / s.E);
  if ((rc = ws.copy(counts, st)) != BRA_OK) return rc;
  g.bias = bias;
  g.y = y;
  g.counts = counts;
  g.status = args->status;
  g.R = s.R;
  g.ldx = cx.pitch;
  g.ldw = cw.pitch;
  g.ldy = s.yp;
  g.E = (int)s.E;
  g.K = (int)s.K;
  g.N = (int)s.N;
  g.dtype = args->dtype;
  g.wt = args->transpose_weight ? 1 : 0;
  log_tile("grouped_matmul", g, grouped_fwd_tile(g));
  return status_of(launch_grouped_fwd(g, st));
}

int grouped_matmul_grad(const void* dy, const void* x, const void* weight, const int64_t* counts,
                        void* dx, void* dweight, void* dbias, const bra_grouped_args* args,
                        bra_stream_t stream) {
  GroupedSizes s;
  int rc = check_sizes(args, &s);
  if (rc != BRA_OK) return rc;
  if (!counts || (!dx && !dweight && !dbias) || (s.R > 0 && !dy) || (dx && !weight) ||
      (dweight && s.R > 0 && !x))
    return BRA_ERR_NULLPTR;
  const int64_t bes = args->dtype == BRA_BF16 ? 4 : 2;
  if (off_by(dy, 1u) || off_by(x, 1u) || off_by(weight, 1u) || off_by(dx, 1u) ||
      off_by(dweight, 1u) || off_by(dbias, bes - 1) || off_by(counts, 7u))
    return BRA_ERR_INVALID;
  const bool wt = args->transpose_weight != 0;
  const Copy cd = copy_of(dy, s.R, s.N, s.yp), cx = copy_of(x, s.R, s.K, s.xp),
             cw = weight_copy(weight, args, s);
  const int64_t wb = s.E * s.K * s.N * 2;
  const Span outs[3] = {{dx, s.R * s.K * 2}, {dweight, wb}, {dbias, s.E * s.N * bes}};
  const Span ins[5] = {{dy, span(s.R, s.yp, s.N, 2)},
                       {x, span(s.R, s.xp, s.K, 2)},
                       {weight, wb},
                       {counts, s.E * 8},
                       {args->workspace, args->workspace_bytes}};
  if (any_overlap(outs, 3, ins, 5)) return BRA_ERR_INVALID;
  const cudaStream_t st = (cudaStream_t)stream;
  if (s.R == 0) {
    if (dweight && cudaMemsetAsync(dweight, 0, (size_t)wb, st) != cudaSuccess) return BRA_ERR_CUDA;
    if (dbias && cudaMemsetAsync(dbias, 0, (size_t)(s.E * s.N * bes), st) != cudaSuccess)
      return BRA_ERR_CUDA;
    return clear_status(args->status, st);
  }
  const int64_t need = (dx || dweight ? cd.bytes : 0) + (dx ? cw.bytes : 0) + (dweight ? cx.bytes : 0);
  if ((rc = check_workspace(args, need)) != BRA_OK) return rc;
  const Span ws_used[1] = {{args->workspace, need}};
  if (any_overlap(ws_used, 1, ins, 4)) return BRA_ERR_INVALID;
  if ((rc = clear_status(args->status, st)) != BRA_OK) return rc;
  Workspace ws{static_cast<uint8_t*>(args->workspace)};
  GroupedProblem g;
  std::memset(&g, 0, sizeof(g));
  g.counts = counts;
  g.status = args->status;
  g.R = s.R;
  g.E = (int)s.E;
  g.dtype = args->dtype;
  const void* d = dx || dweight ? ws.take(dy, cd) : dy;
  const void* w = dx ? ws.take(weight, cw, cw.rows / s.E) : weight;
  const void* xs = dweight ? ws.take(x, cx) : x;
  if ((rc = ws.copy(counts, st)) != BRA_OK) return rc;
  if (dx) {
    // dx = dy W^T: the contraction runs over N, the weight's layout as stored
    // is the other one seen from here
    g.x = d;
    g.w = w;
    g.y = dx;
    g.ldx = cd.pitch;
    g.ldw = cw.pitch;
    g.ldy = s.K;
    g.K = (int)s.N;
    g.N = (int)s.K;
    g.wt = wt ? 0 : 1;
    log_tile("grouped_matmul_grad dx", g, grouped_fwd_tile(g));
    if ((rc = status_of(launch_grouped_fwd(g, st))) != BRA_OK) return rc;
  }
  if (dweight) {
    // (E, N, K) gradients are the same product with the operands exchanged
    g.x = wt ? d : xs;
    g.w = wt ? xs : d;
    g.ldx = wt ? cd.pitch : cx.pitch;
    g.ldw = wt ? cx.pitch : cd.pitch;
    g.y = dweight;
    g.K = (int)(wt ? s.N : s.K);
    g.N = (int)(wt ? s.K : s.N);
    g.ldy = g.N;
    g.wt = 0;
    g.late = dx != nullptr;      // the gradients do not need each other
    log_tile("grouped_matmul_grad dweight", g, grouped_wgrad_tile(g));
    if ((rc = status_of(launch_grouped_wgrad(g, st))) != BRA_OK) return rc;
  }
  if (dbias) {
    BiasGradProblem b = {dy,        dbias,    counts,      args->status,     s.R, s.yp,
                         (int)s.E, (int)s.N, args->dtype, dx || dweight};
    if ((rc = status_of(launch_bias_grad(b, st))) != BRA_OK) return rc;
  }
  return BRA_OK;
}

}  // extern "C"
