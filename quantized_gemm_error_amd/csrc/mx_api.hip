// C ABI of microscaled matrices and of sampling (spear_mx.h, spear_sample.h):
// host-side validation before any launch.
#include <math.h>

#include <algorithm>

#include "api_common.h"
#include "mx_internal.h"

using namespace spear;

namespace {

constexpr int32_t kMaxRows = 1 << 24, kMaxCols = 1 << 20, kMaxHidden = 65536;
constexpr int64_t kMaxStride = int64_t(1) << 40;

bool valid_sizes(int32_t format, int32_t rows, int32_t cols) {
  return (format == SPEAR_MXFP4 || format == SPEAR_MXFP8) && rows >= 0 && rows <= kMaxRows &&
         cols >= 1 && cols <= kMaxCols;
}

spear_status_t check_mx(const char *name, const spear_mx_t *m) {
  if (!m) return fail(SPEAR_ERR_INVALID_ARGUMENT, "%s is NULL", name);
  if (m->format != SPEAR_MXFP4 && m->format != SPEAR_MXFP8)
    return fail(SPEAR_ERR_INVALID_ARGUMENT, "%s: format=%d is not SPEAR_MXFP4 or SPEAR_MXFP8", name, m->format);
  if (m->rows < 0 || m->cols < 1)
    return fail(SPEAR_ERR_INVALID_ARGUMENT, "%s: rows=%d cols=%d", name, m->rows, m->cols);
  if (!valid_sizes(m->format, m->rows, m->cols))
    return fail(SPEAR_ERR_UNSUPPORTED, "%s: rows=%d above %d or cols=%d above %d", name, m->rows, kMaxRows,
                m->cols, kMaxCols);
  const MxDesc d = mx_desc(*m);
  // (a grid of 256 threads for each group of 16 x 512 values stays below 2^32 threads)
  if ((int64_t)d.rb * d.kq >= (1 << 24))
    return fail(SPEAR_ERR_UNSUPPORTED, "%s: %d x %d values in one matrix", name, m->rows, m->cols);
  if (m->rows == 0) return SPEAR_OK;
  if (!m->codes || !m->scales) return fail(SPEAR_ERR_INVALID_ARGUMENT, "%s: codes and scales must not be NULL", name);
  if (!aligned(m->codes, 256) || !aligned(m->scales, 256))
    return fail(SPEAR_ERR_INVALID_ARGUMENT, "%s: codes and scales must be 256-byte aligned", name);
  return SPEAR_OK;
}

spear_status_t check_rows(const char *name, const void *p, int32_t dtype, int64_t stride, int64_t least) {
  if (!p) return fail(SPEAR_ERR_INVALID_ARGUMENT, "%s must not be NULL", name);
  if (!aligned(p, dtype == SPEAR_F32 ? 4 : 2)) return fail(SPEAR_ERR_INVALID_ARGUMENT, "%s is not aligned to its type", name);
  if (stride < least || stride > kMaxStride)
    return fail(SPEAR_ERR_INVALID_ARGUMENT, "%s: stride=%lld below %lld or too large", name, (long long)stride,
                (long long)least);
  return SPEAR_OK;
}

spear_status_t check_type(const char *name, int32_t dtype, bool f32) {
  if (dtype != SPEAR_F16 && dtype != SPEAR_BF16 && !(f32 && dtype == SPEAR_F32))
    return fail(SPEAR_ERR_INVALID_ARGUMENT, "%s=%d is not SPEAR_F16%s SPEAR_BF16%s", name, dtype,
                f32 ? "," : " or", f32 ? " or SPEAR_F32" : "");
  return SPEAR_OK;
}

spear_status_t check_workspace(const void *ws, size_t bytes, size_t need) {
  if (!ws) return fail(SPEAR_ERR_WORKSPACE, "workspace of %zu bytes required, got NULL", need);
  if (!aligned(ws, 256)) return fail(SPEAR_ERR_WORKSPACE, "workspace not 256-byte aligned");
  if (bytes < need) return fail(SPEAR_ERR_WORKSPACE, "workspace of %zu bytes required, got %zu", need, bytes);
  return SPEAR_OK;
}

// Whether `bytes` from p on lie in the `need` bytes of the workspace, which the call writes.
spear_status_t check_apart(const char *name, const void *p, size_t bytes, const void *ws, size_t need) {
  const uintptr_t a = (uintptr_t)p, w = (uintptr_t)ws;
  if (p && a < w + need && w < a + bytes)
    return fail(SPEAR_ERR_INVALID_ARGUMENT, "%s overlaps the workspace", name);
  return SPEAR_OK;
}
// Bytes from the first to the last element of rows of cols elements.
size_t row_bytes(int32_t rows, int64_t stride, int32_t cols, int32_t dtype) {
  return ((size_t)(rows - 1) * stride + cols) * (dtype == SPEAR_F32 ? 4 : 2);
}

size_t code_bytes(int32_t format, const MxDesc &d) {
  return (size_t)d.rb * d.kt * (format == SPEAR_MXFP4 ? 1024 : 2048);
}
size_t scale_bytes(const MxDesc &d) { return (size_t)d.rb * d.kq * 256; }

MxDesc sizes_of(int32_t format, int32_t rows, int32_t cols) {
  return mx_desc(spear_mx_t{format, rows, cols, nullptr, nullptr});
}

}  // namespace

extern "C" {

size_t spear_mx_code_bytes(int32_t format, int32_t rows, int32_t cols) {
  return valid_sizes(format, rows, cols) ? code_bytes(format, sizes_of(format, rows, cols)) : 0;
}

size_t spear_mx_scale_bytes(int32_t format, int32_t rows, int32_t cols) {
  return valid_sizes(format, rows, cols) ? scale_bytes(sizes_of(format, rows, cols)) : 0;
}

spear_status_t spear_mx_quantize(const void *x, int32_t dtype, int64_t stride, const spear_mx_t *out,
                                 spear_stream_t stream) {
  TRY(check_mx("out", out));
  TRY(check_type("dtype", dtype, true));
  if (out->rows == 0) return ok();
  TRY(check_rows("x", x, dtype, stride, 0));
  return hip_status(launch_mx_quantize(x, dtype, stride, out->format, mx_desc(*out), (hipStream_t)stream),
                    "quantize launch");
}

spear_status_t spear_mx_dequantize(const spear_mx_t *x, void *out, int32_t dtype, int64_t stride,
                                   spear_stream_t stream) {
  TRY(check_mx("x", x));
  TRY(check_type("dtype", dtype, true));
  if (x->rows == 0) return ok();
  TRY(check_rows("out", out, dtype, stride, x->rows > 1 ? x->cols : 0));
  return hip_status(launch_mx_dequantize(mx_desc(*x), x->format, out, dtype, stride, (hipStream_t)stream),
                    "dequantize launch");
}

spear_status_t spear_rms_norm(const spear_norm_args_t *a, spear_stream_t stream) {
  if (!a) return fail(SPEAR_ERR_INVALID_ARGUMENT, "args is NULL");
  TRY(check_type("dtype", a->dtype, false));
  if (a->rows < 0 || a->hidden < 1)
    return fail(SPEAR_ERR_INVALID_ARGUMENT, "rows=%d hidden=%d", a->rows, a->hidden);
  if (a->rows > kMaxRows || a->hidden > kMaxHidden)
    return fail(SPEAR_ERR_UNSUPPORTED, "rows=%d above %d or hidden=%d above %d", a->rows, kMaxRows, a->hidden, kMaxHidden);
  if (!(a->eps >= 0) || !isfinite(a->eps)) return fail(SPEAR_ERR_INVALID_ARGUMENT, "eps is negative or not finite");
  // (no rows: an empty array may have no address)
  if ((a->out && a->out_mx) || (a->rows > 0 && !a->out && !a->out_mx))
    return fail(SPEAR_ERR_INVALID_ARGUMENT, "one of out and out_mx must be given");
  if (!a->residual != !a->residual_out)
    return fail(SPEAR_ERR_INVALID_ARGUMENT, "residual and residual_out come together");
  if (a->out_mx) {
    TRY(check_mx("out_mx", a->out_mx));
    if (a->out_mx->rows != a->rows || a->out_mx->cols != a->hidden)
      return fail(SPEAR_ERR_INVALID_ARGUMENT, "out_mx is %d x %d for rows=%d hidden=%d", a->out_mx->rows,
                  a->out_mx->cols, a->rows, a->hidden);
  }
  if (a->rows == 0) return ok();
  const int64_t apart = a->rows > 1 ? a->hidden : 0;
  TRY(check_rows("x", a->x, a->dtype, a->x_stride, 0));
  TRY(check_rows("weight", a->weight, a->dtype, 0, 0));
  if (a->residual) {
    TRY(check_rows("residual", a->residual, a->dtype, a->residual_stride, 0));
    TRY(check_rows("residual_out", a->residual_out, a->dtype, a->residual_out_stride, apart));
    if (a->residual_out == a->out) return fail(SPEAR_ERR_INVALID_ARGUMENT, "out and residual_out are one array");
  }
  if (a->out) TRY(check_rows("out", a->out, a->dtype, a->out_stride, apart));
  // (a row is read whole before any of it is written, so the same rows may be input and output)
  const struct { const void *in, *out; int64_t s_in, s_out; } same[] = {
      {a->x, a->out, a->x_stride, a->out_stride}, {a->x, a->residual_out, a->x_stride, a->residual_out_stride},
      {a->residual, a->out, a->residual_stride, a->out_stride},
      {a->residual, a->residual_out, a->residual_stride, a->residual_out_stride}};
  for (const auto &p : same)
    if (p.in && p.in == p.out && p.s_in != p.s_out && a->rows > 1)
      return fail(SPEAR_ERR_INVALID_ARGUMENT, "an output in an input's place must have its stride");
  NormDesc d{};
  d.rows = a->rows;
  d.hidden = a->hidden;
  d.x = (const uint16_t *)a->x;
  d.residual = (const uint16_t *)a->residual;
  d.weight = (const uint16_t *)a->weight;
  d.x_stride = a->x_stride;
  d.residual_stride = a->residual_stride;
  d.residual_out_stride = a->residual_out_stride;
  d.out_stride = a->out_stride;
  d.residual_out = (uint16_t *)a->residual_out;
  d.out = (uint16_t *)a->out;
  if (a->out_mx) d.mx = mx_desc(*a->out_mx);
  d.eps = a->eps;
  return hip_status(launch_rms_norm(d, a->dtype, a->out_mx ? a->out_mx->format : -1, (hipStream_t)stream),
                    "norm launch");
}

size_t spear_mx_workspace_bytes(const spear_mx_t *w, int32_t n_tokens) {
  if (!w || !valid_sizes(w->format, w->rows, w->cols) || !valid_sizes(SPEAR_MXFP8, n_tokens, w->cols)) return 0;
  const MxDesc x = sizes_of(SPEAR_MXFP8, n_tokens, w->cols);
  return std::max(code_bytes(SPEAR_MXFP8, x) + scale_bytes(x), size_t(256));
}

spear_status_t spear_mx_linear(const spear_mx_linear_args_t *a, void *ws, size_t ws_bytes, spear_stream_t stream) {
  if (!a) return fail(SPEAR_ERR_INVALID_ARGUMENT, "args is NULL");
  TRY(check_mx("w", a->w));
  if (a->w->format != SPEAR_MXFP4) return fail(SPEAR_ERR_UNSUPPORTED, "w must be SPEAR_MXFP4");
  TRY(check_type("y_dtype", a->y_dtype, true));
  if (!a->x_mx == !a->x) {
    if (a->x || a->n_tokens != 0)
      return fail(SPEAR_ERR_INVALID_ARGUMENT, "one of x and x_mx must be given");
    return ok();
  }
  MxLinearDesc d{};
  const int N = a->w->rows, K = a->w->cols;
  int M, x_format;
  spear_mx_t x{};
  if (a->x_mx) {
    TRY(check_mx("x_mx", a->x_mx));
    if (a->x_mx->cols != K) return fail(SPEAR_ERR_INVALID_ARGUMENT, "x_mx has %d columns, w %d", a->x_mx->cols, K);
    x = *a->x_mx;
    M = x.rows;
    x_format = x.format;
  } else {
    TRY(check_type("x_dtype", a->x_dtype, false));
    if (a->x_format != SPEAR_MXFP4 && a->x_format != SPEAR_MXFP8)
      return fail(SPEAR_ERR_INVALID_ARGUMENT, "x_format=%d is not SPEAR_MXFP4 or SPEAR_MXFP8", a->x_format);
    if (a->n_tokens < 0) return fail(SPEAR_ERR_INVALID_ARGUMENT, "n_tokens=%d", a->n_tokens);
    if (!valid_sizes(a->x_format, a->n_tokens, K)) return fail(SPEAR_ERR_UNSUPPORTED, "n_tokens=%d too large", a->n_tokens);
    M = a->n_tokens;
    x_format = a->x_format;
    if (M > 0) TRY(check_rows("x", a->x, a->x_dtype, a->x_stride, 0));
    const MxDesc s = sizes_of(x_format, M, K);
    if ((int64_t)s.rb * s.kq >= (1 << 24)) return fail(SPEAR_ERR_UNSUPPORTED, "%d x %d tokens in one call", M, K);
  }
  if (M == 0 || N == 0) return ok();
  TRY(check_rows("y", a->y, a->y_dtype, a->y_stride, M > 1 ? N : 0));
  if ((int64_t)mx_desc(*a->w).rb * ((M + 15) / 16) >= (1 << 24))
    return fail(SPEAR_ERR_UNSUPPORTED, "%d x %d outputs in one call", M, N);
  if (!a->x_mx) {
    const size_t need = spear_mx_workspace_bytes(a->w, M);
    TRY(check_workspace(ws, ws_bytes, need));
    TRY(check_apart("x", a->x, row_bytes(M, a->x_stride, K, a->x_dtype), ws, need));
    TRY(check_apart("y", a->y, row_bytes(M, a->y_stride, N, a->y_dtype), ws, need));
    TRY(check_apart("w", a->w->codes, code_bytes(SPEAR_MXFP4, mx_desc(*a->w)), ws, need));
    TRY(check_apart("w", a->w->scales, scale_bytes(mx_desc(*a->w)), ws, need));
    const size_t codes = code_bytes(x_format, sizes_of(x_format, M, K));  // (a multiple of 1024)
    x = spear_mx_t{x_format, M, K, ws, (char *)ws + codes};
    if (mx_linear_quantizes(M, K) && aligned(a->x, 16) && a->x_stride % 8 == 0) {
      d.x16 = (const uint16_t *)a->x;
      d.x16_dtype = a->x_dtype;
      d.x16_stride = a->x_stride;
    } else {
      const hipError_t e = launch_mx_quantize(a->x, a->x_dtype, a->x_stride, x_format, mx_desc(x), (hipStream_t)stream);
      if (e != hipSuccess) return hip_status(e, "token quantize launch");
    }
  }
  d.w = mx_desc(*a->w);
  d.x = mx_desc(x);
  d.x_format = x_format;
  d.y = a->y;
  d.y_dtype = a->y_dtype;
  d.y_stride = a->y_stride;
  const size_t elem = a->y_dtype == SPEAR_F32 ? 4 : 2;
  d.y_vec = aligned(a->y, 4 * elem) && a->y_stride % 4 == 0;
  d.y_vec16 = aligned(a->y, 16) && a->y_stride * elem % 16 == 0;
  return hip_status(launch_mx_linear(d, (hipStream_t)stream), "linear launch");
}

size_t spear_sample_workspace_bytes(int32_t rows, int32_t vocab) {
  if (rows < 0 || rows > (1 << 20) || vocab < 1 || vocab > (1 << 18)) return 0;
  return sample_workspace(rows, vocab);
}

spear_status_t spear_sample(const spear_sample_args_t *a, void *ws, size_t ws_bytes, spear_stream_t stream) {
  if (!a) return fail(SPEAR_ERR_INVALID_ARGUMENT, "args is NULL");
  TRY(check_type("dtype", a->dtype, true));
  if (a->rows < 0 || a->vocab < 1) return fail(SPEAR_ERR_INVALID_ARGUMENT, "rows=%d vocab=%d", a->rows, a->vocab);
  const size_t need = spear_sample_workspace_bytes(a->rows, a->vocab);
  if (need == 0) return fail(SPEAR_ERR_UNSUPPORTED, "rows=%d above 2^20 or vocab=%d above 2^18", a->rows, a->vocab);
  if (a->rows == 0) return ok();
  TRY(check_rows("logits", a->logits, a->dtype, a->stride, 0));
  if (!a->u || !a->tokens) return fail(SPEAR_ERR_INVALID_ARGUMENT, "u and tokens must not be NULL");
  if (!aligned(a->u, 4) || !aligned(a->temperature, 4) || !aligned(a->top_k, 4) || !aligned(a->top_p, 4) ||
      !aligned(a->min_p, 4) || !aligned(a->tokens, 4) || !aligned(a->logprobs, 4))
    return fail(SPEAR_ERR_INVALID_ARGUMENT, "the per-row arrays must be 4-byte aligned");
  TRY(check_workspace(ws, ws_bytes, need));
  TRY(check_apart("logits", a->logits, row_bytes(a->rows, a->stride, a->vocab, a->dtype), ws, need));
  const void *const per_row[] = {a->u, a->temperature, a->top_k, a->top_p, a->min_p, a->tokens, a->logprobs};
  for (const void *p : per_row) TRY(check_apart("a per-row array", p, (size_t)a->rows * 4, ws, need));
  return hip_status(launch_sample(*a, ws, (hipStream_t)stream), "sample launch");
}

}  // extern "C"
