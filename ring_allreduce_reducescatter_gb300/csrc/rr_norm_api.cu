// rr_norm_api.cu -- the C ABI of layer norm (include/ringred.h): argument
// checks, all on the host and before any CUDA call, and the parameter blocks of
// the launches.
#include <math.h>

#include "rr_args.h"
#include "rr_norm.h"

namespace {

using rr::aligned16;
using rr::elem_bytes;
using rr::matrix_span;
using rr::share;
using rr::Span;
using rr::span_of;
using rr::valid_type;

constexpr size_t kMaxExtent = 0x7fffff00;

rr_status launched(cudaError_t e) { return rr::note_cuda(e) ? RR_OK : RR_ERR_CUDA; }

// x and its norm's weights: formats and extents that every call has.
bool shape_ok(size_t rows, size_t cols, rr_dtype dtype, rr_dtype wtype) {
  return valid_type(dtype) && (wtype == dtype || wtype == RR_FP32) && rows <= kMaxExtent && cols <= kMaxExtent;
}
// A vector that may be missing.
bool optional_span(const void *p, size_t bytes, size_t align, Span *s) {
  return !p ? (*s = Span{}, true) : span_of(p, bytes, align, s);
}
bool vec16(const void *p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

}  // namespace

extern "C" {

size_t ring_layer_norm_workspace(size_t rows, size_t cols) {
  if (rows > kMaxExtent || cols > kMaxExtent) return 0;
  return (size_t)rr::norm_parts((long long)rows, (long long)cols) * 2 * cols * sizeof(float);
}

rr_status ring_layer_norm(const void *x, size_t ld_x, const void *weight, const void *bias, rr_dtype wtype, double eps,
                          void *out, size_t ld_out, float *mean, float *rstd, size_t rows, size_t cols, rr_dtype dtype,
                          cudaStream_t stream) {
  if (!shape_ok(rows, cols, dtype, wtype) || !(eps >= 0.0) || isinf(eps)) return RR_ERR_INVALID_ARG;
  if (rows == 0 || cols == 0) return RR_OK;
  const size_t E = elem_bytes(dtype), W = elem_bytes(wtype);
  Span sx, so, sw, sb, sm, sr;
  if (!matrix_span(x, rows, cols, ld_x, E, &sx) || !matrix_span(out, rows, cols, ld_out, E, &so) ||
      !optional_span(weight, cols * W, W, &sw) || !optional_span(bias, cols * W, W, &sb) ||
      !optional_span(mean, rows * 4, 4, &sm) || !optional_span(rstd, rows * 4, 4, &sr))
    return RR_ERR_INVALID_ARG;
  if (!(x == out && ld_x == ld_out) && share(sx, ld_x, so, ld_out, cols, E)) return RR_ERR_ALIAS;
  for (const Span &written : {so, sm, sr})
    if (written.overlaps(sw) || written.overlaps(sb)) return RR_ERR_ALIAS;
  if (sm.overlaps(sr) || sm.overlaps(so) || sr.overlaps(so) || sm.overlaps(sx) || sr.overlaps(sx)) return RR_ERR_ALIAS;
  rr::NormParams p{};
  p.x = x, p.weight = weight, p.bias = bias, p.out = out, p.mean = mean, p.rstd = rstd;
  p.rows = (long long)rows, p.cols = (long long)cols, p.ld_x = (long long)ld_x, p.ld_out = (long long)ld_out;
  p.eps = (float)eps;
  p.dtype = dtype, p.wtype = wtype;
  p.vec = cols * E % 16 == 0 && aligned16(x, rows, ld_x, E) && aligned16(out, rows, ld_out, E) && vec16(weight) && vec16(bias);
  const rr_status st = rr::device_info(&p.status, &p.sms);
  if (st != RR_OK) return st;
  return launched(dtype == RR_FP32   ? rr::launch_norm_f32(p, stream)
                  : dtype == RR_FP16 ? rr::launch_norm_f16(p, stream)
                                     : rr::launch_norm_bf16(p, stream));
}

rr_status ring_layer_norm_backward(const void *dy, size_t ld_dy, const void *x, size_t ld_x, const void *weight,
                                   rr_dtype wtype, const float *mean, const float *rstd, void *dx, size_t ld_dx,
                                   void *dweight, void *dbias, size_t rows, size_t cols, rr_dtype dtype, void *workspace,
                                   size_t workspace_bytes, cudaStream_t stream) {
  if (!shape_ok(rows, cols, dtype, wtype)) return RR_ERR_INVALID_ARG;
  if (cols == 0 || !(dx || dweight || dbias)) return RR_OK;
  const size_t E = elem_bytes(dtype), W = elem_bytes(wtype);
  const bool sums = dweight || dbias;
  Span sdy, sx, sdx, sw, sm, sr, sdw, sdb, ws;
  if (!matrix_span(dy, rows, cols, ld_dy, E, &sdy) || !matrix_span(x, rows, cols, ld_x, E, &sx) ||
      (dx && !matrix_span(dx, rows, cols, ld_dx, E, &sdx)) || !optional_span(weight, cols * W, W, &sw) ||
      !span_of(mean, rows * 4, 4, &sm) || !span_of(rstd, rows * 4, 4, &sr) || !optional_span(dweight, cols * W, W, &sdw) ||
      !optional_span(dbias, cols * W, W, &sdb))
    return RR_ERR_INVALID_ARG;
  const size_t need = sums ? ring_layer_norm_workspace(rows, cols) : 0;
  if (need && (workspace_bytes < need || !span_of(workspace, need, 16, &ws))) return RR_ERR_INVALID_ARG;
  if (dx && !(dx == dy && ld_dx == ld_dy) && share(sdy, ld_dy, sdx, ld_dx, cols, E)) return RR_ERR_ALIAS;
  if (dx && !(dx == x && ld_dx == ld_x) && share(sx, ld_x, sdx, ld_dx, cols, E)) return RR_ERR_ALIAS;
  for (const Span &read : {sdy, sx, sw, sm, sr})
    if (read.overlaps(sdw) || read.overlaps(sdb) || read.overlaps(ws)) return RR_ERR_ALIAS;
  if (sdx.overlaps(sw) || sdx.overlaps(sm) || sdx.overlaps(sr) || sdx.overlaps(sdw) || sdx.overlaps(sdb) || sdx.overlaps(ws) ||
      sdw.overlaps(sdb) || sdw.overlaps(ws) || sdb.overlaps(ws))
    return RR_ERR_ALIAS;
  if (rows == 0 && !sums) return RR_OK;
  rr::NormGradParams p{};
  p.dy = dy, p.x = x, p.weight = weight, p.mean = mean, p.rstd = rstd;
  p.dx = dx, p.dweight = dweight, p.dbias = dbias, p.partials = sums ? static_cast<float *>(workspace) : nullptr;
  p.rows = (long long)rows, p.cols = (long long)cols;
  p.ld_dy = (long long)ld_dy, p.ld_x = (long long)ld_x, p.ld_dx = (long long)ld_dx;
  p.parts = (int)rr::norm_parts(p.rows, p.cols);
  p.sums = sums;
  p.dtype = dtype, p.wtype = wtype;
  p.vec = cols * E % 16 == 0 && aligned16(dy, rows, ld_dy, E) && aligned16(x, rows, ld_x, E) &&
          (!dx || aligned16(dx, rows, ld_dx, E)) && vec16(weight);
  const rr_status st = rr::device_info(&p.status, &p.sms);
  if (st != RR_OK) return st;
  return launched(dtype == RR_FP32   ? rr::launch_norm_grad_f32(p, stream)
                  : dtype == RR_FP16 ? rr::launch_norm_grad_f16(p, stream)
                                     : rr::launch_norm_grad_bf16(p, stream));
}

}  // extern "C"
