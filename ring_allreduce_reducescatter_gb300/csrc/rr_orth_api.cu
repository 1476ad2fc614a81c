// rr_orth_api.cu -- the C ABI of the orthogonalised update (include/ringred.h):
// argument checks, all on the host and before any CUDA call, the workspace's
// layout, and the parameter block.
#include <math.h>

#include "rr_args.h"
#include "rr_orth.h"

namespace {

using rr::elem_bytes;
using rr::Span;
using rr::span_of;
using rr::valid_type;

constexpr size_t kMaxExtent = 0x7fffff00, kMaxBatch = 65535;

size_t round_up(size_t n, size_t to) { return (n + to - 1) / to * to; }

struct Layout {
  size_t norms, x[2], s, b, bytes = 0;
  size_t held_rows, held_cols, ld_x, ld_s, stride_x, stride_s;
  size_t take(size_t n) {
    const size_t at = bytes;
    bytes += round_up(n, 256);
    return at;
  }
  Layout(size_t batch, size_t rows, size_t cols) {
    held_rows = (size_t)rr::orth_held((long long)rows, (long long)rows, (long long)cols);
    held_cols = (size_t)rr::orth_held((long long)cols, (long long)rows, (long long)cols);
    const size_t m = held_rows < held_cols ? held_rows : held_cols;
    ld_x = round_up(held_cols, 32), ld_s = round_up(m, 32);
    stride_x = held_rows * ld_x, stride_s = m * ld_s;
    norms = take(batch * (size_t)rr::orth_parts((long long)rows, (long long)cols) * 12);
    for (size_t &at : x) at = take(batch * stride_x * 2);
    s = take(batch * stride_s * 2);
    b = take(batch * stride_s * 2);
  }
};

bool sizes_ok(size_t batch, size_t rows, size_t cols) {
  return batch <= kMaxBatch && rows <= kMaxExtent && cols <= kMaxExtent &&
         (rows == 0 || cols == 0 || batch == 0 || rows <= ((size_t)1 << 40) / cols / batch);
}

// The extent of `batch` strided matrices, each ending before the next begins.
bool batch_span(const void *p, size_t batch, size_t stride, size_t rows, size_t cols, size_t ld, size_t E, Span *s) {
  if (ld < cols || ld > ((size_t)1 << 40) / rows) return false;
  const size_t one = (rows - 1) * ld + cols;
  if (batch > 1 && (stride < one || stride > ((size_t)1 << 44) / batch)) return false;
  return span_of(p, ((batch - 1) * (batch > 1 ? stride : 0) + one) * E, E, s);
}

}  // namespace

extern "C" {

size_t ring_orthogonalize_workspace(size_t batch, size_t rows, size_t cols) {
  if (!sizes_ok(batch, rows, cols) || batch == 0 || rows == 0 || cols == 0) return 0;
  return Layout(batch, rows, cols).bytes;
}

rr_status ring_orthogonalize(const void *g, size_t ld_g, size_t stride_g, rr_dtype dtype, void *out, size_t ld_out,
                             size_t stride_out, rr_dtype out_dtype, size_t batch, size_t rows, size_t cols, int steps, double eps,
                             void *workspace, size_t workspace_bytes, cudaStream_t stream) {
  if (!valid_type(dtype) || !valid_type(out_dtype) || steps < 1 || steps > 1000 || !(eps >= 0.0) || isinf(eps) ||
      !sizes_ok(batch, rows, cols))
    return RR_ERR_INVALID_ARG;
  if (batch == 0 || rows == 0 || cols == 0) return RR_OK;
  Span sg, so, sp;
  if (!batch_span(g, batch, stride_g, rows, cols, ld_g, elem_bytes(dtype), &sg) ||
      !batch_span(out, batch, stride_out, rows, cols, ld_out, elem_bytes(out_dtype), &so))
    return RR_ERR_INVALID_ARG;
  const Layout l(batch, rows, cols);
  if (workspace_bytes < l.bytes || !span_of(workspace, l.bytes, 32, &sp)) return RR_ERR_INVALID_ARG;
  const bool in_place = g == out && ld_g == ld_out && dtype == out_dtype && (batch == 1 || stride_g == stride_out);
  if ((!in_place && sg.overlaps(so)) || sp.overlaps(sg) || sp.overlaps(so)) return RR_ERR_ALIAS;
  rr::OrthParams p{};
  const rr_status st = rr::device_info(&p.status, &p.sms);
  if (st != RR_OK) return st;
  char *ws = static_cast<char *>(workspace);
  p.g = g, p.out = out;
  p.rows = (long long)rows, p.cols = (long long)cols;
  p.ld_g = (long long)ld_g, p.ld_out = (long long)ld_out;
  p.stride_g = batch > 1 ? (long long)stride_g : 0, p.stride_out = batch > 1 ? (long long)stride_out : 0;
  p.batch = (int)batch, p.steps = steps, p.dtype = dtype, p.out_dtype = out_dtype;
  p.eps = (float)eps;
  p.parts = rr::orth_parts(p.rows, p.cols);
  p.vec_out = rr::aligned16(out, rows, ld_out, elem_bytes(out_dtype)) && (batch == 1 || stride_out * elem_bytes(out_dtype) % 16 == 0);
  p.vec = rr::aligned16(g, rows, ld_g, elem_bytes(dtype)) && (batch == 1 || stride_g * elem_bytes(dtype) % 16 == 0);
  p.norms = reinterpret_cast<float *>(ws + l.norms);
  p.x[0] = ws + l.x[0], p.x[1] = ws + l.x[1], p.s = ws + l.s, p.b = ws + l.b;
  p.held_rows = (long long)l.held_rows, p.held_cols = (long long)l.held_cols;
  p.ld_x = (long long)l.ld_x, p.ld_s = (long long)l.ld_s, p.stride_x = (long long)l.stride_x, p.stride_s = (long long)l.stride_s;
  return rr::note_cuda(rr::launch_orth(p, stream)) ? RR_OK : RR_ERR_CUDA;
}

}  // extern "C"
