// rr_mx4_api.cu -- the C ABI of the microscaled 4-bit operators and dropout
// (include/ringred.h): argument checks, all on the host and before any CUDA
// call, and the parameter blocks of the launches.
#include <math.h>

#include "rr_args.h"
#include "rr_mx4.h"

namespace {

using rr::aligned16;
using rr::aligned32;
using rr::ceil_div;
using rr::elem_bytes;
using rr::matrix_span;
using rr::share;
using rr::Span;
using rr::span_of;
using rr::valid_type;

constexpr size_t kMaxExtent = 0x7fffff00;  // rows or columns (tensor-copy coordinates are 32 bits)

bool extents_ok(size_t rows, size_t cols) {
  return rows <= kMaxExtent && cols <= kMaxExtent && (cols == 0 || rows <= (SIZE_MAX / 64) / cols);
}

struct Mx4Spans {
  Span data, scales;
  bool overlaps(const Span &o) const { return data.overlaps(o) || scales.overlaps(o); }
  bool overlaps(const Mx4Spans &o) const { return overlaps(o.data) || overlaps(o.scales); }
};

bool mx4_spans(const rr_mx4 *q, Mx4Spans *s) {
  return extents_ok(q->rows, q->cols) && span_of(q->data, q->rows * ring_mx4_row_bytes(q->cols), 16, &s->data) &&
         span_of(q->scales, ring_mx4_scale_bytes(q->rows, q->cols), 16, &s->scales);
}

rr::Mx4Out mx4_out(const rr_mx4 *q) {
  rr::Mx4Out o{};
  if (!q) return o;
  o.data = static_cast<uint8_t *>(q->data);
  o.scales = static_cast<uint8_t *>(q->scales);
  o.rows = (long long)q->rows;
  o.row_bytes = (long long)ring_mx4_row_bytes(q->cols);
  o.tiles_k = (long long)ceil_div(q->cols, (size_t)rr::kMx4TileCols);
  return o;
}

// The threshold and the scale of a dropout; null or p = 0: nothing is dropped.
bool drop_params(const rr_dropout *d, rr::DropParams *o) {
  *o = rr::DropParams{};
  o->scale = 1.f;
  if (!d) return true;
  if (!(d->p >= 0.0 && d->p < 1.0)) return false;
  const unsigned t = (unsigned)floor(d->p * 65536.0 + 0.5);
  if (t > 65535u) return false;
  o->gen = rr::make_generator(d->seed, d->subsequence);
  o->first = d->first;
  o->cut = t << 16;
  o->scale = (float)(65536.0 / (65536.0 - (double)t));
  return true;
}

rr_status launched(cudaError_t e) { return rr::note_cuda(e) ? RR_OK : RR_ERR_CUDA; }

}  // namespace

extern "C" {

size_t ring_mx4_row_bytes(size_t cols) { return ceil_div(cols, (size_t)rr::kMx4Block) * 16; }

size_t ring_mx4_scale_bytes(size_t rows, size_t cols) {
  return ceil_div(rows, (size_t)rr::kMx4TileRows) * ceil_div(cols, (size_t)rr::kMx4TileCols) * rr::kMx4TileBytes;
}

rr_status ring_mx4_quantize(const void *x, size_t rows, size_t cols, size_t ld, rr_dtype dtype, const rr_mx4 *by_rows,
                            const rr_mx4 *by_cols, rr_mx4_rounding rounding, unsigned long long seed,
                            unsigned long long subsequence, const rr_dropout *drop, cudaStream_t stream) {
  if (!valid_type(dtype) || !(by_rows || by_cols)) return RR_ERR_INVALID_ARG;
  if (rounding != RR_MX4_NEAREST && rounding != RR_MX4_STOCHASTIC) return RR_ERR_INVALID_ARG;
  if (!extents_ok(rows, cols)) return RR_ERR_INVALID_ARG;
  rr::QuantParams p{};
  if (!drop_params(drop, &p.drop)) return RR_ERR_INVALID_ARG;
  if (by_rows && (by_rows->rows != rows || by_rows->cols != cols)) return RR_ERR_INVALID_ARG;
  if (by_cols && (by_cols->rows != cols || by_cols->cols != rows)) return RR_ERR_INVALID_ARG;
  if (rows == 0 || cols == 0) return RR_OK;
  const size_t E = elem_bytes(dtype);
  Span sx;
  Mx4Spans sr, sc;
  if (!matrix_span(x, rows, cols, ld, E, &sx)) return RR_ERR_INVALID_ARG;
  if (by_rows && !mx4_spans(by_rows, &sr)) return RR_ERR_INVALID_ARG;
  if (by_cols && !mx4_spans(by_cols, &sc)) return RR_ERR_INVALID_ARG;
  if (sr.overlaps(sx) || sc.overlaps(sx) || sr.overlaps(sc) || sr.data.overlaps(sr.scales) ||
      sc.data.overlaps(sc.scales))
    return RR_ERR_ALIAS;
  p.x = x;
  p.rows = (long long)rows, p.cols = (long long)cols, p.ld = (long long)ld;
  p.by_rows = mx4_out(by_rows), p.by_cols = mx4_out(by_cols);
  p.gen_rows = rr::make_generator(seed, subsequence);
  p.gen_cols = rr::make_generator(seed, subsequence + (by_rows ? 1 : 0));
  p.dtype = dtype;
  p.stochastic = rounding == RR_MX4_STOCHASTIC;
  p.vec = aligned16(x, rows, ld, E);
  p.vec32 = aligned32(x, rows, ld, E);
  p.x_lo = sx.lo, p.x_hi = sx.hi;
  unsigned *status;
  const rr_status st = rr::device_info(&status, &p.sms);
  if (st != RR_OK) return st;
  return launched(rr::launch_mx4_quantize(p, stream));
}

rr_status ring_mx4_dequantize(const rr_mx4 *q, void *out, size_t ld, rr_dtype dtype, cudaStream_t stream) {
  if (!q || !valid_type(dtype) || !extents_ok(q->rows, q->cols)) return RR_ERR_INVALID_ARG;
  if (q->rows == 0 || q->cols == 0) return RR_OK;
  const size_t E = elem_bytes(dtype);
  Span so;
  Mx4Spans sq;
  if (!mx4_spans(q, &sq) || !matrix_span(out, q->rows, q->cols, ld, E, &so)) return RR_ERR_INVALID_ARG;
  if (sq.overlaps(so)) return RR_ERR_ALIAS;
  const rr::Mx4Out o = mx4_out(q);
  rr::DequantParams p{};
  p.data = o.data, p.scales = o.scales;
  p.rows = o.rows, p.cols = (long long)q->cols, p.row_bytes = o.row_bytes, p.tiles_k = o.tiles_k;
  p.out = out, p.ld = (long long)ld, p.dtype = dtype;
  p.vec = aligned16(out, q->rows, ld, E);
  p.vec32 = aligned32(out, q->rows, ld, E);
  return launched(rr::launch_mx4_dequantize(p, stream));
}

rr_status ring_mx4_matmul(const rr_mx4 *a, const rr_mx4 *b, void *out, size_t ld, rr_dtype dtype, const void *residual,
                          size_t ld_residual, const rr_dropout *drop, cudaStream_t stream) {
  if (!a || !b || !valid_type(dtype) || a->cols != b->cols) return RR_ERR_INVALID_ARG;
  if (!extents_ok(a->rows, a->cols) || !extents_ok(b->rows, b->cols) || !extents_ok(a->rows, b->rows))
    return RR_ERR_INVALID_ARG;
  rr::MatmulParams p{};
  if (!drop_params(drop, &p.drop)) return RR_ERR_INVALID_ARG;
  const size_t m = a->rows, n = b->rows, E = elem_bytes(dtype);
  if (m == 0 || n == 0) return RR_OK;
  Span so, sres;
  Mx4Spans sa, sb;
  if (!mx4_spans(a, &sa) || !mx4_spans(b, &sb) || !matrix_span(out, m, n, ld, E, &so)) return RR_ERR_INVALID_ARG;
  if (residual && !matrix_span(residual, m, n, ld_residual, E, &sres)) return RR_ERR_INVALID_ARG;
  if (sa.overlaps(so) || sb.overlaps(so)) return RR_ERR_ALIAS;
  if (!(residual == out && ld_residual == ld) && share(sres, ld_residual, so, ld, n, E)) return RR_ERR_ALIAS;
  p.m = (long long)m, p.n = (long long)n, p.k = (long long)a->cols;
  const rr::Mx4Out oa = mx4_out(a), ob = mx4_out(b);
  p.a = rr::Mx4Operand{oa.data, oa.scales, oa.rows, oa.row_bytes};
  p.b = rr::Mx4Operand{ob.data, ob.scales, ob.rows, ob.row_bytes};
  p.out = out, p.residual = residual;
  p.ld_out = (long long)ld, p.ld_res = (long long)ld_residual;
  p.dtype = dtype;
  p.vec = aligned16(out, m, ld, E) && (!residual || aligned16(residual, m, ld_residual, E));
  p.vec32 = aligned32(out, m, ld, E) && (!residual || aligned32(residual, m, ld_residual, E));
  const rr_status st = rr::device_info(&p.status, &p.sms);
  if (st != RR_OK) return st;
  return launched(rr::launch_mx4_matmul(p, stream));
}

rr_status ring_dropout(const void *x, size_t ld_x, const void *residual, size_t ld_residual, void *out, size_t ld_out,
                       size_t rows, size_t cols, rr_dtype dtype, const rr_dropout *drop, cudaStream_t stream) {
  if (!valid_type(dtype) || !drop) return RR_ERR_INVALID_ARG;
  rr::DropoutParams p{};
  if (!drop_params(drop, &p.drop)) return RR_ERR_INVALID_ARG;
  if (rows == 0 || cols == 0) return RR_OK;
  if (cols > (SIZE_MAX / 64) / rows) return RR_ERR_INVALID_ARG;
  const size_t E = elem_bytes(dtype);
  Span sx, sr, so;
  if (!matrix_span(x, rows, cols, ld_x, E, &sx) || !matrix_span(out, rows, cols, ld_out, E, &so))
    return RR_ERR_INVALID_ARG;
  if (residual && !matrix_span(residual, rows, cols, ld_residual, E, &sr)) return RR_ERR_INVALID_ARG;
  if (!(x == out && ld_x == ld_out) && share(sx, ld_x, so, ld_out, cols, E)) return RR_ERR_ALIAS;
  if (!(residual == out && ld_residual == ld_out) && share(sr, ld_residual, so, ld_out, cols, E)) return RR_ERR_ALIAS;
  // rows that follow one another everywhere are one long row
  if (ld_x == cols && ld_out == cols && (!residual || ld_residual == cols)) cols *= rows, rows = 1;
  p.x = x, p.residual = residual, p.out = out;
  p.rows = (long long)rows, p.cols = (long long)cols;
  p.ld_x = (long long)ld_x, p.ld_res = (long long)ld_residual, p.ld_out = (long long)ld_out;
  p.dtype = dtype;
  p.vec = aligned16(x, rows, ld_x, E) && aligned16(out, rows, ld_out, E) &&
          (!residual || aligned16(residual, rows, ld_residual, E));
  return launched(rr::launch_dropout(p, stream));
}

rr_status ring_mx4_allreduce(const rr_mx4 *in, void *const *out_bufs, int R, rr_dtype dtype, cudaStream_t stream) {
  if (!in || !out_bufs || R < 1 || R > RR_MAX_RANKS || !valid_type(dtype)) return RR_ERR_INVALID_ARG;
  const size_t rows = in[0].rows, cols = in[0].cols, E = elem_bytes(dtype);
  if (!extents_ok(rows, cols)) return RR_ERR_INVALID_ARG;
  for (int r = 0; r < R; ++r)
    if (in[r].rows != rows || in[r].cols != cols) return RR_ERR_INVALID_ARG;
  if (rows == 0 || cols == 0) return RR_OK;
  rr::Mx4ReduceParams p{};
  Mx4Spans si[RR_MAX_RANKS];
  Span so[RR_MAX_RANKS];
  p.vec = p.vec32 = true;
  for (int r = 0; r < R; ++r) {
    if (!mx4_spans(&in[r], &si[r]) || !span_of(out_bufs[r], rows * cols * E, E, &so[r])) return RR_ERR_INVALID_ARG;
    p.data[r] = static_cast<const uint8_t *>(in[r].data);
    p.scales[r] = static_cast<const uint8_t *>(in[r].scales);
    p.out[r] = out_bufs[r];
    p.vec = p.vec && aligned16(out_bufs[r], 1, cols, E);  // contiguous: one long row
    p.vec32 = p.vec32 && aligned32(out_bufs[r], 1, cols, E);
  }
  for (int r = 0; r < R; ++r)
    for (int s = 0; s < R; ++s)
      if (si[s].overlaps(so[r]) || (s != r && so[s].overlaps(so[r]))) return RR_ERR_ALIAS;
  const rr::Mx4Out o = mx4_out(&in[0]);
  p.rows = o.rows, p.cols = (long long)cols, p.row_bytes = o.row_bytes, p.tiles_k = o.tiles_k;
  p.base = (long long)(rows * cols / (size_t)R);
  p.R = R, p.dtype = dtype;
  return launched(rr::launch_mx4_reduce(p, stream));
}

}  // extern "C"
