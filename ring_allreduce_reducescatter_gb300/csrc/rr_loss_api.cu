// rr_loss_api.cu -- the C ABI of the linear cross entropy (include/ringred.h):
// argument checks, all on the host and before any CUDA call, the workspace's
// layout, and the parameter blocks of the launches.
#include "rr_args.h"
#include "rr_loss.h"

namespace {

using rr::matrix_span;
using rr::Span;
using rr::span_of;

constexpr size_t kMaxExtent = 0x7fffff00;

rr_status launched(cudaError_t e) { return rr::note_cuda(e) ? RR_OK : RR_ERR_CUDA; }

// Parts of a workspace, each on 256 bytes.
struct Layout {
  size_t bytes = 0;
  size_t take(size_t n) {
    const size_t at = bytes;
    bytes += (n + 255) / 256 * 256;
    return at;
  }
};

size_t round_up(size_t n, size_t to) { return (n + to - 1) / to * to; }

// x and w: whether tensor copies read them as they lie, else where their copy goes.
struct Operands {
  bool copy_x, copy_w;
  size_t x_at, w_at, ld;  // of the copies
  size_t rows;            // of x, with the zeros behind it
};
bool readable(const void *p, size_t ld) { return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld % 8 == 0; }
Operands operands(Layout *l, const void *x, size_t ld_x, const void *w, size_t ld_w, size_t tokens, size_t hidden,
                  size_t vocabulary, bool along) {
  Operands o{};
  o.ld = round_up(hidden, 8);
  o.rows = (size_t)rr::loss_rows((long long)tokens, (long long)hidden, along);
  o.copy_x = o.rows != tokens || !readable(x, ld_x), o.copy_w = !readable(w, ld_w);
  if (o.copy_x) o.x_at = l->take(o.rows * o.ld * 2);
  if (o.copy_w) o.w_at = l->take(vocabulary * o.ld * 2);
  return o;
}

struct ForwardLayout : Layout {
  Operands o;
  size_t parts, chosen;
  ForwardLayout(const void *x, size_t ld_x, const void *w, size_t ld_w, size_t tokens, size_t hidden, size_t vocabulary) {
    const size_t group = (size_t)rr::loss_group((long long)tokens);
    parts = take((vocabulary + group - 1) / group * tokens * 8);
    chosen = take(tokens * 4);
    o = operands(this, x, ld_x, w, ld_w, tokens, hidden, vocabulary, true);
  }
};
struct BackwardLayout : Layout {
  Operands o;
  size_t factors, e, sum, piece, ld_sum;
  BackwardLayout(const void *x, size_t ld_x, const void *w, size_t ld_w, size_t tokens, size_t hidden, size_t vocabulary) {
    piece = (size_t)rr::loss_piece((long long)tokens, (long long)vocabulary);
    ld_sum = round_up(hidden, 32);
    factors = take((tokens + 1) * 4);
    e = take((size_t)rr::loss_rows((long long)tokens, (long long)hidden, false) * piece * 2);
    sum = piece < vocabulary ? take(tokens * ld_sum * 4) : 0;
    o = operands(this, x, ld_x, w, ld_w, tokens, hidden, vocabulary, false);
  }
};

bool sizes_ok(size_t tokens, size_t hidden, size_t vocabulary, size_t ld_x, size_t ld_w) {
  return tokens <= kMaxExtent && hidden >= 1 && hidden <= kMaxExtent && vocabulary >= 1 && vocabulary <= kMaxExtent &&
         ld_x >= hidden && ld_w >= hidden && ld_x <= (size_t)1 << 36 && ld_w <= (size_t)1 << 36;
}

// The operands as tensor copies read them, copied where they must be.
rr_status place(const Operands &o, char *ws, const void *x, size_t ld_x, const void *w, size_t ld_w, size_t tokens, size_t hidden,
                size_t vocabulary, rr::LossMatrix *mx, rr::LossMatrix *mw, cudaStream_t stream) {
  *mx = rr::LossMatrix{o.copy_x ? ws + o.x_at : x, (long long)tokens, (long long)o.rows, (long long)(o.copy_x ? o.ld : ld_x)};
  *mw = rr::LossMatrix{o.copy_w ? ws + o.w_at : w, (long long)vocabulary, (long long)vocabulary,
                       (long long)(o.copy_w ? o.ld : ld_w)};
  rr::PadParams p{};
  if (o.copy_x)
    p.copy[p.n++] = rr::Pad{x, ws + o.x_at, (long long)tokens, (long long)hidden, (long long)ld_x, (long long)o.ld, (long long)o.rows};
  if (o.copy_w)
    p.copy[p.n++] = rr::Pad{w, ws + o.w_at, (long long)vocabulary, (long long)hidden, (long long)ld_w, (long long)o.ld,
                            (long long)vocabulary};
  if (p.n > 0 && !rr::note_cuda(rr::launch_pad(p, stream))) return RR_ERR_CUDA;
  return RR_OK;
}

}  // namespace

extern "C" {

size_t ring_linear_cross_entropy_workspace(const void *x, size_t ld_x, const void *w, size_t ld_w, size_t tokens, size_t hidden,
                                           size_t vocabulary) {
  if (!sizes_ok(tokens, hidden, vocabulary, ld_x, ld_w)) return 0;
  return ForwardLayout(x, ld_x, w, ld_w, tokens, hidden, vocabulary).bytes;
}

size_t ring_linear_cross_entropy_backward_workspace(const void *x, size_t ld_x, const void *w, size_t ld_w, size_t tokens,
                                                    size_t hidden, size_t vocabulary) {
  if (!sizes_ok(tokens, hidden, vocabulary, ld_x, ld_w)) return 0;
  return BackwardLayout(x, ld_x, w, ld_w, tokens, hidden, vocabulary).bytes;
}

rr_status ring_linear_cross_entropy(const void *x, size_t ld_x, const void *w, size_t ld_w, const long long *target,
                                    long long ignore_index, float *loss, float *lse, float *sums, size_t tokens, size_t hidden,
                                    size_t vocabulary, rr_dtype dtype, void *workspace, size_t workspace_bytes,
                                    cudaStream_t stream) {
  if (dtype == RR_FP32) return RR_ERR_UNSUPPORTED;
  if (dtype != RR_FP16 && dtype != RR_BF16) return RR_ERR_INVALID_ARG;
  if (!sizes_ok(tokens, hidden, vocabulary, ld_x, ld_w)) return RR_ERR_INVALID_ARG;
  if (tokens == 0 && !sums) return RR_OK;
  Span sx, sw, st, sl, se, ss, sp;
  if (!matrix_span(x, tokens, hidden, ld_x, 2, &sx) || (tokens && !matrix_span(w, vocabulary, hidden, ld_w, 2, &sw)) ||
      !span_of(target, tokens * 8, 8, &st) || !span_of(loss, tokens * 4, 4, &sl) ||
      (lse && !span_of(lse, tokens * 4, 4, &se)) || (sums && !span_of(sums, 12, 4, &ss)))
    return RR_ERR_INVALID_ARG;
  const ForwardLayout l(x, ld_x, w, ld_w, tokens, hidden, vocabulary);
  if (tokens && (workspace_bytes < l.bytes || !span_of(workspace, l.bytes, 16, &sp))) return RR_ERR_INVALID_ARG;
  for (const Span &out : {sl, se, ss, sp})
    if (out.overlaps(sx) || out.overlaps(sw) || out.overlaps(st)) return RR_ERR_ALIAS;
  if (sl.overlaps(se) || sl.overlaps(ss) || sl.overlaps(sp) || se.overlaps(ss) || se.overlaps(sp) || ss.overlaps(sp))
    return RR_ERR_ALIAS;
  rr::LossParams p{};
  rr_status code = rr::device_info(&p.status, &p.sms);
  if (code != RR_OK) return code;
  char *ws = static_cast<char *>(workspace);
  if (tokens && (code = place(l.o, ws, x, ld_x, w, ld_w, tokens, hidden, vocabulary, &p.x, &p.w, stream)) != RR_OK) return code;
  p.hidden = (long long)hidden;
  p.target = target, p.ignore = ignore_index;
  p.loss = loss, p.lse = lse, p.sums = sums;
  p.parts = reinterpret_cast<float2 *>(ws + l.parts), p.chosen = reinterpret_cast<float *>(ws + l.chosen);
  p.dtype = dtype;
  return launched(rr::launch_loss(p, stream));
}

rr_status ring_linear_cross_entropy_backward(const float *grad, size_t grad_step, const void *x, size_t ld_x, const void *w,
                                             size_t ld_w, const long long *target, long long ignore_index, const float *lse,
                                             void *dx, size_t ld_dx, void *dw, size_t ld_dw, size_t tokens, size_t hidden,
                                             size_t vocabulary, rr_dtype dtype, void *workspace, size_t workspace_bytes,
                                             cudaStream_t stream) {
  if (dtype == RR_FP32) return RR_ERR_UNSUPPORTED;
  if ((dtype != RR_FP16 && dtype != RR_BF16) || grad_step > 1) return RR_ERR_INVALID_ARG;
  if (!sizes_ok(tokens, hidden, vocabulary, ld_x, ld_w)) return RR_ERR_INVALID_ARG;
  if (!(dx || dw)) return RR_OK;
  if (tokens == 0 && !dw) return RR_OK;
  Span sg, sx, sw, st, sl, sdx, sdw, sp;
  if (!matrix_span(x, tokens, hidden, ld_x, 2, &sx) || (tokens && !matrix_span(w, vocabulary, hidden, ld_w, 2, &sw)) ||
      !span_of(grad, tokens == 0 ? 0 : grad_step ? tokens * 4 : 4, 4, &sg) || !span_of(target, tokens * 8, 8, &st) ||
      !span_of(lse, tokens * 4, 4, &sl) || (dx && !matrix_span(dx, tokens, hidden, ld_dx, 2, &sdx)) ||
      (dw && !matrix_span(dw, vocabulary, hidden, ld_dw, 2, &sdw)))
    return RR_ERR_INVALID_ARG;
  const BackwardLayout l(x, ld_x, w, ld_w, tokens, hidden, vocabulary);
  if (tokens && (workspace_bytes < l.bytes || !span_of(workspace, l.bytes, 16, &sp))) return RR_ERR_INVALID_ARG;
  for (const Span &out : {sdx, sdw, sp})
    if (out.overlaps(sg) || out.overlaps(sx) || out.overlaps(sw) || out.overlaps(st) || out.overlaps(sl)) return RR_ERR_ALIAS;
  if (sdx.overlaps(sdw) || sdx.overlaps(sp) || sdw.overlaps(sp)) return RR_ERR_ALIAS;
  rr::LossGradParams p{};
  rr_status code = rr::device_info(&p.status, &p.sms);
  if (code != RR_OK) return code;
  if (tokens == 0)  // no token: the gradient of w is zero
    return launched(cudaMemset2DAsync(dw, ld_dw * 2, 0, hidden * 2, vocabulary, stream));
  char *ws = static_cast<char *>(workspace);
  if ((code = place(l.o, ws, x, ld_x, w, ld_w, tokens, hidden, vocabulary, &p.x, &p.w, stream)) != RR_OK) return code;
  p.hidden = (long long)hidden;
  p.target = target, p.ignore = ignore_index;
  p.grad = grad, p.grad_step = (int)grad_step, p.lse = lse;
  p.dx = dx, p.dw = dw, p.ld_dx = (long long)ld_dx, p.ld_dw = (long long)ld_dw;
  p.factors = reinterpret_cast<float *>(ws + l.factors);
  p.e = ws + l.e, p.sum_x = reinterpret_cast<float *>(ws + l.sum);
  p.piece = (long long)l.piece, p.ld_e = (long long)l.piece, p.ld_sum = (long long)l.ld_sum;
  p.dtype = dtype;
  return launched(dtype == RR_FP16 ? rr::launch_loss_grad_f16(p, stream) : rr::launch_loss_grad_bf16(p, stream));
}

}  // extern "C"
