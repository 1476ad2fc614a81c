// rr_loss_grad.cuh -- the gradient of the linear cross entropy, in pieces of the
// vocabulary: with p the softmax and f[t] what token t's loss passes on,
//   e[t, v] = f[t] (p[t, v] - (v == target[t])), dx = e W, dW = e^T x.
// A piece's logits are made again from x and W, and e goes to memory in 16 bits
// as the operand of two products: 8 operations for every 2 of the forward pass,
// where logits kept from it would save 2 and cost tokens times vocabulary of
// memory.  e is rounded to x's format, the operands' format of the tensor cores:
// half a step a term, the same that rounding the outputs costs, and independent
// from term to term.  dx is summed over the pieces in binary32, in order.  8192
// tokens by 4096 by 32000 take 4.0 ms of the 5.1 of both passes: three products of
// 2.1 TFLOP at the power limit.
#pragma once

#include <math.h>

#include "rr_gemm.cuh"
#include "rr_loss.h"

namespace rr {

namespace loss {

constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

template <int DT>
struct LogitGradient {
  static constexpr int kRun = 0;
  struct Params {
    const long long *target;
    const float *lse;
    const float *factors;  // null: `widen` for a token that counts
    long long ignore, vocabulary;
    float widen;
    long long tokens;
    gemm::Out e;      // (rows past the tokens: zeros)
    long long first;  // the piece's first column of the vocabulary
  };
  const Params &p;
  long long row, col, at;
  float lse, factor, *stage;
  __device__ __forceinline__ LogitGradient(const Params &p, long long row, long long col, int, float *stage)
      : p(p), row(row), col(col), at(-1), lse(0.f), factor(0.f), stage(stage) {
    if (row < p.tokens) {
      at = p.target[row], lse = p.lse[row];
      factor = p.factors ? p.factors[row] : at == p.ignore ? 0.f : at >= 0 && at < p.vocabulary ? p.widen : NAN;
      at -= p.first;
    }
  }
  __device__ __forceinline__ void chunk(int c, float v[gemm::kChunk]) {
    const long long first = col + c * gemm::kChunk;
    if (first >= p.e.cols) return;
#pragma unroll
    for (int j = 0; j < gemm::kChunk; ++j) v[j] = __fmul_rn(ex2(__fmul_rn(__fsub_rn(v[j], lse), kLog2e)), factor);
    if (at >= first && at < first + gemm::kChunk) {
      const int j0 = (int)(at - first);
#pragma unroll
      for (int j = 0; j < gemm::kChunk; ++j)
        if (j == j0) v[j] = __fsub_rn(v[j], factor);
    }
    if (factor == 0.f) {  // (also where the logits are no numbers)
#pragma unroll
      for (int j = 0; j < gemm::kChunk; ++j) v[j] = 0.f;
    }
    gemm::store_row<DT>(p.e, row, first, v, stage);
  }
  __device__ __forceinline__ void end() {}
};

// D times the factors' power of two to storage.
template <int DT>
struct Scaled {
  static constexpr int kRun = 0;
  struct Params {
    gemm::Out out;
    const float *scale;
    float narrow;  // scale times this
  };
  const Params &p;
  long long row, col;
  float scale, *stage;
  __device__ __forceinline__ Scaled(const Params &p, long long row, long long col, int, float *stage)
      : p(p), row(row), col(col), scale(__fmul_rn(*p.scale, p.narrow)), stage(stage) {}
  __device__ __forceinline__ void chunk(int c, float v[gemm::kChunk]) {
#pragma unroll
    for (int j = 0; j < gemm::kChunk; ++j) v[j] = __fmul_rn(v[j], scale);
    gemm::store_row<DT>(p.out, row, col + c * gemm::kChunk, v, stage);
  }
  __device__ __forceinline__ void end() {}
};

// The sum over pieces: D onto the pieces before it, to storage with the last.
template <int DT>
struct Summed {
  static constexpr int kRun = 0;
  struct Params {
    gemm::Out out;
    const float *scale;
    float narrow;
    float *sum;  // rows of ld_sum, a multiple of 32
    long long ld_sum;
    bool first, last;
  };
  const Params &p;
  long long row, col;
  float scale, *stage;
  __device__ __forceinline__ Summed(const Params &p, long long row, long long col, int, float *stage)
      : p(p), row(row), col(col), scale(__fmul_rn(*p.scale, p.narrow)), stage(stage) {}
  __device__ __forceinline__ void chunk(int c, float v[gemm::kChunk]) {
    const long long at = col + c * gemm::kChunk;
    if (at >= p.out.cols) return;
    uint4 *q = reinterpret_cast<uint4 *>(p.sum + row * p.ld_sum + at);
    if (!p.first && row < p.out.rows) {
      uint4 raw[8];
#pragma unroll
      for (int j = 0; j < 8; j += 2) ldg32(q + j, raw[j], raw[j + 1]);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        v[4 * j] = __fadd_rn(__uint_as_float(raw[j].x), v[4 * j]);
        v[4 * j + 1] = __fadd_rn(__uint_as_float(raw[j].y), v[4 * j + 1]);
        v[4 * j + 2] = __fadd_rn(__uint_as_float(raw[j].z), v[4 * j + 2]);
        v[4 * j + 3] = __fadd_rn(__uint_as_float(raw[j].w), v[4 * j + 3]);
      }
    }
    if (p.last) {
#pragma unroll
      for (int j = 0; j < gemm::kChunk; ++j) v[j] = __fmul_rn(v[j], scale);
      gemm::store_row<DT>(p.out, row, at, v, stage);
    } else if (row < p.out.rows) {
      uint4 raw[8];
#pragma unroll
      for (int h = 0; h < 4; ++h) narrow8<kF32>(v + 8 * h, raw + 2 * h);
#pragma unroll
      for (int j = 0; j < 8; j += 2) stg32(q + j, raw[j], raw[j + 1]);
    }
  }
  __device__ __forceinline__ void end() {}
};

inline bool rows32(const void *p, long long ld, int bytes) {
  return reinterpret_cast<uintptr_t>(p) % 32 == 0 && ld * bytes % 32 == 0;
}
template <int DT>
cudaError_t backward(const LossGradParams &p, cudaStream_t s) {
  using gemm::Operand;
  const long long tokens = p.x.rows, vocabulary = p.w.rows, hidden = p.hidden;
  // One gradient for all tokens goes to the outputs whole, so that e is p - 1 and p
  // themselves (their common factor rounded into every e put the same error, up to
  // half a step, on all of them: twice the error of dx).  Gradients of their own make
  // factors.  In binary16 e is 2^14 times as large: it neither overflows nor falls
  // among the subnormals, down to probabilities of 2^-28.
  const bool one = p.grad_step == 0;
  const float widen = DT == kF16 ? kLossWiden : 1.f, narrow = one ? 1.f / widen : 1.f;
  cudaError_t err = one ? cudaSuccess : launch_loss_factors(p, s);
  const float *scale = one ? p.grad : p.factors + tokens;
  for (long long v0 = 0; v0 < vocabulary && err == cudaSuccess; v0 += p.piece) {
    const long long n = vocabulary - v0 < p.piece ? vocabulary - v0 : p.piece;
    const void *w = static_cast<const uint16_t *>(p.w.at) + v0 * p.w.ld;
    const Operand x_along{p.x.at, p.x.padded, hidden, p.x.ld, 0, 1, false}, w_along{w, n, hidden, p.w.ld, 0, 1, false};
    // (e's rows are whole chunks: what lies past the piece's columns is written and never read)
    const typename LogitGradient<DT>::Params e{p.target,   p.lse,      one ? nullptr : p.factors,
                                               p.ignore,   vocabulary, widen,
                                               tokens,     gemm::Out{p.e, p.x.padded, p.ld_e, p.ld_e, true}, v0};
    err = gemm::launch_product<false, false, LogitGradient<DT>>(x_along, w_along, false, DT == kBF16, p.status, p.sms, e, s);
    if (err == cudaSuccess && p.dx) {
      const Operand e_along{p.e, p.x.padded, n, p.ld_e, 0, 1, false}, w_across{w, hidden, n, p.w.ld, 0, 1, true};
      const typename Summed<DT>::Params d{gemm::Out{p.dx, tokens, hidden, p.ld_dx, rows32(p.dx, p.ld_dx, 2)}, scale, narrow, p.sum_x,
                                          p.ld_sum, v0 == 0, v0 + n == vocabulary};
      err = gemm::launch_product<false, true, Summed<DT>>(e_along, w_across, false, DT == kBF16, p.status, p.sms, d, s);
    }
    if (err == cudaSuccess && p.dw) {
      const Operand e_across{p.e, n, p.x.padded, p.ld_e, 0, 1, true}, x_across{p.x.at, hidden, p.x.padded, p.x.ld, 0, 1, true};
      void *dw = static_cast<uint16_t *>(p.dw) + v0 * p.ld_dw;
      const typename Scaled<DT>::Params d{gemm::Out{dw, n, hidden, p.ld_dw, rows32(dw, p.ld_dw, 2)}, scale, narrow};
      err = gemm::launch_product<true, true, Scaled<DT>>(e_across, x_across, false, DT == kBF16, p.status, p.sms, d, s);
    }
  }
  return err;
}

}  // namespace loss

}  // namespace rr
