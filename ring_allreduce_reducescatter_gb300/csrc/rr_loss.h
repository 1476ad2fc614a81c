// rr_loss.h -- parameter blocks and launchers of the linear cross entropy,
// between the C ABI (rr_loss_api.cu) and the kernel translation units.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "rr_mx4.h"

namespace rr {

// A 16-bit matrix of rows x hidden that tensor copies can read (16-byte aligned
// rows), ld elements from row to row; behind its rows zeros up to `padded` of them.
struct LossMatrix {
  const void *at;
  long long rows, padded, ld;
};

struct LossParams {
  LossMatrix x, w;
  long long hidden;
  const long long *target;
  long long ignore;
  float *loss, *lse, *sums;  // lse and sums may be null
  float2 *parts;             // [groups][tokens]: maximum and sum of exponentials of a group of columns
  float *chosen;             // [tokens]: the target's logit
  unsigned int *status;
  int dtype, sms;
};

struct LossGradParams {
  LossMatrix x, w;
  long long hidden;
  const long long *target;
  long long ignore;
  const float *grad;
  int grad_step;  // 0: one for all tokens, 1: one each
  const float *lse;
  void *dx, *dw;  // null: not wanted
  long long ld_dx, ld_dw;
  float *factors;     // [tokens], then the outputs' common factor
  void *e;            // [x.padded][ld_e]: one piece of the logits' gradient
  float *sum_x;       // [tokens][ld_sum]: dx over the pieces so far
  long long piece, ld_e, ld_sum;  // columns of the vocabulary a piece
  unsigned int *status;
  int dtype, sms;
};

struct Pad {
  const void *from;
  void *to;
  long long rows, cols, ld_from, ld_to;  // 16-bit elements
  long long rows_to;  // zeros behind the rows, and behind the columns up to ld_to
};
struct PadParams {
  Pad copy[2];
  int n;
};

constexpr float kLossWiden = 16384.f;  // what the logits' gradient is held times in binary16

// The rows that x is held in: few and short ones in whole boxes (rr_gemm.cuh says
// why), with zeros behind them.
// Where x is read along K alone, a box takes as many rows as there are up to 128.
inline long long loss_rows(long long tokens, long long hidden, bool along) {
  return !(along && tokens < 128) && tokens % 128 && tokens * hidden * 2 < (1 << 20) ? ceil_div(tokens, 128ll) * 128 : tokens;
}

// Whether the logits of so many tokens are made in the larger tiles, whose
// epilogue sums up groups of 128 columns; else groups of 64.
inline bool loss_pairs(long long tokens) { return tokens > 128; }
inline long long loss_group(long long tokens) { return loss_pairs(tokens) ? 128 : 64; }

// Columns of the vocabulary a piece: the logits' gradient of a piece takes 256
// MiB at most (or 256 columns), and pieces are about equal.
inline long long loss_piece(long long tokens, long long vocabulary) {
  long long most = (1ll << 27) / (tokens > 0 ? tokens : 1) / 256 * 256;
  if (most < 256) most = 256;
  const long long pieces = ceil_div(vocabulary, most);
  return ceil_div(ceil_div(vocabulary, pieces), 256ll) * 256;
}

cudaError_t launch_pad(const PadParams &p, cudaStream_t s);
cudaError_t launch_loss(const LossParams &p, cudaStream_t s);
cudaError_t launch_loss_grad_f16(const LossGradParams &p, cudaStream_t s);
cudaError_t launch_loss_grad_bf16(const LossGradParams &p, cudaStream_t s);
cudaError_t launch_loss_factors(const LossGradParams &p, cudaStream_t s);

}  // namespace rr
