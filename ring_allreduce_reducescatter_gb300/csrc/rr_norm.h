// rr_norm.h -- parameter blocks and launchers of layer norm, between the C ABI
// (rr_norm_api.cu) and the kernel translation units (rr_norm_*.cu).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "rr_mx4.h"

namespace rr {

struct NormParams {
  const void *x, *weight, *bias;  // weight and bias may be null
  void *out;
  float *mean, *rstd;  // may be null
  long long rows, cols, ld_x, ld_out;
  float eps;
  int dtype, wtype, sms;
  unsigned int *status;
  bool vec;  // 16-byte groups of the rows of x and out, and of weight and bias, are aligned; cols is whole groups
};

struct NormGradParams {
  const void *dy, *x, *weight;  // weight may be null
  const float *mean, *rstd;
  void *dx, *dweight, *dbias;  // null: not wanted
  float *partials;             // [parts][2][cols]: sums over some rows of dy h and of dy (null with no rows)
  long long rows, cols, ld_dy, ld_x, ld_dx;
  int parts, dtype, wtype, sms;
  unsigned int *status;
  bool sums;  // dweight or dbias is wanted
  bool vec;
};

// The most partial sums of the weights' gradients that a backward pass keeps:
// three CTAs an SM of 152 where a CTA holds whole rows, and fewer where rows are
// long and memory would go to the partial sums.
constexpr long long kNormParts = 456, kNormLongParts = 304, kNormLongRow = 4096, kNormOverRow = 16384, kNormOverParts = 32;
inline long long norm_parts(long long rows, long long cols) {
  const long long most = cols <= kNormLongRow ? kNormParts : cols <= kNormOverRow ? kNormLongParts : kNormOverParts;
  return rows < most ? rows : most;
}

cudaError_t launch_norm_f32(const NormParams &p, cudaStream_t s);
cudaError_t launch_norm_f16(const NormParams &p, cudaStream_t s);
cudaError_t launch_norm_bf16(const NormParams &p, cudaStream_t s);
cudaError_t launch_norm_grad_f32(const NormGradParams &p, cudaStream_t s);
cudaError_t launch_norm_grad_f16(const NormGradParams &p, cudaStream_t s);
cudaError_t launch_norm_grad_bf16(const NormGradParams &p, cudaStream_t s);

}  // namespace rr
