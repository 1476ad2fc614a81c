// rr_orth.h -- parameter block and launcher of the orthogonalised update,
// between the C ABI (rr_orth_api.cu) and the kernels (rr_orth.cu).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "rr_mx4.h"

namespace rr {

struct OrthParams {
  const void *g;
  void *out;
  long long rows, cols, ld_g, ld_out, stride_g, stride_out;  // strides: from matrix to matrix
  int batch, steps, dtype, out_dtype, parts;
  bool vec, vec_out;  // 16-byte groups of the rows of g, of out are aligned
  float eps;
  float *norms;       // [batch][parts][3]
  void *x[2], *s, *b; // binary16: two iterates, the Gram matrix and its polynomial
  long long held_rows, held_cols, ld_x, ld_s, stride_x, stride_s;
  unsigned int *status;
  int sms;
};

// Partial sums of a matrix's squares: 2048 elements each at least.
inline int orth_parts(long long rows, long long cols) {
  const long long n = ceil_div(rows * cols, 2048ll);
  return (int)(n < 1024 ? n : 1024);
}

// The sizes that the iterates are held in: small ones in whole boxes of zeros and
// elements (rr_gemm.cuh says why).
inline long long orth_held(long long n, long long rows, long long cols) {
  return rows * cols * 2 < (1 << 20) ? ceil_div(n, 128ll) * 128 : n;
}

// Matrices that one cluster holds, and their launch (rr_orth_short.cu).
bool orth_is_short(long long rows, long long cols);
cudaError_t launch_orth_short(const OrthParams &p, cudaStream_t s);
cudaError_t launch_orth(const OrthParams &p, cudaStream_t s);

}  // namespace rr
