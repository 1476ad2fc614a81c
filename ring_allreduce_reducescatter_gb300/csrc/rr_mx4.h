// rr_mx4.h -- parameter blocks and launchers of the microscaled 4-bit
// operators and dropout, between the C ABI (rr_mx4_api.cu) and the kernel
// translation units (rr_mx4_convert.cu, rr_mx4_matmul.cu).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "ringred.h"
#include "rr_params.h"

namespace rr {

// A block is 32 elements under one scale byte; the scales of 128 rows by
// 8 blocks (256 elements) are one tile of 1024 bytes, in the order the tensor
// cores' scale copies read: two atoms of 512 bytes (4 blocks each), where row
// r of the 128 has 4 bytes at (r % 32) * 16 + (r / 32) * 4.
constexpr int kMx4Block = 32;
constexpr int kMx4TileRows = 128;
constexpr int kMx4TileCols = 256;
constexpr int kMx4TileBytes = 1024;
constexpr int kMx4AtomBytes = 512;

template <class T>
__host__ __device__ constexpr T ceil_div(T a, T b) {
  return (a + b - 1) / b;
}

// Allows a kernel its dynamic shared memory, once a device.
template <auto kKernel>
cudaError_t allow_smem(int bytes) {
  static std::atomic<unsigned long long> done{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 64 && (done.load(std::memory_order_relaxed) >> dev & 1)) return cudaSuccess;
  e = cudaFuncSetAttribute(kKernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess && dev < 64) done.fetch_or(1ull << dev, std::memory_order_relaxed);
  return e;
}

struct Mx4Out {
  uint8_t *data;         // [rows][row_bytes]
  uint8_t *scales;       // [ceil(rows / 128)][tiles_k][1024]
  long long rows;
  long long row_bytes;   // 16 * ceil(cols / 32)
  long long tiles_k;     // ceil(cols / 256)
};

// The generator of one seed and subsequence: the ten rounds' keys, made on the
// host so that each is an operand from the parameter block (made in the
// kernels they cost a fifth of the generator's instructions).
struct Generator {
  unsigned int keys[20];
  unsigned int sub_lo, sub_hi;
};
inline Generator make_generator(unsigned long long seed, unsigned long long subsequence) {
  Generator g;
  unsigned int k0 = (unsigned int)seed, k1 = (unsigned int)(seed >> 32);
  for (int r = 0; r < 10; ++r) {
    g.keys[2 * r] = k0, g.keys[2 * r + 1] = k1;
    k0 += 0x9E3779B9u, k1 += 0xBB67AE85u;
  }
  g.sub_lo = (unsigned int)subsequence, g.sub_hi = (unsigned int)(subsequence >> 32);
  return g;
}

struct DropParams {
  Generator gen;
  unsigned long long first;
  unsigned int cut;  // threshold << 16: kept if the 16-bit number, so shifted, is at least this; 0: everything is kept
  float scale;       // 65536 / (65536 - threshold)
};

struct QuantParams {
  const void *x;
  long long rows, cols, ld;
  Mx4Out by_rows, by_cols;   // data null: not wanted
  Generator gen_rows, gen_cols;  // stochastic rounding
  DropParams drop;
  uintptr_t x_lo, x_hi;  // the bytes of x: [x_lo, x_hi)
  int dtype, sms;
  bool stochastic;
  bool vec, vec32;  // 16- and 32-byte groups of the rows of x are aligned
};

struct DequantParams {
  const uint8_t *data, *scales;
  long long rows, cols, row_bytes, tiles_k;
  void *out;
  long long ld;
  int dtype;
  bool vec, vec32;  // 16- and 32-byte groups of the rows of out are aligned
};

struct DropoutParams {
  const void *x, *residual;  // residual may be null
  void *out;
  long long rows, cols, ld_x, ld_res, ld_out;
  DropParams drop;
  int dtype;
  bool vec;
};

struct Mx4ReduceParams {
  const uint8_t *data[RR_MAX_RANKS], *scales[RR_MAX_RANKS];
  void *out[RR_MAX_RANKS];
  long long rows, cols, row_bytes, tiles_k, base;  // base: floor(rows * cols / R)
  int R, dtype;
  bool vec, vec32;
};

struct Mx4Operand {
  const uint8_t *data, *scales;
  long long rows, row_bytes;
};

struct MatmulParams {
  Mx4Operand a, b;
  long long m, n, k;
  void *out;
  const void *residual;   // may be null
  long long ld_out, ld_res;
  DropParams drop;
  unsigned int *status;
  int dtype, sms;
  bool vec;    // every 16-byte group of the rows of out and residual is aligned
  bool vec32;  // every 32-byte group of them
};

cudaError_t launch_mx4_quantize_f32(const QuantParams &p, cudaStream_t s);
cudaError_t launch_mx4_quantize_f16(const QuantParams &p, cudaStream_t s);
cudaError_t launch_mx4_quantize_bf16(const QuantParams &p, cudaStream_t s);
inline cudaError_t launch_mx4_quantize(const QuantParams &p, cudaStream_t s) {
  return p.dtype == kF32   ? launch_mx4_quantize_f32(p, s)
         : p.dtype == kF16 ? launch_mx4_quantize_f16(p, s)
                           : launch_mx4_quantize_bf16(p, s);
}
cudaError_t launch_mx4_dequantize(const DequantParams &p, cudaStream_t s);
cudaError_t launch_dropout(const DropoutParams &p, cudaStream_t s);
cudaError_t launch_mx4_reduce(const Mx4ReduceParams &p, cudaStream_t s);
cudaError_t launch_mx4_matmul(const MatmulParams &p, cudaStream_t s);

// Defined in rr_api.cu: the current device's status word and SM count, and the
// record behind ring_last_cuda_error.
rr_status device_info(unsigned int **status, int *sms);
bool note_cuda(cudaError_t e);

}  // namespace rr
