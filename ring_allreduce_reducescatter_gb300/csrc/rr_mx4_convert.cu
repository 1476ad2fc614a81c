// rr_mx4_convert.cu -- 4-bit matrices back to values, dropout, and the
// AllReduce fold of 4-bit matrices.  All are bound by memory: each reads its
// inputs once and writes its outputs once.
#include "rr_mx4.cuh"

namespace rr {

namespace {

// A block of 256 threads as tx groups of a row by 256 / tx rows: tx is the
// power of two that covers a row's groups, at most 256.  rows_a_thread rows
// of the grid are left to each thread's loop.
struct Shape {
  dim3 grid, block;
};
Shape shape_of(long long groups, long long rows, int rows_a_thread) {
  int tx = 1;
  while (tx < kFlatThreads && tx < groups) tx *= 2;
  const int ty = kFlatThreads / tx;
  const long long y = ceil_div(rows, (long long)ty * rows_a_thread);
  Shape s;
  s.block = dim3((unsigned)tx, (unsigned)ty);
  s.grid = dim3((unsigned)ceil_div(groups, (long long)tx), (unsigned)(y < 65535 ? y : 65535));
  return s;
}

template <class P>
cudaError_t launch(void (*k)(P), const Shape &sh, const P &p, cudaStream_t s) {
  cudaLaunchConfig_t c = {};
  c.gridDim = sh.grid;
  c.blockDim = sh.block;
  c.stream = s;
  cudaLaunchAttribute a = {};
  a.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  a.val.programmaticStreamSerializationAllowed = 1;
  c.attrs = &a;
  c.numAttrs = 1;
  return cudaLaunchKernelEx(&c, k, p);
}

// Sixteen elements of one row to memory, whole sectors where they are aligned.
template <int DT>
__device__ __forceinline__ void store16(void *base, long long at, int valid, bool vec, bool vec32, const float v[16]) {
  if (vec32 && valid >= 16) {
    using T = typename Fmt<DT>::type;
    uint4 raw[2 * kRaw8<DT>];
    narrow8<DT>(v, raw), narrow8<DT>(v + 8, raw + kRaw8<DT>);
    uint4 *o = reinterpret_cast<uint4 *>(static_cast<T *>(base) + at);
#pragma unroll
    for (int j = 0; j < kRaw8<DT>; ++j) stg32(o + 2 * j, raw[2 * j], raw[2 * j + 1]);
  } else {
    store8<DT>(base, at, valid, vec, v);
    if (valid > 8) store8<DT>(base, at + 8, valid - 8, vec, v + 8);
  }
}

// --------------------------------------------------------------------------
// back to values
// --------------------------------------------------------------------------

// A thread takes sixteen neighbours, half a block.
template <int DT>
__global__ void __launch_bounds__(kFlatThreads) mx4_values_kernel(const __grid_constant__ DequantParams p) {
  grid_dependency_wait();
  grid_dependents_launch();
  const long long c0 = ((long long)blockIdx.x * blockDim.x + threadIdx.x) * 16;
  const int valid = (int)max(0ll, min(16ll, p.cols - c0));
  if (valid == 0) return;
  const long long step = (long long)gridDim.y * blockDim.y;
  constexpr int U = 4;
  for (long long r0 = (long long)blockIdx.y * blockDim.y + threadIdx.y; r0 < p.rows; r0 += U * step) {
    uint2 codes[U];
    uint8_t byte[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const long long r = r0 + u * step;
      if (r >= p.rows) break;
      codes[u] = __ldg(reinterpret_cast<const uint2 *>(p.data + r * p.row_bytes + c0 / 2));
      byte[u] = __ldg(p.scales + scale_offset(r, c0 / kMx4Block, p.tiles_k));
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const long long r = r0 + u * step;
      if (r >= p.rows) break;
      const float scale = scale_value(byte[u]);
      float v[16];
      unpack8(codes[u].x, scale, v), unpack8(codes[u].y, scale, v + 8);
      store16<DT>(p.out, r * p.ld + c0, valid, p.vec, p.vec32, v);
    }
  }
}

// --------------------------------------------------------------------------
// dropout
// --------------------------------------------------------------------------

template <int DT, bool RES>
__device__ __forceinline__ void dropout8(const DropoutParams &p, unsigned long long i, float *v, const float *res) {
  if (p.drop.cut) drop8(p.drop, i, v);
  if constexpr (RES) {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = __fadd_rn(res[j], v[j]);
  }
}

// One long row: a thread takes U groups of eight (one counter of the generator
// each), a block's groups apart, all loaded before the first call of the
// generator.
template <int DT, bool RES, int U>
__global__ void __launch_bounds__(kFlatThreads) dropout_flat_kernel(const __grid_constant__ DropoutParams p) {
  grid_dependency_wait();
  grid_dependents_launch();
  using T = typename Fmt<DT>::type;
  const long long block0 = (long long)blockIdx.x * (kFlatThreads * U * 8), c0 = block0 + threadIdx.x * 8;
  float v[U][8], w[U][8];
  if (p.vec && block0 + kFlatThreads * U * 8 <= p.cols) {  // the same for the whole block
    const T *x = static_cast<const T *>(p.x) + c0, *res = static_cast<const T *>(p.residual) + c0;
    uint4 raw[U][kRaw8<DT>], rawr[U][kRaw8<DT>];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int j = 0; j < kRaw8<DT>; ++j) {
        raw[u][j] = ldg_stream(reinterpret_cast<const uint4 *>(x + u * kFlatThreads * 8) + j);
        if constexpr (RES) rawr[u][j] = ldg_stream(reinterpret_cast<const uint4 *>(res + u * kFlatThreads * 8) + j);
      }
    T *o = static_cast<T *>(p.out) + c0;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      widen8<DT>(raw[u], v[u]);
      if constexpr (RES) widen8<DT>(rawr[u], w[u]);
      dropout8<DT, RES>(p, (unsigned long long)(c0 + u * kFlatThreads * 8), v[u], w[u]);
      narrow8<DT>(v[u], raw[u]);
#pragma unroll
      for (int j = 0; j < kRaw8<DT>; ++j) stg_stream(reinterpret_cast<uint4 *>(o + u * kFlatThreads * 8) + j, raw[u][j]);
    }
    return;
  }
#pragma unroll 1
  for (int u = 0; u < U; ++u) {
    const long long c = c0 + u * kFlatThreads * 8;
    const int valid = (int)max(0ll, min(8ll, p.cols - c));
    if (valid == 0) break;
    load8<DT>(p.x, c, valid, p.vec, v[0]);
    if constexpr (RES) load8<DT>(p.residual, c, valid, p.vec, w[0]);
    dropout8<DT, RES>(p, (unsigned long long)c, v[0], w[0]);
    store8<DT>(p.out, c, valid, p.vec, v[0]);
  }
}

template <int DT, bool RES>
__global__ void __launch_bounds__(kFlatThreads) dropout_rows_kernel(const __grid_constant__ DropoutParams p) {
  grid_dependency_wait();
  grid_dependents_launch();
  const long long c0 = ((long long)blockIdx.x * blockDim.x + threadIdx.x) * 8;
  const int valid = (int)max(0ll, min(8ll, p.cols - c0));
  if (valid == 0) return;
  for (long long r = (long long)blockIdx.y * blockDim.y + threadIdx.y; r < p.rows;
       r += (long long)gridDim.y * blockDim.y) {
    float v[8], w[8];
    load8<DT>(p.x, r * p.ld_x + c0, valid, p.vec, v);
    if constexpr (RES) load8<DT>(p.residual, r * p.ld_res + c0, valid, p.vec, w);
    dropout8<DT, RES>(p, (unsigned long long)(r * p.cols + c0), v, w);
    store8<DT>(p.out, r * p.ld_out + c0, valid, p.vec, v);
  }
}

// --------------------------------------------------------------------------
// the fold of R ranks' 4-bit matrices
// --------------------------------------------------------------------------

// Sixteen values summed over the ranks from rank c on, four ranks' loads in
// flight.
__device__ __forceinline__ void fold16(const Mx4ReduceParams &p, int c, long long at, long long sat, float acc[16]) {
  const int R = p.R;
  int k = c;
  for (int s0 = 0; s0 < R; s0 += 4) {
    uint2 codes[4];
    uint8_t byte[4];
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      if (s0 + b >= R) break;
      codes[b] = __ldg(reinterpret_cast<const uint2 *>(p.data[k] + at));
      byte[b] = __ldg(p.scales[k] + sat);
      k = k + 1 == R ? 0 : k + 1;
    }
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      if (s0 + b >= R) break;
      const float scale = scale_value(byte[b]);
      float v[16];
      unpack8(codes[b].x, scale, v), unpack8(codes[b].y, scale, v + 8);
#pragma unroll
      for (int j = 0; j < 16; ++j) acc[j] = s0 + b == 0 ? v[j] : __fadd_rn(acc[j], v[j]);
    }
  }
}

// Element i = row * cols + column lies in chunk c of the partition of
// rows * cols into R chunks and is folded from rank c on, in binary32, as
// ring_allreduce does on the values; the sum is rounded once to storage.
template <int DT>
__global__ void __launch_bounds__(kFlatThreads) mx4_reduce_kernel(const __grid_constant__ Mx4ReduceParams p) {
  grid_dependency_wait();
  grid_dependents_launch();
  const long long c0 = ((long long)blockIdx.x * blockDim.x + threadIdx.x) * 16;
  const int valid = (int)max(0ll, min(16ll, p.cols - c0));
  if (valid == 0) return;
  const int R = p.R;
  auto chunk = [&](long long i) {
    if (p.base == 0) return R - 1;
    // (a 64-bit division takes several times the instructions of a 32-bit one)
    const long long c = p.rows * p.cols < (1ll << 32) ? (long long)((unsigned)i / (unsigned)p.base) : i / p.base;
    return c < R - 1 ? (int)c : R - 1;
  };
  for (long long r = (long long)blockIdx.y * blockDim.y + threadIdx.y; r < p.rows;
       r += (long long)gridDim.y * blockDim.y) {
    const long long at = r * p.row_bytes + c0 / 2, sat = scale_offset(r, c0 / kMx4Block, p.tiles_k);
    const long long i0 = r * p.cols + c0;
    const int first = chunk(i0);
    float sum[16];
    fold16(p, first, at, sat, sum);
    if (first + 1 < R && i0 + valid > (first + 1) * p.base) {  // the group ends in another chunk, or several
      const int last = chunk(i0 + valid - 1);
      for (int c = first + 1; c <= last; ++c) {
        float acc[16];
        fold16(p, c, at, sat, acc);
#pragma unroll
        for (int j = 0; j < 16; ++j)
          if (chunk(i0 + j) == c) sum[j] = acc[j];
      }
    }
    for (int k = 0; k < R; ++k) store16<DT>(p.out[k], i0, valid, p.vec, p.vec32, sum);
  }
}

}  // namespace

cudaError_t launch_mx4_dequantize(const DequantParams &p, cudaStream_t s) {
  const Shape sh = shape_of(p.row_bytes / 8, p.rows, 4);
  return p.dtype == kF32   ? launch(mx4_values_kernel<kF32>, sh, p, s)
         : p.dtype == kF16 ? launch(mx4_values_kernel<kF16>, sh, p, s)
                           : launch(mx4_values_kernel<kBF16>, sh, p, s);
}

template <int DT>
static cudaError_t dropout_dt(const DropoutParams &p, cudaStream_t s) {
  const long long groups = ceil_div(p.cols, 8ll);
  if (p.rows == 1) {
    constexpr int U = DT == kF32 ? 1 : 2;
    const long long grid = ceil_div(groups, (long long)kFlatThreads * U);
    if (grid > 0x7fffffffll) return cudaErrorInvalidConfiguration;
    const Shape sh{dim3((unsigned)grid), dim3(kFlatThreads)};
    return p.residual ? launch(dropout_flat_kernel<DT, true, U>, sh, p, s)
                      : launch(dropout_flat_kernel<DT, false, U>, sh, p, s);
  }
  const Shape sh = shape_of(groups, p.rows, 1);
  return p.residual ? launch(dropout_rows_kernel<DT, true>, sh, p, s)
                    : launch(dropout_rows_kernel<DT, false>, sh, p, s);
}

cudaError_t launch_dropout(const DropoutParams &p, cudaStream_t s) {
  return p.dtype == kF32 ? dropout_dt<kF32>(p, s) : p.dtype == kF16 ? dropout_dt<kF16>(p, s) : dropout_dt<kBF16>(p, s);
}

cudaError_t launch_mx4_reduce(const Mx4ReduceParams &p, cudaStream_t s) {
  const Shape sh = shape_of(p.row_bytes / 8, p.rows, 1);
  return p.dtype == kF32   ? launch(mx4_reduce_kernel<kF32>, sh, p, s)
         : p.dtype == kF16 ? launch(mx4_reduce_kernel<kF16>, sh, p, s)
                           : launch(mx4_reduce_kernel<kBF16>, sh, p, s);
}

}  // namespace rr
