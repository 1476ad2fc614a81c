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
// generator.  (The output may be x or the residual: what a thread stores, it has
// loaded itself.)
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
        raw[u][j] = ld16_stream(reinterpret_cast<const uint4 *>(x + u * kFlatThreads * 8) + j);
        if constexpr (RES) rawr[u][j] = ld16_stream(reinterpret_cast<const uint4 *>(res + u * kFlatThreads * 8) + j);
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
// the fold of R ranks' 4-bit matrices into contiguous outputs
// --------------------------------------------------------------------------

// Element i = row * cols + column lies in chunk c of the partition of
// rows * cols into R chunks and is folded from rank c on, in binary32, as
// ring_allreduce does on the values; the sum is rounded once to storage.  A
// thread takes sixteen neighbours of the flat output, so its stores are whole
// aligned sectors whatever the number of columns; where columns are no
// multiple of 16 it shifts its codes into place and may meet two scales.  (A
// thread by sixteen columns of a row instead stored rows of odd length element
// by element: 46 us for the values of 5003 x 1999, now 14.)  With R = 1 it
// is the values of one matrix.

// Where the sixteen elements of a thread lie: from column `col` of row `row`
// on, the first `here` of them in that row, the rest at the start of the next
// one (cols >= 16).
struct Group {
  long long row, col;
  int here;    // 16: all
  bool next;   // some lie in the next row
};

// The sum over the ranks from rank c on, kB ranks' loads in flight.  kAligned:
// the group is half a block.  Otherwise its codes are shifted into place and
// its scales are up to three: the block of its first element, the one after
// it, and the next row's first.
template <bool kAligned, bool kOne, int kB>
__device__ __forceinline__ void fold16(const Mx4ReduceParams &p, int c, const Group &g, float sum[16]) {
  const int R = kOne ? 1 : p.R;
  const long long at = g.row * p.row_bytes + g.col / 8 * 4;
  const long long sat = scale_offset(g.row, g.col / kMx4Block, p.tiles_k);
  const int sh = (int)(g.col & 7) * 4, edge = kMx4Block - (int)(g.col & 31);  // edge: first element of the second block
  const int words = (int)((g.col & 7) + g.here + 7) / 8;                      // of this row's codes
  const bool two = edge < g.here;
  const long long sat1 = !kAligned && two ? scale_offset(g.row, g.col / kMx4Block + 1, p.tiles_k) : sat;
  const long long next = (g.row + 1) * p.row_bytes, snext = g.next ? scale_offset(g.row + 1, 0, p.tiles_k) : sat;
  int k = c;
  for (int s0 = 0; s0 < R; s0 += kB) {
    uint32_t w[kB][3], n[kB][2];
    uint8_t y[kB][3];
#pragma unroll
    for (int b = 0; b < kB; ++b) {
      if (s0 + b >= R) break;
      const uint32_t *q = reinterpret_cast<const uint32_t *>(p.data[k] + at);
      if constexpr (kAligned) {
        const uint2 u = __ldg(reinterpret_cast<const uint2 *>(q));
        w[b][0] = u.x, w[b][1] = u.y;
      } else {
        w[b][0] = __ldg(q);
        w[b][1] = words > 1 ? __ldg(q + 1) : 0u;
        w[b][2] = words > 2 ? __ldg(q + 2) : 0u;
        y[b][1] = __ldg(p.scales[k] + sat1);
        n[b][0] = n[b][1] = 0;
        y[b][2] = 0;
        if (g.next) {
          const uint2 u = __ldg(reinterpret_cast<const uint2 *>(p.data[k] + next));
          n[b][0] = u.x, n[b][1] = u.y;
          y[b][2] = __ldg(p.scales[k] + snext);
        }
      }
      y[b][0] = __ldg(p.scales[k] + sat);
      k = k + 1 == R ? 0 : k + 1;
    }
#pragma unroll
    for (int b = 0; b < kB; ++b) {
      if (s0 + b >= R) break;
      float v[16];
      const float scale = scale_value(y[b][0]);
      if constexpr (kAligned) {
        unpack8(w[b][0], scale, v), unpack8(w[b][1], scale, v + 8);
      } else {
        // (columns past the last are stored as zeros, so the codes only need joining)
        uint32_t lo = __funnelshift_r(w[b][0], w[b][1], sh), hi = __funnelshift_r(w[b][1], w[b][2], sh);
        if (g.next) {
          const unsigned long long m = (((unsigned long long)n[b][1] << 32) | n[b][0]) << (4 * g.here);
          lo |= (uint32_t)m, hi |= (uint32_t)(m >> 32);
        }
        unpack8(lo, 1.f, v), unpack8(hi, 1.f, v + 8);
        const float scale1 = scale_value(y[b][1]), scale2 = scale_value(y[b][2]);
#pragma unroll
        for (int j = 0; j < 16; ++j) v[j] = __fmul_rn(v[j], j >= g.here ? scale2 : j < edge ? scale : scale1);
      }
#pragma unroll
      for (int j = 0; j < 16; ++j) sum[j] = s0 + b == 0 ? v[j] : __fadd_rn(sum[j], v[j]);
    }
  }
}

// An aligned group that meets several chunks: each chunk's fold, an element from its own.
__device__ __noinline__ void fold_chunks(const Mx4ReduceParams &p, int first, long long i0, int valid, const Group &g,
                                         float sum[16]) {
#pragma unroll 1
  for (int c = first; c < p.R; ++c) {
    if (c > first && i0 + valid <= c * p.base) break;
    float more[16];
    fold16<true, false, 4>(p, c, g, more);
#pragma unroll
    for (int j = 0; j < 16; ++j) sum[j] = c == first || i0 + j >= c * p.base ? more[j] : sum[j];
  }
}

// One element, for rows shorter than sixteen.
__device__ __noinline__ float fold_element(const Mx4ReduceParams &p, int c, long long row, long long col) {
  float acc = 0.f;
  int k = c;
  for (int s = 0; s < p.R; ++s) {
    const uint32_t byte = __ldg(p.data[k] + row * p.row_bytes + col / 2);
    const uint32_t code = (col & 1) ? byte >> 4 : byte & 15u;
    float v[8];
    unpack8(code, scale_value(__ldg(p.scales[k] + scale_offset(row, col / kMx4Block, p.tiles_k))), v);
    acc = s == 0 ? v[0] : __fadd_rn(acc, v[0]);
    k = k + 1 == p.R ? 0 : k + 1;
  }
  return acc;
}

// kOne: R = 1, the values of one matrix.  Eight ranks of 4096 x 4096 to
// bfloat16: 55 us with eight ranks in flight, 0.92 of the copy rate (four: 60).
template <int DT, bool kAligned, bool kOne>
__global__ void __launch_bounds__(kFlatThreads, kAligned || kOne ? 4 : 2) mx4_fold_kernel(const __grid_constant__ Mx4ReduceParams p) {
  grid_dependency_wait();
  grid_dependents_launch();
  const long long total = p.rows * p.cols, i0 = ((long long)blockIdx.x * kFlatThreads + threadIdx.x) * 16;
  if (i0 >= total) return;
  // (a 64-bit division takes several times the instructions of a 32-bit one)
  const bool narrow = total < (1ll << 32);
  auto chunk = [&](long long i) {
    if (kOne || p.base == 0) return p.R - 1;
    const long long c = narrow ? (long long)((unsigned)i / (unsigned)p.base) : i / p.base;
    return c < p.R - 1 ? (int)c : p.R - 1;
  };
  const int valid = (int)min(16ll, total - i0);
  Group g;
  g.row = narrow ? (long long)((unsigned)i0 / (unsigned)p.cols) : i0 / p.cols;
  g.col = i0 - g.row * p.cols;
  g.here = kAligned ? 16 : (int)min(16ll, p.cols - g.col);
  g.next = !kAligned && g.here < 16 && g.row + 1 < p.rows;
  float sum[16];
  if (kAligned || p.cols >= 16) {
    const int first = chunk(i0);
    if constexpr (kOne) {
      fold16<kAligned, true, 1>(p, first, g, sum);
    } else if constexpr (kAligned) {
      if (first == p.R - 1 || i0 + valid <= (first + 1) * p.base) {
        fold16<true, false, 8>(p, first, g, sum);
      } else {
        float v[16];  // (in local memory: its address is taken)
        fold_chunks(p, first, i0, valid, g, v);
#pragma unroll
        for (int j = 0; j < 16; ++j) sum[j] = v[j];
      }
    } else {
      // one pass, but for a group over a chunk boundary (or several); here the
      // loop was faster than the call (1001 x 1003 over eight ranks: 16 us
      // against 19; with four ranks in flight instead of two 12), in the
      // aligned kernel slower
#pragma unroll 1
      for (int c = first; c < p.R; ++c) {
        if (c > first && i0 + valid <= c * p.base) break;
        float more[16];
        fold16<false, false, 4>(p, c, g, more);
#pragma unroll
        for (int j = 0; j < 16; ++j) sum[j] = c == first || i0 + j >= c * p.base ? more[j] : sum[j];
      }
    }
  } else {
    long long r = g.row, c = g.col;
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      sum[j] = j < valid ? fold_element(p, chunk(i0 + j), r, c) : 0.f;
      if (++c == p.cols) c = 0, ++r;
    }
  }
  for (int k = 0; k < (kOne ? 1 : p.R); ++k) store16<DT>(p.out[k], i0, valid, p.vec, p.vec32, sum);
}

template <int DT>
cudaError_t fold_dt(const Mx4ReduceParams &p, cudaStream_t s) {
  const long long grid = ceil_div(ceil_div(p.rows * p.cols, 16ll), (long long)kFlatThreads);
  if (grid > 0x7fffffffll) return cudaErrorInvalidConfiguration;
  const Shape sh{dim3((unsigned)grid), dim3(kFlatThreads)};
  if (p.R == 1 && p.cols % 16 != 0) return launch(mx4_fold_kernel<DT, false, true>, sh, p, s);
  return p.cols % 16 == 0 ? launch(mx4_fold_kernel<DT, true, false>, sh, p, s)
                          : launch(mx4_fold_kernel<DT, false, false>, sh, p, s);
}

}  // namespace

cudaError_t launch_mx4_dequantize(const DequantParams &p, cudaStream_t s) {
  if (p.ld == p.cols && p.cols % 16 != 0) {  // contiguous rows of odd length
    Mx4ReduceParams q{};
    q.data[0] = p.data, q.scales[0] = p.scales, q.out[0] = p.out;
    q.rows = p.rows, q.cols = p.cols, q.row_bytes = p.row_bytes, q.tiles_k = p.tiles_k, q.base = p.rows * p.cols;
    q.R = 1, q.dtype = p.dtype;
    q.vec = reinterpret_cast<uintptr_t>(p.out) % 16 == 0, q.vec32 = reinterpret_cast<uintptr_t>(p.out) % 32 == 0;
    return launch_mx4_reduce(q, s);
  }
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
  return p.dtype == kF32 ? fold_dt<kF32>(p, s) : p.dtype == kF16 ? fold_dt<kF16>(p, s) : fold_dt<kBF16>(p, s);
}

}  // namespace rr
