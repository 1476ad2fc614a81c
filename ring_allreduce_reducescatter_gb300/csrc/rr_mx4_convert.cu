// rr_mx4_convert.cu -- quantisation to microscaled 4 bits and back, dropout,
// and the AllReduce fold of 4-bit matrices.
//
// All four are bound by memory: each reads its inputs once and writes its
// outputs once.
#include "rr_mx4.cuh"

namespace rr {

namespace {

template <class K, class P>
cudaError_t launch(K *k, long long grid, int threads, const P &p, cudaStream_t s) {
  if (grid > 0x7fffffffll) return cudaErrorInvalidConfiguration;
  cudaLaunchConfig_t c = {};
  c.gridDim = dim3((unsigned)grid);
  c.blockDim = dim3((unsigned)threads);
  c.stream = s;
  cudaLaunchAttribute a = {};
  a.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  a.val.programmaticStreamSerializationAllowed = 1;
  c.attrs = &a;
  c.numAttrs = 1;
  return cudaLaunchKernelEx(&c, k, p);
}

// --------------------------------------------------------------------------
// quantisation along the rows
// --------------------------------------------------------------------------

// One CTA: 128 rows by 256 columns, the extent of one scale tile.  Warp w
// takes rows w, w + 8, ...; a lane takes eight neighbours of a row (one
// counter of the generator, one 32-bit word of codes), four lanes a block.
// The scales gather in shared memory, so the tile is written whole, its
// padding as zeros.
constexpr int kRowsThreads = 256;

template <int DT, bool SR, bool DROP>
__global__ void __launch_bounds__(kRowsThreads) mx4_rows_kernel(const __grid_constant__ QuantParams p) {
  grid_dependency_wait();
  __shared__ __align__(16) uint8_t tile[kMx4TileBytes];
  const Mx4Out &o = p.by_rows;
  const long long tk = blockIdx.x % o.tiles_k, tr = blockIdx.x / o.tiles_k;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const long long c0 = tk * kMx4TileCols + lane * 8;
  const int valid = (int)max(0ll, min(8ll, p.cols - c0));
  const bool in_row = c0 < o.row_bytes * 2;
#pragma unroll 4
  for (int k = 0; k < kMx4TileRows / 8; ++k) {
    const int rl = warp + 8 * k;
    const long long r = tr * kMx4TileRows + rl;
    uint32_t byte = 0;
    if (r < p.rows) {
      float v[8];
      load8<DT>(p.x, r * p.ld + c0, valid, p.vec, v);
      if constexpr (DROP) drop8(p.drop, (unsigned long long)(r * p.cols + c0), v);
      uint32_t m = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(v[j]) & 0x7fffffffu);
      m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
      m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
      byte = scale_byte(m);
      const float inv = inverse_scale(byte);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = __fmul_rn(v[j], inv);
      uint32_t codes;
      if constexpr (SR)
        codes = pack8_stochastic(v, philox(p.seed, p.subsequence, (unsigned long long)(r * o.row_bytes * 2 + c0) >> 3));
      else
        codes = pack8_nearest(v);
      if (byte == 255u) codes = 0;
      if (in_row) *reinterpret_cast<uint32_t *>(o.data + r * o.row_bytes + c0 / 2) = codes;
    }
    if ((lane & 3) == 0) tile[(lane >> 4) * kMx4AtomBytes + (rl & 31) * 16 + (rl >> 5) * 4 + ((lane >> 2) & 3)] = (uint8_t)byte;
  }
  __syncthreads();
  if (threadIdx.x < kMx4TileBytes / 16)
    reinterpret_cast<uint4 *>(o.scales + (tr * o.tiles_k + tk) * kMx4TileBytes)[threadIdx.x] =
        reinterpret_cast<const uint4 *>(tile)[threadIdx.x];
}

// --------------------------------------------------------------------------
// quantisation along the columns (the result is the transpose), with or
// without the rows
// --------------------------------------------------------------------------

// One CTA: 128 rows by 32 * E columns (E elements in 16 bytes), a warp 32 of
// the rows.  A lane keeps 32 rows of its E columns in registers as they were
// loaded, so each of its columns is a whole block: no exchange between lanes
// for the columns, and the rows' quantisation reads the same registers.  The
// transposed codes (16 bytes a column and warp) go through shared memory to
// be written 64 bytes a column at a time.
constexpr int kTileThreads = 128;

template <int DT>
struct Packed16 {  // 16 bytes of storage elements
  static constexpr int E = 16 / Fmt<DT>::bytes;
  // element j as binary32
  static __device__ __forceinline__ float get(const uint4 &r, int j) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
    if constexpr (DT == kF32) {
      return __uint_as_float(w[j]);
    } else if constexpr (DT == kF16) {
      const float2 f = __half22float2(as_h2(w[j / 2]));
      return (j & 1) ? f.y : f.x;
    } else {
      return __uint_as_float((j & 1) ? w[j / 2] & 0xffff0000u : w[j / 2] << 16);
    }
  }
  static __device__ __forceinline__ uint4 load(const void *base, long long at, int valid, bool vec) {
    const uint8_t *p = static_cast<const uint8_t *>(base) + at * Fmt<DT>::bytes;
    if (vec && valid >= E) return ldg_stream(p);
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int j = 0; j < E; ++j)
      if (j < valid) {
        if constexpr (DT == kF32) w[j] = reinterpret_cast<const uint32_t *>(p)[j];
        else w[j / 2] |= (uint32_t)reinterpret_cast<const uint16_t *>(p)[j] << (16 * (j & 1));
      }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
  // zeroes the elements whose bit in `keep` is clear
  static __device__ __forceinline__ void mask(uint4 &r, uint32_t keep) {
    uint32_t *w = &r.x;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (DT == kF32) {
        if (!(keep >> j & 1)) w[j] = 0;
      } else {
        w[j] &= ((keep >> (2 * j) & 1) ? 0xffffu : 0u) | ((keep >> (2 * j + 1) & 1) ? 0xffff0000u : 0u);
      }
    }
  }
};

// Running maximum of magnitudes: of the two halves of a word apart for 16-bit
// formats (their bit patterns order like the values), of the word for binary32.
template <int DT>
__device__ __forceinline__ uint32_t max_mag(uint32_t m, uint32_t w) {
  if constexpr (DT == kF32) return max(m, w & 0x7fffffffu);
  else return __vmaxu2(m, w & 0x7fff7fffu);
}
template <int DT>
__device__ __forceinline__ uint32_t mag_bits(uint32_t m, int half) {  // as binary32 bits
  if constexpr (DT == kF32) return m;
  const uint32_t h = half ? m >> 16 : m & 0xffffu;
  if constexpr (DT == kBF16) return h << 16;
  return __float_as_uint(__half2float(__ushort_as_half((unsigned short)h)));
}

template <int DT, bool SR, bool DROP, bool ROWS>
__global__ void __launch_bounds__(kTileThreads) mx4_tile_kernel(const __grid_constant__ QuantParams p, int tiles_r) {
  grid_dependency_wait();
  constexpr int E = Packed16<DT>::E;   // columns a lane
  constexpr int W = 32 * E;            // columns a CTA
  __shared__ __align__(16) uint4 codes_t[W * 4];            // [column][64 bytes], 16-byte units swizzled
  __shared__ __align__(16) uint8_t scales_r[W / 128][kMx4AtomBytes];
  __shared__ __align__(16) uint8_t scales_c[W / 128][kMx4AtomBytes];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const long long tr = blockIdx.x % tiles_r, tc = blockIdx.x / tiles_r;
  const long long r0 = tr * kMx4TileRows + warp * 32, c0 = tc * W + lane * E;
  const int valid = (int)max(0ll, min((long long)E, p.cols - c0));
  const float dscale = DROP ? p.drop.scale : 1.f;

  uint4 x[32];
#pragma unroll
  for (int r = 0; r < 32; ++r)
    x[r] = r0 + r < p.rows ? Packed16<DT>::load(p.x, (r0 + r) * p.ld + c0, valid, p.vec) : make_uint4(0, 0, 0, 0);
  if constexpr (DROP) {
#pragma unroll
    for (int r = 0; r < 32; ++r) {
      const uint4 u = numbers8(p.drop.seed, p.drop.subsequence,
                               p.drop.first + (unsigned long long)((r0 + r) * p.cols + c0));
      uint32_t keep = 0;
#pragma unroll
      for (int j = 0; j < E; ++j) keep |= (number_of(u, j) >= p.drop.threshold ? 1u : 0u) << j;
      Packed16<DT>::mask(x[r], keep);
    }
  }

  if constexpr (ROWS) {
    const Mx4Out &o = p.by_rows;
#pragma unroll
    for (int r = 0; r < 32; ++r) {
      uint32_t m = max_mag<DT>(max_mag<DT>(max_mag<DT>(max_mag<DT>(0, x[r].x), x[r].y), x[r].z), x[r].w);
      m = DT == kF32 ? m : max(m & 0xffffu, m >> 16);
#pragma unroll
      for (int d = 1; d < 32 / E; d *= 2) m = max(m, __shfl_xor_sync(0xffffffffu, m, d));
      m = mag_bits<DT>(m, 0);
      if constexpr (DROP) m = __float_as_uint(__fmul_rn(__uint_as_float(m), dscale));
      const uint32_t byte = scale_byte(m);
      const float inv = inverse_scale(byte);
      float v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        v[j] = j < E ? Packed16<DT>::get(x[r], j < E ? j : 0) : 0.f;
        if constexpr (DROP) v[j] = __fmul_rn(v[j], dscale);
        v[j] = __fmul_rn(v[j], inv);
      }
      uint32_t codes;
      const long long i = (r0 + r) * o.row_bytes * 2 + c0;
      if constexpr (SR) {
        uint4 u = philox(p.seed, p.subsequence, (unsigned long long)i >> 3);
        if (E == 4 && (i & 4)) u.x = u.z, u.y = u.w;
        codes = pack8_stochastic(v, u);
      } else {
        codes = pack8_nearest(v);
      }
      if (byte == 255u) codes = 0;
      if (r0 + r < p.rows && c0 < o.row_bytes * 2) {
        uint8_t *q = o.data + i / 2;
        if constexpr (E == 8) *reinterpret_cast<uint32_t *>(q) = codes;
        else *reinterpret_cast<uint16_t *>(q) = (uint16_t)codes;
      }
      constexpr int LB = 32 / E;  // lanes a block
      if (lane % LB == 0) {
        const int j = lane / LB;  // block of the CTA's columns
        scales_r[j / 4][r * 16 + warp * 4 + (j & 3)] = r0 + r < p.rows ? (uint8_t)byte : 0;
      }
    }
  }

  const Mx4Out &o = p.by_cols;
  const unsigned long long sub = p.subsequence + (ROWS ? 1 : 0);
#pragma unroll
  for (int j = 0; j < E; ++j) {
    uint32_t m = 0;
#pragma unroll
    for (int r = 0; r < 32; ++r) m = max_mag<DT>(m, (&x[r].x)[DT == kF32 ? j : j / 2]);
    m = mag_bits<DT>(m, j & 1);
    if constexpr (DROP) m = __float_as_uint(__fmul_rn(__uint_as_float(m), dscale));
    const uint32_t byte = scale_byte(m);
    const float inv = inverse_scale(byte);
    uint32_t q[4];
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      float v[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        v[e] = Packed16<DT>::get(x[8 * g + e], j);
        if constexpr (DROP) v[e] = __fmul_rn(v[e], dscale);
        v[e] = __fmul_rn(v[e], inv);
      }
      if constexpr (SR)
        q[g] = pack8_stochastic(v, philox(p.seed, sub, (unsigned long long)((c0 + j) * o.row_bytes * 2 + r0 + 8 * g) >> 3));
      else
        q[g] = pack8_nearest(v);
      if (byte == 255u) q[g] = 0;
    }
    const int c = lane * E + j;  // column of the CTA
    codes_t[(c * 4 + warp) ^ (lane & 7)] = make_uint4(q[0], q[1], q[2], q[3]);
    scales_c[c / 128][(c & 31) * 16 + ((c >> 5) & 3) * 4 + warp] = (uint8_t)byte;
  }
  __syncthreads();

  // 64 bytes of codes a column: four lanes of 16 bytes
#pragma unroll
  for (int k = 0; k < W * 4 / kTileThreads; ++k) {
    const int unit = threadIdx.x + k * kTileThreads, c = unit / 4, part = unit % 4;
    const long long col = tc * W + c, row = tr * kMx4TileRows + part * 32;
    if (col < p.cols && row < p.rows)
      *reinterpret_cast<uint4 *>(o.data + col * o.row_bytes + row / 2) = codes_t[unit ^ ((c / E) & 7)];
  }
  // the scales: an atom is 128 columns by this CTA's four blocks
  for (int k = threadIdx.x; k < W / 128 * (kMx4AtomBytes / 16); k += kTileThreads) {
    const int a = k / (kMx4AtomBytes / 16), w = k % (kMx4AtomBytes / 16);
    const long long rb = tc * (W / 128) + a;  // 128 rows of the result
    if (rb * kMx4TileRows < p.cols)
      reinterpret_cast<uint4 *>(o.scales + (rb * o.tiles_k + tr / 2) * kMx4TileBytes + (tr & 1) * kMx4AtomBytes)[w] =
          reinterpret_cast<const uint4 *>(scales_c[a])[w];
    if constexpr (ROWS) {
      const Mx4Out &q = p.by_rows;
      const long long atom = tc * (W / 128) + a;  // 128 columns
      if (tr * kMx4TileRows < p.rows && atom / 2 < q.tiles_k)
        reinterpret_cast<uint4 *>(q.scales + (tr * q.tiles_k + atom / 2) * kMx4TileBytes + (atom & 1) * kMx4AtomBytes)[w] =
            reinterpret_cast<const uint4 *>(scales_r[a])[w];
    }
  }
}

template <int DT, bool SR, bool DROP>
cudaError_t quantize_dt(const QuantParams &p, cudaStream_t s) {
  if (!p.by_cols.data) {
    const long long grid = ((p.rows + kMx4TileRows - 1) / kMx4TileRows) * p.by_rows.tiles_k;
    return launch(mx4_rows_kernel<DT, SR, DROP>, grid, kRowsThreads, p, s);
  }
  // tiles of 128 rows, an even number of them (a scale tile of the result
  // spans 256 rows), and columns to whole scale tiles of both results
  constexpr int W = 32 * Packed16<DT>::E;
  const long long tiles_r = 2 * p.by_cols.tiles_k;
  const long long tiles_c = (p.cols + kMx4TileCols - 1) / kMx4TileCols * (kMx4TileCols / W);
  const long long grid = tiles_r * tiles_c;
  if (grid > 0x7fffffffll) return cudaErrorInvalidConfiguration;
  cudaLaunchConfig_t c = {};
  c.gridDim = dim3((unsigned)grid);
  c.blockDim = dim3(kTileThreads);
  c.stream = s;
  cudaLaunchAttribute a = {};
  a.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  a.val.programmaticStreamSerializationAllowed = 1;
  c.attrs = &a;
  c.numAttrs = 1;
  if (p.by_rows.data) return cudaLaunchKernelEx(&c, mx4_tile_kernel<DT, SR, DROP, true>, p, (int)tiles_r);
  return cudaLaunchKernelEx(&c, mx4_tile_kernel<DT, SR, DROP, false>, p, (int)tiles_r);
}

template <int DT>
cudaError_t quantize_any(const QuantParams &p, cudaStream_t s) {
  const bool drop = p.drop.threshold != 0;
  if (p.stochastic) return drop ? quantize_dt<DT, true, true>(p, s) : quantize_dt<DT, true, false>(p, s);
  return drop ? quantize_dt<DT, false, true>(p, s) : quantize_dt<DT, false, false>(p, s);
}

// --------------------------------------------------------------------------
// back to values
// --------------------------------------------------------------------------

constexpr int kFlatThreads = 256;

template <int DT>
__global__ void __launch_bounds__(kFlatThreads) mx4_values_kernel(const __grid_constant__ DequantParams p) {
  grid_dependency_wait();
  const long long gpr = p.row_bytes / 4;  // groups of eight a row
  const long long g = (long long)blockIdx.x * kFlatThreads + threadIdx.x;
  const long long r = g / gpr;
  if (r >= p.rows) return;
  const long long c0 = (g - r * gpr) * 8;
  const int valid = (int)min(8ll, p.cols - c0);
  if (valid <= 0) return;
  const uint32_t codes = __ldg(reinterpret_cast<const uint32_t *>(p.data + r * p.row_bytes + c0 / 2));
  float v[8];
  unpack8(codes, scale_value(__ldg(p.scales + scale_offset(r, c0 / kMx4Block, p.tiles_k))), v);
  store8<DT>(p.out, r * p.ld + c0, valid, p.vec, v);
}

// --------------------------------------------------------------------------
// dropout
// --------------------------------------------------------------------------

template <int DT, bool RES>
__global__ void __launch_bounds__(kFlatThreads) dropout_kernel(const __grid_constant__ DropoutParams p) {
  grid_dependency_wait();
  const long long gpr = ceil_div(p.cols, 8ll);
  const long long g = (long long)blockIdx.x * kFlatThreads + threadIdx.x;
  const long long r = g / gpr;
  if (r >= p.rows) return;
  const long long c0 = (g - r * gpr) * 8;
  const int valid = (int)min(8ll, p.cols - c0);
  float v[8];
  load8<DT>(p.x, r * p.ld_x + c0, valid, p.vec, v);
  if (p.drop.threshold) drop8(p.drop, (unsigned long long)(r * p.cols + c0), v);
  if constexpr (RES) {
    float w[8];
    load8<DT>(p.residual, r * p.ld_res + c0, valid, p.vec, w);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = __fadd_rn(w[j], v[j]);
  }
  store8<DT>(p.out, r * p.ld_out + c0, valid, p.vec, v);
}

// --------------------------------------------------------------------------
// the fold of R ranks' 4-bit matrices
// --------------------------------------------------------------------------

// Element i = row * cols + column lies in chunk c of the partition of
// rows * cols into R chunks and is folded from rank c on, in binary32, as
// ring_allreduce does on the values; the sum is rounded once to storage.  A
// thread takes eight neighbours of a row.
template <int DT>
__global__ void __launch_bounds__(kFlatThreads) mx4_reduce_kernel(const __grid_constant__ Mx4ReduceParams p) {
  grid_dependency_wait();
  const long long gpr = p.row_bytes / 4;
  const long long g = (long long)blockIdx.x * kFlatThreads + threadIdx.x;
  const long long r = g / gpr;
  if (r >= p.rows) return;
  const long long c0 = (g - r * gpr) * 8;
  const int valid = (int)min(8ll, p.cols - c0);
  if (valid <= 0) return;
  const long long at = r * p.row_bytes + c0 / 2, sat = scale_offset(r, c0 / kMx4Block, p.tiles_k);
  const long long i0 = r * p.cols + c0;
  const int R = p.R;
  auto chunk = [&](long long i) { return p.base == 0 ? R - 1 : (int)min((long long)(R - 1), i / p.base); };
  const int first = chunk(i0), last = chunk(i0 + valid - 1);
  float sum[8];
  for (int c = first; c <= last; ++c) {  // one pass, but for a group over a chunk boundary
    float acc[8];
    int k = c;
    for (int s = 0; s < R; ++s) {
      float v[8];
      unpack8(__ldg(reinterpret_cast<const uint32_t *>(p.data[k] + at)), scale_value(__ldg(p.scales[k] + sat)), v);
#pragma unroll
      for (int j = 0; j < 8; ++j) acc[j] = s == 0 ? v[j] : __fadd_rn(acc[j], v[j]);
      k = k + 1 == R ? 0 : k + 1;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (c == first || chunk(i0 + j) == c) sum[j] = acc[j];
  }
  for (int k = 0; k < R; ++k) store8<DT>(p.out[k], i0, valid, p.vec, sum);
}

}  // namespace

cudaError_t launch_mx4_quantize(const QuantParams &p, cudaStream_t s) {
  return p.dtype == kF32 ? quantize_any<kF32>(p, s) : p.dtype == kF16 ? quantize_any<kF16>(p, s) : quantize_any<kBF16>(p, s);
}

cudaError_t launch_mx4_dequantize(const DequantParams &p, cudaStream_t s) {
  const long long groups = p.rows * (p.row_bytes / 4), grid = (groups + kFlatThreads - 1) / kFlatThreads;
  return p.dtype == kF32   ? launch(mx4_values_kernel<kF32>, grid, kFlatThreads, p, s)
         : p.dtype == kF16 ? launch(mx4_values_kernel<kF16>, grid, kFlatThreads, p, s)
                           : launch(mx4_values_kernel<kBF16>, grid, kFlatThreads, p, s);
}

template <int DT>
static cudaError_t dropout_dt(const DropoutParams &p, cudaStream_t s) {
  const long long groups = p.rows * ((p.cols + 7) / 8), grid = (groups + kFlatThreads - 1) / kFlatThreads;
  return p.residual ? launch(dropout_kernel<DT, true>, grid, kFlatThreads, p, s)
                    : launch(dropout_kernel<DT, false>, grid, kFlatThreads, p, s);
}

cudaError_t launch_dropout(const DropoutParams &p, cudaStream_t s) {
  return p.dtype == kF32 ? dropout_dt<kF32>(p, s) : p.dtype == kF16 ? dropout_dt<kF16>(p, s) : dropout_dt<kBF16>(p, s);
}

cudaError_t launch_mx4_reduce(const Mx4ReduceParams &p, cudaStream_t s) {
  const long long groups = p.rows * (p.row_bytes / 4), grid = (groups + kFlatThreads - 1) / kFlatThreads;
  return p.dtype == kF32   ? launch(mx4_reduce_kernel<kF32>, grid, kFlatThreads, p, s)
         : p.dtype == kF16 ? launch(mx4_reduce_kernel<kF16>, grid, kFlatThreads, p, s)
                           : launch(mx4_reduce_kernel<kBF16>, grid, kFlatThreads, p, s);
}

}  // namespace rr
