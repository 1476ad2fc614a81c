// rr_mx4_quantize.cuh -- quantisation to microscaled 4 bits of one storage
// format (compiled once for each by rr_mx4_quantize_*.cu).
//
// Bound by memory where the rounding is to nearest, on the 16-byte grid: the
// input is read once, 17/32 of a byte an element and direction written.
// Stochastic rounding takes twice the instructions (8192 x 4096 bfloat16 along
// the rows: 20.9 an element for 9.5, of which the generator's, one call for every
// eight elements and direction, are 5) and two to four times the memory's time.
// Two thirds of the issue slots are busy then, so neither the issue rate nor
// memory is used up: a tile waits for all its loads before it computes, and
// every thread sets up its addresses for 64 elements.
#pragma once

#include "rr_mx4.cuh"

namespace rr {

namespace mx4q {

__device__ __forceinline__ void copy_async16(void *smem_dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_addr(smem_dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_async_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// Sixteen bytes kN times, neighbouring elements of x from q on, of which the
// first `valid` exist (the rest read as zero), element by element.
template <int DT, int kN>
__device__ __forceinline__ void load_ends(const uint8_t *q, int valid, uint4 out[kN]) {
  constexpr int E = 16 / Fmt<DT>::bytes;
#pragma unroll
  for (int n = 0; n < kN; ++n) {
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int j = 0; j < E; ++j)
      if (n * E + j < valid) {
        if constexpr (DT == kF32) w[j] = reinterpret_cast<const uint32_t *>(q)[n * E + j];
        else w[j / 2] |= (uint32_t)reinterpret_cast<const uint16_t *>(q)[n * E + j] << (16 * (j & 1));
      }
    out[n] = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// The same for rows off the 16-byte grid, in two steps so that several rows'
// loads can be in flight: the aligned vectors around the elements (where all
// exist and the vectors lie inside x), then the elements out of them.
template <int DT, int kN>
__device__ __forceinline__ bool load_around(const QuantParams &p, long long at, int valid, uint4 v[kN + 1]) {
  const uintptr_t q = reinterpret_cast<uintptr_t>(p.x) + (uintptr_t)(at * Fmt<DT>::bytes), a = q & ~(uintptr_t)15;
  if (valid < kN * 16 / Fmt<DT>::bytes || a < p.x_lo || a + 16 * (kN + 1) > p.x_hi) return false;
#pragma unroll
  for (int j = 0; j <= kN; ++j) v[j] = ldg_l1(reinterpret_cast<const void *>(a + 16 * j));
  return true;
}
template <int DT, int kN>
__device__ __forceinline__ void take_from(const QuantParams &p, long long at, int valid, bool around,
                                          const uint4 v[kN + 1], uint4 out[kN]) {
  if (around) {
    const int sh = (int)((reinterpret_cast<uintptr_t>(p.x) + (uintptr_t)(at * Fmt<DT>::bytes)) & 15);
#pragma unroll
    for (int j = 0; j < kN; ++j) out[j] = funnel16(v[j], v[j + 1], sh);
  } else {
    load_ends<DT, kN>(static_cast<const uint8_t *>(p.x) + at * Fmt<DT>::bytes, valid, out);
  }
}

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
// The largest magnitude of eight elements, as its own bits.
template <int DT>
__device__ __forceinline__ uint32_t max_mag8(const uint4 *raw) {
  uint32_t m = 0;
#pragma unroll
  for (int j = 0; j < kRaw8<DT>; ++j)
    m = max_mag<DT>(max_mag<DT>(max_mag<DT>(max_mag<DT>(m, raw[j].x), raw[j].y), raw[j].z), raw[j].w);
  return DT == kF32 ? m : max(m & 0xffffu, m >> 16);
}

// Zeroes the dropped ones of eight elements, whose numbers are u.
template <int DT>
__device__ __forceinline__ void mask8(const uint4 &u, uint32_t cut, uint4 *raw) {
  uint32_t *w = &raw[0].x;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const bool lo = kept(u, 2 * j, cut), hi = kept(u, 2 * j + 1, cut);
    if constexpr (DT == kF32) {
      if (!lo) w[2 * j] = 0;
      if (!hi) w[2 * j + 1] = 0;
    } else {
      w[j] &= (lo ? 0xffffu : 0u) | (hi ? 0xffff0000u : 0u);
    }
  }
}
// Of sixteen elements, from element i of the tensor on.
template <int DT>
__device__ __forceinline__ void mask16(const DropParams &d, unsigned long long i, uint4 *raw) {
  i += d.first;
  const unsigned long long g = i >> 3;
  const int sh = (int)(i & 7) * 2;
  uint4 a = philox(d.gen, g), b = philox(d.gen, g + 1);
  if (sh != 0) {
    a = funnel16(a, b, sh);
    b = funnel16(b, philox(d.gen, g + 2), sh);
  }
  mask8<DT>(a, d.cut, raw);
  mask8<DT>(b, d.cut, raw + kRaw8<DT>);
}

// Eight elements of one block to codes.
template <bool SR, bool DROP>
__device__ __forceinline__ uint32_t codes8(float v[8], uint32_t byte, float inv, float dscale, const Generator &gen,
                                           unsigned long long group) {
  if constexpr (DROP) {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = __fmul_rn(v[j], dscale);
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = __fmul_rn(v[j], inv);
  uint32_t q;
  if constexpr (SR) q = pack8_stochastic(v, philox(gen, group));
  else q = pack8_nearest(v);
  return byte == 255u ? 0u : q;
}

// --------------------------------------------------------------------------
// along the rows
// --------------------------------------------------------------------------

// One CTA: 128 rows by 256 columns, the extent of one scale tile.  A lane takes
// sixteen neighbours, half a block (two counters of the generator, one store
// of eight bytes), so a warp takes two rows at a time; warp w the pairs w,
// w + warps, ...  Eight a lane, four lanes a block, took 12 instructions an
// element instead of 7.  The scales gather in shared memory, so the tile is
// written whole, its padding as zeros.
template <int DT, bool SR, bool DROP>
__global__ void __launch_bounds__(512) mx4_rows_kernel(const __grid_constant__ QuantParams p) {
  grid_dependency_wait();
  grid_dependents_launch();
  using T = typename Fmt<DT>::type;
  constexpr int N = 2 * kRaw8<DT>;        // 16-byte loads a lane and row
  constexpr int U = DT == kF32 ? 2 : 4;   // pairs of rows in flight
  __shared__ __align__(16) uint8_t tile[kMx4TileBytes];
  const Mx4Out &o = p.by_rows;
  const unsigned tk = blockIdx.x % (unsigned)o.tiles_k, tr = blockIdx.x / (unsigned)o.tiles_k;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, warps = blockDim.x / 32;
  const int cl = lane % 16 * 16, rl0 = warp * 2 + lane / 16;
  const long long c0 = (long long)tk * kMx4TileCols + cl, r0 = (long long)tr * kMx4TileRows + rl0;
  const int valid = (int)max(0ll, min(16ll, p.cols - c0));
  const bool in_row = c0 < o.row_bytes * 2;
  const int left = (int)max(-1ll, min((long long)kMx4TileRows, p.rows - r0));  // rows from this lane's first on
  // everything below steps from one pair of rows to the warp's next
  const uint8_t *src = static_cast<const uint8_t *>(p.x) + (r0 * p.ld + c0) * (int)sizeof(T);  // read only where it exists
  const long long src_step = 2 * warps * p.ld * (int)sizeof(T);
  uint8_t *dst = o.data + r0 * o.row_bytes + c0 / 2;
  const long long dst_step = 2 * warps * o.row_bytes;
  unsigned long long group = (unsigned long long)(r0 * o.row_bytes * 2 + c0) >> 3, element = (unsigned long long)(r0 * p.cols + c0);
  const unsigned long long group_step = (unsigned long long)dst_step / 4, element_step = 2ull * warps * p.cols;
  uint8_t *scale = tile + (cl >> 7) * kMx4AtomBytes + ((cl >> 5) & 3);
#pragma unroll 1
  for (int k = 0; k < kMx4TileRows; k += 2 * U * warps) {
    uint4 raw[U][N];
#pragma unroll
    for (int u = 0; u < U; ++u, src += src_step) {
      const int dr = k + u * 2 * warps;
      if (valid == 16 && dr < left) {
        // (whole sectors: 16-byte loads of a lane's 32 bytes fetched each twice)
#pragma unroll
        for (int j = 0; j < N; j += 2) {
          if (p.vec32) ldg32_stream(src + 16 * j, raw[u][j], raw[u][j + 1]);
          else raw[u][j] = ldg_l1(src + 16 * j), raw[u][j + 1] = ldg_l1(src + 16 * j + 16);
        }
      } else {
        load_ends<DT, N>(src, dr < left ? valid : 0, raw[u]);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u, dst += dst_step, group += group_step, element += element_step) {
      const int dr = k + u * 2 * warps, rl = rl0 + dr;
      uint32_t byte = 0;
      if (dr < left + lane / 16) {  // the warp's first row exists
        if constexpr (DROP) {
          mask16<DT>(p.drop, element, raw[u]);
        }
        uint32_t m = max(max_mag8<DT>(raw[u]), max_mag8<DT>(raw[u] + kRaw8<DT>));
        m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
        m = mag_bits<DT>(m, 0);
        if constexpr (DROP) m = __float_as_uint(__fmul_rn(__uint_as_float(m), p.drop.scale));
        byte = scale_byte(m);
        const float inv = inverse_scale(byte);
        uint2 q;
        float v[8];
        widen8<DT>(raw[u], v);
        q.x = codes8<SR, DROP>(v, byte, inv, p.drop.scale, p.gen_rows, group);
        widen8<DT>(raw[u] + kRaw8<DT>, v);
        q.y = codes8<SR, DROP>(v, byte, inv, p.drop.scale, p.gen_rows, group + 1);
        if (dr < left && in_row) *reinterpret_cast<uint2 *>(dst) = q;
      }
      if ((lane & 1) == 0) scale[(rl & 31) * 16 + (rl >> 5) * 4] = (uint8_t)byte;
    }
  }
  __syncthreads();
  if (threadIdx.x < kMx4TileBytes / 16)
    reinterpret_cast<uint4 *>(o.scales + ((long long)tr * o.tiles_k + tk) * kMx4TileBytes)[threadIdx.x] =
        reinterpret_cast<const uint4 *>(tile)[threadIdx.x];
}

// --------------------------------------------------------------------------
// along the columns (the result is the transpose), with or without the rows
// --------------------------------------------------------------------------

// One CTA: 64 rows (16 where the rows' result alone is wanted) by W columns (512
// bytes a row), brought to shared memory by asynchronous copies, 24 warps an SM
// in several CTAs, so that one's loads run under another's arithmetic.  First the rows (a lane sixteen neighbours, two
// lanes a block; dropout is applied in place here), then the columns: a lane
// takes the 32-bit word of one column, or two, down 32 rows, a whole block in
// registers.  Four warps to nearest, each two blocks one after the other, so
// that a lane stores 32 bytes, a whole sector (eight warps: columns of
// 8192 x 4096 bfloat16 18.5 us instead of 14.7); eight where the generator
// is called, whose long chains want more warps a tile (2048 x 4096 both ways
// 16 us instead of 22).  (Holding the tile in
// registers instead, 32 rows a lane, spilled: 47 us for both ways of
// 8192 x 4096 bfloat16, now 21.  Tiles of 128 rows leave SMs idle at the end:
// 4096 x 4096 stochastic both ways 30 us, now 28; of the rows alone, tiles of 64
// and of 16 rows: stochastic 15.8 and 15.0 us, 5003 x 1999 binary32 to nearest
// 19.2 and 14.5.)
constexpr int kTileRowBytes = 512;

// Rows and warps of a tile.
__host__ __device__ constexpr int tile_rows(bool cols) { return cols ? 64 : 16; }
__host__ __device__ constexpr int tile_warps(bool generator, bool cols) { return cols ? (generator ? 8 : 4) : 2; }

template <int DT, bool SR, bool DROP, bool ROWS, bool COLS>
__global__ void __launch_bounds__(32 * tile_warps(SR || DROP, COLS), 24 / tile_warps(SR || DROP, COLS)) mx4_tile_kernel(const __grid_constant__ QuantParams p,
                                                                  unsigned tiles_c, bool out32) {
  grid_dependency_wait();
  grid_dependents_launch();
  constexpr int E = 16 / Fmt<DT>::bytes;              // elements in 16 bytes
  constexpr int W = kTileRowBytes / Fmt<DT>::bytes;   // columns of the CTA
  constexpr int C = 4 / Fmt<DT>::bytes;               // columns in 32 bits
  constexpr int kWarps = tile_warps(SR || DROP, COLS), kThreads = 32 * kWarps;
  constexpr int kTileRows = tile_rows(COLS), kTiles = kMx4TileRows / kTileRows;  // of a scale tile's rows
  constexpr int kWarpRows = kTileRows / kWarps;       // of the rows' part, a warp's rows
  constexpr int kWarpBlocks = 8 / kWarps;             // of the columns' part, a warp's blocks of a fourth of the columns
  extern __shared__ __align__(16) unsigned char x[];  // [kTileRows][kTileRowBytes]
  __shared__ __align__(16) uint8_t scales_r[W / 128][kTileRows][4];  // of the rows, 128 columns each
  __shared__ __align__(4) uint8_t scales_c[W][2];                     // of the columns, this CTA's two blocks
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const unsigned tc = blockIdx.x % tiles_c, tr = blockIdx.x / tiles_c;
  const long long row0 = (long long)tr * kTileRows, col0 = (long long)tc * W;
  const float dscale = DROP ? p.drop.scale : 1.f;

  {
    const int c = (threadIdx.x % 32) * E;
    const int valid = (int)max(0ll, min((long long)E, p.cols - col0 - c));
    unsigned char *dst = x + warp * kTileRowBytes + (threadIdx.x % 32) * 16;
    const long long at = (row0 + warp) * p.ld + col0 + c;
    const long long left = p.rows - row0 - warp;  // rows from this warp's first on
    if (p.vec && valid == E) {
#pragma unroll
      for (int k = 0; k < kTileRows; k += kWarps) {
        if (k < left)
          copy_async16(dst + k * kTileRowBytes, static_cast<const uint8_t *>(p.x) + (at + k * p.ld) * Fmt<DT>::bytes);
        else
          *reinterpret_cast<uint4 *>(dst + k * kTileRowBytes) = make_uint4(0, 0, 0, 0);
      }
    } else {
      constexpr int U = 4;
#pragma unroll 1
      for (int k = 0; k < kTileRows; k += kWarps * U) {
        uint4 v[U][2], out[U];
        bool around[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
          around[u] = load_around<DT, 1>(p, at + (k + kWarps * u) * p.ld, k + kWarps * u < left ? valid : 0, v[u]);
#pragma unroll
        for (int u = 0; u < U; ++u) {
          take_from<DT, 1>(p, at + (k + kWarps * u) * p.ld, k + kWarps * u < left ? valid : 0, around[u], v[u], &out[u]);
          *reinterpret_cast<uint4 *>(dst + (k + kWarps * u) * kTileRowBytes) = out[u];
        }
      }
    }
    copy_async_wait();
  }
  __syncthreads();

  if constexpr (ROWS || DROP) {
    constexpr int L = W / 16;  // lanes a row, sixteen neighbours each
    constexpr int N = 2 * kRaw8<DT>;
    const Mx4Out &o = p.by_rows;
    constexpr int S = 32 / L;   // rows a warp takes at once
    const int cl = lane % L * 16, rl0 = warp * kWarpRows + lane / L;
    const long long c0 = col0 + cl, r0 = row0 + rl0;
    const bool in_row = c0 < o.row_bytes * 2;
    const int left = (int)max(-16ll, min((long long)kTileRows, p.rows - r0));  // rows from this lane's first on
    uint4 *at = reinterpret_cast<uint4 *>(x + rl0 * kTileRowBytes + cl * Fmt<DT>::bytes);
    uint8_t *dst = o.data + r0 * o.row_bytes + c0 / 2;
    unsigned long long group = (unsigned long long)(r0 * o.row_bytes * 2 + c0) >> 3, element = (unsigned long long)(r0 * p.cols + c0);
    uint8_t *scale = &scales_r[cl >> 7][rl0][(cl >> 5) & 3];
#pragma unroll 1
    for (int k = 0; k < kWarpRows; k += S, at += S * kTileRowBytes / 16, dst += S * o.row_bytes, group += S * o.row_bytes / 4,
             element += S * p.cols, scale += S * 4) {
      if (k >= left + lane / L) {  // none of the warp's rows exist
        if (ROWS && (lane & 1) == 0) *scale = 0;
        continue;
      }
      uint4 raw[N];
#pragma unroll
      for (int j = 0; j < N; ++j) raw[j] = at[j];
      if constexpr (DROP) {
        mask16<DT>(p.drop, element, raw);
#pragma unroll
        for (int j = 0; j < N; ++j) at[j] = raw[j];
      }
      if constexpr (ROWS) {
        uint32_t m = max(max_mag8<DT>(raw), max_mag8<DT>(raw + kRaw8<DT>));
        m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
        m = mag_bits<DT>(m, 0);
        if constexpr (DROP) m = __float_as_uint(__fmul_rn(__uint_as_float(m), dscale));
        const uint32_t byte = scale_byte(m);
        const float inv = inverse_scale(byte);
        uint2 q;
        float v[8];
        widen8<DT>(raw, v);
        q.x = codes8<SR, DROP>(v, byte, inv, dscale, p.gen_rows, group);
        widen8<DT>(raw + kRaw8<DT>, v);
        q.y = codes8<SR, DROP>(v, byte, inv, dscale, p.gen_rows, group + 1);
        if (k < left && in_row) *reinterpret_cast<uint2 *>(dst) = q;
        if ((lane & 1) == 0) *scale = (uint8_t)byte;
      }
    }
    if constexpr (DROP && COLS) __syncthreads();
  }

  if constexpr (COLS) {
    const Mx4Out &o = p.by_cols;
    // the lane's first column, the warp's first block
    const int cl = warp / (kWarps / 4) * 32 * C + lane * C, b0 = warp % (kWarps / 4);
    uint4 codes[C][kWarpBlocks];
#pragma unroll
    for (int b = 0; b < kWarpBlocks; ++b) {
      const int rl = (b0 + b) * 32;
      if (row0 + rl >= p.rows) {  // no such block
#pragma unroll
        for (int c = 0; c < C; ++c) scales_c[cl + c][b0 + b] = 0;
        continue;
      }
      uint32_t w[32];
      uint32_t m4[4] = {0, 0, 0, 0};  // four chains
#pragma unroll
      for (int r = 0; r < 32; ++r) {
        w[r] = *reinterpret_cast<const uint32_t *>(x + (rl + r) * kTileRowBytes + cl * Fmt<DT>::bytes);
        m4[r % 4] = max_mag<DT>(m4[r % 4], w[r]);
      }
      const uint32_t m = max_mag<DT>(max_mag<DT>(m4[0], m4[1]), max_mag<DT>(m4[2], m4[3]));
#pragma unroll
      for (int c = 0; c < C; ++c) {
        uint32_t mc = mag_bits<DT>(m, c);
        if constexpr (DROP) mc = __float_as_uint(__fmul_rn(__uint_as_float(mc), dscale));
        const uint32_t byte = scale_byte(mc);
        const float inv = inverse_scale(byte);
        const unsigned long long group = (unsigned long long)((col0 + cl + c) * o.row_bytes * 2 + row0 + rl) >> 3;
        uint32_t q[4];
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          float v[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const uint32_t y = w[8 * g + e];
            if constexpr (DT == kF32) v[e] = __uint_as_float(y);
            else if constexpr (DT == kBF16) v[e] = __uint_as_float(c ? y & 0xffff0000u : y << 16);
            else v[e] = c ? __high2float(as_h2(y)) : __low2float(as_h2(y));
          }
          q[g] = codes8<SR, DROP>(v, byte, inv, dscale, p.gen_cols, group + g);
        }
        codes[c][b] = make_uint4(q[0], q[1], q[2], q[3]);
        scales_c[cl + c][b0 + b] = (uint8_t)byte;
      }
    }
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const long long col = col0 + cl + c;
      const long long row = row0 + b0 * 32;
      if (col >= p.cols || row >= p.rows) continue;
      uint8_t *q = o.data + col * o.row_bytes + row / 2;
      if (kWarpBlocks == 2 && out32 && row + 32 < p.rows) {
        stg32(q, codes[c][0], codes[c][kWarpBlocks - 1]);
      } else {
        *reinterpret_cast<uint4 *>(q) = codes[c][0];
        if (kWarpBlocks == 2 && row + 32 < p.rows) *reinterpret_cast<uint4 *>(q + 16) = codes[c][kWarpBlocks - 1];
      }
    }
  }
  __syncthreads();
  // the scales: of a column two neighbouring bytes, of a row four for every
  // 128 columns
  if constexpr (COLS) {
    const Mx4Out &q = p.by_cols;
    for (int c = threadIdx.x; c < W; c += kThreads) {
      const long long rb = (col0 + c) / kMx4TileRows;
      if (rb * kMx4TileRows < p.cols)
        *reinterpret_cast<uint16_t *>(q.scales + (rb * q.tiles_k + tr / 4) * kMx4TileBytes + (tr >> 1 & 1) * kMx4AtomBytes +
                                      (c & 31) * 16 + (c >> 5 & 3) * 4 + (tr & 1) * 2) =
            *reinterpret_cast<const uint16_t *>(scales_c[c]);
    }
  }
  if constexpr (ROWS) {
    const Mx4Out &q = p.by_rows;
    for (int k = threadIdx.x; k < W / 128 * kTileRows; k += kThreads) {
      const int a = k / kTileRows, r = k % kTileRows, rt = (int)(tr % kTiles) * kTileRows + r;  // rt: of the scale tile's rows
      const long long atom = (long long)tc * (W / 128) + a;
      if ((row0 - tr % kTiles * kTileRows) < p.rows && atom / 2 < q.tiles_k)
        *reinterpret_cast<uint32_t *>(q.scales + (tr / kTiles * q.tiles_k + atom / 2) * kMx4TileBytes + (atom & 1) * kMx4AtomBytes +
                                      (rt & 31) * 16 + (rt >> 5) * 4) = *reinterpret_cast<const uint32_t *>(scales_r[a][r]);
    }
  }
}

template <auto kKernel, class... Args>
cudaError_t launch(long long grid, int threads, int smem, cudaStream_t s, const Args &...args) {
  if (grid > 0x7fffffffll) return cudaErrorInvalidConfiguration;
  if (smem > 0) {
    const cudaError_t e = allow_smem<kKernel>(smem);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t c = {};
  c.gridDim = dim3((unsigned)grid);
  c.blockDim = dim3((unsigned)threads);
  c.dynamicSmemBytes = (size_t)smem;
  c.stream = s;
  cudaLaunchAttribute a = {};
  a.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  a.val.programmaticStreamSerializationAllowed = 1;
  c.attrs = &a;
  c.numAttrs = 1;
  return cudaLaunchKernelEx(&c, kKernel, args...);
}

template <int DT, bool SR, bool DROP>
cudaError_t quantize_dt(const QuantParams &p, cudaStream_t s) {
  constexpr int W = kTileRowBytes / Fmt<DT>::bytes;
  const bool rows = p.by_rows.data, cols = p.by_cols.data;
  // rows and columns to whole scale tiles of the results (256 rows for the
  // columns' result, 128 for the rows')
  const long long tiles_r = cols ? 4 * p.by_cols.tiles_k : kMx4TileRows / tile_rows(false) * ceil_div(p.rows, (long long)kMx4TileRows);
  const long long tiles_c = ceil_div(p.cols, (long long)kMx4TileCols) * (kMx4TileCols / W);
  const long long tiles = tiles_r * tiles_c;
  // Rows alone.  Off the 16-byte grid they go through the tiles too (binary32
  // 5003 x 1999: 26 us element by element a lane, 14.5 so), and up to 16 of them
  // (1 x 4096: 1.7 us, 2.5 with a warp for every pair of 128).  Else by the tiles
  // an SM, figures being through the tiles and straight from memory, for 4096
  // columns: their 24 warps an SM serve the generator better and few rows spread
  // further, straight loads have less to do where memory is the bound.
  //   16 bits, nearest: up to 48 (300 rows 2.3 and 2.9 us, 4096 8.8 and 9.3, 6000
  //   11.5 and 12.3; 8192 14.8 and 14.3).  Stochastic: all (4096 rows 15.0 and
  //   17.7, 8192 26.9 and 29.3).  With dropout: but seven or eight, which is a
  //   second turn of warps on some schedulers (800 rows 6.2 and 7.4, 1024 10.0 and
  //   7.3, 2048 13.2 and 13.8).
  //   binary32, nearest: up to eight (450 rows 3.1 and 3.6, 600 4.4 and 3.6).  With
  //   the generator: up to 96 (1400 rows 8.0 and 10.9, 6000 25.4 and 28.5, with
  //   dropout 34.4 and 37.6; 1200 7.3 and 7.1, 8192 33.3 and 29.4).
  const long long an_sm = ceil_div(tiles, (long long)p.sms);
  constexpr bool kTiled = SR && !DROP && DT != kF32;
  const bool tiled = kTiled || !p.vec || p.rows <= 16 ||
                     (DT == kF32 ? an_sm <= (SR || DROP ? 96 : 8)
                      : DROP     ? an_sm <= 6 || an_sm > 8
                                 : an_sm <= 48);
  if constexpr (!kTiled) if (!cols && !tiled) {
    const long long grid = ceil_div(p.rows, (long long)kMx4TileRows) * p.by_rows.tiles_k;
    // More warps a tile where tiles are few.  To nearest: sixteen below two
    // tiles an SM (binary32 1024 x 4096: 4.7 us, 5.9 with eight, 8.8 with four),
    // else eight (8192 x 4096: bfloat16 14.3 us, 16.1 with sixteen, 16.6 with four;
    // binary32 24.3, 24.7 and 25.8).  The kernels that call the generator hold 110
    // registers a thread and want about twelve warps an SM (binary32 stochastic
    // 8192 x 4096: 29.5 us with four warps a tile, 30.6 with eight, 38.5 with
    // sixteen; bfloat16 1024 x 4096 stochastic with dropout: 7.4 us with sixteen, 8.4
    // with eight, 13.8 with four).
    int threads = 128;
    if constexpr (SR || DROP) {
      while (threads < 512 && grid * threads < 12 * 32ll * p.sms) threads *= 2;
    } else {
      threads = grid >= 2ll * p.sms ? 256 : 512;
    }
    return launch<mx4_rows_kernel<DT, SR, DROP>>(grid, threads, 0, s, p);
  }
  constexpr int kThreads = 32 * tile_warps(SR || DROP, true), kSmem = tile_rows(true) * kTileRowBytes;
  const bool out32 = (reinterpret_cast<uintptr_t>(p.by_cols.data) | (uintptr_t)p.by_cols.row_bytes) % 32 == 0;
  const unsigned tc = (unsigned)tiles_c;
  if (!cols)
    return launch<mx4_tile_kernel<DT, SR, DROP, true, false>>(tiles, 32 * tile_warps(SR || DROP, false),
                                                              tile_rows(false) * kTileRowBytes, s, p, tc, out32);
  if (rows) return launch<mx4_tile_kernel<DT, SR, DROP, true, true>>(tiles, kThreads, kSmem, s, p, tc, out32);
  return launch<mx4_tile_kernel<DT, SR, DROP, false, true>>(tiles, kThreads, kSmem, s, p, tc, out32);
}

template <int DT>
cudaError_t quantize_any(const QuantParams &p, cudaStream_t s) {
  const bool drop = p.drop.cut != 0;
  if (p.stochastic) return drop ? quantize_dt<DT, true, true>(p, s) : quantize_dt<DT, true, false>(p, s);
  return drop ? quantize_dt<DT, false, true>(p, s) : quantize_dt<DT, false, false>(p, s);
}

}  // namespace mx4q

}  // namespace rr
