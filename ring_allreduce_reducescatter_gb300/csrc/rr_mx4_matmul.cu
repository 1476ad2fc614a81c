// rr_mx4_matmul.cu -- the product of two microscaled 4-bit matrices,
//   out[i, j] = (residual[i, j] +) drop(sum_k A[i, k] B[j, k]),
// on the block-scaled tensor cores.
#include "rr_mx4.cuh"
#include "rr_tcgen05.cuh"
#include "rr_turns.h"

namespace rr {

namespace {

// K goes in steps of 256 elements: 128 bytes a row, one scale tile.
constexpr int kBK = 256;
constexpr int kRowBytes = kBK / 2;
constexpr int kHalfBytes = 128 * kRowBytes;  // 128 rows of an operand, one step

struct MatmulKernelParams {
  // the operands by their sides of the tensor cores' product: P gives the rows
  // of the accumulators, Q the columns
  CUtensorMap map_p, map_q;
  CUtensorMap map_sp, map_sq;  // their scale tiles (pair kernel)
  CUtensorMap map_qh, map_sqh;  // Q and its scales in half the rows a box (pair kernel, halved tiles)
  const uint8_t *scales_p, *scales_q;
  long long m, n;
  int steps;  // of K
  int tiles_p, tiles_q;
  long long items, whole;  // pair kernel: pieces of work, of which the first are whole tiles, the rest halves
  void *out;
  const void *residual;
  long long ld_out, ld_res;
  DropParams drop;
  unsigned int *status;
  bool vec, vec32;  // 16- and 32-byte groups of the rows of out and residual are aligned
};

// The limit of a wait for what has come already, unless another wait gave up.
constexpr unsigned long long kLateLimitNs = 10000000ull;  // 10 ms

// Waits, each time up to the limit, for the turns before `end` that may still be
// in flight on these barriers of a ring of S stages.
template <int S>
__device__ __forceinline__ void wait_turns(uint64_t *bars, unsigned end, unsigned long long limit_ns) {
  each_open_turn(end, S, [&](unsigned stage, unsigned parity) { mbar_wait_bounded(&bars[stage], parity, limit_ns); });
}

// Masks kN accumulators of one row, from column `col` on.
template <int kN>
__device__ __forceinline__ void drop_row(const MatmulKernelParams &p, long long row, long long col, float v[kN]) {
  const unsigned long long i = p.drop.first + (unsigned long long)(row * p.n + col), g = i >> 3;
  const int sh = (int)(i & 7) * 2;
  if (sh == 0) {  // apart, so that the calls, which do not depend on one another, run together
    uint4 u[kN / 8];
#pragma unroll
    for (int h = 0; h < kN / 8; ++h) u[h] = philox(p.drop.gen, g + h);
#pragma unroll
    for (int h = 0; h < kN / 8; ++h) drop8(p.drop, u[h], v + 8 * h);
    return;
  }
  uint4 u = philox(p.drop.gen, g);
#pragma unroll
  for (int h = 0; h < kN / 8; ++h) {
    const uint4 next = philox(p.drop.gen, g + h + 1);
    drop8(p.drop, funnel16(u, next, sh), v + 8 * h);
    u = next;
  }
}

// A warp's 32 rows of kN accumulators each, a row a lane, to the output.
// rows0, col: the block's first row and column; res: the lane's part of the
// residual, loaded ahead by load_residual (aligned blocks only).
// stage: kStageFloats of shared memory of this warp's own.
constexpr int kStageFloats = 32 * 17;

// Whether a block of kN columns takes the vector path.
template <int kN>
__device__ __forceinline__ bool aligned_block(const MatmulKernelParams &p, long long col) {
  return p.vec && col + kN <= p.n;
}
template <int DT, int kN>
__device__ __forceinline__ void load_residual(const MatmulKernelParams &p, long long row, long long col, uint4 *res) {
  using T = typename Fmt<DT>::type;
  const uint4 *q = reinterpret_cast<const uint4 *>(static_cast<const T *>(p.residual) + row * p.ld_res + col);
#pragma unroll
  for (int j = 0; j < kN / 8 * kRaw8<DT>; j += 2) {
    if (row >= p.m) {
      res[j] = res[j + 1] = make_uint4(0, 0, 0, 0);
    } else if (p.vec32) {
      ldg32(q + j, res[j], res[j + 1]);
    } else {
      res[j] = ld16(q + j), res[j + 1] = ld16(q + j + 1);
    }
  }
}

template <int DT, int kN>
__device__ __forceinline__ void finish_aligned(const MatmulKernelParams &p, long long row, long long col,
                                               const uint32_t *acc, const uint4 *res) {
  using T = typename Fmt<DT>::type;
  if (row >= p.m) return;
  float v[kN];
#pragma unroll
  for (int j = 0; j < kN; ++j) v[j] = __uint_as_float(acc[j]);
  if (p.drop.cut) drop_row<kN>(p, row, col, v);
  if (p.residual) {
#pragma unroll
    for (int h = 0; h < kN / 8; ++h) {
      float w[8];
      widen8<DT>(res + h * kRaw8<DT>, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[8 * h + j] = __fadd_rn(w[j], v[8 * h + j]);
    }
  }
  uint4 raw[kN / 8 * kRaw8<DT>];
#pragma unroll
  for (int h = 0; h < kN / 8; ++h) narrow8<DT>(v + 8 * h, raw + h * kRaw8<DT>);
  uint4 *o = reinterpret_cast<uint4 *>(static_cast<T *>(p.out) + row * p.ld_out + col);
#pragma unroll
  for (int j = 0; j < kN / 8 * kRaw8<DT>; j += 2) {
    if (p.vec32) {
      stg32(o + j, raw[j], raw[j + 1]);
    } else {
      stg_stream(o + j, raw[j]);
      stg_stream(o + j + 1, raw[j + 1]);
    }
  }
}

// Sixteen columns of a block whose rows are not aligned, or end inside it: the
// block is turned in shared memory so that sixteen lanes take neighbours of a row
// (a lane storing its own row by single elements made such products twice as long).
template <int DT>
__device__ __forceinline__ void finish_ragged(const MatmulKernelParams &p, long long rows0, long long col,
                                              const uint32_t *acc, float *stage) {
  using T = typename Fmt<DT>::type;
  const int lane = threadIdx.x % 32;
  if (col >= p.n || rows0 >= p.m) return;  // the same for the whole warp
  float v[16];
#pragma unroll
  for (int j = 0; j < 16; ++j) v[j] = __uint_as_float(acc[j]);
  if (p.drop.cut) drop_row<16>(p, rows0 + lane, col, v);
#pragma unroll
  for (int j = 0; j < 16; ++j) stage[lane * 17 + j] = v[j];
  __syncwarp();
  const long long c = col + lane % 16, r0 = rows0 + lane / 16;
  const int left = c < p.n ? (int)min(32ll, p.m - r0) : 0;  // rows from r0 on
  const float *from = stage + lane / 16 * 17 + lane % 16;
  T *o = static_cast<T *>(p.out) + r0 * p.ld_out + c;
  const long long step = 2 * p.ld_out;
  if (p.residual) {
    const T *q = static_cast<const T *>(p.residual) + r0 * p.ld_res + c;
    T w[16];
#pragma unroll
    for (int k = 0; k < 16; ++k, q += 2 * p.ld_res) w[k] = 2 * k < left ? *q : from_f32<DT>(0.f);
#pragma unroll
    for (int k = 0; k < 16; ++k, o += step)
      if (2 * k < left) *o = from_f32<DT>(__fadd_rn(to_f32<DT>(w[k]), from[2 * k * 17]));
  } else {
#pragma unroll
    for (int k = 0; k < 16; ++k, o += step)
      if (2 * k < left) *o = from_f32<DT>(from[2 * k * 17]);
  }
  __syncwarp();
}

template <int DT>
__device__ __forceinline__ void finish16(const MatmulKernelParams &p, long long row, long long col, const uint32_t *acc,
                                         float *stage) {
  if (aligned_block<16>(p, col)) {
    uint4 res[2 * kRaw8<DT>];
    if (p.residual) load_residual<DT, 16>(p, row, col, res);
    finish_aligned<DT, 16>(p, row, col, acc, res);
  } else {
    finish_ragged<DT>(p, row - threadIdx.x % 32, col, acc, stage);
  }
}

// One accumulator to the output (the element's own random number: a whole
// counter for one element, for the few columns of a small batch).
template <int DT>
__device__ __forceinline__ void finish1(const MatmulKernelParams &p, long long row, long long col, float v) {
  using T = typename Fmt<DT>::type;
  if (row >= p.m || col >= p.n) return;
  if (p.drop.cut) {
    const unsigned long long i = p.drop.first + (unsigned long long)(row * p.n + col);
    const uint4 u = philox(p.drop.gen, i >> 3);
    v = kept(u, (int)(i & 7), p.drop.cut) ? __fmul_rn(v, p.drop.scale) : 0.f;
  }
  if (p.residual) v = __fadd_rn(to_f32<DT>(static_cast<const T *>(p.residual)[row * p.ld_res + col]), v);
  static_cast<T *>(p.out)[row * p.ld_out + col] = from_f32<DT>(v);
}

// --------------------------------------------------------------------------
// small products: K split over a cluster
// --------------------------------------------------------------------------

// A cluster of S CTAs computes one tile of 128 rows of P by BN rows of Q, each
// CTA a contiguous part of K.  Each CTA sends its sums, a group of columns to
// each CTA in turn, to a place of its own in that CTA's shared memory; one
// barrier later every CTA adds up the groups it received, in rank order (so
// the result does not depend on timing), and finishes them.  Reading the
// operands bounds these products, and a grid of whole tiles would leave most
// SMs without a share of the memory; split_of below says how S is chosen.  (Reading the other CTAs' sums instead of sending them
// took a second barrier and the latency of a remote load: 33 rows by 4096 by
// 11008 took 9.3 us.)
// kSwap: P is B (a weight matrix, 128 rows a tile) and Q is A (the few tokens
// of a small batch, BN of them): no operand row is padded beyond BN tokens.

template <int BN>
struct Split {
  static constexpr int kStageBytes = kHalfBytes + BN * kRowBytes + 2 * kMx4TileBytes;
  static constexpr int kStages = BN <= 32 ? 4 : 3;  // two CTAs an SM, with the groups of a split
  static constexpr int kGroup = BN <= 64 ? 4 : 16;                 // columns a group
  static constexpr int kGroups = BN / kGroup;
  // epilogue warps first (four quarters of the rows, once or, each with every
  // second 16 columns, twice), then one for the copies and one for the products
  static constexpr int kHalves = BN <= 32 ? 1 : 2;
  static constexpr int kEpilogue = 4 * kHalves;
  static constexpr int kThreads = 32 * (kEpilogue + 2);
  static constexpr int kGroupBytes = kGroup * 128 * 4;
  // the stages, then the groups received: [split][slots][kGroup / 4][128][4]
  static __host__ __device__ constexpr int slots(int split) { return (kGroups + split - 1) / split; }
  static __host__ __device__ constexpr int smem_bytes(int split) {
    return 1024 + kStages * kStageBytes + (split > 1 ? split * slots(split) * kGroupBytes : 0);
  }
  static constexpr uint32_t kScales = BN;                          // first column of the scales
  static constexpr uint32_t kColumns = BN <= 64 ? 128 : 256;       // accumulators and the scales of every stage
  static_assert(kScales + kStages * 16 <= kColumns, "they fit");
  static_assert(kStages * kStageBytes >= kEpilogue * kStageFloats * 4, "the ragged epilogue fits the stages");
};

// The groups of columns that this CTA received, added up and finished.
template <int DT, int BN, bool kSwap>
__device__ __forceinline__ void finish_split(const MatmulKernelParams &p, const float *got, int split, int rank, int row,
                                             int half, long long prow, long long q0, float *stage) {
  using L = Split<BN>;
  const int slots = L::slots(split);
  for (int slot = half, g = rank + half * split; g < L::kGroups; slot += L::kHalves, g += split * L::kHalves) {
    const long long col = q0 + g * L::kGroup;
    if (kSwap && col >= p.m) break;
    float v[L::kGroup];
#pragma unroll
    for (int j = 0; j < L::kGroup; ++j) v[j] = 0.f;
#pragma unroll 2
    for (int r = 0; r < split; ++r) {
      const float4 *w = reinterpret_cast<const float4 *>(got + (r * slots + slot) * (L::kGroup * 128)) + row;
#pragma unroll
      for (int j = 0; j < L::kGroup; j += 4) {
        const float4 x = w[j / 4 * 128];
        v[j] = r == 0 ? x.x : __fadd_rn(v[j], x.x);
        v[j + 1] = r == 0 ? x.y : __fadd_rn(v[j + 1], x.y);
        v[j + 2] = r == 0 ? x.z : __fadd_rn(v[j + 2], x.z);
        v[j + 3] = r == 0 ? x.w : __fadd_rn(v[j + 3], x.w);
      }
    }
    if constexpr (kSwap) {
#pragma unroll
      for (int j = 0; j < L::kGroup; ++j) finish1<DT>(p, col + j, prow, v[j]);
    } else {
      uint32_t acc[16];
#pragma unroll
      for (int j = 0; j < 16; ++j) acc[j] = __float_as_uint(v[j % L::kGroup]);
      finish16<DT>(p, prow, col, acc, stage);
    }
  }
}

template <int DT, int BN, bool kSwap>
__global__ void __launch_bounds__(Split<BN>::kThreads, 2) mx4_split_kernel(const __grid_constant__ MatmulKernelParams p,
                                                                    int split) {
  using L = Split<BN>;
  extern __shared__ unsigned char smem_raw[];
  __shared__ __align__(8) uint64_t full[L::kStages], empty[L::kStages], done;
  __shared__ uint32_t tmem_slot;
  __shared__ int failed;
  unsigned char *smem = smem_raw + ((1024 - (smem_addr(smem_raw) & 1023)) & 1023);
  const int warp = uniform(threadIdx.x / 32), lane = threadIdx.x % 32;

  if (threadIdx.x == 0) {
    for (int s = 0; s < L::kStages; ++s) mbar_init(&full[s], 1), mbar_init(&empty[s], 1);
    mbar_init(&done, 1);
    failed = 0;
    fence_mbar_init();
  }
  if (split > 1) cluster_arrive();  // waited for before the first remote store: by then every CTA runs
  if (warp == L::kEpilogue + 1) tmem_alloc<1>(&tmem_slot, L::kColumns);
  tcgen05_fence_before();
  __syncthreads();
  tcgen05_fence_after();
  const uint32_t tmem = (uint32_t)uniform((int)tmem_slot);
  const int rank = blockIdx.x % split, tile = blockIdx.x / split;
  const int tp = tile % p.tiles_p, tq = tile / p.tiles_p;
  const int k0 = (int)((long long)p.steps * rank / split), n_steps = (int)((long long)p.steps * (rank + 1) / split) - k0;
  grid_dependency_wait();
  grid_dependents_launch();

  if (warp == L::kEpilogue) {
    const uint64_t pol = l2_evict_normal_policy();
    const bool one = elect_one();
    int k = 0;
    for (; k < n_steps; ++k) {
      const int s = k % L::kStages;
      if (!__all_sync(0xffffffffu, mbar_wait_bounded(&empty[s], ((k / L::kStages) & 1) ^ 1, kWaitLimitNs))) break;
      unsigned char *st = smem + s * L::kStageBytes, *sc = st + kHalfBytes + BN * kRowBytes;
      if (one) {
        mbar_arrive_expect_tx(&full[s], L::kStageBytes);
        tensor_load(st, &p.map_p, (k0 + k) * kRowBytes, tp * 128, &full[s], pol);
        tensor_load(st + kHalfBytes, &p.map_q, (k0 + k) * kRowBytes, tq * BN, &full[s], pol);
        bulk_load(sc, p.scales_p + ((long long)tp * p.steps + k0 + k) * kMx4TileBytes, kMx4TileBytes, &full[s], pol);
        bulk_load(sc + kMx4TileBytes, p.scales_q + ((long long)tq * p.steps + k0 + k) * kMx4TileBytes, kMx4TileBytes,
                  &full[s], pol);
      }
      __syncwarp();
    }
    if (k < n_steps && one) {
      atomicOr(p.status, kStatusWaitTimeout);
      atomicExch(&failed, 1);
    }
    // the copies in flight land before shared memory is given back, also where
    // it is the products that give up
    wait_turns<L::kStages>(full, k, kWaitLimitNs);
  } else if (warp == L::kEpilogue + 1) {
    const bool one = elect_one();
    int k = 0;
    for (; k < n_steps; ++k) {
      const int s = k % L::kStages;
      if (!__all_sync(0xffffffffu, mbar_wait_bounded(&full[s], (k / L::kStages) & 1, kWaitLimitNs))) break;
      tcgen05_fence_after();
      const uint32_t a = smem_addr(smem) + s * L::kStageBytes, b = a + kHalfBytes, sc = b + BN * kRowBytes;
      // the scales of a step: P's eight columns, then Q's; a place for each stage
      const uint32_t sa = tmem + L::kScales + s * 16, sb = sa + 8;
      if (one) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          scale_copy<1>(sa + 4 * j, scale_desc(sc + j * kMx4AtomBytes));
          scale_copy<1>(sb + 4 * j, scale_desc(sc + kMx4TileBytes + j * kMx4AtomBytes));
        }
#pragma unroll
        for (int j = 0; j < kBK / 64; ++j)
          mx4_mma<1>(tmem, operand_desc(a + 32 * j), operand_desc(b + 32 * j), mx4_instr_desc(128, BN, (j & 1) * 2),
                     sa + 4 * (j / 2), sb + 4 * (j / 2), k > 0 || j > 0);
        tcgen05_commit<1>(&empty[s]);
      }
      __syncwarp();
    }
    if (one) {
      if (k < n_steps) {
        atomicOr(p.status, kStatusWaitTimeout);
        atomicExch(&failed, 1);
      }
      tcgen05_commit<1>(&done);
    }
  }
  __syncwarp();
  // every warp waits here for the last product, so none leaves tensor memory
  // or shared memory while they are in use
  if (!mbar_wait_bounded(&done, 0, 2 * kWaitLimitNs) && lane == 0) {
    atomicOr(p.status, kStatusWaitTimeout);
    atomicExch(&failed, 1);
  }
  __syncwarp();
  tcgen05_fence_after();
  __syncthreads();

  const int row = warp % 4 * 32 + lane, half = warp / 4;  // of the tile (epilogue warps)
  const long long prow = (long long)tp * 128 + row, q0 = (long long)tq * BN;
  float *stage = reinterpret_cast<float *>(smem) + warp % L::kEpilogue * kStageFloats;
  float *got = reinterpret_cast<float *>(smem + L::kStages * L::kStageBytes);
  if (split > 1) cluster_wait();
  if (warp < L::kEpilogue) {
    const int slots = L::slots(split);
#pragma unroll 1
    for (int c = 16 * half; c < BN; c += 16 * L::kHalves) {
      if (kSwap && q0 + c >= p.m) break;
      uint32_t acc[16];
      tmem_load16(tmem + ((uint32_t)(warp % 4 * 32) << 16) + c, acc);
      tmem_load_wait();
      if (n_steps == 0) {
#pragma unroll
        for (int j = 0; j < 16; ++j) acc[j] = 0;
      }
      if (split > 1) {
#pragma unroll
        for (int j = 0; j < 16; j += 4) {
          const int g = (c + j) / L::kGroup;
          if (kSwap && q0 + c + j >= p.m) break;
          const float *to = got + (rank * slots + g / split) * (L::kGroup * 128) + (((c + j) % L::kGroup) / 4 * 128 + row) * 4;
          cluster_store4(cluster_addr(to, g % split), make_uint4(acc[j], acc[j + 1], acc[j + 2], acc[j + 3]));
        }
      } else if (!failed) {
        if constexpr (kSwap) {
#pragma unroll
          for (int j = 0; j < 16; ++j) finish1<DT>(p, q0 + c + j, prow, __uint_as_float(acc[j]));
        } else {
          finish16<DT>(p, prow, q0 + c, acc, stage);
        }
      }
    }
  } else if (warp == L::kEpilogue) {
    // the commits of the last turns come before the CTA goes: later ones would
    // meet another's barrier
    wait_turns<L::kStages>(empty, n_steps, kLateLimitNs);
  }
  tcgen05_fence_before();
  __syncthreads();
  tcgen05_fence_after();
  if (split > 1) cluster_arrive();
  if (warp == L::kEpilogue + 1) tmem_free<1>(tmem, L::kColumns);
  if (split > 1) {
    cluster_wait();
    if (warp < L::kEpilogue && !failed) finish_split<DT, BN, kSwap>(p, got, split, rank, row, half, prow, q0, stage);
  }
}

// --------------------------------------------------------------------------
// large products: a pair of CTAs a tile
// --------------------------------------------------------------------------

// A pair of CTAs on two SMs computes 256 x 256 tiles: each CTA holds 128 rows
// of A and 128 of B, and the tensor cores of both read both halves of B.  One
// CTA's 128 x 256 tile would need A and B tiles of 12 KB for every 128 cycles
// of products, read and written in shared memory, 192 bytes a cycle of the 128
// it has; the pair needs 128.  The grid is one CTA per SM and loops over
// tiles; eight warps take a finished tile from tensor memory into registers at
// once (128 accumulators a thread) and store it while the next tile's products
// run.  Where the tiles left for the last turn are no more than half the pairs,
// they are halved along the columns (4096^3, 3 turns and 28 tiles for 76 pairs).
constexpr int kPM = 256, kPN = 256;
constexpr int kPairStages = 5;
constexpr int kPairStageBytes = 2 * kHalfBytes + 3 * kMx4TileBytes;  // + scales of 128 rows of A, 256 of B
constexpr int kPairSmemBytes = kPairStages * kPairStageBytes + 8 * kStageFloats * 4 + 1024;
constexpr int kPairThreads = 384;  // warps 0-7 epilogue, 8 copies, 9 products, 10 and 11 idle
// registers a thread: 168 at launch (384 threads), 216 for the two warpgroups
// of the epilogue and 72 for the third: 2 * 216 + 72 = 3 * 168
constexpr uint32_t kPairScales = kPN;  // first tensor-memory column of the scales

// Piece t of the work: a tile, or half of one (side 0 or 1 of its columns).
struct PairItem {
  int tp, tq, side;
  bool whole;
};
__device__ __forceinline__ PairItem pair_item(const MatmulKernelParams &p, long long t) {
  PairItem i;
  i.whole = t < p.whole;
  const long long u = i.whole ? t : p.whole + (t - p.whole) / 2;
  i.side = i.whole ? 0 : (int)((t - p.whole) & 1);
  i.tp = (int)(u % p.tiles_p), i.tq = (int)(u / p.tiles_p);
  return i;
}

template <int DT>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPairThreads, 1)
    mx4_pair_kernel(const __grid_constant__ MatmulKernelParams p) {
  extern __shared__ unsigned char smem_raw[];
  __shared__ __align__(8) uint64_t full[kPairStages], empty[kPairStages], acc_full, acc_empty;
  __shared__ uint32_t tmem_slot;
  unsigned char *smem = smem_raw + ((1024 - (smem_addr(smem_raw) & 1023)) & 1023);
  const int warp = uniform(threadIdx.x / 32), lane = threadIdx.x % 32;
  const uint32_t rank = cluster_rank();

  if (threadIdx.x == 0) {
    for (int s = 0; s < kPairStages; ++s) mbar_init(&full[s], 1), mbar_init(&empty[s], 1);
    mbar_init(&acc_full, 1);
    mbar_init(&acc_empty, 16);
    fence_mbar_init();
  }
  if (warp == 9) tmem_alloc<2>(&tmem_slot, 512);
  tcgen05_fence_before();
  __syncthreads();
  cluster_sync_all();
  tcgen05_fence_after();
  const uint32_t tmem = (uint32_t)uniform((int)tmem_slot);
  const int pairs = gridDim.x / 2, pair = blockIdx.x / 2;
  grid_dependency_wait();
  grid_dependents_launch();

  if (warp < 8) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
    // The residual comes 64 bytes a row ahead of the columns being finished, the
    // first before the tile is complete, in whole sectors (16-byte loads of a
    // lane's own row made 4096^3 with residual and dropout 42 us, now 36; more
    // of it ahead takes registers and was no faster).
    constexpr int kChunk = DT == kF32 ? 16 : 32, kAhead = 1;
    const int quarter = warp % 4, half = warp / 4;
    float *stage = reinterpret_cast<float *>(smem + kPairStages * kPairStageBytes) + warp * kStageFloats;
    unsigned i = 0;
    for (long long t = pair; t < p.items; t += pairs, ++i) {
      const PairItem w = pair_item(p, t);
      const bool mine = w.whole || half == 0;  // a half tile is one half's warps' work
      const long long rows0 = (long long)w.tp * kPM + rank * 128 + quarter * 32, row = rows0 + lane;
      const long long col0 = (long long)w.tq * kPN + (w.whole ? half : w.side) * 128;
      const bool aligned = aligned_block<128>(p, col0);
      uint4 res[kAhead][kChunk / 8 * kRaw8<DT>];
      if (p.residual && aligned && mine) {
#pragma unroll
        for (int c = 0; c < kAhead; ++c) load_residual<DT, kChunk>(p, row, col0 + c * kChunk, res[c]);
      }
      if (!__all_sync(0xffffffffu, mbar_wait_bounded(&acc_full, i & 1, kWaitLimitNs))) {
        if (lane == 0) atomicOr(p.status, kStatusWaitTimeout);
        break;
      }
      tcgen05_fence_after();
      uint32_t acc[128];
#pragma unroll
      for (int c = 0; c < 4; ++c)
        tmem_load32(tmem + ((uint32_t)(quarter * 32) << 16) + half * 128 + 32 * c, acc + 32 * c);
      tmem_load_wait();
      tcgen05_fence_before();
      __syncwarp();
      if (lane == 0) cluster_arrive_remote(cluster_addr(&acc_empty, 0));
      if (!mine) continue;
      if (aligned) {
#pragma unroll
        for (int c = 0; c < 128 / kChunk; ++c) {
          finish_aligned<DT, kChunk>(p, row, col0 + c * kChunk, acc + c * kChunk, res[c % kAhead]);
          if (p.residual && c + kAhead < 128 / kChunk)
            load_residual<DT, kChunk>(p, row, col0 + (c + kAhead) * kChunk, res[c % kAhead]);
        }
      } else {
#pragma unroll
        for (int c = 0; c < 8; ++c) finish_ragged<DT>(p, rows0, col0 + 16 * c, acc + 16 * c, stage);
      }
    }
    // The commits of the last turns have come, to both CTAs, before they go: one
    // that came later would meet another's barrier.  (Here, after the stores, they
    // are there already; by the copy warp, which polled for them while the last
    // products ran, 4096^3 took 27.9 us for 27.6.)
    if (warp == 0) wait_turns<kPairStages>(empty, i * (unsigned)p.steps, kLateLimitNs);
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    if (warp == 8) {
      const uint64_t pol = l2_evict_normal_policy();
      const bool one = elect_one();
      unsigned g = 0;
      bool ok = true;
      for (long long t = pair; t < p.items && ok; t += pairs) {
        const PairItem w = pair_item(p, t);
        const uint32_t bytes = 2 * (w.whole ? kPairStageBytes : kHalfBytes * 3 / 2 + 2 * kMx4TileBytes);
        const int row_a = w.tp * kPM + (int)rank * 128, row_b = w.tq * kPN + (w.whole ? (int)rank * 128 : w.side * 128 + (int)rank * 64);
        for (int k = 0; k < p.steps; ++k, ++g) {
          const unsigned s = g % kPairStages;
          if (!(ok = __all_sync(0xffffffffu, mbar_wait_bounded(&empty[s], ((g / kPairStages) & 1) ^ 1, kWaitLimitNs)))) break;
          unsigned char *st = smem + s * kPairStageBytes;
          const uint32_t bar = cluster_addr(&full[s], 0);
          if (one) {
            // (rows past the last, of the operands and of the scale tiles, read as zeros)
            if (rank == 0) mbar_arrive_expect_tx(&full[s], bytes);
            tensor_load_pair(st, &p.map_p, k * kRowBytes, row_a, bar, pol);
            tensor_load_pair(st + kHalfBytes, w.whole ? &p.map_q : &p.map_qh, k * kRowBytes, row_b, bar, pol);
            tensor_load_pair(st + 2 * kHalfBytes, &p.map_sp, 0, k, w.tp * 2 + (int)rank, bar, pol);
            tensor_load_pair(st + 2 * kHalfBytes + kMx4TileBytes, w.whole ? &p.map_sq : &p.map_sqh, 0, k, w.tq * 2 + w.side, bar, pol);
          }
          __syncwarp();
        }
      }
      if (!ok && one) atomicOr(p.status, kStatusWaitTimeout);
      // The copies in flight land before shared memory is given back: both CTAs'
      // count on rank 0, for whose last barrier below rank 1 waits.
      if (rank == 0) wait_turns<kPairStages>(full, g, kWaitLimitNs);
    } else if (warp == 9 && rank == 0) {
      const bool one = elect_one();
      unsigned g = 0, i = 0;
      bool ok = true;
      for (long long t = pair; t < p.items && ok; t += pairs, ++i) {
        const bool whole = t < p.whole;
        const uint32_t idesc = whole ? mx4_instr_desc(kPM, kPN, 0) : mx4_instr_desc(kPM, kPN / 2, 0);
        if (i > 0 && !(ok = __all_sync(0xffffffffu, mbar_wait_bounded(&acc_empty, (i - 1) & 1, kWaitLimitNs)))) break;
        tcgen05_fence_after();
        for (int k = 0; k < p.steps; ++k, ++g) {
          const unsigned s = g % kPairStages;
          if (!(ok = __all_sync(0xffffffffu, mbar_wait_bounded(&full[s], (g / kPairStages) & 1, kWaitLimitNs)))) break;
          tcgen05_fence_after();
          const uint32_t a = smem_addr(smem) + s * kPairStageBytes, b = a + kHalfBytes, sc = b + kHalfBytes;
          // the scales of a step: A's eight columns, then B's sixteen; a place for each stage
          const uint32_t sa = tmem + kPairScales + s * 24, sb = sa + 8;
          if (one) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              scale_copy<2>(sa + 4 * j, scale_desc(sc + j * kMx4AtomBytes));
              scale_copy<2>(sb + 8 * j, scale_desc(sc + kMx4TileBytes + j * kMx4AtomBytes));
              if (whole) scale_copy<2>(sb + 8 * j + 4, scale_desc(sc + 2 * kMx4TileBytes + j * kMx4AtomBytes));
            }
#pragma unroll
            for (int j = 0; j < kBK / 64; ++j)
              mx4_mma<2>(tmem, operand_desc(a + 32 * j), operand_desc(b + 32 * j), idesc | mx4_scale_at((j & 1) * 2),
                         sa + 4 * (j / 2), sb + 8 * (j / 2), k > 0 || j > 0);
            tcgen05_commit<2>(&empty[s]);
          }
          __syncwarp();
        }
        if (ok && one) tcgen05_commit<2>(&acc_full);  // a tile that was given up is not stored
      }
      if (!ok) {
        if (one) atomicOr(p.status, kStatusWaitTimeout);
        // the products issued so far end before tensor memory is given back (a
        // turn's commit covers all before it)
        if (g > 0) mbar_wait_bounded(&empty[(g - 1) % kPairStages], turn_parity(g - 1, kPairStages), kWaitLimitNs);
      }
    }
  }
  __syncwarp();
  tcgen05_fence_before();
  cluster_sync_all();
  tcgen05_fence_after();
  if (warp == 9) tmem_free<2>(tmem, 512);
}

using EncodeTiled = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                 const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encode_tiled() {
  static const EncodeTiled fn = [] {
    void *f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      f = nullptr;
    return reinterpret_cast<EncodeTiled>(f);
  }();
  return fn;
}

// The map of an operand's bytes: boxes of `box_rows` rows by 128 bytes, with
// the 128-byte swizzle; outside the matrix a load reads zeros.
bool make_map(CUtensorMap *map, const Mx4Operand &o, int box_rows) {
  const EncodeTiled fn = encode_tiled();
  if (!fn) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)o.row_bytes, (cuuint64_t)o.rows};
  const cuuint64_t strides[1] = {(cuuint64_t)o.row_bytes};
  const cuuint32_t box[2] = {(cuuint32_t)kRowBytes, (cuuint32_t)box_rows};
  const cuuint32_t unit[2] = {1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t *>(o.data), dims, strides, box, unit,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The map of an operand's scale tiles: [rows / 128][steps][1024 bytes], boxes of
// one step of `box_tiles` row tiles.
bool make_scale_map(CUtensorMap *map, const uint8_t *scales, long long row_tiles, int steps, int box_tiles) {
  const EncodeTiled fn = encode_tiled();
  if (!fn) return false;
  constexpr int kWords = kMx4TileBytes / 4;
  const cuuint64_t dims[3] = {kWords, (cuuint64_t)steps, (cuuint64_t)row_tiles};
  const cuuint64_t strides[2] = {kMx4TileBytes, (cuuint64_t)steps * kMx4TileBytes};
  const cuuint32_t box[3] = {kWords, 1, (cuuint32_t)box_tiles};
  const cuuint32_t unit[3] = {1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT32, 3, const_cast<uint8_t *>(scales), dims, strides, box, unit,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

constexpr int kMaxSmem = 227 * 1024 - 1024;  // a CTA's dynamic shared memory at most, less its static part

// cluster: CTAs a cluster (given as a launch attribute where the kernel has no
// size of its own).
template <auto kKernel, class... Args>
cudaError_t launch_matmul(long long grid, int threads, int smem, int cluster, cudaStream_t s, const Args &...args) {
  if (grid > 0x7fffffffll) return cudaErrorInvalidConfiguration;
  const cudaError_t e = allow_smem<kKernel>(kMaxSmem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t c = {};
  c.gridDim = dim3((unsigned)grid);
  c.blockDim = dim3((unsigned)threads);
  c.dynamicSmemBytes = smem;
  c.stream = s;
  cudaLaunchAttribute a[2] = {};
  a[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  a[0].val.programmaticStreamSerializationAllowed = 1;
  a[1].id = cudaLaunchAttributeClusterDimension;
  a[1].val.clusterDim.x = (unsigned)cluster, a[1].val.clusterDim.y = 1, a[1].val.clusterDim.z = 1;
  c.attrs = a;
  c.numAttrs = cluster > 0 ? 2 : 1;
  return cudaLaunchKernelEx(&c, kKernel, args...);
}

// CTAs a tile.  Up to 64 columns: as many as fit the GPU at two an SM, each with
// a step or more (33 x 4096 x 11008: 20.2 us whole, 13.0, 9.4 and 8.8 us at 2, 4
// and 8; 1 x 11008 x 4096, 86 tiles: 8.1 us whole, 8.7, 8.4 and, past two an SM,
// 10.5 us at 2, 3 and 4; where both 4 and 8 fit and K is short, 4 is the faster:
// 1 x 4096 x 4096 6.2 us whole, 4.8, 4.3 and 4.9, 64 x 4096 x 4096 9.8 us, 7.9, 6.1
// and 6.8).  At 128 columns a tile has 64 KB of sums to exchange and there is one
// CTA an SM, so at most that many, and four steps or more each (128 x 1024 x 4096:
// 6.8 us whole, 6.6, 5.9 and 6.7 at 2, 4 and 8; 1024^3, 64 tiles of four steps:
// 4.4 us whole, 5.8 in two).  The rule is not the faster side everywhere: eight
// steps are faster whole (128 x 4096 x 2048: 5.2 us, 6.0 in two; 1024 x 1024 x 2048:
// 5.2 and 6.4), and clusters of seven or eight with one CTA an SM do not all run
// at once (512 x 512 x 8192: 10.2 us whole, 6.9 at 4, 7.4 at 6, 13.0 at 7 and 13.6
// at 8, which the rule takes).
template <int BN>
int split_of(long long tiles, int steps, int sms) {
  constexpr int kTwoAnSm = (228 * 1024) / 2 - 1024 - 256;  // shared memory of a CTA of which two fit an SM
  const long long most = BN <= 64 ? 2ll * sms : sms;
  const int least = BN <= 64 ? 1 : 4;
  int best = 1;
  for (int s = 2; s <= 8; ++s)
    if (tiles * s <= most && s * least <= steps && (BN > 64 || Split<BN>::smem_bytes(s) <= kTwoAnSm)) best = s;
  return best;
}

template <int DT, int BN, bool kSwap>
cudaError_t split_bn(MatmulKernelParams &q, const Mx4Operand &op, const Mx4Operand &oq, int sms, cudaStream_t s) {
  q.tiles_p = (int)ceil_div(op.rows, 128ll), q.tiles_q = (int)ceil_div(oq.rows, (long long)BN);
  if (q.steps > 0 && (!make_map(&q.map_p, op, 128) || !make_map(&q.map_q, oq, BN))) return cudaErrorInvalidValue;
  q.scales_p = op.scales, q.scales_q = oq.scales;
  const long long tiles = (long long)q.tiles_p * q.tiles_q;
  const int split = split_of<BN>(tiles, q.steps, sms);
  return launch_matmul<mx4_split_kernel<DT, BN, kSwap>>(tiles * split, Split<BN>::kThreads, Split<BN>::smem_bytes(split), split, s,
                                                        q, split);
}

template <int DT>
cudaError_t matmul_dt(const MatmulParams &p, cudaStream_t s) {
  MatmulKernelParams q;
  q.m = p.m, q.n = p.n;
  q.steps = (int)((p.k + kBK - 1) / kBK);
  q.out = p.out, q.residual = p.residual, q.ld_out = p.ld_out, q.ld_res = p.ld_res;
  q.drop = p.drop, q.status = p.status;
  q.vec = p.vec, q.vec32 = p.vec32;
  if (p.m <= 16) return split_bn<DT, 16, true>(q, p.b, p.a, p.sms, s);
  if (p.m <= 32) return split_bn<DT, 32, true>(q, p.b, p.a, p.sms, s);
  if (p.m <= 64) return split_bn<DT, 64, true>(q, p.b, p.a, p.sms, s);
  // Pairs once they have a tile each; for K above 1024 once whole tiles of
  // 128 x 128 are more than the SMs (2048 x 2048 x 4096, 64 pair tiles: 10.6 us
  // against 13.0; 2048 x 2048 x 512: 6.2 against 5.6); and for K from 4096 once
  // there are sixteen pair tiles, each then halved (512 x 4096 x 4096, 32: 8.3 us
  // against 9.1; 1024^2 x 4096, 16: 7.3 against 7.5; 1024^3: 4.8 against 4.4).
  const long long pair_tiles = ceil_div(p.m, (long long)kPM) * ceil_div(p.n, (long long)kPN);
  const long long whole_tiles = ceil_div(p.m, 128ll) * ceil_div(p.n, 128ll);
  const bool by_pairs = pair_tiles >= p.sms / 2 || (q.steps > 4 && whole_tiles > p.sms) ||
                        (q.steps >= 16 && pair_tiles >= 16);
  if (q.steps == 0 || !by_pairs)
    return split_bn<DT, 128, false>(q, p.a, p.b, p.sms, s);
  const long long ra = ceil_div(p.m, (long long)kMx4TileRows), rb = ceil_div(p.n, (long long)kMx4TileRows);
  if (!make_map(&q.map_p, p.a, 128) || !make_map(&q.map_q, p.b, 128) ||
      !make_scale_map(&q.map_sp, p.a.scales, ra, q.steps, 1) || !make_scale_map(&q.map_sq, p.b.scales, rb, q.steps, 2))
    return cudaErrorInvalidValue;
  q.tiles_p = (int)ceil_div(p.m, (long long)kPM), q.tiles_q = (int)ceil_div(p.n, (long long)kPN);
  const long long pairs = p.sms / 2, last = pair_tiles % pairs;
  q.whole = 2 * last <= pairs ? pair_tiles - last : pair_tiles;
  q.items = q.whole + 2 * (pair_tiles - q.whole);
  if (q.items > q.whole && (!make_map(&q.map_qh, p.b, 64) || !make_scale_map(&q.map_sqh, p.b.scales, rb, q.steps, 1)))
    return cudaErrorInvalidValue;
  const long long grid = 2 * (q.items < pairs ? q.items : pairs);
  return launch_matmul<mx4_pair_kernel<DT>>(grid, kPairThreads, kPairSmemBytes, 0, s, q);
}

}  // namespace

cudaError_t launch_mx4_matmul(const MatmulParams &p, cudaStream_t s) {
  return p.dtype == kF32 ? matmul_dt<kF32>(p, s) : p.dtype == kF16 ? matmul_dt<kF16>(p, s) : matmul_dt<kBF16>(p, s);
}

}  // namespace rr
