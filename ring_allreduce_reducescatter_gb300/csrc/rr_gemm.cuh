// rr_gemm.cuh -- products of two matrices in 16 bits on the tensor cores, with
// an epilogue of the caller's: D[i, j] = sum_k A[i, k] B[j, k], sums in binary32.
//
// Either operand may lie in memory along K or along its rows (the "MN-major"
// form: a matrix times another's transpose needs no copy of a transpose), in
// batches of equal matrices.  The grid is persistent: a CTA (or a pair of CTAs
// on two SMs, whose tensor cores read both halves of B) loops over tiles; one
// warp brings operand tiles of 64 elements of K by tensor copies into a ring of
// stages, one issues the products, eight take a finished tile out of tensor
// memory while the next one's products run into the other of two accumulators.
//
// What bounds it: the tensor cores take 128 cycles for 256 x 256 x 16 on a pair;
// a pair reads 64 KB of operands a step of 512 cycles, 64 bytes a cycle and SM.  8192
// x 32000 x 4096 in bfloat16 takes 1.06 ms alone (2.0 PFLOP/s, the tensor pipe 93 %
// busy) and, one after another, what the power limit leaves, 1.65-1.69 PFLOP/s.
#pragma once

#include "rr_mx4.cuh"
#include "rr_tcgen05.cuh"
#include "rr_turns.h"

namespace rr {

namespace gemm {

constexpr int kStep = 64;      // elements of K a stage: 128 bytes
constexpr int kThreads = 384;  // warps 0-7 epilogue, 8 copies, 9 products, 10 and 11 idle
constexpr int kChunk = 32;     // columns of a row that an epilogue takes at a time
// The epilogue's shared memory: a warp's 32 rows by 16 columns, padded.
constexpr int kPitch = 17, kStageFloats = 32 * kPitch;

// G CTAs on a tile of 128 G rows by BN columns.
template <int G, int BN>
struct Shape {
  static constexpr int kBM = 128 * G, kBN = BN;
  static constexpr int kRowsB = BN / G;  // of B, in a CTA
  static constexpr int kBytesA = 128 * 128, kBytesB = kRowsB * 128;
  static constexpr int kStageBytes = kBytesA + kBytesB;
  static constexpr int kStages = 6;
  static constexpr int kSmem = kStages * kStageBytes + 8 * kStageFloats * 4 + 1024;
  static constexpr uint32_t kColumns = 2 * BN;  // two accumulators
  static constexpr int kHalf = BN / 2;          // columns of one epilogue warp
  static_assert(kRowsB % 64 == 0 && kHalf % kChunk == 0 && kColumns <= 512, "whole boxes and chunks");
};
using Pair = Shape<2, 256>;
using Single = Shape<1, 128>;

struct Product {
  CUtensorMap a, b;  // (inner axis, outer axis, batch)
  CUtensorMap b_half;  // b in half the rows a box (halved tiles of pairs)
  long long m, n;
  int steps;  // of K
  int tiles_m, tiles_n;
  long long per_batch;         // tiles of one product
  long long items, whole;      // pieces of work, of which the first are whole tiles, the rest halves
  uint32_t format;             // of the operands: 0 binary16, 1 bfloat16
  uint32_t bytes_a;            // of A's box of one step (single tiles of few rows: the rows there are)
  int upper;                   // D is symmetric: only tiles on and above the diagonal
  unsigned int *status;
};

struct Place {
  int batch, tm, tn;
  bool whole;
  int side;  // of the columns of a halved tile
};
// Piece t of the work: a tile, or half of one.  Eight rows of tiles go together, column after column, so that the
// tiles in flight share their operands in L2; of a symmetric product, the
// columns of the upper triangle.
__device__ __forceinline__ Place place_of(const Product &p, long long t) {
  Place w;
  w.whole = t < p.whole, w.side = w.whole ? 0 : (int)((t - p.whole) & 1);
  if (!w.whole) t = p.whole + (t - p.whole) / 2;
  w.batch = (int)(t / p.per_batch);
  const int u = (int)(t - w.batch * p.per_batch);
  if (p.upper) {
    int j = (int)((__fsqrt_rn(8.f * (float)u + 1.f) - 1.f) * 0.5f);
    while ((long long)j * (j + 1) / 2 > u) --j;
    while ((long long)(j + 1) * (j + 2) / 2 <= u) ++j;
    w.tn = j, w.tm = u - (int)((long long)j * (j + 1) / 2);
    return w;
  }
  constexpr int kBand = 8;
  const int band = u / (kBand * p.tiles_n), first = band * kBand;
  const int high = p.tiles_m - first < kBand ? p.tiles_m - first : kBand, v = u - first * p.tiles_n;
  w.tm = first + v % high, w.tn = v / high;
  return w;
}

// --------------------------------------------------------------------------
// PTX
// --------------------------------------------------------------------------

// Instruction descriptor of a product of 16-bit operands into binary32: bits
// 4-5 the accumulators' format (1: binary32), 7-9 and 10-12 the operands', 15
// and 16 set where A and B lie along their rows, 17-22 N / 8, 24-28 M / 16.
__device__ __forceinline__ constexpr uint32_t instr_desc(uint32_t format, bool mn_a, bool mn_b, int M, int N) {
  return (1u << 4) | (format << 7) | (format << 10) | ((uint32_t)mn_a << 15) | ((uint32_t)mn_b << 16) |
         ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
// An operand along its rows: boxes of 64 elements (128 bytes, the 128-byte
// swizzle) by 64 of K, 8192 bytes each; groups of eight of K are 1024 bytes
// apart, the next 64 elements a box.
__device__ __forceinline__ uint64_t rows_desc(uint32_t smem) {
  return (uint64_t)((smem >> 4) & 0x3fff) | (512ull << 16) | (64ull << 32) | (1ull << 46) | (2ull << 61);
}
// D += A B^T over 16 elements of K.
template <int G>
__device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool accumulate) {
  if constexpr (G == 1)
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)accumulate)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)accumulate)
        : "memory");
}
// A box of a three-dimensional map; the bytes count on the barrier at this
// cluster address (G = 2) or of this CTA (G = 1).
template <int G>
__device__ __forceinline__ void load_box(void *dst, const CUtensorMap *map, int x, int y, int z, uint64_t *bar,
                                         uint32_t cluster_bar, uint64_t pol) {
  if constexpr (G == 2) {
    tensor_load_pair(dst, map, x, y, z, cluster_bar, pol);
  } else {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint "
        "[%0], [%1, {%2, %3, %4}], [%5], %6;" ::"r"(smem_addr(dst)),
        "l"(map), "r"(x), "r"(y), "r"(z), "r"(smem_addr(bar)), "l"(pol)
        : "memory");
  }
}

// Brings a tensor map to where the copies read it, ahead of the first (one thread).
__device__ __forceinline__ void prefetch_map(const CUtensorMap *map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}

// Waits for this warp's tensor-memory loads; the values, named here, cannot be
// used before.
__device__ __forceinline__ void tmem_loaded32(uint32_t r[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]),
                 "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]),
                 "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]), "+r"(r[24]),
                 "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])::"memory");
}

// The limit of a wait for what has come already, unless another wait gave up.
constexpr unsigned long long kLateLimitNs = 10000000ull;  // 10 ms
template <int S>
__device__ __forceinline__ void wait_turns(uint64_t *bars, unsigned end, unsigned long long limit_ns) {
  each_open_turn(end, S, [&](unsigned stage, unsigned parity) { mbar_wait_bounded(&bars[stage], parity, limit_ns); });
}

// --------------------------------------------------------------------------
// the kernel
// --------------------------------------------------------------------------

// An epilogue is a struct made for each tile by one thread, which owns one row
// of it and half its columns:
//   Epi(params, row, col, batch, stage)  the row and first column in D (the
//                  warp's lanes have consecutive rows); stage: kStageFloats
//                  floats of the warp's own
//   chunk(c, v)    32 accumulators from column col + 32 c on (the whole warp
//                  calls it; rows and columns past the product's are zero)
//   end()          after the last chunk
// kRun: steps of K after which the sums so far move to registers (0: none).  The
// tensor cores cut a sum at every addition, always towards zero; a run's sums are
// added up in binary32 rounded to nearest, while the next run's products go on in
// the other accumulator.
template <class S, int G, bool kMnA, bool kMnB, class Epi>
__device__ __forceinline__ void product_body(const Product &p, const typename Epi::Params &e) {
  extern __shared__ unsigned char smem_raw[];
  __shared__ __align__(8) uint64_t full[S::kStages], empty[S::kStages], acc_full[2], acc_empty[2];
  __shared__ uint32_t tmem_slot;
  unsigned char *smem = smem_raw + ((1024 - (smem_addr(smem_raw) & 1023)) & 1023);
  const int warp = uniform(threadIdx.x / 32), lane = threadIdx.x % 32;
  const uint32_t rank = G == 2 ? cluster_rank() : 0;

  if (threadIdx.x == 0) {
    for (int s = 0; s < S::kStages; ++s) mbar_init(&full[s], 1), mbar_init(&empty[s], 1);
    for (int s = 0; s < 2; ++s) mbar_init(&acc_full[s], 1), mbar_init(&acc_empty[s], 8 * G);
    fence_mbar_init();
  }
  if (threadIdx.x == 256) prefetch_map(&p.a), prefetch_map(&p.b);
  if (warp == 9) tmem_alloc<G>(&tmem_slot, S::kColumns);
  tcgen05_fence_before();
  __syncthreads();
  if constexpr (G == 2) cluster_sync_all();
  tcgen05_fence_after();
  const uint32_t tmem = (uint32_t)uniform((int)tmem_slot);
  const int workers = gridDim.x / G, worker = blockIdx.x / G;
  grid_dependency_wait();
  grid_dependents_launch();

  if (warp < 8) {
    // registers a thread: 168 at launch (384 threads); 2 * 216 + 72 = 3 * 168
    asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
    const int quarter = warp % 4, half = warp / 4;
    float *stage = reinterpret_cast<float *>(smem + S::kStages * S::kStageBytes) + warp * kStageFloats;
    unsigned i = 0;
    bool ok = true;
    unsigned steps = 0;
    for (long long t = worker; t < p.items && ok; t += workers) {
      const Place w = place_of(p, t);
      const bool mine = G == 1 || w.whole || half == 0;  // a half tile is one half's warps' work
      Epi epi(e, (long long)w.tm * S::kBM + rank * 128 + quarter * 32 + lane,
              (long long)w.tn * S::kBN + (G == 1 || w.whole ? half : w.side) * S::kHalf, w.batch, stage);
      constexpr int kChunks = S::kHalf / kChunk;
      float total[Epi::kRun ? kChunks : 1][kChunk];
      for (int k = 0; k < p.steps; k += Epi::kRun ? Epi::kRun : p.steps, ++i) {
        const unsigned buf = i & 1;
        const bool last = !Epi::kRun || k + Epi::kRun >= p.steps;
        if (!(ok = __all_sync(0xffffffffu, mbar_wait_bounded(&acc_full[buf], (i >> 1) & 1, kWaitLimitNs)))) {
          if (lane == 0) atomicOr(p.status, kStatusWaitTimeout);
          break;
        }
        tcgen05_fence_after();
        const uint32_t at = tmem + ((uint32_t)(quarter * 32) << 16) + buf * S::kBN + half * S::kHalf;
        const auto release = [&] {
          tcgen05_fence_before();
          __syncwarp();
          if (lane == 0) {
            if constexpr (G == 2) cluster_arrive_remote(cluster_addr(&acc_empty[buf], 0));
            else asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(&acc_empty[buf])) : "memory");
          }
        };
        if (!mine) {
          release();
          continue;
        }
        uint32_t acc[2][kChunk];  // a chunk is on its way while the one before is worked on
        tmem_load32(at, acc[0]);
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
          tmem_loaded32(acc[c & 1]);
          if (c + 1 < kChunks) tmem_load32(at + (c + 1) * kChunk, acc[(c + 1) & 1]);
          else release();
          if constexpr (Epi::kRun > 0) {
            if (k == 0) {
#pragma unroll
              for (int j = 0; j < kChunk; ++j) total[c][j] = __uint_as_float(acc[c & 1][j]);
            } else {
#pragma unroll
              for (int j = 0; j < kChunk; ++j) total[c][j] = __fadd_rn(total[c][j], __uint_as_float(acc[c & 1][j]));
            }
            if (last) epi.chunk(c, total[c]);
          } else {
            float v[kChunk];
#pragma unroll
            for (int j = 0; j < kChunk; ++j) v[j] = __uint_as_float(acc[c & 1][j]);
            epi.chunk(c, v);
          }
        }
        if (last) epi.end();
      }
      if (ok) steps += (unsigned)p.steps;
    }
    // the commits of the last turns come before the CTA goes: one that came later
    // would meet another's barrier
    if (warp == 0) wait_turns<S::kStages>(empty, steps, kLateLimitNs);
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    if (warp == 8) {
      const uint64_t pol = l2_evict_normal_policy();
      const bool one = elect_one();
      unsigned g = 0;
      bool ok = true;
      for (long long t = worker; t < p.items && ok; t += workers) {
        const Place w = place_of(p, t);
        const int row_a = w.tm * S::kBM + (int)rank * 128, row_b = w.tn * S::kBN + (G == 1 || w.whole ? (int)rank * S::kRowsB : w.side * S::kHalf + (int)rank * S::kRowsB / 2);
        const bool whole = G == 1 || w.whole;
        const uint32_t bytes = G * (p.bytes_a + (whole ? S::kBytesB : S::kBytesB / 2));
        for (int k = 0; k < p.steps; ++k, ++g) {
          const unsigned s = g % S::kStages;
          if (!(ok = __all_sync(0xffffffffu, mbar_wait_bounded(&empty[s], ((g / S::kStages) & 1) ^ 1, kWaitLimitNs)))) break;
          unsigned char *a = smem + s * S::kStageBytes, *b = a + S::kBytesA;
          const uint32_t bar = G == 2 ? cluster_addr(&full[s], 0) : 0;
          if (one) {
            // (what lies past the operands' ends reads as zeros and counts)
            if (rank == 0) mbar_arrive_expect_tx(&full[s], bytes);
            if constexpr (kMnA) {
#pragma unroll
              for (int j = 0; j < 2; ++j) load_box<G>(a + 8192 * j, &p.a, row_a + 64 * j, k * kStep, w.batch, &full[s], bar, pol);
            } else {
              load_box<G>(a, &p.a, k * kStep, row_a, w.batch, &full[s], bar, pol);
            }
            if constexpr (kMnB) {
#pragma unroll
              for (int j = 0; j < S::kRowsB / 64; ++j)
                if (j == 0 || whole) load_box<G>(b + 8192 * j, &p.b, row_b + 64 * j, k * kStep, w.batch, &full[s], bar, pol);
            } else {
              load_box<G>(b, whole ? &p.b : &p.b_half, k * kStep, row_b, w.batch, &full[s], bar, pol);
            }
          }
          __syncwarp();
        }
      }
      if (!ok && one) atomicOr(p.status, kStatusWaitTimeout);
      // The copies in flight land before shared memory is given back: a pair's all
      // count on rank 0, for whose last barrier below rank 1 waits.
      if (rank == 0) wait_turns<S::kStages>(full, g, kWaitLimitNs);
    } else if (warp == 9 && rank == 0) {
      const bool one = elect_one();
      unsigned g = 0, i = 0;
      bool ok = true;
      for (long long t = worker; t < p.items && ok; t += workers) {
        const uint32_t idesc = G == 1 || t < p.whole ? instr_desc(p.format, kMnA, kMnB, S::kBM, S::kBN)
                                                     : instr_desc(p.format, kMnA, kMnB, S::kBM, S::kBN / 2);
        for (int from = 0; from < p.steps && ok; from += Epi::kRun ? Epi::kRun : p.steps, ++i) {
          const unsigned buf = i & 1;
          const int end = Epi::kRun && from + Epi::kRun < p.steps ? from + Epi::kRun : p.steps;
          if (!(ok = __all_sync(0xffffffffu, mbar_wait_bounded(&acc_empty[buf], ((i >> 1) & 1) ^ 1, kWaitLimitNs)))) break;
          tcgen05_fence_after();
          const uint32_t d = tmem + buf * S::kBN;
          for (int k = from; k < end; ++k, ++g) {
            const unsigned s = g % S::kStages;
            if (!(ok = __all_sync(0xffffffffu, mbar_wait_bounded(&full[s], (g / S::kStages) & 1, kWaitLimitNs)))) break;
            tcgen05_fence_after();
            const uint32_t a = smem_addr(smem) + s * S::kStageBytes, b = a + S::kBytesA;
            if (one) {
#pragma unroll
              for (int j = 0; j < kStep / 16; ++j)
                mma<G>(d, kMnA ? rows_desc(a + 2048 * j) : operand_desc(a + 32 * j),
                       kMnB ? rows_desc(b + 2048 * j) : operand_desc(b + 32 * j), idesc, k > from || j > 0);
              tcgen05_commit<G>(&empty[s]);
            }
            __syncwarp();
          }
          if (ok && one) tcgen05_commit<G>(&acc_full[buf]);  // a tile that was given up is not stored
        }
      }
      if (!ok) {
        if (one) atomicOr(p.status, kStatusWaitTimeout);
        // the products issued so far end before tensor memory is given back (a
        // turn's commit covers all before it)
        if (g > 0) mbar_wait_bounded(&empty[(g - 1) % S::kStages], turn_parity(g - 1, S::kStages), kWaitLimitNs);
      }
    }
  }
  __syncwarp();
  tcgen05_fence_before();
  if constexpr (G == 2) cluster_sync_all();
  else __syncthreads();
  tcgen05_fence_after();
  if (warp == 9) tmem_free<G>(tmem, S::kColumns);
}

// --------------------------------------------------------------------------
// few tiles: K split over a cluster
// --------------------------------------------------------------------------

// A cluster of S CTAs (2, 4 or 8) computes one tile of 128 x 128, each CTA a
// contiguous part of K.  Each sends its sums, 32 columns (64 for two CTAs) to each
// of up to four owners, to a place of its own in the owner's shared memory; one
// barrier later the owners add up what they received, in rank order (the result
// does not depend on timing), and finish it.  A grid of whole tiles would leave most
// SMs without a share of the work: 33 x 1024 by K of 8000 took 30 us whole.
struct Split {
  static constexpr int kStages = 3, kStageBytes = 2 * 128 * 128;
  static constexpr int kThreads = 320;  // warps 0-7 epilogue, 8 copies, 9 products
  static constexpr uint32_t kColumns = 128;
  static __host__ __device__ constexpr int owners(int split) { return split < 4 ? split : 4; }
  static __host__ __device__ constexpr int part_bytes(int split) { return 128 * 128 * 4 / owners(split); }
  static __host__ __device__ constexpr int smem(int split) { return 1024 + kStages * kStageBytes + split * part_bytes(split); }
  static_assert(kStages * kStageBytes >= 8 * kStageFloats * 4, "the ragged epilogue fits the stages");
};

template <bool kMnA, bool kMnB, class Epi>
__global__ void __launch_bounds__(Split::kThreads, 1)
    product_split_kernel(const __grid_constant__ Product p, const __grid_constant__ typename Epi::Params e, int split) {
  extern __shared__ unsigned char smem_raw[];
  __shared__ __align__(8) uint64_t full[Split::kStages], empty[Split::kStages], done;
  __shared__ uint32_t tmem_slot;
  __shared__ int failed;
  unsigned char *smem = smem_raw + ((1024 - (smem_addr(smem_raw) & 1023)) & 1023);
  const int warp = uniform(threadIdx.x / 32), lane = threadIdx.x % 32;
  if (threadIdx.x == 0) {
    for (int s = 0; s < Split::kStages; ++s) mbar_init(&full[s], 1), mbar_init(&empty[s], 1);
    mbar_init(&done, 1);
    failed = 0;
    fence_mbar_init();
  }
  cluster_arrive();  // waited for before the first remote store: by then every CTA runs
  if (threadIdx.x == 256) prefetch_map(&p.a), prefetch_map(&p.b);
  if (warp == 9) tmem_alloc<1>(&tmem_slot, Split::kColumns);
  tcgen05_fence_before();
  __syncthreads();
  tcgen05_fence_after();
  const uint32_t tmem = (uint32_t)uniform((int)tmem_slot);
  const int rank = blockIdx.x % split;
  const Place w = place_of(p, blockIdx.x / split);
  const int k0 = (int)((long long)p.steps * rank / split), n_steps = (int)((long long)p.steps * (rank + 1) / split) - k0;
  grid_dependency_wait();
  grid_dependents_launch();

  if (warp == 8) {
    const uint64_t pol = l2_evict_normal_policy();
    const bool one = elect_one();
    int k = 0;
    for (; k < n_steps; ++k) {
      const int s = k % Split::kStages;
      if (!__all_sync(0xffffffffu, mbar_wait_bounded(&empty[s], ((k / Split::kStages) & 1) ^ 1, kWaitLimitNs))) break;
      unsigned char *a = smem + s * Split::kStageBytes, *b = a + 128 * 128;
      if (one) {
        mbar_arrive_expect_tx(&full[s], p.bytes_a + 128 * 128);
        if constexpr (kMnA) {
#pragma unroll
          for (int j = 0; j < 2; ++j) load_box<1>(a + 8192 * j, &p.a, w.tm * 128 + 64 * j, (k0 + k) * kStep, w.batch, &full[s], 0, pol);
        } else {
          load_box<1>(a, &p.a, (k0 + k) * kStep, w.tm * 128, w.batch, &full[s], 0, pol);
        }
        if constexpr (kMnB) {
#pragma unroll
          for (int j = 0; j < 2; ++j) load_box<1>(b + 8192 * j, &p.b, w.tn * 128 + 64 * j, (k0 + k) * kStep, w.batch, &full[s], 0, pol);
        } else {
          load_box<1>(b, &p.b, (k0 + k) * kStep, w.tn * 128, w.batch, &full[s], 0, pol);
        }
      }
      __syncwarp();
    }
    if (k < n_steps && one) {
      atomicOr(p.status, kStatusWaitTimeout);
      atomicExch(&failed, 1);
    }
    // the copies in flight land before shared memory is given back
    wait_turns<Split::kStages>(full, k, kWaitLimitNs);
  } else if (warp == 9) {
    const bool one = elect_one();
    const uint32_t idesc = instr_desc(p.format, kMnA, kMnB, 128, 128);
    int k = 0;
    for (; k < n_steps; ++k) {
      const int s = k % Split::kStages;
      if (!__all_sync(0xffffffffu, mbar_wait_bounded(&full[s], (k / Split::kStages) & 1, kWaitLimitNs))) break;
      tcgen05_fence_after();
      const uint32_t a = smem_addr(smem) + s * Split::kStageBytes, b = a + 128 * 128;
      if (one) {
#pragma unroll
        for (int j = 0; j < kStep / 16; ++j)
          mma<1>(tmem, kMnA ? rows_desc(a + 2048 * j) : operand_desc(a + 32 * j),
                 kMnB ? rows_desc(b + 2048 * j) : operand_desc(b + 32 * j), idesc, k > 0 || j > 0);
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
  // every warp waits here for the last product, so none leaves tensor memory or
  // shared memory while they are in use
  if (!mbar_wait_bounded(&done, 0, 2 * kWaitLimitNs) && lane == 0) {
    atomicOr(p.status, kStatusWaitTimeout);
    atomicExch(&failed, 1);
  }
  __syncwarp();
  tcgen05_fence_after();
  __syncthreads();

  const int quarter = warp % 4, half = warp / 4, row = quarter * 32 + lane, owners = Split::owners(split);
  float *got = reinterpret_cast<float *>(smem + Split::kStages * Split::kStageBytes);
  const int part = Split::part_bytes(split) / 4;  // floats: [columns / 4][128 rows][4]
  cluster_wait();
  if (warp < 8) {
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      uint32_t acc[kChunk];
      tmem_load32(tmem + ((uint32_t)(quarter * 32) << 16) + half * 64 + c * kChunk, acc);
      tmem_loaded32(acc);
      const int g = half * 2 + c, owner = owners == 4 ? g : g / 2, at = owners == 4 ? 0 : g % 2;
      const uint32_t to = cluster_addr(got + rank * part + at * (kChunk * 128) + row * 4, owner);
#pragma unroll
      for (int j = 0; j < kChunk; j += 4) cluster_store4(to + j * 128 * 4, make_uint4(acc[j], acc[j + 1], acc[j + 2], acc[j + 3]));
    }
  } else if (warp == 8) {
    // the commits of the last turns come before the CTA goes: later ones would
    // meet another's barrier
    wait_turns<Split::kStages>(empty, n_steps, kLateLimitNs);
  }
  tcgen05_fence_before();
  __syncthreads();
  tcgen05_fence_after();
  cluster_arrive();
  if (warp == 9) tmem_free<1>(tmem, Split::kColumns);
  cluster_wait();
  if (rank < owners && half < 4 / owners && warp < 8 && !failed) {
    const int first = rank * (128 / owners) + half * kChunk;
    Epi epi(e, (long long)w.tm * 128 + row, (long long)w.tn * 128 + first, w.batch, reinterpret_cast<float *>(smem) + warp * kStageFloats);
    float v[kChunk];
#pragma unroll
    for (int j = 0; j < kChunk; ++j) v[j] = 0.f;
    for (int r = 0; r < split; ++r) {
      const float4 *from = reinterpret_cast<const float4 *>(got + r * part + half * (kChunk * 128)) + row;
#pragma unroll
      for (int j = 0; j < kChunk; j += 4) {
        const float4 x = from[j / 4 * 128];
        v[j] = __fadd_rn(v[j], x.x), v[j + 1] = __fadd_rn(v[j + 1], x.y);
        v[j + 2] = __fadd_rn(v[j + 2], x.z), v[j + 3] = __fadd_rn(v[j + 3], x.w);
      }
    }
    epi.chunk(0, v);
    epi.end();
  }
}

template <bool kMnA, bool kMnB, class Epi>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    product_pair_kernel(const __grid_constant__ Product p, const __grid_constant__ typename Epi::Params e) {
  product_body<Pair, 2, kMnA, kMnB, Epi>(p, e);
}
template <bool kMnA, bool kMnB, class Epi>
__global__ void __launch_bounds__(kThreads, 1)
    product_single_kernel(const __grid_constant__ Product p, const __grid_constant__ typename Epi::Params e) {
  product_body<Single, 1, kMnA, kMnB, Epi>(p, e);
}

// --------------------------------------------------------------------------
// what epilogues store
// --------------------------------------------------------------------------

// A strided output and whether its rows' 32-byte groups are aligned.
struct Out {
  void *at;
  long long rows, cols, ld;
  bool vec32;
};

// 32 values of this lane's row from column col on, to storage: whole sectors
// where rows are aligned, else the block is turned in shared memory, sixteen
// columns at a time, so that sixteen lanes take neighbours of a row.
template <int DT>
__device__ __forceinline__ void store_row(const Out &o, long long row, long long col, const float v[kChunk], float *stage) {
  using T = typename Fmt<DT>::type;
  T *base = static_cast<T *>(o.at);
  if (o.vec32 && col + kChunk <= o.cols) {
    if (row >= o.rows) return;
    uint4 *q = reinterpret_cast<uint4 *>(base + row * o.ld + col);
    uint4 raw[4 * kRaw8<DT>];
#pragma unroll
    for (int h = 0; h < 4; ++h) narrow8<DT>(v + 8 * h, raw + h * kRaw8<DT>);
#pragma unroll
    for (int j = 0; j < 4 * kRaw8<DT>; j += 2) stg32(q + j, raw[j], raw[j + 1]);
    return;
  }
  const int lane = threadIdx.x % 32;
  const long long rows0 = row - lane;
  if (col >= o.cols || rows0 >= o.rows) return;  // the same for the whole warp
#pragma unroll
  for (int half = 0; half < 2; ++half) {
#pragma unroll
    for (int j = 0; j < 16; ++j) stage[lane * kPitch + j] = v[16 * half + j];
    __syncwarp();
    const long long c = col + 16 * half + lane % 16, r0 = rows0 + lane / 16;
    const long long most = o.rows - r0;
    const int left = c < o.cols ? (int)(most < 32 ? most : 32) : 0;  // rows from r0 on
    const float *from = stage + lane / 16 * kPitch + lane % 16;
    T *q = base + r0 * o.ld + c;
#pragma unroll
    for (int k = 0; k < 16; ++k, q += 2 * o.ld)
      if (2 * k < left) *q = from_f32<DT>(from[2 * k * kPitch]);
    __syncwarp();
  }
}

// --------------------------------------------------------------------------
// launches
// --------------------------------------------------------------------------

// An operand in memory: `rows` rows by K, along K (ld elements from row to row)
// or, mn, along its rows (ld from one of K to the next).
struct Operand {
  const void *at;
  long long rows, k, ld, batch_stride;
  int batch;
  bool mn;
};

// Boxes that lie partly past the end of a small operand are slow to read when all
// SMs read it: 16 rows by 1024 (32 KB) in boxes of 128 rows took a product with
// 131072 rows 252 us, in an array of 256 KB 77 us, 128 whole rows 66 us.  Small
// operands therefore lie in whole boxes, of rows and of zeros, or the box is as high
// as the operand.
constexpr long long kSmallOperand = 1 << 20;  // bytes

// Defined in rr_gemm.cu: the map of an operand's boxes; `box` rows a box along K.
bool make_operand_map(CUtensorMap *map, const Operand &o, int box);

template <class S>
bool fill_product(Product *q, const Operand &a, const Operand &b, bool upper, uint32_t format, unsigned int *status) {
  q->m = a.rows, q->n = b.rows;
  // (rows of A that are not there leave what shared memory held in rows of D that
  // no epilogue stores)
  const int box = !a.mn && S::kBM == 128 && a.rows < 128 ? (int)a.rows : 128;
  if (!make_operand_map(&q->a, a, box) || !make_operand_map(&q->b, b, S::kRowsB)) return false;
  q->bytes_a = (uint32_t)box * 128;
  q->steps = (int)ceil_div(a.k, (long long)kStep);
  q->tiles_m = (int)ceil_div(q->m, (long long)S::kBM), q->tiles_n = (int)ceil_div(q->n, (long long)S::kBN);
  q->per_batch = upper ? (long long)q->tiles_n * (q->tiles_n + 1) / 2 : (long long)q->tiles_m * q->tiles_n;
  q->items = q->whole = q->per_batch * b.batch;
  q->format = format, q->upper = upper, q->status = status;
  return true;
}

template <auto kKernel, class S, int G, class Params>
cudaError_t launch_shape(const Operand &a, const Operand &b, bool upper, uint32_t format, unsigned int *status, int sms,
                         const Params &e, cudaStream_t s) {
  Product q;
  if (!fill_product<S>(&q, a, b, upper, format, status)) return cudaErrorInvalidValue;
  if constexpr (G == 2) {
    // the last turn's tiles are halved where they are no more than half the pairs
    const long long last = q.items % (sms / 2);
    if (last > 0 && 2 * last <= sms / 2) {
      if (!make_operand_map(&q.b_half, b, S::kRowsB / 2)) return cudaErrorInvalidValue;
      q.whole = q.items - last, q.items += last;
    }
  }
  const long long most = sms / G, workers = q.items < most ? q.items : most;
  const cudaError_t err = allow_smem<kKernel>(S::kSmem);
  if (err != cudaSuccess) return err;
  cudaLaunchConfig_t c = {};
  c.gridDim = dim3((unsigned)(workers * G));
  c.blockDim = dim3(kThreads);
  c.dynamicSmemBytes = S::kSmem;
  c.stream = s;
  cudaLaunchAttribute at = {};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  c.attrs = &at;
  c.numAttrs = 1;
  return cudaLaunchKernelEx(&c, kKernel, q, e);
}

// CTAs a tile: none is split where the tiles fill the SMs, or K is short (an
// exchange costs about 1.5 us, a step of K 0.15).
inline int split_of(long long tiles, long long steps, int sms) {
  if (tiles * 8 <= 64 && steps >= 32) return 8;
  if (tiles * 4 <= sms && steps >= 12) return 4;
  if (tiles * 2 <= sms && steps >= 16) return 2;
  return 1;
}

template <bool kMnA, bool kMnB, class Epi>
cudaError_t launch_split(const Operand &a, const Operand &b, bool upper, int split, uint32_t format, unsigned int *status,
                         const typename Epi::Params &e, cudaStream_t s) {
  Product q;
  if (!fill_product<Single>(&q, a, b, upper, format, status)) return cudaErrorInvalidValue;
  if (q.items * split > 0x7fffffffll) return cudaErrorInvalidConfiguration;
  const cudaError_t err = allow_smem<product_split_kernel<kMnA, kMnB, Epi>>(Split::smem(8));
  if (err != cudaSuccess) return err;
  cudaLaunchConfig_t c = {};
  c.gridDim = dim3((unsigned)(q.items * split));
  c.blockDim = dim3(Split::kThreads);
  c.dynamicSmemBytes = Split::smem(split);
  c.stream = s;
  cudaLaunchAttribute at[2] = {};
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = (unsigned)split, at[1].val.clusterDim.y = 1, at[1].val.clusterDim.z = 1;
  c.attrs = at;
  c.numAttrs = 2;
  return cudaLaunchKernelEx(&c, product_split_kernel<kMnA, kMnB, Epi>, q, e, split);
}

// Which of the three a product takes: beyond one turn of the smaller tiles, the
// larger ones unless their turns cost more (half a turn of a pair takes 1.33 of a
// single's: 32 KB a step for 128 x 128 come at 64 bytes a cycle, and 24 for twice that).
enum Kind { kSingle, kPair, kSplit };
inline Kind kind_of(long long m, long long n, long long k, int batch, bool upper, int sms, int *split) {
  const auto tiles = [&](long long side) {
    const long long tm = ceil_div(m, side), tn = ceil_div(n, side);
    return (upper ? tn * (tn + 1) / 2 : tm * tn) * batch;
  };
  const long long pairs = tiles(256), singles = tiles(128);
  *split = split_of(singles, ceil_div(k, (long long)kStep), sms);
  if (*split > 1) return kSplit;
  if (singles <= sms) return kSingle;
  const long long last = pairs % (sms / 2), turns = 2 * (pairs / (sms / 2)) + (last == 0 ? 0 : 2 * last <= sms / 2 ? 1 : 2);  // halves
  return 3 * turns <= 4 * ceil_div(singles, (long long)sms) ? kPair : kSingle;
}

// A product of a (its rows are D's rows) and b (D's columns).  upper: D is
// symmetric, a and b the same matrix.
template <bool kMnA, bool kMnB, class Epi>
cudaError_t launch_product(const Operand &a, const Operand &b, bool upper, uint32_t format, unsigned int *status, int sms,
                           const typename Epi::Params &e, cudaStream_t s) {
  int split;
  switch (kind_of(a.rows, b.rows, a.k, b.batch, upper, sms, &split)) {
    case kSplit:
      return launch_split<kMnA, kMnB, Epi>(a, b, upper, split, format, status, e, s);
    case kPair:
      return launch_shape<product_pair_kernel<kMnA, kMnB, Epi>, Pair, 2>(a, b, upper, format, status, sms, e, s);
    default:
      return launch_shape<product_single_kernel<kMnA, kMnB, Epi>, Single, 1>(a, b, upper, format, status, sms, e, s);
  }
}

}  // namespace gemm

}  // namespace rr
