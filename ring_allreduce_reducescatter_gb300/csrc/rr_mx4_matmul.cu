// rr_mx4_matmul.cu -- the product of two microscaled 4-bit matrices,
//   out[i, j] = (residual[i, j] +) drop(sum_k A[i, k] B[j, k]),
// on the block-scaled tensor cores.
#include "rr_mx4.cuh"
#include "rr_tcgen05.cuh"

namespace rr {

namespace {

// Tile of a CTA: 128 rows of A by kBN rows of B, K in steps of 256 elements
// (128 bytes a row, one scale tile).
constexpr int kBM = 128, kBN = 128, kBK = 256;
constexpr int kStages = 6;
constexpr int kRowBytes = kBK / 2;
constexpr int kStageA = kBM * kRowBytes, kStageB = kBN * kRowBytes;
constexpr int kStageBytes = kStageA + kStageB + 2 * kMx4TileBytes;
constexpr int kSmemBytes = kStages * kStageBytes + 1024;
constexpr int kMatmulThreads = 192;  // warps 0-3 epilogue, 4 copies, 5 products
constexpr uint32_t kTmemColumns = 256;  // kBN accumulators, then the scales of two steps
constexpr uint32_t kTmemScales = kBN;

struct MatmulKernelParams {
  CUtensorMap map_a, map_b;
  CUtensorMap map_sa, map_sb;  // the scale tiles, 8 rows of 128 bytes each (pair kernel)
  const uint8_t *scales_a, *scales_b;
  long long m, n;
  int steps;  // of K
  int tiles_m, tiles_n;
  void *out;
  const void *residual;
  long long ld_out, ld_res;
  DropParams drop;
  unsigned int *status;
  bool vec, vec32;  // 16- and 32-byte groups of the rows of out (and residual, for vec) are aligned
};

// Sixteen accumulators of one row, from column `col` on, to the output.
template <int DT>
__device__ __forceinline__ void finish16(const MatmulKernelParams &p, long long row, long long col,
                                         const uint32_t *acc) {
  const long long left = p.n - col;
  if (row >= p.m || left <= 0) return;
  float v[16];
#pragma unroll
  for (int j = 0; j < 16; ++j) v[j] = __uint_as_float(acc[j]);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int valid = (int)min(8ll, left - 8 * h);
    if (valid <= 0) break;
    if (p.drop.threshold) drop8(p.drop, (unsigned long long)(row * p.n + col + 8 * h), v + 8 * h);
    if (p.residual) {
      float w[8];
      load8<DT>(p.residual, row * p.ld_res + col + 8 * h, valid, p.vec, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[8 * h + j] = __fadd_rn(w[j], v[8 * h + j]);
    }
  }
  if (p.vec32 && left >= 16) {
    using T = typename Fmt<DT>::type;
    T *o = static_cast<T *>(p.out) + row * p.ld_out + col;
    uint4 raw[2 * kRaw8<DT>];
    narrow8<DT>(v, raw), narrow8<DT>(v + 8, raw + kRaw8<DT>);
#pragma unroll
    for (int j = 0; j < kRaw8<DT>; ++j) stg32(reinterpret_cast<uint4 *>(o) + 2 * j, raw[2 * j], raw[2 * j + 1]);
  } else {
    store8<DT>(p.out, row * p.ld_out + col, (int)min(8ll, left), p.vec, v);
    if (left > 8) store8<DT>(p.out, row * p.ld_out + col + 8, (int)min(8ll, left - 8), p.vec, v + 8);
  }
}

template <int DT>
__global__ void __launch_bounds__(kMatmulThreads, 1) mx4_matmul_kernel(const __grid_constant__ MatmulKernelParams p) {
  extern __shared__ unsigned char smem_raw[];
  __shared__ __align__(8) uint64_t full[kStages], empty[kStages], done;
  __shared__ uint32_t tmem_slot;
  __shared__ int failed;
  unsigned char *smem = smem_raw + ((1024 - (smem_addr(smem_raw) & 1023)) & 1023);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) mbar_init(&full[s], 1), mbar_init(&empty[s], 1);
    mbar_init(&done, 1);
    failed = 0;
    fence_mbar_init();
  }
  if (warp == 5) tmem_alloc<1>(&tmem_slot, kTmemColumns);
  tcgen05_fence_before();
  __syncthreads();
  tcgen05_fence_after();
  const uint32_t tmem = tmem_slot;
  const int tm = blockIdx.x % p.tiles_m, tn = blockIdx.x / p.tiles_m;
  grid_dependency_wait();

  if (warp == 4 && lane == 0) {
    const uint64_t pol = l2_evict_normal_policy();
    int k = 0;
    for (; k < p.steps; ++k) {
      const int s = k % kStages;
      if (!mbar_wait_bounded(&empty[s], ((k / kStages) & 1) ^ 1, kWaitLimitNs)) break;
      unsigned char *st = smem + s * kStageBytes;
      mbar_arrive_expect_tx(&full[s], kStageBytes);
      tensor_load(st, &p.map_a, k * kRowBytes, tm * kBM, &full[s], pol);
      tensor_load(st + kStageA, &p.map_b, k * kRowBytes, tn * kBN, &full[s], pol);
      bulk_load(st + kStageA + kStageB, p.scales_a + ((long long)tm * p.steps + k) * kMx4TileBytes, kMx4TileBytes, &full[s], pol);
      bulk_load(st + kStageA + kStageB + kMx4TileBytes, p.scales_b + ((long long)tn * p.steps + k) * kMx4TileBytes,
                kMx4TileBytes, &full[s], pol);
    }
    if (k < p.steps) {  // gave up: wait for the copies still in flight
      atomicOr(p.status, kStatusWaitTimeout);
      atomicExch(&failed, 1);
      for (int q = k > kStages ? k - kStages : 0; q < k; ++q)
        mbar_wait_bounded(&full[q % kStages], (q / kStages) & 1, kWaitLimitNs);
    }
  } else if (warp == 5 && lane == 0) {
    int k = 0;
    for (; k < p.steps; ++k) {
      const int s = k % kStages;
      if (!mbar_wait_bounded(&full[s], (k / kStages) & 1, kWaitLimitNs)) break;
      tcgen05_fence_after();
      const uint32_t a = smem_addr(smem + s * kStageBytes), b = a + kStageA, sc = b + kStageB;
      // the scales of a step: A's eight columns, then B's; steps alternate
      const uint32_t sa = tmem + kTmemScales + (k & 1) * 16, sb = sa + 8;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        scale_copy<1>(sa + 4 * j, scale_desc(sc + j * kMx4AtomBytes));
        scale_copy<1>(sb + 4 * j, scale_desc(sc + kMx4TileBytes + j * kMx4AtomBytes));
      }
#pragma unroll
      for (int j = 0; j < kBK / 64; ++j)
        mx4_mma<1>(tmem, operand_desc(a + 32 * j), operand_desc(b + 32 * j), mx4_instr_desc(kBM, kBN, (j & 1) * 2),
                sa + 4 * (j / 2), sb + 4 * (j / 2), k > 0 || j > 0);
      tcgen05_commit<1>(&empty[s]);
    }
    if (k < p.steps) {
      atomicOr(p.status, kStatusWaitTimeout);
      atomicExch(&failed, 1);
    }
    tcgen05_commit<1>(&done);
  }
  __syncwarp();
  // every warp waits here for the last product, so none leaves tensor memory
  // or shared memory while they are in use
  if (!mbar_wait_bounded(&done, 0, 2 * kWaitLimitNs)) {
    if (lane == 0) {
      atomicOr(p.status, kStatusWaitTimeout);
      atomicExch(&failed, 1);
    }
  }
  tcgen05_fence_after();
  __syncthreads();

  if (warp < 4 && !failed) {
    const long long row = (long long)tm * kBM + warp * 32 + lane;
#pragma unroll 1
    for (int c = 0; c < kBN; c += 32) {
      uint32_t acc[32];
      tmem_load32(tmem + ((uint32_t)(warp * 32) << 16) + c, acc);
      tmem_load_wait();
if (p.steps == 0) {
#pragma unroll
        for (int j = 0; j < 32; ++j) acc[j] = 0;
      }
      finish16<DT>(p, row, (long long)tn * kBN + c, acc);
      finish16<DT>(p, row, (long long)tn * kBN + c + 16, acc + 16);
    }
  }
  tcgen05_fence_before();
  __syncthreads();
  tcgen05_fence_after();
  if (warp == 5) tmem_free<1>(tmem, kTmemColumns);
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
// run.
constexpr int kPM = 256, kPN = 256;
constexpr int kPairStages = 6;
constexpr int kPairHalf = 128 * kRowBytes;  // 128 rows of A or of B
constexpr int kPairStageBytes = 2 * kPairHalf + 3 * kMx4TileBytes;  // + scales of 128 rows of A, 256 of B
constexpr int kPairSmemBytes = kPairStages * kPairStageBytes + 1024;
constexpr int kPairThreads = 320;  // warps 0-7 epilogue, 8 copies, 9 products
constexpr uint32_t kPairScales = kPN;  // first tensor-memory column of the scales

template <int DT>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPairThreads, 1)
    mx4_pair_kernel(const __grid_constant__ MatmulKernelParams p) {
  extern __shared__ unsigned char smem_raw[];
  __shared__ __align__(8) uint64_t full[kPairStages], empty[kPairStages], acc_full, acc_empty;
  __shared__ uint32_t tmem_slot;
  unsigned char *smem = smem_raw + ((1024 - (smem_addr(smem_raw) & 1023)) & 1023);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
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
  const uint32_t tmem = tmem_slot;
  const int pairs = gridDim.x / 2, pair = blockIdx.x / 2;
  const long long tiles = (long long)p.tiles_m * p.tiles_n;
  grid_dependency_wait();

  if (warp == 8 && lane == 0) {
    const uint64_t pol = l2_evict_normal_policy();
    const int row_tiles_b = (int)ceil_div(p.n, (long long)kMx4TileRows);
    unsigned g = 0;
    bool ok = true;
    for (long long t = pair; t < tiles && ok; t += pairs) {
      const int tm = (int)(t % p.tiles_m), tn = (int)(t / p.tiles_m);
      // a scale tile past the end reads as zeros
      const int ra = tm * 2 + (int)rank, rb = tn * 2, rb1 = rb + 1 < row_tiles_b ? rb + 1 : rb;
      for (int k = 0; k < p.steps; ++k, ++g) {
        const unsigned s = g % kPairStages;
        if (!(ok = mbar_wait_bounded(&empty[s], ((g / kPairStages) & 1) ^ 1, kWaitLimitNs))) break;
        unsigned char *st = smem + s * kPairStageBytes;
        const uint32_t bar = cluster_addr(&full[s], 0);
        if (rank == 0) mbar_arrive_expect_tx(&full[s], 2 * kPairStageBytes);
        tensor_load_pair(st, &p.map_a, k * kRowBytes, tm * kPM + (int)rank * 128, bar, pol);
        tensor_load_pair(st + kPairHalf, &p.map_b, k * kRowBytes, tn * kPN + (int)rank * 128, bar, pol);
        tensor_load_pair(st + 2 * kPairHalf, &p.map_sa, 0, (ra * p.steps + k) * 8, bar, pol);
        tensor_load_pair(st + 2 * kPairHalf + kMx4TileBytes, &p.map_sb, 0, (rb * p.steps + k) * 8, bar, pol);
        tensor_load_pair(st + 2 * kPairHalf + 2 * kMx4TileBytes, &p.map_sb, 0, (rb1 * p.steps + k) * 8, bar, pol);
      }
    }
    if (!ok) {  // gave up: let the copies in flight land (a limit, not a wait on them)
      atomicOr(p.status, kStatusWaitTimeout);
      for (int s = 0; s < kPairStages; ++s) mbar_wait_bounded(&full[s], 0, 10000000ull);
    }
  } else if (warp == 9 && lane == 0 && rank == 0) {
    unsigned g = 0, i = 0;
    bool ok = true;
    for (long long t = pair; t < tiles && ok; t += pairs, ++i) {
      if (i > 0 && !(ok = mbar_wait_bounded(&acc_empty, (i - 1) & 1, kWaitLimitNs))) break;
      tcgen05_fence_after();
      for (int k = 0; k < p.steps; ++k, ++g) {
        const unsigned s = g % kPairStages;
        if (!(ok = mbar_wait_bounded(&full[s], (g / kPairStages) & 1, kWaitLimitNs))) break;
        tcgen05_fence_after();
        const uint32_t a = smem_addr(smem + s * kPairStageBytes), b = a + kPairHalf, sc = b + kPairHalf;
        // the scales of a step: A's eight columns, then B's sixteen; steps alternate
        const uint32_t sa = tmem + kPairScales + (g & 1) * 32, sb = sa + 8;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          scale_copy<2>(sa + 4 * j, scale_desc(sc + j * kMx4AtomBytes));
          scale_copy<2>(sb + 8 * j, scale_desc(sc + kMx4TileBytes + j * kMx4AtomBytes));
          scale_copy<2>(sb + 8 * j + 4, scale_desc(sc + 2 * kMx4TileBytes + j * kMx4AtomBytes));
        }
#pragma unroll
        for (int j = 0; j < kBK / 64; ++j)
          mx4_mma<2>(tmem, operand_desc(a + 32 * j), operand_desc(b + 32 * j), mx4_instr_desc(kPM, kPN, (j & 1) * 2),
                     sa + 4 * (j / 2), sb + 8 * (j / 2), k > 0 || j > 0);
        tcgen05_commit<2>(&empty[s]);
      }
      tcgen05_commit<2>(&acc_full);
    }
    if (!ok) atomicOr(p.status, kStatusWaitTimeout);
  } else if (warp < 8) {
    const int quarter = warp % 4, half = warp / 4;
    unsigned i = 0;
    for (long long t = pair; t < tiles; t += pairs, ++i) {
      const int tm = (int)(t % p.tiles_m), tn = (int)(t / p.tiles_m);
      if (!mbar_wait_bounded(&acc_full, i & 1, kWaitLimitNs)) {
        if (lane == 0) atomicOr(p.status, kStatusWaitTimeout);
        break;
      }
      __syncwarp();
      tcgen05_fence_after();
      uint32_t acc[128];
#pragma unroll
      for (int c = 0; c < 4; ++c)
        tmem_load32(tmem + ((uint32_t)(quarter * 32) << 16) + half * 128 + 32 * c, acc + 32 * c);
      tmem_load_wait();
      tcgen05_fence_before();
      __syncwarp();
      if (lane == 0) cluster_arrive_remote(cluster_addr(&acc_empty, 0));
      const long long row = (long long)tm * kPM + rank * 128 + quarter * 32 + lane;
#pragma unroll
      for (int c = 0; c < 8; ++c) finish16<DT>(p, row, (long long)tn * kPN + half * 128 + 16 * c, acc + 16 * c);
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

// The map of an operand's scale tiles, 1024 bytes each as 8 rows of 128.
bool make_scale_map(CUtensorMap *map, const uint8_t *scales, long long tiles) {
  const EncodeTiled fn = encode_tiled();
  if (!fn) return false;
  const cuuint64_t dims[2] = {128, (cuuint64_t)tiles * 8};
  const cuuint64_t strides[1] = {128};
  const cuuint32_t box[2] = {128, 8};
  const cuuint32_t unit[2] = {1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t *>(scales), dims, strides, box, unit,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <class K>
cudaError_t launch_matmul(K *k, long long grid, int threads, int smem, const MatmulKernelParams &q, cudaStream_t s) {
  if (grid > 0x7fffffffll) return cudaErrorInvalidConfiguration;
  cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t c = {};
  c.gridDim = dim3((unsigned)grid);
  c.blockDim = dim3((unsigned)threads);
  c.dynamicSmemBytes = smem;
  c.stream = s;
  cudaLaunchAttribute a = {};
  a.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  a.val.programmaticStreamSerializationAllowed = 1;
  c.attrs = &a;
  c.numAttrs = 1;
  return cudaLaunchKernelEx(&c, k, q);
}

template <int DT>
cudaError_t matmul_dt(const MatmulParams &p, cudaStream_t s) {
  MatmulKernelParams q;
  q.scales_a = p.a.scales, q.scales_b = p.b.scales;
  q.m = p.m, q.n = p.n;
  q.steps = (int)((p.k + kBK - 1) / kBK);
  q.out = p.out, q.residual = p.residual, q.ld_out = p.ld_out, q.ld_res = p.ld_res;
  q.drop = p.drop, q.status = p.status;
  q.vec = p.vec, q.vec32 = p.vec32;
  const long long ra = ceil_div(p.m, (long long)kMx4TileRows), rb = ceil_div(p.n, (long long)kMx4TileRows);
  if (p.k > 0 && (!make_map(&q.map_a, p.a, kBM) || !make_map(&q.map_b, p.b, kBN) ||
                  !make_scale_map(&q.map_sa, p.a.scales, ra * q.steps) ||
                  !make_scale_map(&q.map_sb, p.b.scales, rb * q.steps)))
    return cudaErrorInvalidValue;
  const long long pair_tiles = ceil_div(p.m, (long long)kPM) * ceil_div(p.n, (long long)kPN);
  if (p.k > 0 && pair_tiles >= p.sms / 2) {
    q.tiles_m = (int)ceil_div(p.m, (long long)kPM), q.tiles_n = (int)ceil_div(p.n, (long long)kPN);
    const long long grid = 2 * (pair_tiles < p.sms / 2 ? pair_tiles : p.sms / 2);
    return launch_matmul(mx4_pair_kernel<DT>, grid, kPairThreads, kPairSmemBytes, q, s);
  }
  q.tiles_m = (int)ra, q.tiles_n = (int)rb;
  return launch_matmul(mx4_matmul_kernel<DT>, ra * rb, kMatmulThreads, kSmemBytes, q, s);
}

}  // namespace

cudaError_t launch_mx4_matmul(const MatmulParams &p, cudaStream_t s) {
  return p.dtype == kF32 ? matmul_dt<kF32>(p, s) : p.dtype == kF16 ? matmul_dt<kF16>(p, s) : matmul_dt<kBF16>(p, s);
}

}  // namespace rr
