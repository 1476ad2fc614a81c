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
  const uint8_t *scales_a, *scales_b;
  long long m, n;
  int steps;  // of K
  int tiles_m, tiles_n;
  void *out;
  const void *residual;
  long long ld_out, ld_res;
  DropParams drop;
  unsigned int *status;
  bool vec;
};

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
  if (warp == 5) tmem_alloc(&tmem_slot, kTmemColumns);
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
        scale_copy(sa + 4 * j, scale_desc(sc + j * kMx4AtomBytes));
        scale_copy(sb + 4 * j, scale_desc(sc + kMx4TileBytes + j * kMx4AtomBytes));
      }
#pragma unroll
      for (int j = 0; j < kBK / 64; ++j)
        mx4_mma(tmem, operand_desc(a + 32 * j), operand_desc(b + 32 * j), mx4_instr_desc(kBM, kBN, (j & 1) * 2),
                sa + 4 * (j / 2), sb + 4 * (j / 2), k > 0 || j > 0);
      tcgen05_commit(&empty[s]);
    }
    if (k < p.steps) {
      atomicOr(p.status, kStatusWaitTimeout);
      atomicExch(&failed, 1);
    }
    tcgen05_commit(&done);
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
      if (row >= p.m) continue;
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const long long col = (long long)tn * kBN + c + 8 * g;
        const int valid = (int)min(8ll, p.n - col);
        if (valid <= 0) continue;
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = p.steps > 0 ? __uint_as_float(acc[8 * g + j]) : 0.f;
        if (p.drop.threshold) drop8(p.drop, (unsigned long long)(row * p.n + col), v);
        if (p.residual) {
          float w[8];
          load8<DT>(p.residual, row * p.ld_res + col, valid, p.vec, w);
#pragma unroll
          for (int j = 0; j < 8; ++j) v[j] = __fadd_rn(w[j], v[j]);
        }
        store8<DT>(p.out, row * p.ld_out + col, valid, p.vec, v);
      }
    }
  }
  tcgen05_fence_before();
  __syncthreads();
  tcgen05_fence_after();
  if (warp == 5) tmem_free(tmem, kTmemColumns);
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

template <int DT>
cudaError_t matmul_dt(const MatmulParams &p, cudaStream_t s) {
  MatmulKernelParams q;
  if (p.k > 0 && (!make_map(&q.map_a, p.a, kBM) || !make_map(&q.map_b, p.b, kBN))) return cudaErrorInvalidValue;
  q.scales_a = p.a.scales, q.scales_b = p.b.scales;
  q.m = p.m, q.n = p.n;
  q.steps = (int)((p.k + kBK - 1) / kBK);
  q.tiles_m = (int)((p.m + kBM - 1) / kBM), q.tiles_n = (int)((p.n + kBN - 1) / kBN);
  q.out = p.out, q.residual = p.residual, q.ld_out = p.ld_out, q.ld_res = p.ld_res;
  q.drop = p.drop, q.status = p.status;
  q.vec = p.vec;
  const long long grid = (long long)q.tiles_m * q.tiles_n;
  if (grid > 0x7fffffffll) return cudaErrorInvalidConfiguration;
  auto *k = mx4_matmul_kernel<DT>;
  cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t c = {};
  c.gridDim = dim3((unsigned)grid);
  c.blockDim = dim3(kMatmulThreads);
  c.dynamicSmemBytes = kSmemBytes;
  c.stream = s;
  cudaLaunchAttribute a = {};
  a.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  a.val.programmaticStreamSerializationAllowed = 1;
  c.attrs = &a;
  c.numAttrs = 1;
  return cudaLaunchKernelEx(&c, k, q);
}

}  // namespace

cudaError_t launch_mx4_matmul(const MatmulParams &p, cudaStream_t s) {
  return p.dtype == kF32 ? matmul_dt<kF32>(p, s) : p.dtype == kF16 ? matmul_dt<kF16>(p, s) : matmul_dt<kBF16>(p, s);
}

}  // namespace rr
