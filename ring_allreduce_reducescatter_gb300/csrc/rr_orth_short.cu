// rr_orth_short.cu -- the orthogonalised update of matrices whose shorter side is
// at most 128: all steps in one launch.
//
// A cluster of up to eight CTAs holds a matrix in shared memory, 128 rows (the
// shorter side) by 128 or 256 columns each.  A step: every CTA multiplies its
// columns with themselves; the sums go to their owners (a part of S's columns
// each), which add them up in rank order and send S in binary16 to all;
// S^2, the polynomial and the CTA's own columns of the update need nobody else.
// X lies once in shared memory, 64 columns in 128-byte swizzled rows: along K it is
// the operand of S, along its rows that of the update.
//
// The general path takes fifteen products and two launches before them, each bound
// by the latency of a launch, first loads and an epilogue (4.3 us): eight matrices
// of 128 x 512 took it 73 us.
#include <math.h>

#include "rr_gemm.cuh"
#include "rr_orth.cuh"

namespace rr {

namespace orth {

namespace {

constexpr int kShortThreads = 256, kTile = 128 * 128;  // bytes of 64 columns by 128 rows
// NS: slices of 128 columns a CTA.
template <int NS>
struct Short {
  static constexpr int kX = 2 * NS * kTile, kS = 2 * kTile, kGot = 7 * 128 * 24 * 4;  // the most over 1 .. 8 CTAs
  static constexpr int kSmem = 1024 + kX + 2 * kS + kGot;
  static constexpr uint32_t kColumns = 128 * NS;
};
// Columns of S, in eights, that an owner adds up: sixteen over the CTAs.
constexpr int owned(int ctas) { return (16 + ctas - 1) / ctas; }
static_assert(7 * owned(7) >= 8 * owned(8) && 7 * owned(7) >= 6 * owned(6) && 7 * owned(7) >= 5 * owned(5) &&
                  7 * owned(7) >= 4 * owned(4) && 7 * owned(7) >= 3 * owned(3) && 7 * owned(7) >= 2 * owned(2),
              "their sums fit");

// The place of eight columns (8 c8 on) of a row.
__device__ __forceinline__ uint32_t swizzled(int row, int c8) {
  return (uint32_t)((c8 / 8) * kTile + row * 128 + (((c8 & 7) ^ (row & 7)) << 4));
}
// An operand along its rows whose next 64 elements are a whole tile on.
__device__ __forceinline__ uint64_t tile_rows_desc(uint32_t smem) {
  return (uint64_t)((smem >> 4) & 0x3fff) | ((uint64_t)(kTile / 16) << 16) | (64ull << 32) | (1ull << 46) | (2ull << 61);
}

__device__ __forceinline__ float load_any(const void *p, long long i, int dtype) {
  return dtype == kF32   ? static_cast<const float *>(p)[i]
         : dtype == kF16 ? __half2float(static_cast<const __half *>(p)[i])
                         : __bfloat162float(static_cast<const __nv_bfloat16 *>(p)[i]);
}
// Eight neighbours to a 16-byte aligned place.
__device__ __forceinline__ void store8_any(void *p, int dtype, const float v[8]) {
  uint4 raw[2];
  if (dtype == kF32) {
    narrow8<kF32>(v, raw);
    stg_stream(p, raw[0]), stg_stream(static_cast<char *>(p) + 16, raw[1]);
  } else {
    if (dtype == kF16) narrow8<kF16>(v, raw);
    else narrow8<kBF16>(v, raw);
    stg_stream(p, raw[0]);
  }
}
__device__ __forceinline__ void store_any(void *p, long long i, int dtype, float v) {
  if (dtype == kF32) static_cast<float *>(p)[i] = v;
  else if (dtype == kF16) static_cast<__half *>(p)[i] = __float2half_rn(v);
  else static_cast<__nv_bfloat16 *>(p)[i] = __float2bfloat16_rn(v);
}

template <int NS>
__global__ void __launch_bounds__(kShortThreads, 1) orth_short_kernel(const __grid_constant__ OrthParams p, int ctas, int eights) {
  using L = Short<NS>;
  extern __shared__ unsigned char smem_raw[];
  __shared__ Squares slots[8], sums[8];
  __shared__ __align__(8) uint64_t done;
  __shared__ uint32_t tmem_slot;
  unsigned char *smem = smem_raw + ((1024 - (smem_addr(smem_raw) & 1023)) & 1023);
  unsigned char *sx = smem, *ss = sx + L::kX, *sb = ss + L::kS;
  float *got = reinterpret_cast<float *>(sb + L::kS);
  const int warp = uniform(threadIdx.x / 32), lane = threadIdx.x % 32, row = warp % 4 * 32 + lane, half = warp / 4;
  const int rank = blockIdx.x % ctas, matrix = blockIdx.x / ctas;
  if (threadIdx.x == 0) {
    mbar_init(&done, 1);
    fence_mbar_init();
  }
  if (ctas > 1) cluster_arrive();  // waited for before the first remote store: by then every CTA runs
  if (warp == 0) tmem_alloc<1>(&tmem_slot, L::kColumns);
  tcgen05_fence_before();
  __syncthreads();
  tcgen05_fence_after();
  const uint32_t tmem = (uint32_t)uniform((int)tmem_slot), lanes = tmem + ((uint32_t)(warp % 4 * 32) << 16);
  grid_dependency_wait();
  grid_dependents_launch();

  // this thread's row of the shorter side, and its columns: eight at a time
  const bool tall = p.rows > p.cols;
  const long long m = tall ? p.cols : p.rows, n = tall ? p.rows : p.cols, n0 = (long long)rank * 128 * NS;
  const int e_in = p.dtype == kF32 ? 4 : 2, e_out = p.out_dtype == kF32 ? 4 : 2;
  const char *g = static_cast<const char *>(p.g) + matrix * p.stride_g * e_in;
  char *out = static_cast<char *>(p.out) + matrix * p.stride_out * e_out;
  constexpr int kEights = 8 * NS;  // of this thread: c8 = half * kEights + i
  const auto read = [&](int c8, float x[8]) {
    const long long c = n0 + 8 * c8;
    if (p.vec && !tall && row < m && c + 8 <= n) {
      const char *at = g + (row * p.ld_g + c) * e_in;
      uint4 raw[2];
      raw[0] = ld16(at);  // (out may be g)
      if (p.dtype == kF32) raw[1] = ld16(at + 16), widen8<kF32>(raw, x);
      else if (p.dtype == kF16) widen8<kF16>(raw, x);
      else widen8<kBF16>(raw, x);
      return;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)
      x[j] = row < m && c + j < n ? load_any(g, tall ? (c + j) * p.ld_g + row : row * p.ld_g + c + j, p.dtype) : 0.f;
  };
  Squares v{0.f, 0.f, 0.f};
#pragma unroll 4
  for (int i = 0; i < kEights; ++i) {
    float x[8];
    read(half * kEights + i, x);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float d = __fmul_rn(x[j], kDown), u = __fmul_rn(x[j], kUp);
      v.mid = __fmaf_rn(x[j], x[j], v.mid), v.big = __fmaf_rn(d, d, v.big), v.small = __fmaf_rn(u, u, v.small);
    }
  }
  v = block_sum(v, slots);
  if (ctas > 1) {
    cluster_wait();
    if (threadIdx.x < ctas) {
      const uint32_t to = cluster_addr(&sums[rank], threadIdx.x);
      asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(to), "f"(v.mid) : "memory");
      asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(to + 4), "f"(v.big) : "memory");
      asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(to + 8), "f"(v.small) : "memory");
    }
    cluster_sync_all();
    v = sums[0];
    for (int r = 1; r < ctas; ++r)
      v.mid = __fadd_rn(v.mid, sums[r].mid), v.big = __fadd_rn(v.big, sums[r].big), v.small = __fadd_rn(v.small, sums[r].small);
  }
  const Scale scale = scale_of(v, p.eps, p.dtype);
#pragma unroll 4
  for (int i = 0; i < kEights; ++i) {
    const int c8 = half * kEights + i;
    float x[8];
    read(c8, x);
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = __fmul_rn(__fmul_rn(x[j], scale.before), scale.after);
    uint4 raw;
    narrow8<kF16>(x, &raw);
    *reinterpret_cast<uint4 *>(sx + swizzled(row, c8)) = raw;
  }

  const bool one = warp == 0 && elect_one();
  const uint32_t ax = smem_addr(sx), as = smem_addr(ss), ab = smem_addr(sb);
  const int width = 8 * eights;  // columns of S that an owner adds up
  const int inverse = (256 + eights - 1) / eights;  // q / eights is q * inverse / 256 for q below 16
  unsigned turn = 0;
  bool ok = true;
  // what shared memory holds to the tensor cores, and what they made of it
  const auto multiply = [&](auto issue) {
    fence_proxy_async_smem();
    tcgen05_fence_before();
    __syncthreads();
    tcgen05_fence_after();
    if (one) {
      issue();
      tcgen05_commit<1>(&done);
    }
    __syncwarp();
    ok = mbar_wait_bounded(&done, turn & 1, ok ? kWaitLimitNs : 0) && ok;
    ++turn;
    __syncwarp();
    tcgen05_fence_after();
  };
  for (int k = 0; k < p.steps; ++k) {
    multiply([&] {
#pragma unroll
      for (int q = 0; q < 8 * NS; ++q) {
        const uint64_t d = operand_desc(ax + q / 4 * kTile + q % 4 * 32);
        gemm::mma<1>(tmem, d, d, gemm::instr_desc(0, false, false, 128, 128), q > 0);
      }
    });
    constexpr float into_s = kHeldS / (kHeldX * kHeldX);
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int first = half * 64 + c * 32;
      uint32_t acc[32];
      tmem_load32(lanes + first, acc);
      gemm::tmem_loaded32(acc);
      if (ctas > 1) {
#pragma unroll
        for (int j = 0; j < 32; j += 4) {
          const int col = first + j, owner = col / 8 * inverse >> 8;
          const uint32_t to = cluster_addr(got + rank * (128 * width) + (col - owner * width) / 4 * 512 + row * 4, owner);
          cluster_store4(to, make_uint4(acc[j], acc[j + 1], acc[j + 2], acc[j + 3]));
        }
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float s[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) s[i] = __fmul_rn(__uint_as_float(acc[8 * j + i]), into_s);
          uint4 raw;
          narrow8<kF16>(s, &raw);
          *reinterpret_cast<uint4 *>(ss + swizzled(row, first / 8 + j)) = raw;
        }
      }
    }
    if (ctas > 1) {
      cluster_sync_all();
      for (int c8 = half; c8 < eights && rank * eights + c8 < 16; c8 += 2) {
        float s[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) s[i] = 0.f;
#pragma unroll 4
        for (int r = 0; r < ctas; ++r) {
          const float4 *from = reinterpret_cast<const float4 *>(got + r * (128 * width) + c8 * 1024) + row;
          const float4 a = from[0], b = from[128];
          s[0] = __fadd_rn(s[0], a.x), s[1] = __fadd_rn(s[1], a.y), s[2] = __fadd_rn(s[2], a.z), s[3] = __fadd_rn(s[3], a.w);
          s[4] = __fadd_rn(s[4], b.x), s[5] = __fadd_rn(s[5], b.y), s[6] = __fadd_rn(s[6], b.z), s[7] = __fadd_rn(s[7], b.w);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) s[i] = __fmul_rn(s[i], into_s);
        uint4 raw;
        narrow8<kF16>(s, &raw);
        const unsigned char *to = ss + swizzled(row, rank * eights + c8);
#pragma unroll 4
        for (int r = 0; r < ctas; ++r) cluster_store4(cluster_addr(to, r), raw);
      }
      cluster_sync_all();
    }
    // b S + c S^2
    multiply([&] {
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const uint64_t d = operand_desc(as + q / 4 * kTile + q % 4 * 32);
        gemm::mma<1>(tmem, d, d, gemm::instr_desc(0, false, false, 128, 128), q > 0);
      }
    });
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int first = half * 64 + c * 32;
      uint32_t acc[32];
      tmem_load32(lanes + first, acc);
      gemm::tmem_loaded32(acc);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t at = swizzled(row, first / 8 + j);
        const uint4 old = *reinterpret_cast<const uint4 *>(ss + at);
        float w[8], s[8];
        widen8<kF16>(&old, s);
#pragma unroll
        for (int i = 0; i < 8; ++i)
          w[i] = __fmaf_rn(s[i], kB * kHeldB / kHeldS, __fmul_rn(__uint_as_float(acc[8 * j + i]), kC * kHeldB / (kHeldS * kHeldS)));
        uint4 raw;
        narrow8<kF16>(w, &raw);
        *reinterpret_cast<uint4 *>(sb + at) = raw;
      }
    }
    // a X + (b S + c S^2) X
    multiply([&] {
#pragma unroll
      for (int q = 0; q < 8; ++q)
        gemm::mma<1>(tmem, operand_desc(ab + q / 4 * kTile + q % 4 * 32), tile_rows_desc(ax + q * 2048),
                     gemm::instr_desc(0, false, true, 128, 128 * NS), q > 0);
    });
    const bool last = k + 1 == p.steps;
#pragma unroll
    for (int c = 0; c < 2 * NS; ++c) {
      const int first = half * 64 * NS + c * 32;
      uint32_t acc[32];
      tmem_load32(lanes + first, acc);
      gemm::tmem_loaded32(acc);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        unsigned char *at = sx + swizzled(row, first / 8 + j);
        const uint4 old = *reinterpret_cast<const uint4 *>(at);
        float x[8];
        widen8<kF16>(&old, x);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = __fmaf_rn(x[i], kA, __fmul_rn(__uint_as_float(acc[8 * j + i]), 1.f / kHeldB));
        if (!last) {
          uint4 raw;
          narrow8<kF16>(x, &raw);
          *reinterpret_cast<uint4 *>(at) = raw;
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) x[i] = __fmul_rn(x[i], 1.f / kHeldX);
          const long long col = n0 + first + 8 * j;
          if (tall) {
            // (a warp's rows are neighbours in memory)
#pragma unroll
            for (int i = 0; i < 8; ++i)
              if (row < m && col + i < n && ok) store_any(out, (col + i) * p.ld_out + row, p.out_dtype, x[i]);
          } else if (p.vec_out && col + 8 <= n) {
            if (row < m && ok) store8_any(out + (row * p.ld_out + col) * e_out, p.out_dtype, x);
          } else {
            // eight columns of 32 rows, turned so that eight lanes take neighbours
            float *stage = got + warp * (32 * 9);
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 8; ++i) stage[lane * 9 + i] = x[i];
            __syncwarp();
            const long long at = col + lane % 8;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const int r = 4 * i + lane / 8, to = warp % 4 * 32 + r;
              if (to < m && at < n && ok) store_any(out, to * p.ld_out + at, p.out_dtype, stage[r * 9 + lane % 8]);
            }
          }
        }
      }
    }
  }
  if (!ok) {
    // the products end before tensor memory is given back
    if (lane == 0) atomicOr(p.status, kStatusWaitTimeout);
    mbar_wait_bounded(&done, (turn - 1) & 1, kWaitLimitNs);
  }
  tcgen05_fence_before();
  __syncthreads();
  tcgen05_fence_after();
  if (warp == 0) tmem_free<1>(tmem, L::kColumns);
}

template <int NS>
cudaError_t launch_short_of(const OrthParams &p, int ctas, cudaStream_t s) {
  using L = Short<NS>;
  const cudaError_t err = allow_smem<orth_short_kernel<NS>>(L::kSmem);
  if (err != cudaSuccess) return err;
  cudaLaunchConfig_t c = {};
  c.gridDim = dim3((unsigned)(ctas * p.batch));
  c.blockDim = dim3(kShortThreads);
  c.dynamicSmemBytes = L::kSmem;
  c.stream = s;
  cudaLaunchAttribute at[2] = {};
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = (unsigned)ctas, at[1].val.clusterDim.y = 1, at[1].val.clusterDim.z = 1;
  c.attrs = at;
  c.numAttrs = 2;
  return cudaLaunchKernelEx(&c, orth_short_kernel<NS>, p, ctas, owned(ctas));
}

}  // namespace

}  // namespace orth

bool orth_is_short(long long rows, long long cols) {
  return (rows < cols ? rows : cols) <= 128 && (rows < cols ? cols : rows) <= 8 * 256;
}

cudaError_t launch_orth_short(const OrthParams &p, cudaStream_t s) {
  const long long n = p.rows < p.cols ? p.cols : p.rows;
  return n <= 8 * 128 ? orth::launch_short_of<1>(p, (int)ceil_div(n, 128ll), s)
                      : orth::launch_short_of<2>(p, (int)ceil_div(n, 256ll), s);
}

}  // namespace rr
