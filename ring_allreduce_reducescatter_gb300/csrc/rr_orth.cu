// rr_orth.cu -- an update brought near the orthogonal matrix that has its
// singular vectors (Muon's Newton-Schulz iteration; Jordan et al., "Muon: An
// optimizer for hidden layers in neural networks", 2024):
//   X = G / (|G| + eps); five (or more) times X <- a X + (b S + c S^2) X with
//   S = X X^T (where G is tall, X <- a X + X (b S + c S^2) with S = X^T X),
// (a, b, c) = (3.4445, -4.7750, 2.0315): every singular value s goes to a s + b
// s^3 + c s^5, which brings (0.003, 1] to about 0.7 .. 1.2 in five turns.
//
// Each turn is three products on the tensor cores.  S and S^2 are symmetric:
// their tiles above the diagonal are computed and stored twice, so a square turn
// costs 4 n^3 operations for 6 n^3.  Where a product sums over the other axis of
// X it reads X along its rows; no transpose is ever made.
//
// The iterates are held in binary16, which has eight times bfloat16's precision
// and whose range they cannot leave: |X| <= 1 in the Frobenius norm at the
// start and every singular value stays below 1.21.  X is held times 2^6, S times
// 2^14, b S + c S^2 times 2^13, so that the entries of large matrices (S of a
// 4096 x 4096 starts at 2^-12 on and 2^-18 off the diagonal) stay above the
// subnormals; none of the three reaches 2^15.  Sums and the terms around them are
// in binary32.  On gradients of a few strong directions and noise the five turns
// leave 0.0013 of the result (0.011 with bfloat16's rounding).
//
// Bound by the tensor cores: 4096 x 4096 is 1.37 TFLOP over 67 MB.
#include <math.h>

#include "rr_gemm.cuh"
#include "rr_orth.cuh"

namespace rr {

namespace {

using namespace orth;

// Eight columns of a row, zeros past the last.
template <int DT>
__device__ __forceinline__ void eight(const OrthParams &p, const typename Fmt<DT>::type *row, long long c, float x[8]) {
  if (p.vec && c + 8 <= p.cols) {
    uint4 raw[kRaw8<DT>];
#pragma unroll
    for (int j = 0; j < kRaw8<DT>; ++j) raw[j] = ldg_stream(reinterpret_cast<const uint4 *>(row + c) + j);
    widen8<DT>(raw, x);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = c + j < p.cols ? to_f32<DT>(row[c + j]) : 0.f;
  }
}
// Group i of `each` a row: its row.
__device__ __forceinline__ long long row_of(long long i, long long each) {
  return i < 0x7fffffff ? (long long)((unsigned)i / (unsigned)each) : i / each;
}

// blockIdx.x: one of p.parts parts of a matrix; blockIdx.y: the matrix.
template <int DT>
__global__ void __launch_bounds__(256) orth_squares_kernel(const __grid_constant__ OrthParams p) {
  using T = typename Fmt<DT>::type;
  __shared__ Squares slots[8];
  grid_dependency_wait();
  grid_dependents_launch();
  const T *g = static_cast<const T *>(p.g) + blockIdx.y * p.stride_g;
  const long long each = (p.cols + 7) / 8, all = each * p.rows, step = (long long)p.parts * 256;
  Squares v{0.f, 0.f, 0.f};
#pragma unroll 4
  for (long long i = blockIdx.x * 256ll + threadIdx.x; i < all; i += step) {
    const long long row = row_of(i, each);
    float x[8];
    eight<DT>(p, g + row * p.ld_g, (i - row * each) * 8, x);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      v.mid = __fmaf_rn(x[j], x[j], v.mid);
      if constexpr (DT != kF16) {
        const float d = __fmul_rn(x[j], kDown), u = __fmul_rn(x[j], kUp);
        v.big = __fmaf_rn(d, d, v.big), v.small = __fmaf_rn(u, u, v.small);
      }
    }
  }
  v = block_sum(v, slots);
  if (threadIdx.x == 0) {
    float *out = p.norms + (blockIdx.y * (long long)p.parts + blockIdx.x) * 3;
    out[0] = v.mid, out[1] = v.big, out[2] = v.small;
  }
}

// X = G / (|G| + eps) in the form it is held in, zeros behind its rows and columns.
template <int DT>
__global__ void __launch_bounds__(256) orth_start_kernel(const __grid_constant__ OrthParams p) {
  using T = typename Fmt<DT>::type;
  __shared__ Squares slots[8];
  grid_dependency_wait();
  grid_dependents_launch();
  Squares v{0.f, 0.f, 0.f};
  const float *part = p.norms + blockIdx.y * (long long)p.parts * 3;
  for (int i = threadIdx.x; i < p.parts; i += 256)
    v.mid = __fadd_rn(v.mid, part[3 * i]), v.big = __fadd_rn(v.big, part[3 * i + 1]), v.small = __fadd_rn(v.small, part[3 * i + 2]);
  v = block_sum(v, slots);
  const Scale scale = scale_of(v, p.eps, DT);
  const T *g = static_cast<const T *>(p.g) + blockIdx.y * p.stride_g;
  __half *x = static_cast<__half *>(p.x[0]) + blockIdx.y * p.stride_x;
  const long long each = p.ld_x / 8, all = each * p.held_rows, step = gridDim.x * 256ll;
#pragma unroll 2
  for (long long i = blockIdx.x * 256ll + threadIdx.x; i < all; i += step) {
    const long long row = row_of(i, each), c = (i - row * each) * 8;
    float w[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] = 0.f;
    if (row < p.rows && c < p.cols) eight<DT>(p, g + row * p.ld_g, c, w);
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] = __fmul_rn(__fmul_rn(w[j], scale.before), scale.after);
    uint4 raw;
    narrow8<kF16>(w, &raw);
    *reinterpret_cast<uint4 *>(x + row * p.ld_x + c) = raw;
  }
}

// alpha D + beta C to storage; of a symmetric D also its mirror image.
template <int DT>
struct Combined {
  static constexpr int kRun = 0;
  struct Params {
    gemm::Out out;
    long long out_stride;
    const __half *c;  // null: none
    long long ld_c, c_stride;
    float alpha, beta;
    int tile;  // rows of a tile of a symmetric D (else 0)
    int half;  // columns of an epilogue
  };
  const Params &p;
  gemm::Out out;
  const __half *c0;
  long long row, col;
  float *stage;
  bool mirror;
  uint4 next[4];  // C's chunk that comes next, on its way since the one before
  __device__ __forceinline__ Combined(const Params &p, long long row, long long col, int batch, float *stage)
      : p(p), out(p.out), c0(p.c ? p.c + batch * p.c_stride + row * p.ld_c + col : nullptr), row(row), col(col), stage(stage),
        mirror(p.tile && row / p.tile != col / p.tile) {
    out.at = static_cast<typename Fmt<DT>::type *>(p.out.at) + batch * p.out_stride;
    fetch(0);
  }
  // (C's rows are whole chunks)
  __device__ __forceinline__ void fetch(int c) {
    if (!c0 || row >= out.rows || col + c * gemm::kChunk >= out.cols) return;
    ldg32(c0 + c * gemm::kChunk, next[0], next[1]);
    ldg32(c0 + c * gemm::kChunk + 16, next[2], next[3]);
  }
  __device__ __forceinline__ void chunk(int c, float v[gemm::kChunk]) {
    const long long at = col + c * gemm::kChunk;
    if (at >= out.cols) return;
#pragma unroll
    for (int j = 0; j < gemm::kChunk; ++j) v[j] = __fmul_rn(v[j], p.alpha);
    if (c0 && row < out.rows) {
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        float w[8];
        widen8<kF16>(next + h, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[8 * h + j] = __fmaf_rn(w[j], p.beta, v[8 * h + j]);
      }
      if ((c + 1) * gemm::kChunk < p.half) fetch(c + 1);
    }
    gemm::store_row<DT>(out, row, at, v, stage);
    if (mirror && row < out.rows) {
      typename Fmt<DT>::type *q = static_cast<typename Fmt<DT>::type *>(out.at) + at * out.ld + row;
#pragma unroll
      for (int j = 0; j < gemm::kChunk; ++j, q += out.ld)
        if (at + j < out.rows) *q = from_f32<DT>(v[j]);
    }
  }
  __device__ __forceinline__ void end() {}
};

template <class... P, class... Args>
cudaError_t launch(void (*k)(P...), dim3 grid, int block, cudaStream_t s, const Args &...args) {
  cudaLaunchConfig_t c = {};
  c.gridDim = grid;
  c.blockDim = dim3((unsigned)block);
  c.stream = s;
  cudaLaunchAttribute a = {};
  a.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  a.val.programmaticStreamSerializationAllowed = 1;
  c.attrs = &a;
  c.numAttrs = 1;
  return cudaLaunchKernelEx(&c, k, args...);
}

template <int DT>
cudaError_t start(const OrthParams &p, cudaStream_t s) {
  cudaError_t e = launch(orth_squares_kernel<DT>, dim3((unsigned)p.parts, p.batch), 256, s, p);
  if (e != cudaSuccess) return e;
  const long long groups = ceil_div(p.held_rows * (p.ld_x / 8), 256ll), most = 8ll * p.sms;
  return launch(orth_start_kernel<DT>, dim3((unsigned)(groups < most ? groups : most), p.batch), 256, s, p);
}

template <bool kMnA, bool kMnB, int DT>
cudaError_t product(const OrthParams &p, const gemm::Operand &a, const gemm::Operand &b, bool upper,
                    typename Combined<DT>::Params e, cudaStream_t s) {
  int split;
  const gemm::Kind kind = gemm::kind_of(a.rows, b.rows, a.k, b.batch, upper, p.sms, &split);
  if (upper) e.tile = kind == gemm::kPair ? 256 : 128;
  e.half = kind == gemm::kPair ? gemm::Pair::kHalf : kind == gemm::kSingle ? gemm::Single::kHalf : gemm::kChunk;
  return gemm::launch_product<kMnA, kMnB, Combined<DT>>(a, b, upper, 0, p.status, p.sms, e, s);
}

// X <- a X + (b S + c S^2) X, or the same from the right, to `out`.
template <int DT>
cudaError_t update(const OrthParams &p, const void *x, const gemm::Out &out, long long out_stride, float alpha, float beta,
                   cudaStream_t s) {
  using gemm::Operand;
  const long long m = p.held_rows < p.held_cols ? p.held_rows : p.held_cols;
  const typename Combined<DT>::Params e{out, out_stride, static_cast<const __half *>(x), p.ld_x, p.stride_x, alpha, beta, 0, 0};
  const Operand poly{p.b, m, m, p.ld_s, p.stride_s, p.batch, false};
  if (p.rows > p.cols) {
    const Operand along{x, p.held_rows, p.held_cols, p.ld_x, p.stride_x, p.batch, false};
    return product<false, false, DT>(p, along, poly, false, e, s);
  }
  const Operand across{x, p.held_cols, p.held_rows, p.ld_x, p.stride_x, p.batch, true};
  return product<false, true, DT>(p, poly, across, false, e, s);
}

}  // namespace

cudaError_t launch_orth(const OrthParams &p, cudaStream_t s) {
  using gemm::Operand;
  using gemm::Out;
  if (orth_is_short(p.rows, p.cols)) return launch_orth_short(p, s);
  cudaError_t err = p.dtype == kF32 ? start<kF32>(p, s) : p.dtype == kF16 ? start<kF16>(p, s) : start<kBF16>(p, s);
  const bool tall = p.rows > p.cols;
  const long long m = tall ? p.held_cols : p.held_rows;
  const Out held_s{p.s, m, p.ld_s, p.ld_s, true}, held_b{p.b, m, p.ld_s, p.ld_s, true};
  const float into_s = kHeldS / (kHeldX * kHeldX);
  for (int k = 0; k < p.steps && err == cudaSuccess; ++k) {
    const void *x = p.x[k & 1];
    const Combined<kF16>::Params es{held_s, p.stride_s, nullptr, 0, 0, into_s, 0.f, 0, 0};
    if (tall) {
      const Operand across{x, p.held_cols, p.held_rows, p.ld_x, p.stride_x, p.batch, true};
      err = product<true, true, kF16>(p, across, across, true, es, s);
    } else {
      const Operand along{x, p.held_rows, p.held_cols, p.ld_x, p.stride_x, p.batch, false};
      err = product<false, false, kF16>(p, along, along, true, es, s);
    }
    if (err != cudaSuccess) return err;
    const Operand gram{p.s, m, m, p.ld_s, p.stride_s, p.batch, false};
    const Combined<kF16>::Params eb{held_b, p.stride_s, static_cast<const __half *>(p.s), p.ld_s, p.stride_s,
                                    kC * kHeldB / (kHeldS * kHeldS), kB * kHeldB / kHeldS, 0, 0};
    if ((err = product<false, false, kF16>(p, gram, gram, true, eb, s)) != cudaSuccess) return err;
    if (k + 1 < p.steps) {
      err = update<kF16>(p, x, Out{p.x[(k + 1) & 1], p.held_rows, p.ld_x, p.ld_x, true}, p.stride_x, 1.f / kHeldB, kA, s);
    } else {
      const int bytes = p.out_dtype == kF32 ? 4 : 2;
      const bool vec32 = reinterpret_cast<uintptr_t>(p.out) % 32 == 0 && p.ld_out * bytes % 32 == 0 &&
                         (p.batch == 1 || p.stride_out * bytes % 32 == 0);
      const Out out{p.out, p.rows, p.cols, p.ld_out, vec32};
      const float alpha = 1.f / (kHeldB * kHeldX), beta = kA / kHeldX;
      err = p.out_dtype == kF32   ? update<kF32>(p, x, out, p.stride_out, alpha, beta, s)
            : p.out_dtype == kF16 ? update<kF16>(p, x, out, p.stride_out, alpha, beta, s)
                                  : update<kBF16>(p, x, out, p.stride_out, alpha, beta, s);
    }
  }
  return err;
}

}  // namespace rr
