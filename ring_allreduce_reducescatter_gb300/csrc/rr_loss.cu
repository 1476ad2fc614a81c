// rr_loss.cu -- the softmax cross entropy of logits l = x W^T that are never
// stored:
//   lse[t] = log(sum_v exp(l[t, v])), loss[t] = lse[t] - l[t, target[t]].
// The product's epilogue keeps, of a row and 128 (64) columns, the maximum and
// the sum of exponentials around it, 8 bytes for 256 of logits, and the target's
// logit where it passes; loss_rows_kernel joins them.  The product bounds it: for
// 8192 tokens by 32000 by 4096, 2.1 TFLOP of tensor work for 16 MB of sums.
#include <math.h>

#include "rr_gemm.cuh"
#include "rr_loss.h"

namespace rr {

namespace {

constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// exp(a - b) for b >= a or b finite: 0 where a is minus infinity, whatever b.
__device__ __forceinline__ float exp_above(float a, float b) {
  return a == -INFINITY ? 0.f : ex2(__fmul_rn(__fsub_rn(a, b), kLog2e));
}

struct Statistics {
  static constexpr int kRun = 8;  // 512 elements of K (whole, a loss of 8 was off by 1e-5 at 4096)
  struct Params {
    const long long *target;
    float2 *parts;
    float *chosen;
    long long tokens, vocabulary, group;
  };
  const Params &p;
  long long row, col, at;
  float top, sum;
  __device__ __forceinline__ Statistics(const Params &p, long long row, long long col, int, float *)
      : p(p), row(row), col(col), at(row < p.tokens ? p.target[row] : -1), top(-INFINITY), sum(0.f) {}
  // One pass with a running maximum: the sum so far is scaled down where it rises.
  __device__ __forceinline__ void chunk(int c, float v[gemm::kChunk]) {
    const long long first = col + c * gemm::kChunk;
    if (first >= p.vocabulary) return;
    if (at >= first && at < first + gemm::kChunk && at < p.vocabulary) {
      const int j0 = (int)(at - first);
#pragma unroll
      for (int j = 0; j < gemm::kChunk; ++j)
        if (j == j0) p.chosen[row] = v[j];
    }
    if (first + gemm::kChunk > p.vocabulary) {
#pragma unroll
      for (int j = 0; j < gemm::kChunk; ++j) v[j] = first + j < p.vocabulary ? v[j] : -INFINITY;
    }
    float m[4] = {v[0], v[1], v[2], v[3]};
#pragma unroll
    for (int j = 4; j < gemm::kChunk; ++j) m[j % 4] = fmaxf(m[j % 4], v[j]);
    const float high = fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
    if (high > top) sum = __fmul_rn(sum, exp_above(top, high)), top = high;
    // (with nothing above minus infinity yet, every term is 0: around 0, not around top)
    const float around = top == -INFINITY ? 0.f : top;
    float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int j = 0; j < gemm::kChunk; ++j) s[j % 4] = __fadd_rn(s[j % 4], ex2(__fmul_rn(__fsub_rn(v[j], around), kLog2e)));
    sum = __fadd_rn(sum, __fadd_rn(__fadd_rn(s[0], s[1]), __fadd_rn(s[2], s[3])));
  }
  __device__ __forceinline__ void end() {
    if (row < p.tokens && col < p.vocabulary) p.parts[col / p.group * p.tokens + row] = make_float2(top, sum);
  }
};

// The groups of a row joined: kRows rows a CTA of 256 threads, 256 / kRows
// threads each a part of a row's groups, joined in a fixed tree (one thread that
// joined 256 parts in turn took 12 us).
struct Part {
  float top, sum;
  __device__ __forceinline__ void join(float top2, float sum2) {
    if (top2 > top) sum = __fmul_rn(sum, exp_above(top, top2)), top = top2;
    // (a sum that is no number stays one, whatever its maximum)
    sum = sum2 == sum2 ? __fadd_rn(sum, __fmul_rn(sum2, exp_above(top2, top))) : sum2;
  }
};
template <int kRows>
__global__ void __launch_bounds__(256) loss_rows_kernel(const __grid_constant__ LossParams p, long long groups) {
  constexpr int kEach = 256 / kRows;
  __shared__ Part got[8][kRows];
  grid_dependency_wait();
  grid_dependents_launch();
  const int r = threadIdx.x % kRows, g0 = threadIdx.x / kRows;
  const long long row = (long long)blockIdx.x * kRows + r, tokens = p.x.rows;
  Part v{-INFINITY, 0.f};
  if (row < tokens) {
#pragma unroll 4
    for (long long g = g0; g < groups; g += kEach) {
      const float2 w = p.parts[g * tokens + row];
      v.join(w.x, w.y);
    }
  }
#pragma unroll
  for (int d = 16; d >= kRows; d /= 2) {
    const float top = __shfl_xor_sync(0xffffffffu, v.top, d), sum = __shfl_xor_sync(0xffffffffu, v.sum, d);
    v.join(top, sum);
  }
  if (threadIdx.x % 32 < kRows) got[threadIdx.x / 32][r] = v;
  __syncthreads();
  if (g0 != 0 || row >= tokens) return;
#pragma unroll
  for (int q = 1; q < 8; ++q) v.join(got[q][r].top, got[q][r].sum);
  const float lse = v.top == -INFINITY ? (v.sum == v.sum ? -INFINITY : v.sum) : __fadd_rn(v.top, logf(v.sum));
  const long long t = p.target[row];
  const bool valid = t >= 0 && t < p.w.rows;
  if (p.lse) p.lse[row] = lse;
  p.loss[row] = t == p.ignore ? 0.f : valid ? __fsub_rn(lse, p.chosen[row]) : NAN;
}

// sums: the losses' total, how many tokens count, and the mean over those (0
// with none), by one CTA in a fixed order.
__global__ void __launch_bounds__(1024) loss_sums_kernel(const __grid_constant__ LossParams p) {
  __shared__ float totals[32];
  __shared__ int counts[32];
  grid_dependency_wait();
  grid_dependents_launch();
  float total = 0.f;
  int count = 0;
#pragma unroll 4
  for (long long t = threadIdx.x; t < p.x.rows; t += 1024) {
    total = __fadd_rn(total, p.loss[t]);
    count += p.target[t] != p.ignore;
  }
#pragma unroll
  for (int d = 16; d > 0; d /= 2) {
    total = __fadd_rn(total, __shfl_xor_sync(0xffffffffu, total, d));
    count += __shfl_xor_sync(0xffffffffu, count, d);
  }
  if (threadIdx.x % 32 == 0) totals[threadIdx.x / 32] = total, counts[threadIdx.x / 32] = count;
  __syncthreads();
  if (threadIdx.x != 0) return;
  for (int w = 1; w < 32; ++w) total = __fadd_rn(total, totals[w]), count += counts[w];
  p.sums[0] = total, p.sums[1] = (float)count;
  p.sums[2] = count ? __fdiv_rn(total, (float)count) : 0.f;
}

// The factors of the rows of the logits' gradient for tokens that have gradients of
// their own: over a common power of two, that of the largest, 0 for a token that
// does not count and NaN for a target outside the vocabulary.  The outputs get the
// power of two back.
__global__ void __launch_bounds__(1024) loss_factors_kernel(const __grid_constant__ LossGradParams p) {
  __shared__ float tops[32];
  grid_dependency_wait();
  grid_dependents_launch();
  const long long tokens = p.x.rows;
  const float widen = p.dtype == kF16 ? kLossWiden : 1.f;
  float top = 0.f;
#pragma unroll 4
  for (long long t = threadIdx.x; t < tokens; t += 1024)
    if (p.target[t] != p.ignore) top = fmaxf(top, fabsf(p.grad[t]));
#pragma unroll
  for (int d = 16; d > 0; d /= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
  if (threadIdx.x % 32 == 0) tops[threadIdx.x / 32] = top;
  __syncthreads();
  for (int w = 0; w < 32; ++w) top = fmaxf(top, tops[w]);
  // 2^k with top <= 2^k, k in -100 .. 100; 1 where there is nothing to scale
  int k = 0;
  if (top > 0.f && top < INFINITY) frexpf(top, &k);
  k = k < -100 ? -100 : k > 100 ? 100 : k;
  const float down = __fmul_rn(__int_as_float((127 - k) << 23), widen), up = __fdiv_rn(__int_as_float((127 + k) << 23), widen);
#pragma unroll 4
  for (long long t = threadIdx.x; t < tokens; t += 1024) {
    const long long at = p.target[t];
    p.factors[t] = at == p.ignore ? 0.f : at >= 0 && at < p.w.rows ? __fmul_rn(p.grad[t], down) : NAN;
  }
  if (threadIdx.x == 0) p.factors[tokens] = up;
}

// A copy in rows of ld_to, for operands that tensor copies do not read as they lie:
// eight elements a thread, put together from the aligned 16-byte groups around them
// where those lie inside the matrix.  blockIdx.y: which of the copies.
__global__ void __launch_bounds__(256) pad_kernel(const __grid_constant__ PadParams both) {
  grid_dependency_wait();
  grid_dependents_launch();
  const Pad &p = both.copy[blockIdx.y];
  const uint16_t *from = static_cast<const uint16_t *>(p.from);
  uint16_t *to = static_cast<uint16_t *>(p.to);
  const uintptr_t lo = reinterpret_cast<uintptr_t>(from), hi = lo + (uintptr_t)(((p.rows - 1) * p.ld_from + p.cols) * 2);
  const long long each = p.ld_to / 8, all = each * p.rows_to, step = gridDim.x * 256ll;
#pragma unroll 2
  for (long long i = blockIdx.x * 256ll + threadIdx.x; i < all; i += step) {
    const long long row = i < 0x7fffffff ? (long long)((unsigned)i / (unsigned)each) : i / each, c = (i - row * each) * 8;
    uint4 v = make_uint4(0, 0, 0, 0);
    if (row < p.rows) {
      const uint16_t *at = from + row * p.ld_from + c;
      const uintptr_t a = reinterpret_cast<uintptr_t>(at), group = a & ~(uintptr_t)15;
      if (c + 8 <= p.cols && group >= lo && group + 32 <= hi) {
        v = funnel16(ldg_l1(reinterpret_cast<const void *>(group)), ldg_l1(reinterpret_cast<const void *>(group + 16)), (int)(a & 15));
      } else {
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t x = c + 2 * j < p.cols ? at[2 * j] : 0, y = c + 2 * j + 1 < p.cols ? at[2 * j + 1] : 0;
          w[j] = x | y << 16;
        }
        v = make_uint4(w[0], w[1], w[2], w[3]);
      }
    }
    *reinterpret_cast<uint4 *>(to + row * p.ld_to + c) = v;
  }
}

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

}  // namespace

cudaError_t launch_pad(const PadParams &p, cudaStream_t s) {
  long long groups = 0;
  for (int i = 0; i < p.n; ++i) {
    const long long each = ceil_div(p.copy[i].rows_to * (p.copy[i].ld_to / 8), 256ll);
    groups = groups > each ? groups : each;
  }
  return launch(pad_kernel, dim3((unsigned)(groups < 2048 ? groups : 2048), (unsigned)p.n), 256, s, p);
}

cudaError_t launch_loss(const LossParams &p, cudaStream_t s) {
  const long long tokens = p.x.rows, vocabulary = p.w.rows, group = loss_group(tokens), groups = ceil_div(vocabulary, group);
  if (tokens == 0) return launch(loss_sums_kernel, dim3(1), 1024, s, p);
  const gemm::Operand a{p.x.at, p.x.padded, p.hidden, p.x.ld, 0, 1, false}, b{p.w.at, vocabulary, p.hidden, p.w.ld, 0, 1, false};
  const Statistics::Params e{p.target, p.parts, p.chosen, tokens, vocabulary, group};
  // (groups of columns go by the tiles' width: the tokens alone choose)
  const uint32_t format = p.dtype == kBF16;
  cudaError_t err =
      loss_pairs(tokens) ? gemm::launch_shape<gemm::product_pair_kernel<false, false, Statistics>, gemm::Pair, 2>(
                               a, b, false, format, p.status, p.sms, e, s)
                         : gemm::launch_shape<gemm::product_single_kernel<false, false, Statistics>, gemm::Single, 1>(
                               a, b, false, format, p.status, p.sms, e, s);
  if (err != cudaSuccess) return err;
  // few rows: a CTA on each (one token of 131072 has 2048 groups)
  err = tokens <= 4 * p.sms ? launch(loss_rows_kernel<1>, dim3((unsigned)tokens), 256, s, p, groups)
                            : launch(loss_rows_kernel<8>, dim3((unsigned)ceil_div(tokens, 8ll)), 256, s, p, groups);
  if (err != cudaSuccess || !p.sums) return err;
  return launch(loss_sums_kernel, dim3(1), 1024, s, p);
}

cudaError_t launch_loss_factors(const LossGradParams &p, cudaStream_t s) {
  return launch(loss_factors_kernel, dim3(1), 1024, s, p);
}

}  // namespace rr
