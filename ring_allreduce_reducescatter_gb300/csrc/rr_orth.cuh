// rr_orth.cuh -- what the two paths of the orthogonalised update share: its
// constants and the scale of a matrix.
#pragma once

#include <math.h>

#include "rr_mx4.cuh"
#include "rr_orth.h"

namespace rr {

namespace orth {

constexpr float kA = 3.4445f, kB = -4.7750f, kC = 2.0315f;
constexpr float kHeldX = 64.f, kHeldS = 16384.f, kHeldB = 8192.f;  // what each is held times

// Sums of squares of x, x 2^-60 and x 2^60: one of them neither overflows nor
// loses its terms, whatever the matrix's scale.
constexpr float kDown = 0x1p-60f, kUp = 0x1p60f;

struct Squares {
  float mid, big, small;
};
__device__ __forceinline__ Squares block_sum(Squares v, Squares *slots) {
#pragma unroll
  for (int d = 16; d > 0; d /= 2) {
    v.mid = __fadd_rn(v.mid, __shfl_xor_sync(0xffffffffu, v.mid, d));
    v.big = __fadd_rn(v.big, __shfl_xor_sync(0xffffffffu, v.big, d));
    v.small = __fadd_rn(v.small, __shfl_xor_sync(0xffffffffu, v.small, d));
  }
  if (threadIdx.x % 32 == 0) slots[threadIdx.x / 32] = v;
  __syncthreads();
  v = slots[0];
#pragma unroll
  for (int w = 1; w < 8; ++w) {
    v.mid = __fadd_rn(v.mid, slots[w].mid);
    v.big = __fadd_rn(v.big, slots[w].big);
    v.small = __fadd_rn(v.small, slots[w].small);
  }
  return v;
}

// What brings a matrix with these sums to |X| = kHeldX: x times `before` times `after`.
struct Scale {
  float before, after;
};
__device__ __forceinline__ Scale scale_of(const Squares &v, float eps, int dtype) {
  const bool big = dtype != kF16 && !(v.mid < 1e30f), small = dtype != kF16 && v.mid < 1e-20f;
  const float before = big ? kDown : small ? kUp : 1.f;
  const float norm = __fadd_rn(__fsqrt_rn(big ? v.big : small ? v.small : v.mid), __fmul_rn(eps, before));
  return Scale{before, __fdiv_rn(kHeldX, norm)};
}

}  // namespace orth

}  // namespace rr
