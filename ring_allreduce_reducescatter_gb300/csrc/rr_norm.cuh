// rr_norm.cuh -- layer norm and its backward pass, over the rows of a matrix:
//   mean = sum(x) / n, rstd = 1 / sqrt(sum((x - mean)^2) / n + eps),
//   h = (x - mean) rstd, y = h weight + bias;
//   g = dy weight, dx = (g - sum(g) / n - h sum(g h) / n) rstd,
//   dweight = sum over rows of dy h, dbias = sum over rows of dy.
// All arithmetic is in binary32 with one rounding to storage.  The variance is
// summed around the mean (a second pass over the row in registers): the
// difference of the squares' mean and the mean's square loses every digit where
// the mean is large.  Everything here is bound by memory: x is read once and y
// written once, and in the backward pass x and dy are read once and dx written
// once; a row stays in the registers of 32 to 1024 threads between its passes.
#pragma once

#include "rr_mx4.cuh"
#include "rr_norm.h"

namespace rr {

namespace norm {

// Elements a thread takes at a time: 16 bytes, or one where rows are not aligned.
template <int DT, bool kVec>
constexpr int kWide = kVec ? 16 / Fmt<DT>::bytes : 1;

// kN elements in storage and in binary32.
template <int DT, int kN>
struct Raw {
  static constexpr int kWords = kN * Fmt<DT>::bytes >= 4 ? kN * Fmt<DT>::bytes / 4 : 1;
  uint32_t w[kWords];
};
template <int DT, int kN>
__device__ __forceinline__ void zero(Raw<DT, kN> &r) {
#pragma unroll
  for (int j = 0; j < Raw<DT, kN>::kWords; ++j) r.w[j] = 0;
}
// What is read once (and may be the output): no L1 allocation, not the read-only path.
template <int DT, int kN>
__device__ __forceinline__ Raw<DT, kN> load_stream(const void *base, long long at) {
  using T = typename Fmt<DT>::type;
  Raw<DT, kN> r;
  const T *p = static_cast<const T *>(base) + at;
  if constexpr (kN == 1) {
    T v = *p;
    r.w[0] = 0;
    memcpy(r.w, &v, sizeof(T));
  } else {
    const uint4 v = ld16_stream(p);
    r.w[0] = v.x, r.w[1] = v.y, r.w[2] = v.z, r.w[3] = v.w;
  }
  return r;
}
template <int DT, int kN>
__device__ __forceinline__ void widen(const Raw<DT, kN> &r, float v[kN]) {
  if constexpr (kN == 1) {
    typename Fmt<DT>::type t;
    memcpy(&t, r.w, sizeof(t));
    v[0] = to_f32<DT>(t);
  } else if constexpr (DT == kF32) {
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = __uint_as_float(r.w[j]);
  } else {
    const uint4 u = make_uint4(r.w[0], r.w[1], r.w[2], r.w[3]);
    widen8<DT>(&u, v);
  }
}
// 16 bytes from shared memory.
template <int DT>
__device__ __forceinline__ void widen_shared(const unsigned char *from, float v[16 / Fmt<DT>::bytes]) {
  const uint4 u = *reinterpret_cast<const uint4 *>(from);
  Raw<DT, 16 / Fmt<DT>::bytes> r;
  r.w[0] = u.x, r.w[1] = u.y, r.w[2] = u.z, r.w[3] = u.w;
  widen<DT, 16 / Fmt<DT>::bytes>(r, v);
}
template <int DT, int kN>
__device__ __forceinline__ void store(void *base, long long at, const float v[kN]) {
  using T = typename Fmt<DT>::type;
  T *p = static_cast<T *>(base) + at;
  if constexpr (kN == 1) {
    *p = from_f32<DT>(v[0]);
  } else if constexpr (DT == kF32) {
    stg_stream(p, make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])));
  } else {
    uint4 u;
    narrow8<DT>(v, &u);
    stg_stream(p, u);
  }
}
// kN elements of a weight vector of format WT (the same for every row: it stays
// in L1), `fill` where there is none.
template <int WT, int kN>
__device__ __forceinline__ void load_weight(const void *base, long long at, float fill, float v[kN]) {
  using T = typename Fmt<WT>::type;
  if (!base) {
#pragma unroll
    for (int j = 0; j < kN; ++j) v[j] = fill;
    return;
  }
  const T *p = static_cast<const T *>(base) + at;
  if constexpr (kN == 1) {
    v[0] = to_f32<WT>(*p);
  } else if constexpr (WT == kF32) {
#pragma unroll
    for (int j = 0; j < kN; j += 4) {
      const uint4 u = ldg_l1(p + j);
      v[j] = __uint_as_float(u.x), v[j + 1] = __uint_as_float(u.y), v[j + 2] = __uint_as_float(u.z), v[j + 3] = __uint_as_float(u.w);
    }
  } else {
    const uint4 u = ldg_l1(p);
    widen8<WT>(&u, v);
  }
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int d = 16; d > 0; d /= 2) v = __fadd_rn(v, __shfl_xor_sync(0xffffffffu, v, d));
  return v;
}
// The sum over the kRow threads of a row (32, or a whole number of warps: then
// every thread of the CTA takes part, and `slot` is not written again before
// another barrier).
template <int kRow>
__device__ __forceinline__ float row_sum(float v, float *slot) {
  v = warp_sum(v);
  if constexpr (kRow == 32) return v;
  const int warp = threadIdx.x / 32;
  if (threadIdx.x % 32 == 0) slot[warp] = v;
  __syncthreads();
  constexpr int kWarps = kRow / 32;
  const float *s = slot + warp / kWarps * kWarps;
  float t = s[0];
#pragma unroll
  for (int j = 1; j < kWarps; ++j) t = __fadd_rn(t, s[j]);
  return t;
}

template <int kRow>
constexpr int kThreads = kRow < 128 ? 128 : kRow;

// A row on kRow threads, kNv groups of kWide elements each.
template <int DT, int WT, bool kVec, int kRow, int kNv>
__global__ void __launch_bounds__(kThreads<kRow>) norm_kernel(const __grid_constant__ NormParams p) {
  constexpr int kW = kWide<DT, kVec>, kRows = kThreads<kRow> / kRow;
  __shared__ float slots[2][32];
  grid_dependency_wait();
  grid_dependents_launch();
  const int t = threadIdx.x % kRow;
  const long long row = (long long)blockIdx.x * kRows + threadIdx.x / kRow;
  const bool live = row < p.rows;
  float v[kNv][kW], sum = 0.f;
  bool in[kNv];
#pragma unroll
  for (int k = 0; k < kNv; ++k) {
    const long long c = (long long)(t + k * kRow) * kW;
    in[k] = live && c < p.cols;
    Raw<DT, kW> r;
    zero(r);
    if (in[k]) r = load_stream<DT, kW>(p.x, row * p.ld_x + c);
    widen<DT, kW>(r, v[k]);
  }
#pragma unroll
  for (int k = 0; k < kNv; ++k)
#pragma unroll
    for (int j = 0; j < kW; ++j) sum = __fadd_rn(sum, v[k][j]);
  const float n = (float)p.cols;
  const float mean = __fdiv_rn(row_sum<kRow>(sum, slots[0]), n);
  float sq = 0.f;
#pragma unroll
  for (int k = 0; k < kNv; ++k)
#pragma unroll
    for (int j = 0; j < kW; ++j) {
      v[k][j] = in[k] ? __fsub_rn(v[k][j], mean) : 0.f;
      sq = __fmaf_rn(v[k][j], v[k][j], sq);
    }
  const float rstd = __frsqrt_rn(__fadd_rn(__fdiv_rn(row_sum<kRow>(sq, slots[1]), n), p.eps));
  if (t == 0 && live) {
    if (p.mean) p.mean[row] = mean;
    if (p.rstd) p.rstd[row] = rstd;
  }
#pragma unroll
  for (int k = 0; k < kNv; ++k) {
    if (!in[k]) continue;
    const long long c = (long long)(t + k * kRow) * kW;
    float w[kW], b[kW];
    load_weight<WT, kW>(p.weight, c, 1.f, w);
    load_weight<WT, kW>(p.bias, c, 0.f, b);
#pragma unroll
    for (int j = 0; j < kW; ++j) w[j] = __fmaf_rn(__fmul_rn(v[k][j], rstd), w[j], b[j]);
    store<DT, kW>(p.out, row * p.ld_out + c, w);
  }
}

// A row longer than the registers hold: three passes over it by one CTA, the
// later two from L2.
template <int DT, int WT, bool kVec>
__global__ void __launch_bounds__(1024) norm_long_kernel(const __grid_constant__ NormParams p) {
  constexpr int kW = kWide<DT, kVec>;
  __shared__ float slots[2][32];
  grid_dependency_wait();
  grid_dependents_launch();
  const long long row = blockIdx.x, step = 1024ll * kW;
  float sum = 0.f;
#pragma unroll 4
  for (long long c = (long long)threadIdx.x * kW; c < p.cols; c += step) {
    float v[kW], s = 0.f;
    widen<DT, kW>(load_stream<DT, kW>(p.x, row * p.ld_x + c), v);
#pragma unroll
    for (int j = 0; j < kW; ++j) s = __fadd_rn(s, v[j]);
    sum = __fadd_rn(sum, s);
  }
  const float n = (float)p.cols;
  const float mean = __fdiv_rn(row_sum<1024>(sum, slots[0]), n);
  float sq = 0.f;
#pragma unroll 4
  for (long long c = (long long)threadIdx.x * kW; c < p.cols; c += step) {
    float v[kW], s = 0.f;
    widen<DT, kW>(load_stream<DT, kW>(p.x, row * p.ld_x + c), v);
#pragma unroll
    for (int j = 0; j < kW; ++j) {
      const float d = __fsub_rn(v[j], mean);
      s = __fmaf_rn(d, d, s);
    }
    sq = __fadd_rn(sq, s);
  }
  const float rstd = __frsqrt_rn(__fadd_rn(__fdiv_rn(row_sum<1024>(sq, slots[1]), n), p.eps));
  if (threadIdx.x == 0) {
    if (p.mean) p.mean[row] = mean;
    if (p.rstd) p.rstd[row] = rstd;
  }
  // (out may be x: each element is read and then written by the same thread)
#pragma unroll 4
  for (long long c = (long long)threadIdx.x * kW; c < p.cols; c += step) {
    float v[kW], w[kW], b[kW];
    widen<DT, kW>(load_stream<DT, kW>(p.x, row * p.ld_x + c), v);
    load_weight<WT, kW>(p.weight, c, 1.f, w);
    load_weight<WT, kW>(p.bias, c, 0.f, b);
#pragma unroll
    for (int j = 0; j < kW; ++j) v[j] = __fmaf_rn(__fmul_rn(__fsub_rn(v[j], mean), rstd), w[j], b[j]);
    store<DT, kW>(p.out, row * p.ld_out + c, v);
  }
}

// --------------------------------------------------------------------------
// backward
// --------------------------------------------------------------------------

// A row on kRow threads, two groups of 16 bytes each; 256 threads or a row's a CTA.
template <int kRow>
constexpr int kRingThreads = kRow < 256 ? 256 : kRow;
// Rows of x and dy wait in a ring of shared memory: a stage is the rows that a CTA
// takes at once.
template <int kRow>
struct Ring {
  static constexpr int kThreads = kRingThreads<kRow>, kRows = kThreads / kRow, kNv = 2;
  static constexpr int kRowBytes = kRow * kNv * 16;      // at most
  static constexpr int kHalf = kRows * kRowBytes;        // x, or dy
  static constexpr int kStages = kRow <= 256 ? 4 : 3;
  static constexpr int kCtas = kThreads == 256 ? 3 : kThreads == 512 ? 2 : 1;  // an SM
  static constexpr int kSmem = kStages * 2 * kHalf;
};

// Sums of two values over kRow threads, to all of them.  slots: this turn's; the
// barrier in here also ends the CTA's reads of the turn before.
template <int kRow>
__device__ __forceinline__ void row_sums(float &a, float &b, float (*slots)[32]) {
#pragma unroll
  for (int d = kRow < 32 ? kRow / 2 : 16; d > 0; d /= 2)
    a = __fadd_rn(a, __shfl_xor_sync(0xffffffffu, a, d)), b = __fadd_rn(b, __shfl_xor_sync(0xffffffffu, b, d));
  constexpr int kWarps = kRow / 32;
  if constexpr (kWarps > 1) {
    const int warp = threadIdx.x / 32, from = warp / kWarps * kWarps;
    if (threadIdx.x % 32 == 0) slots[0][warp] = a, slots[1][warp] = b;
    __syncthreads();
    if constexpr (kWarps == 2) {
      a = __fadd_rn(slots[0][from], slots[0][from + 1]), b = __fadd_rn(slots[1][from], slots[1][from + 1]);
    } else {
      a = b = 0.f;
#pragma unroll
      for (int j = 0; j < kWarps; j += 4) {
        const float4 u = *reinterpret_cast<const float4 *>(&slots[0][from + j]), v = *reinterpret_cast<const float4 *>(&slots[1][from + j]);
        a = __fadd_rn(a, __fadd_rn(__fadd_rn(u.x, u.y), __fadd_rn(u.z, u.w)));
        b = __fadd_rn(b, __fadd_rn(__fadd_rn(v.x, v.y), __fadd_rn(v.z, v.w)));
      }
    }
  } else {
    __syncthreads();
  }
}

// Rows whose 16-byte groups are aligned.  Persistent CTAs walk the rows; bulk
// copies bring the next ones into the ring while these are finished, so what is in
// flight does not depend on registers (holding it there left 16384 x 4096 bfloat16
// at 132 us of the 59 that memory takes).  A thread keeps its columns throughout,
// and with them their part of dweight and dbias in registers: the sums over rows
// cost one write of two rows a CTA, and the rest is norm_sums_kernel's.  Rows go to
// CTAs by their index, so the order of the sums does not depend on timing.
template <int DT, int WT, int kRow>
__global__ void __launch_bounds__(Ring<kRow>::kThreads, Ring<kRow>::kCtas)
    norm_grad_ring_kernel(const __grid_constant__ NormGradParams p) {
  using R = Ring<kRow>;
  using T = typename Fmt<DT>::type;
  constexpr int kW = kWide<DT, true>, kNv = R::kNv;
  extern __shared__ __align__(128) unsigned char ring[];
  __shared__ __align__(16) float slots[2][2][32];
  __shared__ __align__(8) uint64_t full[R::kStages];
  if (threadIdx.x == 0) {
    for (int s = 0; s < R::kStages; ++s) mbar_init(&full[s], 1);
    fence_mbar_init();
  }
  __syncthreads();
  grid_dependency_wait();
  grid_dependents_launch();
  const int t = threadIdx.x % kRow, group = threadIdx.x / kRow;
  const int cols = (int)p.cols, row_bytes = cols * (int)sizeof(T);
  const float inv = __fdiv_rn(1.f, (float)cols);
  float dw[kNv][kW], db[kNv][kW];
#pragma unroll
  for (int k = 0; k < kNv; ++k)
#pragma unroll
    for (int j = 0; j < kW; ++j) dw[k][j] = db[k][j] = 0.f;
  const long long step = (long long)gridDim.x * R::kRows, start = (long long)blockIdx.x * R::kRows;
  const unsigned turns = start < p.rows ? (unsigned)((p.rows - start + step - 1) / step) : 0;
  // turn q's rows into its stage, by thread 0
  auto fetch = [&](unsigned q) {
    const long long first = start + q * step;
    const int n = (int)(p.rows - first < R::kRows ? p.rows - first : R::kRows);
    const unsigned s = q % R::kStages;
    const uint64_t pol = l2_evict_first_policy();
    unsigned char *to = ring + s * 2 * R::kHalf;
    mbar_arrive_expect_tx(&full[s], (uint32_t)(2 * n * row_bytes));
    for (int r = 0; r < n; ++r) {
      bulk_load(to + r * R::kRowBytes, static_cast<const T *>(p.x) + (first + r) * p.ld_x, row_bytes, &full[s], pol);
      bulk_load(to + R::kHalf + r * R::kRowBytes, static_cast<const T *>(p.dy) + (first + r) * p.ld_dy, row_bytes, &full[s], pol);
    }
  };
  if (threadIdx.x == 0)
    for (unsigned q = 0; q + 1 < R::kStages && q < turns; ++q) fetch(q);
  long long row = start + group;
  float mean = 0.f, rstd = 0.f;
  if (row < p.rows) mean = p.mean[row], rstd = p.rstd[row];
  bool ok = true;
  for (unsigned q = 0; q < turns; ++q, row += step) {
    const bool live = row < p.rows;
    const float shift = mean, scale = live ? rstd : 0.f;
    if (row + step < p.rows) mean = p.mean[row + step], rstd = p.rstd[row + step];
    const unsigned s = q % R::kStages;
    // (a wait that gave up: every thread still comes to every barrier, and stores nothing more)
    ok = mbar_wait_bounded(&full[s], (q / R::kStages) & 1, ok ? kWaitLimitNs : 0) && ok;
    const unsigned char *from = ring + s * 2 * R::kHalf + group * R::kRowBytes + t * 16;
    float s1 = 0.f, s2 = 0.f;
#pragma unroll
    for (int k = 0; k < kNv; ++k) {
      const int c = (t + k * kRow) * kW;
      if (c >= cols || !live) continue;
      float x[kW], d[kW], w[kW];
      widen_shared<DT>(from + k * kRow * 16, x);
      widen_shared<DT>(from + R::kHalf + k * kRow * 16, d);
      load_weight<WT, kW>(p.weight, c, 1.f, w);
#pragma unroll
      for (int j = 0; j < kW; ++j) {
        const float h = __fmul_rn(__fsub_rn(x[j], shift), scale), g = __fmul_rn(d[j], w[j]);
        dw[k][j] = __fmaf_rn(d[j], h, dw[k][j]);
        db[k][j] = __fadd_rn(db[k][j], d[j]);
        s1 = __fadd_rn(s1, g);
        s2 = __fmaf_rn(g, h, s2);
      }
    }
    row_sums<kRow>(s1, s2, slots[q & 1]);
    // every thread is past the turn before: its stage is free
    if (threadIdx.x == 0 && q + R::kStages - 1 < turns) fetch(q + R::kStages - 1);
    if (!p.dx || !live || !ok) continue;
    s1 = __fmul_rn(s1, inv), s2 = __fmul_rn(s2, inv);
#pragma unroll
    for (int k = 0; k < kNv; ++k) {
      const int c = (t + k * kRow) * kW;
      if (c >= cols) continue;
      float x[kW], d[kW], w[kW];
      widen_shared<DT>(from + k * kRow * 16, x);
      widen_shared<DT>(from + R::kHalf + k * kRow * 16, d);
      load_weight<WT, kW>(p.weight, c, 1.f, w);
#pragma unroll
      for (int j = 0; j < kW; ++j) {
        const float h = __fmul_rn(__fsub_rn(x[j], shift), scale);
        d[j] = __fmul_rn(__fsub_rn(__fmaf_rn(-h, s2, __fmul_rn(d[j], w[j])), s1), scale);
      }
      store<DT, kW>(p.dx, row * p.ld_dx + c, d);
    }
  }
  if (!ok) {
    // what is in flight lands before shared memory is given back
    if (threadIdx.x % 32 == 0) atomicOr(p.status, kStatusWaitTimeout);
    for (unsigned u = turns > R::kStages ? turns - R::kStages : 0; u < turns; ++u)
      mbar_wait_bounded(&full[u % R::kStages], (u / R::kStages) & 1, kWaitLimitNs);
  }
  if (!p.sums) return;
  float *out = p.partials + (long long)blockIdx.x * 2 * p.cols;
  float *sums = reinterpret_cast<float *>(ring);
#pragma unroll
  for (int half = 0; half < 2; ++half, out += p.cols) {
    if constexpr (R::kRows > 1) {
      // the groups' sums in their order
      __syncthreads();
#pragma unroll
      for (int k = 0; k < kNv; ++k)
#pragma unroll
        for (int j = 0; j < kW; ++j) sums[group * (kRow * kNv * kW) + (t + k * kRow) * kW + j] = half ? db[k][j] : dw[k][j];
      __syncthreads();
      for (int c = threadIdx.x; c < cols; c += R::kThreads) {
        float v = sums[c];
        for (int g = 1; g < R::kRows; ++g) v = __fadd_rn(v, sums[g * (kRow * kNv * kW) + c]);
        out[c] = v;
      }
    } else {
#pragma unroll
      for (int k = 0; k < kNv; ++k) {
        const int c = (t + k * kRow) * kW;
        if (c >= cols) continue;
#pragma unroll
        for (int j = 0; j < kW; j += 4) {
          const float *v = half ? &db[k][j] : &dw[k][j];
          *reinterpret_cast<float4 *>(out + c + j) = make_float4(v[0], v[1], v[2], v[3]);
        }
      }
    }
  }
}

template <int kRow>
constexpr int kGradThreads = kRow < 256 ? 256 : kRow;

// The same by single elements, for rows that are not aligned: x and dy stay in
// storage format between the sums and dx, and weight comes from L1 both times.
template <int DT, int WT, int kRow, int kNv>
__global__ void __launch_bounds__(kGradThreads<kRow>, kGradThreads<kRow> <= 512 ? 1024 / kGradThreads<kRow> : 1)
    norm_grad_kernel(const __grid_constant__ NormGradParams p) {
  constexpr int kW = 1, kCta = kGradThreads<kRow>, kRows = kCta / kRow;
  __shared__ float slots[2][2][32];
  __shared__ float sums[kRows > 1 ? kCta * kNv * kW : 1];
  grid_dependency_wait();
  grid_dependents_launch();
  const int t = threadIdx.x % kRow, group = threadIdx.x / kRow;
  const int cols = (int)p.cols;  // (longer rows are not this kernel's)
  const float n = (float)cols;
  float dw[kNv][kW], db[kNv][kW];
#pragma unroll
  for (int k = 0; k < kNv; ++k)
#pragma unroll
    for (int j = 0; j < kW; ++j) dw[k][j] = db[k][j] = 0.f;
  const long long step = (long long)gridDim.x * kRows;
  Raw<DT, kW> rx[kNv], rd[kNv];
  float mean = 0.f, rstd = 0.f;
  auto fetch = [&](long long r) {
    const bool live = r < p.rows;
    mean = live ? p.mean[r] : 0.f, rstd = live ? p.rstd[r] : 0.f;
    const long long at_x = r * p.ld_x, at_d = r * p.ld_dy;
#pragma unroll
    for (int k = 0; k < kNv; ++k) {
      const int c = (t + k * kRow) * kW;
      zero(rx[k]), zero(rd[k]);
      if (live && c < cols) {
        rx[k] = load_stream<DT, kW>(p.x, at_x + c);
        rd[k] = load_stream<DT, kW>(p.dy, at_d + c);
      }
    }
  };
  long long row = (long long)blockIdx.x * kRows + group;
  int turn = 0;
  for (long long first = (long long)blockIdx.x * kRows; first < p.rows; first += step, row += step, turn ^= 1) {
    fetch(row);
    Raw<DT, kW> cx[kNv], cd[kNv];
    const float scale = rstd, shift = mean;
    float s1 = 0.f, s2 = 0.f;
#pragma unroll
    for (int k = 0; k < kNv; ++k) {
      const int c = (t + k * kRow) * kW;
      cx[k] = rx[k], cd[k] = rd[k];
      if (c >= cols) continue;
      float x[kW], d[kW], w[kW];
      widen<DT, kW>(cx[k], x);
      widen<DT, kW>(cd[k], d);
      load_weight<WT, kW>(p.weight, c, 1.f, w);
#pragma unroll
      for (int j = 0; j < kW; ++j) {
        const float h = __fmul_rn(__fsub_rn(x[j], shift), scale), g = __fmul_rn(d[j], w[j]);
        dw[k][j] = __fmaf_rn(d[j], h, dw[k][j]);
        db[k][j] = __fadd_rn(db[k][j], d[j]);
        s1 = __fadd_rn(s1, g);
        s2 = __fmaf_rn(g, h, s2);
      }
    }
    if (!p.dx) continue;
    s1 = warp_sum(s1), s2 = warp_sum(s2);
    if constexpr (kRow > 32) {
      // (two places in turn: a warp that is ahead writes the other)
      const int warp = threadIdx.x / 32;
      if (threadIdx.x % 32 == 0) slots[turn][0][warp] = s1, slots[turn][1][warp] = s2;
      __syncthreads();
      constexpr int kWarps = kRow / 32;
      const int from = warp / kWarps * kWarps;
      s1 = slots[turn][0][from], s2 = slots[turn][1][from];
#pragma unroll
      for (int j = 1; j < kWarps; ++j) s1 = __fadd_rn(s1, slots[turn][0][from + j]), s2 = __fadd_rn(s2, slots[turn][1][from + j]);
    }
    s1 = __fdiv_rn(s1, n), s2 = __fdiv_rn(s2, n);
    if (row >= p.rows) continue;
#pragma unroll
    for (int k = 0; k < kNv; ++k) {
      const int c = (t + k * kRow) * kW;
      if (c >= cols) continue;
      float x[kW], d[kW], w[kW];
      widen<DT, kW>(cx[k], x);
      widen<DT, kW>(cd[k], d);
      load_weight<WT, kW>(p.weight, c, 1.f, w);
#pragma unroll
      for (int j = 0; j < kW; ++j) {
        const float h = __fmul_rn(__fsub_rn(x[j], shift), scale), g = __fmul_rn(d[j], w[j]);
        d[j] = __fmul_rn(__fsub_rn(__fsub_rn(g, s1), __fmul_rn(h, s2)), scale);
      }
      store<DT, kW>(p.dx, row * p.ld_dx + c, d);
    }
  }
  if (!p.sums) return;
  float *out = p.partials + (long long)blockIdx.x * 2 * p.cols;
#pragma unroll
  for (int half = 0; half < 2; ++half, out += p.cols) {
    if constexpr (kRows > 1) {
      // the groups' sums in their order
      __syncthreads();
#pragma unroll
      for (int k = 0; k < kNv; ++k)
#pragma unroll
        for (int j = 0; j < kW; ++j) sums[group * (kRow * kNv * kW) + (t + k * kRow) * kW + j] = half ? db[k][j] : dw[k][j];
      __syncthreads();
      for (int c = threadIdx.x; c < cols; c += kCta) {
        float s = sums[c];
        for (int q = 1; q < kRows; ++q) s = __fadd_rn(s, sums[q * (kRow * kNv * kW) + c]);
        out[c] = s;
      }
    } else {
#pragma unroll
      for (int k = 0; k < kNv; ++k) {
        const int c = (t + k * kRow) * kW;
        if (c >= cols) continue;
#pragma unroll
        for (int j = 0; j < kW; ++j) out[c + j] = half ? db[k][j] : dw[k][j];
      }
    }
  }
}

// Rows longer than the registers hold.  dx: two passes over a row by one CTA.
template <int DT, int WT, bool kVec>
__global__ void __launch_bounds__(1024) norm_grad_long_kernel(const __grid_constant__ NormGradParams p) {
  constexpr int kW = kWide<DT, kVec>;
  __shared__ float slots[2][32];
  grid_dependency_wait();
  grid_dependents_launch();
  const long long row = blockIdx.x, step = 1024ll * kW;
  const float n = (float)p.cols, mean = p.mean[row], rstd = p.rstd[row];
  float s1 = 0.f, s2 = 0.f;
#pragma unroll 2
  for (long long c = (long long)threadIdx.x * kW; c < p.cols; c += step) {
    float x[kW], d[kW], w[kW], a = 0.f, b = 0.f;
    widen<DT, kW>(load_stream<DT, kW>(p.x, row * p.ld_x + c), x);
    widen<DT, kW>(load_stream<DT, kW>(p.dy, row * p.ld_dy + c), d);
    load_weight<WT, kW>(p.weight, c, 1.f, w);
#pragma unroll
    for (int j = 0; j < kW; ++j) {
      const float g = __fmul_rn(d[j], w[j]);
      a = __fadd_rn(a, g);
      b = __fmaf_rn(g, __fmul_rn(__fsub_rn(x[j], mean), rstd), b);
    }
    s1 = __fadd_rn(s1, a), s2 = __fadd_rn(s2, b);
  }
  s1 = __fdiv_rn(row_sum<1024>(s1, slots[0]), n);
  s2 = __fdiv_rn(row_sum<1024>(s2, slots[1]), n);
  // (dx may be dy or x: each element is read and then written by the same thread)
#pragma unroll 2
  for (long long c = (long long)threadIdx.x * kW; c < p.cols; c += step) {
    float x[kW], d[kW], w[kW];
    widen<DT, kW>(load_stream<DT, kW>(p.x, row * p.ld_x + c), x);
    widen<DT, kW>(load_stream<DT, kW>(p.dy, row * p.ld_dy + c), d);
    load_weight<WT, kW>(p.weight, c, 1.f, w);
#pragma unroll
    for (int j = 0; j < kW; ++j) {
      const float h = __fmul_rn(__fsub_rn(x[j], mean), rstd);
      d[j] = __fmul_rn(__fsub_rn(__fsub_rn(__fmul_rn(d[j], w[j]), s1), __fmul_rn(h, s2)), rstd);
    }
    store<DT, kW>(p.dx, row * p.ld_dx + c, d);
  }
}
// The sums over rows: 128 threads a CTA, each a group of columns, over every
// parts-th row.
template <int DT, bool kVec>
__global__ void __launch_bounds__(128) norm_columns_kernel(const __grid_constant__ NormGradParams p) {
  constexpr int kW = kWide<DT, kVec>;
  grid_dependency_wait();
  grid_dependents_launch();
  const long long c = ((long long)blockIdx.x * 128 + threadIdx.x) * kW;
  if (c >= p.cols) return;
  float dw[kW], db[kW];
#pragma unroll
  for (int j = 0; j < kW; ++j) dw[j] = db[j] = 0.f;
#pragma unroll 4
  for (long long row = blockIdx.y; row < p.rows; row += gridDim.y) {
    const float mean = p.mean[row], rstd = p.rstd[row];
    float x[kW], d[kW];
    widen<DT, kW>(load_stream<DT, kW>(p.x, row * p.ld_x + c), x);
    widen<DT, kW>(load_stream<DT, kW>(p.dy, row * p.ld_dy + c), d);
#pragma unroll
    for (int j = 0; j < kW; ++j) {
      dw[j] = __fmaf_rn(d[j], __fmul_rn(__fsub_rn(x[j], mean), rstd), dw[j]);
      db[j] = __fadd_rn(db[j], d[j]);
    }
  }
  float *out = p.partials + (long long)blockIdx.y * 2 * p.cols + c;
#pragma unroll
  for (int j = 0; j < kW; ++j) out[j] = dw[j], out[p.cols + j] = db[j];
}

// The partial sums of a column, in one order: sixteen threads a column take every
// sixteenth one, and their sums are added up in turn.  A thread takes kC columns
// (four where a row of the partial sums is whole groups of 16 bytes); blockIdx.y:
// dweight or dbias.
template <int WT, int kC>
__global__ void __launch_bounds__(256) norm_sums_kernel(const float *partials, int parts, long long cols, void *dweight,
                                                        void *dbias) {
  __shared__ float s[16][16 * kC + 1];
  grid_dependency_wait();
  grid_dependents_launch();
  void *out = blockIdx.y ? dbias : dweight;
  if (!out) return;
  const long long c = ((long long)blockIdx.x * 16 + threadIdx.x) * kC;
  float v[kC];
#pragma unroll
  for (int j = 0; j < kC; ++j) v[j] = 0.f;
  if (c < cols) {
    const float *from = partials + blockIdx.y * cols + c;
#pragma unroll 8
    for (int q = threadIdx.y; q < parts; q += 16) {
      const float *at = from + (long long)q * 2 * cols;
      if constexpr (kC == 4) {
        const float4 u = *reinterpret_cast<const float4 *>(at);
        v[0] = __fadd_rn(v[0], u.x), v[1] = __fadd_rn(v[1], u.y), v[2] = __fadd_rn(v[2], u.z), v[3] = __fadd_rn(v[3], u.w);
      } else {
        v[0] = __fadd_rn(v[0], *at);
      }
    }
  }
#pragma unroll
  for (int j = 0; j < kC; ++j) s[threadIdx.y][threadIdx.x * kC + j] = v[j];
  __syncthreads();
  const int tid = threadIdx.y * 16 + threadIdx.x;
  const long long at = (long long)blockIdx.x * 16 * kC + tid;
  if (tid >= 16 * kC || at >= cols) return;
  float total = s[0][tid];
#pragma unroll
  for (int j = 1; j < 16; ++j) total = __fadd_rn(total, s[j][tid]);
  static_cast<typename Fmt<WT>::type *>(out)[at] = from_f32<WT>(total);
}

// --------------------------------------------------------------------------
// launches
// --------------------------------------------------------------------------

template <class... P, class... Args>
cudaError_t launch_smem(void (*k)(P...), dim3 grid, dim3 block, int smem, cudaStream_t s, const Args &...args) {
  cudaLaunchConfig_t c = {};
  c.gridDim = grid;
  c.blockDim = block;
  c.dynamicSmemBytes = smem;
  c.stream = s;
  cudaLaunchAttribute a = {};
  a.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  a.val.programmaticStreamSerializationAllowed = 1;
  c.attrs = &a;
  c.numAttrs = 1;
  return cudaLaunchKernelEx(&c, k, args...);
}

template <class... P, class... Args>
cudaError_t launch(void (*k)(P...), dim3 grid, dim3 block, cudaStream_t s, const Args &...args) {
  return launch_smem(k, grid, block, 0, s, args...);
}

template <int DT, int WT, bool kVec, int kRow, int kNv>
cudaError_t forward_of(const NormParams &p, cudaStream_t s) {
  constexpr int kRows = kThreads<kRow> / kRow;
  return launch(norm_kernel<DT, WT, kVec, kRow, kNv>, dim3((unsigned)ceil_div(p.rows, (long long)kRows)),
                dim3(kThreads<kRow>), s, p);
}
// The fewest threads a row that hold it: with up to four groups of 16 bytes a
// thread, enough loads are in flight at any number of rows.
template <int DT, int WT>
cudaError_t forward(const NormParams &p, cudaStream_t s) {
  if (p.vec) {
    const long long g = p.cols / kWide<DT, true>;
    if (g <= 32) return forward_of<DT, WT, true, 32, 1>(p, s);
    if (g <= 64) return forward_of<DT, WT, true, 32, 2>(p, s);
    if (g <= 128) return forward_of<DT, WT, true, 32, 4>(p, s);
    if (g <= 256) return forward_of<DT, WT, true, 128, 2>(p, s);
    if (g <= 512) return forward_of<DT, WT, true, 128, 4>(p, s);
    if (g <= 1024) return forward_of<DT, WT, true, 256, 4>(p, s);
    if (g <= 2048) return forward_of<DT, WT, true, 512, 4>(p, s);
    if (g <= 4096) return forward_of<DT, WT, true, 1024, 4>(p, s);
    return launch(norm_long_kernel<DT, WT, true>, dim3((unsigned)p.rows), dim3(1024), s, p);
  }
  if (p.cols <= 256) return forward_of<DT, WT, false, 32, 8>(p, s);
  if (p.cols <= 512) return forward_of<DT, WT, false, 64, 8>(p, s);
  if (p.cols <= 1024) return forward_of<DT, WT, false, 128, 8>(p, s);
  if (p.cols <= 2048) return forward_of<DT, WT, false, 256, 8>(p, s);
  if (p.cols <= 4096) return forward_of<DT, WT, false, 512, 8>(p, s);
  if (p.cols <= 8192) return forward_of<DT, WT, false, 1024, 8>(p, s);
  if (p.cols <= 16384) return forward_of<DT, WT, false, 1024, 16>(p, s);
  return launch(norm_long_kernel<DT, WT, false>, dim3((unsigned)p.rows), dim3(1024), s, p);
}

template <int WT>
cudaError_t finish_sums(const NormGradParams &p, int parts, cudaStream_t s) {
  return p.cols % 4 == 0 ? launch(norm_sums_kernel<WT, 4>, dim3((unsigned)ceil_div(p.cols, 64ll), 2), dim3(16, 16), s,
                                  (const float *)p.partials, parts, p.cols, p.dweight, p.dbias)
                         : launch(norm_sums_kernel<WT, 1>, dim3((unsigned)ceil_div(p.cols, 16ll), 2), dim3(16, 16), s,
                                  (const float *)p.partials, parts, p.cols, p.dweight, p.dbias);
}
// One launch over the rows and, where they are wanted, one for the sums.
template <int WT, class K>
cudaError_t backward_by(K kernel, int rows_a_cta, int threads, int ctas, int smem, const NormGradParams &p, cudaStream_t s) {
  long long grid = ceil_div(p.rows, (long long)rows_a_cta);
  if (grid > (long long)p.sms * ctas) grid = (long long)p.sms * ctas;
  if (grid > p.parts) grid = p.parts;
  const cudaError_t e = launch_smem(kernel, dim3((unsigned)grid), dim3((unsigned)threads), smem, s, p);
  return e != cudaSuccess || !p.sums ? e : finish_sums<WT>(p, (int)grid, s);
}
template <int DT, int WT, int kRow, int kNv>
cudaError_t backward_of(const NormGradParams &p, cudaStream_t s) {
  constexpr int kCta = kGradThreads<kRow>;
  return backward_by<WT>(norm_grad_kernel<DT, WT, kRow, kNv>, kCta / kRow, kCta, kCta <= 512 ? 1024 / kCta : 1, 0, p, s);
}
template <int DT, int WT, int kRow>
cudaError_t backward_ring(const NormGradParams &p, cudaStream_t s) {
  using R = Ring<kRow>;
  const cudaError_t e = allow_smem<norm_grad_ring_kernel<DT, WT, kRow>>(R::kSmem);
  if (e != cudaSuccess) return e;
  return backward_by<WT>(norm_grad_ring_kernel<DT, WT, kRow>, R::kRows, R::kThreads, R::kCtas, R::kSmem, p, s);
}
template <int DT, int WT, bool kVec>
cudaError_t backward_long(const NormGradParams &p, cudaStream_t s) {
  cudaError_t e = cudaSuccess;
  if (p.sums) {  // first: dx may be x or dy
    const long long groups = ceil_div(p.cols, (long long)kWide<DT, kVec>);
    e = launch(norm_columns_kernel<DT, kVec>, dim3((unsigned)ceil_div(groups, 128ll), (unsigned)p.parts), dim3(128), s, p);
    if (e == cudaSuccess) e = finish_sums<WT>(p, p.parts, s);
  }
  if (e == cudaSuccess && p.dx) e = launch(norm_grad_long_kernel<DT, WT, kVec>, dim3((unsigned)p.rows), dim3(1024), s, p);
  return e;
}
template <int DT, int WT>
cudaError_t backward(const NormGradParams &p, cudaStream_t s) {
  if (p.rows == 0) return p.sums ? finish_sums<WT>(p, 0, s) : cudaSuccess;
  if (p.vec) {
    const long long g = p.cols / kWide<DT, true>;
    if (g <= 32) return backward_ring<DT, WT, 16>(p, s);
    if (g <= 64) return backward_ring<DT, WT, 32>(p, s);
    if (g <= 128) return backward_ring<DT, WT, 64>(p, s);
    if (g <= 256) return backward_ring<DT, WT, 128>(p, s);
    if (g <= 512) return backward_ring<DT, WT, 256>(p, s);
    if (g <= 1024) return backward_ring<DT, WT, 512>(p, s);
    if (g <= 2048) return backward_ring<DT, WT, 1024>(p, s);
    return backward_long<DT, WT, true>(p, s);
  }
  if (p.cols <= 256) return backward_of<DT, WT, 32, 8>(p, s);
  if (p.cols <= 1024) return backward_of<DT, WT, 128, 8>(p, s);
  if (p.cols <= 2048) return backward_of<DT, WT, 256, 8>(p, s);
  if (p.cols <= 4096) return backward_of<DT, WT, 512, 8>(p, s);
  if (p.cols <= 8192) return backward_of<DT, WT, 1024, 8>(p, s);
  return backward_long<DT, WT, false>(p, s);
}

}  // namespace norm

}  // namespace rr
