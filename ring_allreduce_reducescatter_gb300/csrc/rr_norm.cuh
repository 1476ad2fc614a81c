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

// Two binary32 values and the operations on both at once (each rounded by itself).
struct Two {
  uint64_t v;
};
__device__ __forceinline__ Two two(float a, float b) {
  Two r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 split(Two a) {
  float2 f;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(a.v));
  return f;
}
__device__ __forceinline__ Two add2(Two a, Two b) {
  Two r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ Two mul2(Two a, Two b) {
  Two r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ Two fma2(Two a, Two b, Two c) {
  Two r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}
template <int kN>
__device__ __forceinline__ void pair_up(const float v[kN], Two p[kN / 2]) {
#pragma unroll
  for (int j = 0; j < kN / 2; ++j) p[j] = two(v[2 * j], v[2 * j + 1]);
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

// A row on kRow threads, kNv groups of kWide elements each; short rows several at a
// time, so that their loads are in flight together (131072 x 256 bfloat16 one by one
// 35 us).
template <int kRow, int kNv>
constexpr int kTogether = kRow == 32 && kNv < 4 ? 4 / kNv : 1;
template <int DT, int WT, bool kVec, int kRow, int kNv>
__global__ void __launch_bounds__(kThreads<kRow>) norm_kernel(const __grid_constant__ NormParams p) {
  constexpr int kW = kWide<DT, kVec>, kRows = kThreads<kRow> / kRow, kT = kTogether<kRow, kNv>;
  __shared__ float slots[2][32];
  grid_dependency_wait();
  grid_dependents_launch();
  const int t = threadIdx.x % kRow;
  const long long row0 = (long long)blockIdx.x * (kRows * kT) + threadIdx.x / kRow;
  float v[kT][kNv][kW];
  Raw<DT, kW> raw[kT][kNv];
  bool in[kNv];
#pragma unroll
  for (int k = 0; k < kNv; ++k) in[k] = (long long)(t + k * kRow) * kW < p.cols;
#pragma unroll
  for (int i = 0; i < kT; ++i)
#pragma unroll
    for (int k = 0; k < kNv; ++k) {
      const long long row = row0 + i * kRows;
      zero(raw[i][k]);
      if (in[k] && row < p.rows) raw[i][k] = load_stream<DT, kW>(p.x, row * p.ld_x + (t + k * kRow) * kW);
    }
#pragma unroll
  for (int i = 0; i < kT; ++i)
#pragma unroll
    for (int k = 0; k < kNv; ++k) widen<DT, kW>(raw[i][k], v[i][k]);
  const float n = (float)p.cols;
#pragma unroll
  for (int i = 0; i < kT; ++i) {
    const long long row = row0 + i * kRows;
    float sum = 0.f;
#pragma unroll
    for (int k = 0; k < kNv; ++k)
#pragma unroll
      for (int j = 0; j < kW; ++j) sum = __fadd_rn(sum, v[i][k][j]);
    const float mean = __fdiv_rn(row_sum<kRow>(sum, slots[0]), n);
    float sq = 0.f;
#pragma unroll
    for (int k = 0; k < kNv; ++k)
#pragma unroll
      for (int j = 0; j < kW; ++j) {
        v[i][k][j] = in[k] ? __fsub_rn(v[i][k][j], mean) : 0.f;
        sq = __fmaf_rn(v[i][k][j], v[i][k][j], sq);
      }
    const float rstd = __frsqrt_rn(__fadd_rn(__fdiv_rn(row_sum<kRow>(sq, slots[1]), n), p.eps));
    if (row >= p.rows) break;  // (the whole warp; a CTA's later barriers are only where kT is 1)
    if (t == 0) {
      if (p.mean) p.mean[row] = mean;
      if (p.rstd) p.rstd[row] = rstd;
    }
#pragma unroll
    for (int k = 0; k < kNv; ++k) {
      if (!in[k]) continue;
      const int c = (t + k * kRow) * kW;
      float w[kW], b[kW];
      load_weight<WT, kW>(p.weight, c, 1.f, w);
      load_weight<WT, kW>(p.bias, c, 0.f, b);
#pragma unroll
      for (int j = 0; j < kW; ++j) w[j] = __fmaf_rn(__fmul_rn(v[i][k][j], rstd), w[j], b[j]);
      store<DT, kW>(p.out, row * p.ld_out + c, w);
    }
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

// A row on kRow threads, kNv groups of 16 bytes each, or as many single elements
// where rows are not aligned; 128 threads or a row's a CTA.  Four groups (with two,
// the sums over twice the threads took 16384 x 4096 bfloat16 backward to 97 us for
// 79), but two for long rows of 16-bit elements, whose sums over rows would not fit
// the registers (8192 x 8192 bfloat16 123 us).  Rows of kTensors tensors wait in a
// ring of shared memory: a stage is the rows that a CTA takes at once.
template <int kRow, int kNv_, int kTensors>
struct Ring {
  static constexpr int kThreads = kRow < 128 ? 128 : kRow, kRows = kThreads / kRow, kNv = kNv_;
  static constexpr int kAll = kThreads + 32;              // with the warp that brings the rows
  static constexpr int kRowBytes = kRow * kNv * 16 + 16;  // at most, and what an unaligned row adds
  static constexpr int kTensor = kRows * kRowBytes;
  static constexpr int kCtas = kThreads == 128 ? 3 : kThreads == 256 ? 2 : 1;  // an SM: 112 registers a thread or more
  static constexpr int kStages = kThreads == 128 ? 4 : kNv == 2 && kThreads == 512 ? 6 : 3;
  static constexpr int kSmem = kStages * kTensors * kTensor;
  static_assert(kSmem * kCtas <= 220 * 1024, "they fit an SM");
};

// The 16-byte groups that hold a row, as far as they lie inside the tensor: what a
// bulk copy brings.  A tensor's first and last elements may lie outside of them.
struct Window {
  uintptr_t at, lo, hi;  // the row's first byte, the groups
};
template <int DT, bool kVec>
__device__ __forceinline__ Window window_of(const void *base, long long row, long long ld, long long rows, int cols) {
  constexpr int E = Fmt<DT>::bytes;
  Window w;
  w.at = reinterpret_cast<uintptr_t>(base) + (uintptr_t)(row * ld * E);
  w.lo = w.at, w.hi = w.at + (uintptr_t)cols * E;
  if constexpr (!kVec) {
    const uintptr_t first = reinterpret_cast<uintptr_t>(base), last = first + (uintptr_t)(((rows - 1) * ld + cols) * E);
    w.lo &= ~(uintptr_t)15, w.hi = (w.hi + 15) & ~(uintptr_t)15;
    if (w.lo < first) w.lo += 16;
    if (w.hi > last) w.hi -= 16;
    if (w.hi < w.lo) w.hi = w.lo;
  }
  return w;
}
// Brings a row to its place in the ring (at its offset from the 16-byte grid) and
// says how many bytes that is.
template <int DT, bool kVec>
__device__ __forceinline__ void bring(const Window &w, unsigned char *to, uint64_t *bar, uint64_t pol) {
  if (w.hi > w.lo)
    bulk_load(to + (w.lo - (w.at & ~(uintptr_t)15)), reinterpret_cast<const void *>(w.lo), (uint32_t)(w.hi - w.lo), bar, pol);
}
// How far past the 16-byte grid a row begins, and with it its place in the ring.
template <int DT, bool kVec>
__device__ __forceinline__ int shift_of(const void *base, long long row, long long ld) {
  return kVec ? 0 : (int)((reinterpret_cast<uintptr_t>(base) + (uintptr_t)(row * ld * Fmt<DT>::bytes)) & 15);
}
// A thread's group k of its row: sixteen bytes' worth of elements, neighbours (kVec)
// or kRow apart; zeros past the last column.  from: the row in the ring.
template <int DT, bool kVec, int kRow>
__device__ __forceinline__ void take(const unsigned char *from, int t, int k, int cols, float v[16 / Fmt<DT>::bytes]) {
  constexpr int kW = 16 / Fmt<DT>::bytes;
  if constexpr (kVec) {
    widen_shared<DT>(from + (t + k * kRow) * 16, v);
  } else {
#pragma unroll
    for (int j = 0; j < kW; ++j) {
      const int c = t + (k * kW + j) * kRow;
      v[j] = c < cols ? to_f32<DT>(reinterpret_cast<const typename Fmt<DT>::type *>(from)[c]) : 0.f;
    }
  }
}
template <int WT, int kW, bool kVec, int kRow>
__device__ __forceinline__ void take_weight(const void *base, int t, int k, int cols, float fill, float v[kW]) {
  if constexpr (kVec) {
    load_weight<WT, kW>(base, (t + k * kRow) * kW, fill, v);
  } else {
#pragma unroll
    for (int j = 0; j < kW; ++j) {
      const int c = t + (k * kW + j) * kRow;
      v[j] = 0.f;
      if (c < cols) load_weight<WT, 1>(base, c, fill, v + j);
    }
  }
}
template <int DT, bool kVec, int kRow>
__device__ __forceinline__ void put(void *base, long long row_at, int t, int k, int cols, const float v[16 / Fmt<DT>::bytes]) {
  constexpr int kW = 16 / Fmt<DT>::bytes;
  if constexpr (kVec) {
    store<DT, kW>(base, row_at + (t + k * kRow) * kW, v);
  } else {
#pragma unroll
    for (int j = 0; j < kW; ++j) {
      const int c = t + (k * kW + j) * kRow;
      if (c < cols) store<DT, 1>(base, row_at + c, v + j);
    }
  }
}
// Whether a thread's group k holds a column (of neighbours: all or none).
template <int kW, bool kVec, int kRow>
__device__ __forceinline__ bool holds(int t, int k, int cols) {
  return (kVec ? (t + k * kRow) * kW : t + k * kW * kRow) < cols;
}

// A barrier of the threads that work on rows.
template <int kThreads>
__device__ __forceinline__ void work_sync() {
  asm volatile("bar.sync 1, %0;" ::"n"(kThreads) : "memory");
}
// Sums of two values over kRow threads, to all of them.  slots: this turn's (the
// turn after takes others: a warp that is ahead writes those).
template <int kRow>
__device__ __forceinline__ void row_sums(float &a, float &b, float (*slots)[32]) {
#pragma unroll
  for (int d = kRow < 32 ? kRow / 2 : 16; d > 0; d /= 2)
    a = __fadd_rn(a, __shfl_xor_sync(0xffffffffu, a, d)), b = __fadd_rn(b, __shfl_xor_sync(0xffffffffu, b, d));
  constexpr int kWarps = kRow / 32;
  if constexpr (kWarps > 1) {
    const int warp = threadIdx.x / 32, from = warp / kWarps * kWarps;
    if (threadIdx.x % 32 == 0) slots[0][warp] = a, slots[1][warp] = b;
    work_sync<(kRow < 128 ? 128 : kRow)>();
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
  }
}

// The rows of a persistent CTA and their ring.  One warp brings the rows (by a
// thread of the working warps every turn waited 900 cycles for the copies' set-up).
template <class R, int DT, bool kVec, int kTensors>
struct Walk {
  long long start, step, rows;
  int cols;
  unsigned turns;
  const void *base[kTensors];
  long long ld[kTensors];
  unsigned char *ring;
  uint64_t *full, *empty;
  __device__ __forceinline__ Walk(long long rows, long long cols, unsigned char *ring, uint64_t *full, uint64_t *empty)
      : start((long long)blockIdx.x * R::kRows), step((long long)gridDim.x * R::kRows), rows(rows), cols((int)cols),
        turns(start < rows ? (unsigned)((rows - start + step - 1) / step) : 0), ring(ring), full(full), empty(empty) {}
  // The whole CTA: the barriers, and zeros in the ring (past an aligned row's last
  // column they stay, and count nothing).
  __device__ __forceinline__ void init() const {
    if (threadIdx.x == 0) {
      for (int s = 0; s < R::kStages; ++s) mbar_init(&full[s], 1), mbar_init(&empty[s], R::kThreads / 32);
      fence_mbar_init();
    }
    for (int i = threadIdx.x * 16; i < R::kSmem; i += R::kAll * 16) *reinterpret_cast<uint4 *>(ring + i) = make_uint4(0, 0, 0, 0);
    fence_proxy_async_smem();
    __syncthreads();
  }
  // One thread: every turn's rows into their stages.
  __device__ __forceinline__ void bring_all(unsigned *status) const {
    const uint64_t pol = l2_evict_first_policy();
    for (unsigned q = 0; q < turns; ++q) {
      const unsigned s = q % R::kStages;
      if (!mbar_wait_bounded(&empty[s], ((q / R::kStages) & 1) ^ 1, kWaitLimitNs)) {
        atomicOr(status, kStatusWaitTimeout);
        break;
      }
      const long long first = start + q * step;
      const int n = (int)(rows - first < R::kRows ? rows - first : R::kRows);
      uint32_t bytes = 0;
      if (kVec) {
        bytes = (uint32_t)(n * kTensors * cols * Fmt<DT>::bytes);
      } else {
        for (int r = 0; r < n; ++r)
#pragma unroll
          for (int i = 0; i < kTensors; ++i) {
            const Window w = window_of<DT, kVec>(base[i], first + r, ld[i], rows, cols);
            bytes += (uint32_t)(w.hi - w.lo);
          }
      }
      mbar_arrive_expect_tx(&full[s], bytes);
      for (int r = 0; r < n; ++r)
#pragma unroll
        for (int i = 0; i < kTensors; ++i)
          bring<DT, kVec>(window_of<DT, kVec>(base[i], first + r, ld[i], rows, cols), slot(q, i, r), &full[s], pol);
    }
  }
  __device__ __forceinline__ unsigned char *slot(unsigned q, int i, int group) const {
    return ring + ((q % R::kStages) * kTensors + i) * R::kTensor + group * R::kRowBytes;
  }
  // Tensor i's row of turn q.
  __device__ __forceinline__ const unsigned char *at(unsigned q, int i, int group, long long row) const {
    return slot(q, i, group) + shift_of<DT, kVec>(base[i], row, ld[i]);
  }
  // The elements of a tensor's first and last row that lie outside of the 16-byte
  // groups inside the tensor, by a thread each; all working threads call it.
  __device__ __forceinline__ void edges(unsigned q) const {
    if constexpr (!kVec) {
      using T = typename Fmt<DT>::type;
      const long long first = start + q * step;
      if (first > 0 && first + R::kRows < rows) return;
      for (int r = 0; r < R::kRows; ++r) {
        const long long row = first + r;
        if (row != 0 && row != rows - 1) continue;
#pragma unroll
        for (int i = 0; i < kTensors; ++i) {
          const Window w = window_of<DT, kVec>(base[i], row, ld[i], rows, cols);
          T *to = reinterpret_cast<T *>(slot(q, i, r) + (w.at & 15));
          const T *from = reinterpret_cast<const T *>(w.at);
          const int lo = w.lo > w.at ? (int)((w.lo - w.at) / sizeof(T)) : 0;
          const int hi = w.hi > w.at ? (int)((w.hi - w.at) / sizeof(T)) : 0;
          for (int c = threadIdx.x; c < lo && c < cols; c += R::kThreads) to[c] = from[c];
          for (int c = (hi > lo ? hi : lo) + threadIdx.x; c < cols; c += R::kThreads) to[c] = from[c];
        }
      }
      work_sync<R::kThreads>();
    }
  }
  // (a wait that gave up: every thread still comes to every barrier, and stores nothing more)
  __device__ __forceinline__ bool wait(unsigned q, bool ok) const {
    return mbar_wait_bounded(&full[q % R::kStages], (q / R::kStages) & 1, ok ? kWaitLimitNs : 0) && ok;
  }
  // A working warp is done with turn q's rows.
  __device__ __forceinline__ void done(unsigned q) const {
    __syncwarp();
    if (threadIdx.x % 32 == 0)
      asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(&empty[q % R::kStages])) : "memory");
  }
  // What is in flight lands before shared memory is given back.
  __device__ __forceinline__ void give_up(unsigned *status) const {
    if (threadIdx.x % 32 == 0) atomicOr(status, kStatusWaitTimeout);
    for (unsigned u = turns > R::kStages ? turns - R::kStages : 0; u < turns; ++u)
      mbar_wait_bounded(&full[u % R::kStages], (u / R::kStages) & 1, kWaitLimitNs);
  }
};

// Backward.  Persistent CTAs walk the rows; bulk copies bring the next ones into
// the ring while these are finished, so what is in flight does not depend on
// registers (holding it there left 16384 x 4096 bfloat16 at 132 us of the 59 that
// memory takes).  The arithmetic goes two values an instruction.  A thread keeps its
// columns throughout, and with them their weights (as stored, where they fit) and
// their part of dweight and dbias in registers: the sums over rows cost one write of
// two rows a CTA, and the rest is norm_sums_kernel's.  Rows go to CTAs by their
// index, so the order of the sums does not depend on timing.  16384 x 4096 takes 79
// us (and 7 for the sums) in bfloat16, 126 in binary32, 0.75 and 0.94 of the copy
// rate: twelve working warps an SM leave half the issue slots empty, but threads
// with half the columns and twice the warps took 93.
template <int DT, int WT, bool kVec, int kRow, int kNv>
__global__ void __launch_bounds__(Ring<kRow, kNv, 2>::kAll, Ring<kRow, kNv, 2>::kCtas)
    norm_grad_ring_kernel(const __grid_constant__ NormGradParams p) {
  using R = Ring<kRow, kNv, 2>;
  constexpr int kW = kWide<DT, true>, kP = kW / 2;
  extern __shared__ __align__(128) unsigned char ring[];
  __shared__ __align__(16) float slots[2][2][32];
  __shared__ __align__(8) uint64_t full[R::kStages], empty[R::kStages];
  Walk<R, DT, kVec, 2> walk(p.rows, p.cols, ring, full, empty);
  walk.base[0] = p.x, walk.ld[0] = p.ld_x, walk.base[1] = p.dy, walk.ld[1] = p.ld_dy;
  walk.init();
  grid_dependency_wait();
  grid_dependents_launch();
  if (threadIdx.x >= R::kThreads) {
    if (threadIdx.x == R::kThreads) walk.bring_all(p.status);
    return;
  }
  const int t = threadIdx.x % kRow, group = threadIdx.x / kRow, cols = walk.cols;
  const float inv = __fdiv_rn(1.f, (float)cols);
  // the weights as they are stored: 16 bits two a word, binary32 one (where the
  // registers do not reach, from L1 every time)
  constexpr bool kHold = DT == kF32 || (WT != kF32 && kNv * kRow <= 1024);
  constexpr int kWords = kHold ? kW * Fmt<WT>::bytes / 4 : 1;
  uint32_t held[kNv][kWords];
  Two dw[kNv][kP], db[kNv][kP];
#pragma unroll
  for (int k = 0; k < kNv; ++k) {
#pragma unroll
    for (int j = 0; j < kP; ++j) dw[k][j] = db[k][j] = two(0.f, 0.f);
    if constexpr (kHold) {
      float v[kW];
#pragma unroll
      for (int j = 0; j < kW; ++j) v[j] = 0.f;
      if (holds<kW, kVec, kRow>(t, k, cols)) take_weight<WT, kW, kVec, kRow>(p.weight, t, k, cols, 1.f, v);
#pragma unroll
      for (int j = 0; j < kWords; ++j) {
        if constexpr (WT == kF32) held[k][j] = __float_as_uint(v[j]);
        else if constexpr (WT == kF16) held[k][j] = as_u32(__floats2half2_rn(v[2 * j], v[2 * j + 1]));
        else held[k][j] = as_u32(__floats2bfloat162_rn(v[2 * j], v[2 * j + 1]));
      }
    }
  }
  long long row = walk.start + group;
  float mean = 0.f, rstd = 0.f;
  if (row < p.rows) mean = p.mean[row], rstd = p.rstd[row];
  bool ok = true;
  for (unsigned q = 0; q < walk.turns; ++q, row += walk.step) {
    const bool live = row < p.rows;
    const Two shifts = two(-mean, -mean), scales = two(rstd, rstd);
    if (row + walk.step < p.rows) mean = p.mean[row + walk.step], rstd = p.rstd[row + walk.step];
    ok = walk.wait(q, ok);
    walk.edges(q);
    const unsigned char *from_x = walk.at(q, 0, group, row), *from_d = walk.at(q, 1, group, row);
    // a thread's group k of h, dy and weight (past the last column dy is 0)
    auto get = [&](int k, Two h[kP], Two d[kP], Two w[kP]) {
      float v[kW];
      take<DT, kVec, kRow>(from_x, t, k, cols, v);
      pair_up<kW>(v, h);
      take<DT, kVec, kRow>(from_d, t, k, cols, v);
      pair_up<kW>(v, d);
      if constexpr (kHold) {
#pragma unroll
        for (int j = 0; j < kP; ++j) {
          if constexpr (WT == kF32) {
            w[j] = two(__uint_as_float(held[k][2 * j]), __uint_as_float(held[k][2 * j + 1]));
          } else {
            const float2 f = WT == kF16 ? __half22float2(as_h2(held[k][j])) : __bfloat1622float2(as_b2(held[k][j]));
            w[j] = two(f.x, f.y);
          }
        }
      } else {
#pragma unroll
        for (int j = 0; j < kW; ++j) v[j] = 0.f;
        if (holds<kW, kVec, kRow>(t, k, cols)) take_weight<WT, kW, kVec, kRow>(p.weight, t, k, cols, 1.f, v);
        pair_up<kW>(v, w);
      }
#pragma unroll
      for (int j = 0; j < kP; ++j) h[j] = mul2(add2(h[j], shifts), scales);
    };
    Two sum1 = two(0.f, 0.f), sum2 = sum1;
    if (live) {
#pragma unroll
      for (int k = 0; k < kNv; ++k) {
        Two h[kP], d[kP], w[kP];
        get(k, h, d, w);
#pragma unroll
        for (int j = 0; j < kP; ++j) {
          dw[k][j] = fma2(d[j], h[j], dw[k][j]);
          db[k][j] = add2(db[k][j], d[j]);
          const Two g = mul2(d[j], w[j]);
          sum1 = add2(sum1, g);
          sum2 = fma2(g, h[j], sum2);
        }
      }
    }
    const float2 f1 = split(sum1), f2 = split(sum2);
    float s1 = __fadd_rn(f1.x, f1.y), s2 = __fadd_rn(f2.x, f2.y);
    row_sums<kRow>(s1, s2, slots[q & 1]);
    if (p.dx && live && ok) {
      s1 = __fmul_rn(s1, inv), s2 = __fmul_rn(s2, inv);
      const Two off = two(-s1, -s1), slope = two(-s2, -s2);
      const long long at = row * p.ld_dx;
#pragma unroll
      for (int k = 0; k < kNv; ++k) {
        Two h[kP], d[kP], w[kP];
        get(k, h, d, w);
        float v[kW];
#pragma unroll
        for (int j = 0; j < kP; ++j) {
          const float2 f = split(mul2(add2(fma2(h[j], slope, mul2(d[j], w[j])), off), scales));
          v[2 * j] = f.x, v[2 * j + 1] = f.y;
        }
        if (holds<kW, kVec, kRow>(t, k, cols)) put<DT, kVec, kRow>(p.dx, at, t, k, cols, v);
      }
    }
    walk.done(q);
  }
  if (!ok) walk.give_up(p.status);
  if (!p.sums) return;
  // the groups' sums in their order, through the ring, a column a place
  float *out = p.partials + (long long)blockIdx.x * 2 * p.cols;
  float *sums = reinterpret_cast<float *>(ring);
  constexpr int kWidth = kRow * kNv * kW;
#pragma unroll
  for (int half = 0; half < 2; ++half, out += p.cols) {
    work_sync<R::kThreads>();
#pragma unroll
    for (int k = 0; k < kNv; ++k)
#pragma unroll
      for (int j = 0; j < kP; ++j) {
        const float2 f = split(half ? db[k][j] : dw[k][j]);
        float *to = sums + group * kWidth;
        if constexpr (kVec) reinterpret_cast<float2 *>(to + (t + k * kRow) * kW)[j] = f;
        else to[t + (k * kW + 2 * j) * kRow] = f.x, to[t + (k * kW + 2 * j + 1) * kRow] = f.y;
      }
    work_sync<R::kThreads>();
    for (int c = threadIdx.x; c < cols; c += R::kThreads) {
      float v = sums[c];
#pragma unroll
      for (int g = 1; g < R::kRows; ++g) v = __fadd_rn(v, sums[g * kWidth + c]);
      out[c] = v;
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
  constexpr int kRows = kThreads<kRow> / kRow * kTogether<kRow, kNv>;
  return launch(norm_kernel<DT, WT, kVec, kRow, kNv>, dim3((unsigned)ceil_div(p.rows, (long long)kRows)),
                dim3(kThreads<kRow>), s, p);
}
// Threads that hold a row with four groups of 16 bytes (or as many elements) each.
template <int DT>
long long row_threads(long long cols) {
  return ceil_div(cols, 4ll * kWide<DT, true>);
}
// A CTA a row (of rows that one warp holds, a CTA for several), whose loads start at
// once: the fewest threads that hold a row in up to four groups of 16 bytes, or eight
// or sixteen single elements, each (16384 x 4096 binary32 on 512 threads instead of
// 256: 137 us for 79).
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
  if (p.cols <= 8192) return forward_of<DT, WT, false, 512, 16>(p, s);
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
template <int DT, int WT, bool kVec, int kRow, int kNv>
cudaError_t backward_ring(const NormGradParams &p, cudaStream_t s) {
  using R = Ring<kRow, kNv, 2>;
  const cudaError_t e = allow_smem<norm_grad_ring_kernel<DT, WT, kVec, kRow, kNv>>(R::kSmem);
  if (e != cudaSuccess) return e;
  return backward_by<WT>(norm_grad_ring_kernel<DT, WT, kVec, kRow, kNv>, R::kRows, R::kAll, R::kCtas, R::kSmem, p, s);
}
template <int DT, int WT, bool kVec>
cudaError_t backward_rings(const NormGradParams &p, long long threads, cudaStream_t s) {
  if (threads <= 8) return backward_ring<DT, WT, kVec, 8, 4>(p, s);
  if (threads <= 16) return backward_ring<DT, WT, kVec, 16, 4>(p, s);
  if (threads <= 32) return backward_ring<DT, WT, kVec, 32, 4>(p, s);
  if (threads <= 64) return backward_ring<DT, WT, kVec, 64, 4>(p, s);
  if (threads <= 128) return backward_ring<DT, WT, kVec, 128, 4>(p, s);
  if constexpr (DT == kF32) {
    return threads <= 256 ? backward_ring<DT, WT, kVec, 256, 4>(p, s) : backward_ring<DT, WT, kVec, 512, 4>(p, s);
  } else {
    return threads <= 256 ? backward_ring<DT, WT, kVec, 512, 2>(p, s) : backward_ring<DT, WT, kVec, 512, 4>(p, s);
  }
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
  const long long threads = row_threads<DT>(p.cols);
  if (threads > 512) return p.vec ? backward_long<DT, WT, true>(p, s) : backward_long<DT, WT, false>(p, s);
  return p.vec ? backward_rings<DT, WT, true>(p, threads, s) : backward_rings<DT, WT, false>(p, threads, s);
}

}  // namespace norm

}  // namespace rr
