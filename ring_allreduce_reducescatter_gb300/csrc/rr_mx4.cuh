// rr_mx4.cuh -- device building blocks of the microscaled 4-bit operators and
// dropout: the counter-based generator, block scales, the 4-bit rounding and
// 8-element vectors of the storage formats.
#pragma once

#include "rr_device.cuh"
#include "rr_mx4.h"

namespace rr {

// --------------------------------------------------------------------------
// Philox4x32-10 (Salmon, Moraes, Dror, Shaw: "Parallel random numbers: as easy
// as 1, 2, 3", 2011).  The seed is the key, (i / 8, subsequence) the counter;
// the 128 bits are the 16-bit numbers of elements i .. i + 7, low half first.
// 16 bits an element: one call per 8 elements costs about 5 instructions an
// element, where 32 bits would cost 10 and bound dropout below the memory rate.
// --------------------------------------------------------------------------

__device__ __forceinline__ uint4 philox(const Generator &gen, unsigned long long group) {
  uint32_t c0 = (uint32_t)group, c1 = (uint32_t)(group >> 32), c2 = gen.sub_lo, c3 = gen.sub_hi;
#pragma unroll
  for (int r = 0; r < 10; ++r) {
    const unsigned long long p0 = (unsigned long long)c0 * 0xD2511F53u, p1 = (unsigned long long)c2 * 0xCD9E8D57u;
    c0 = (uint32_t)(p1 >> 32) ^ c1 ^ gen.keys[2 * r];
    c1 = (uint32_t)p1;
    c2 = (uint32_t)(p0 >> 32) ^ c3 ^ gen.keys[2 * r + 1];
    c3 = (uint32_t)p0;
  }
  return make_uint4(c0, c1, c2, c3);
}

// The numbers of elements i .. i + 7 for any i (two counters where i is not a
// multiple of 8).
__device__ __forceinline__ uint4 numbers8(const Generator &gen, unsigned long long i) {
  const unsigned long long g = i >> 3;
  const int sh = (int)(i & 7) * 2;
  uint4 a = philox(gen, g);
  if (sh == 0) return a;
  return funnel16(a, philox(gen, g + 1), sh);
}

// Whether element j of eight is kept: its number, in the high half of a word,
// against the cut (what lies below the high half cannot change the answer).
__device__ __forceinline__ bool kept(const uint4 &u, int j, uint32_t cut) {
  const uint32_t w = j < 2 ? u.x : j < 4 ? u.y : j < 6 ? u.z : u.w;
  return ((j & 1) ? w : w << 16) >= cut;
}

// --------------------------------------------------------------------------
// storage formats, eight elements at a time
// --------------------------------------------------------------------------

template <int DT>
__device__ __forceinline__ float to_f32(typename Fmt<DT>::type x) {
  if constexpr (DT == kF32) return x;
  else if constexpr (DT == kF16) return __half2float(x);
  else return __bfloat162float(x);
}
template <int DT>
__device__ __forceinline__ typename Fmt<DT>::type from_f32(float x) {
  if constexpr (DT == kF32) return x;
  else if constexpr (DT == kF16) return __float2half_rn(x);
  else return __float2bfloat16_rn(x);
}

template <int DT>
__device__ __forceinline__ void widen8(const uint4 *raw, float v[8]) {
  if constexpr (DT == kF32) {
    v[0] = __uint_as_float(raw[0].x), v[1] = __uint_as_float(raw[0].y);
    v[2] = __uint_as_float(raw[0].z), v[3] = __uint_as_float(raw[0].w);
    v[4] = __uint_as_float(raw[1].x), v[5] = __uint_as_float(raw[1].y);
    v[6] = __uint_as_float(raw[1].z), v[7] = __uint_as_float(raw[1].w);
  } else {
    const uint32_t w[4] = {raw[0].x, raw[0].y, raw[0].z, raw[0].w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float2 f;
      if constexpr (DT == kF16) f = __half22float2(as_h2(w[j]));
      else f = __bfloat1622float2(as_b2(w[j]));
      v[2 * j] = f.x, v[2 * j + 1] = f.y;
    }
  }
}
template <int DT>
__device__ __forceinline__ void narrow8(const float v[8], uint4 *raw) {
  if constexpr (DT == kF32) {
    raw[0] = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
    raw[1] = make_uint4(__float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]), __float_as_uint(v[7]));
  } else {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (DT == kF16) w[j] = as_u32(__floats2half2_rn(v[2 * j], v[2 * j + 1]));
      else w[j] = as_u32(__floats2bfloat162_rn(v[2 * j], v[2 * j + 1]));
    }
    raw[0] = make_uint4(w[0], w[1], w[2], w[3]);
  }
}
// uint4s that hold eight elements
template <int DT>
constexpr int kRaw8 = DT == kF32 ? 2 : 1;

// 32 bytes from a 32-byte aligned address; the kernel may write them too.
__device__ __forceinline__ void ldg32(const void *p, uint4 &a, uint4 &b) {
  asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(a.x), "=r"(a.y), "=r"(a.z), "=r"(a.w), "=r"(b.x), "=r"(b.y), "=r"(b.z), "=r"(b.w)
               : "l"(p));
}

// The same through the read-only path without an L1 allocation.
__device__ __forceinline__ void ldg32_stream(const void *p, uint4 &a, uint4 &b) {
  asm volatile("ld.global.nc.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(a.x), "=r"(a.y), "=r"(a.z), "=r"(a.w), "=r"(b.x), "=r"(b.y), "=r"(b.z), "=r"(b.w)
               : "l"(p));
}

// 16 bytes that the same kernel may write: an output may be its input, and the
// read-only path is for memory that nothing writes while the kernel runs.
__device__ __forceinline__ uint4 ld16(const void *p) {
  uint4 v;
  asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}
// The same without an L1 allocation, for what is read once.
__device__ __forceinline__ uint4 ld16_stream(const void *p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

// Eight elements from p, of which the first `valid` exist (the others read as
// zero), where the output may be written; vec: all eight exist and p is 16-byte
// aligned.
template <int DT>
__device__ __forceinline__ void load8(const void *base, long long at, int valid, bool vec, float v[8]) {
  using T = typename Fmt<DT>::type;
  const T *p = static_cast<const T *>(base) + at;
  if (vec && valid >= 8) {
    uint4 raw[kRaw8<DT>];
#pragma unroll
    for (int j = 0; j < kRaw8<DT>; ++j) raw[j] = ld16_stream(reinterpret_cast<const uint4 *>(p) + j);
    widen8<DT>(raw, v);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = j < valid ? to_f32<DT>(p[j]) : 0.f;
  }
}
template <int DT>
__device__ __forceinline__ void store8(void *base, long long at, int valid, bool vec, const float v[8]) {
  using T = typename Fmt<DT>::type;
  T *p = static_cast<T *>(base) + at;
  if (vec && valid >= 8) {
    uint4 raw[kRaw8<DT>];
    narrow8<DT>(v, raw);
#pragma unroll
    for (int j = 0; j < kRaw8<DT>; ++j) stg_stream(reinterpret_cast<uint4 *>(p) + j, raw[j]);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < valid) p[j] = from_f32<DT>(v[j]);
  }
}

// 32 bytes to a 32-byte aligned address: a whole sector from one thread.
__device__ __forceinline__ void stg32(void *p, uint4 a, uint4 b) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(a.x), "r"(a.y), "r"(a.z),
               "r"(a.w), "r"(b.x), "r"(b.y), "r"(b.z), "r"(b.w)
               : "memory");
}

// v[j] *= scale where element i + j is kept, 0 where it is dropped.
__device__ __forceinline__ void drop8(const DropParams &d, const uint4 &u, float v[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = kept(u, j, d.cut) ? __fmul_rn(v[j], d.scale) : 0.f;
}
__device__ __forceinline__ void drop8(const DropParams &d, unsigned long long i, float v[8]) {
  drop8(d, numbers8(d.gen, d.first + i), v);
}

// Threads of the element-by-element kernels: tx groups of a row by 256 / tx
// rows a block, rows beyond the grid in a loop.
constexpr int kFlatThreads = 256;

// --------------------------------------------------------------------------
// block scales and 4-bit elements
// --------------------------------------------------------------------------

// The scale byte X + 127 of a block whose largest magnitude has these binary32
// bits: X is the smallest exponent >= -127 with amax <= 6 * 2^X, so nothing is
// ever clipped (the floor(log2 amax) - 2 rule clips up to a quarter off the
// largest element, which would bias stochastic rounding).  With amax = m 2^e,
// 1 <= m < 2: X = e - 2 if m <= 1.5, else e - 1.  255 (not a number) for a
// block that holds an infinity or a NaN.
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax_bits) {
  if (amax_bits >= 0x7f800000u) return 255u;
  const int x = (int)(amax_bits >> 23) - 2 + ((amax_bits & 0x7fffffu) > 0x400000u ? 1 : 0);
  return x < 0 ? 0u : (uint32_t)x;
}
// 2^-X for a scale byte below 255 (at most 253 here); 0 for 255.
__device__ __forceinline__ float inverse_scale(uint32_t byte) {
  return byte == 255u ? 0.f : __uint_as_float((254u - byte) << 23);
}
// 2^X, NaN for 255.
__device__ __forceinline__ float scale_value(uint32_t byte) {
  return __uint_as_float(byte == 0u ? 0x00400000u : byte == 255u ? 0x7fffffffu : byte << 23);
}

// Eight scaled elements to eight 4-bit codes, nearest (ties to even).
__device__ __forceinline__ uint32_t pack8_nearest(const float v[8]) {
  uint32_t r;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(r)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return r;
}
// The same with stochastic rounding.  |v| * 2^-126, rounded toward zero, puts
// the code in the top bits of a binary32 word: exponent 1 is the code's
// exponent 1, and the code's subnormal step falls on binary32's subnormals.
// The 22 bits below are the fraction f of a grid step; adding the number to
// their top 16 carries into the code exactly when floor(f 2^16) + u >= 2^16.
// Two bits further up the sum leaves the code in the top byte, and byte
// permutations gather four codes, or four signs, at a time.
__device__ __forceinline__ uint32_t pack8_stochastic(const float v[8], const uint4 &u) {
  const uint32_t n[4] = {u.x, u.y, u.z, u.w};
  uint32_t s[8];
#pragma unroll
  for (int j = 0; j < 8; ++j)
    s[j] = __float_as_uint(__fmul_rz(fabsf(v[j]), __uint_as_float(0x00800000u))) * 4 +
           __byte_perm(n[j / 2], 0, (j & 1) ? 0x4324 : 0x4104);
  uint32_t even = __byte_perm(__byte_perm(s[0], s[2], 0x0073), __byte_perm(s[4], s[6], 0x0073), 0x5410);
  uint32_t odd = __byte_perm(__byte_perm(s[1], s[3], 0x0073), __byte_perm(s[5], s[7], 0x0073), 0x5410);
#pragma unroll
  for (int j = 0; j < 8; ++j) s[j] = __float_as_uint(v[j]);
  const uint32_t se = __byte_perm(__byte_perm(s[0], s[2], 0x0073), __byte_perm(s[4], s[6], 0x0073), 0x5410);
  const uint32_t so = __byte_perm(__byte_perm(s[1], s[3], 0x0073), __byte_perm(s[5], s[7], 0x0073), 0x5410);
  even |= (se & 0x80808080u) >> 4;
  odd = odd * 16 | (so & 0x80808080u);
  return even | odd;
}

// The values of eight 4-bit codes, times a scale.
__device__ __forceinline__ void unpack8(uint32_t codes, float scale, float v[8]) {
  uint32_t h[4];
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "mov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(codes));
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 f = __half22float2(as_h2(h[j]));
    v[2 * j] = __fmul_rn(f.x, scale), v[2 * j + 1] = __fmul_rn(f.y, scale);
  }
}

// Byte offset of the scale of (row, block) in the tiled scales.
__device__ __forceinline__ long long scale_offset(long long row, long long block, long long tiles_k) {
  const int r = (int)(row & 127), j = (int)(block & 7);
  return ((row >> 7) * tiles_k + (block >> 3)) * kMx4TileBytes + (j >> 2) * kMx4AtomBytes + (r & 31) * 16 +
         (r >> 5) * 4 + (j & 3);
}

}  // namespace rr
