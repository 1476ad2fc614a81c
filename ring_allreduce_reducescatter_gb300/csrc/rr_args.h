// rr_args.h -- checks of the arguments that the operators' entry points share:
// extents of strided matrices, overlap, alignment.  Host only, no CUDA call.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "ringred.h"

namespace rr {

inline size_t elem_bytes(int t) { return t == RR_FP32 ? 4 : 2; }
inline bool valid_type(int t) { return t == RR_FP32 || t == RR_FP16 || t == RR_BF16; }

struct Span {
  uintptr_t lo = 0, hi = 0;
  bool overlaps(const Span &o) const { return lo < hi && o.lo < o.hi && lo < o.hi && o.lo < hi; }
};

inline bool span_of(const void *ptr, size_t bytes, size_t align, Span *s) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(ptr);
  if (bytes == 0) return *s = Span{}, true;
  if (a == 0 || a % align != 0 || a > UINTPTR_MAX - bytes) return false;
  *s = Span{a, a + bytes};
  return true;
}

// A strided matrix: its extent, and whether 16-byte groups of its rows are aligned.
inline bool matrix_span(const void *ptr, size_t rows, size_t cols, size_t ld, size_t E, Span *s) {
  if (rows == 0 || cols == 0) return *s = Span{}, true;
  if (ld < cols || ld > (SIZE_MAX / 8) / E / rows) return false;
  return span_of(ptr, ((rows - 1) * ld + cols) * E, E, s);
}
// Whether two strided matrices of rows x cols share an element.  Of one ld they
// may lie beside one another in the rows of one array: the second begins `at`
// bytes into a row of the first, past its last column, and ends in that row.
inline bool share(const Span &a, size_t ld_a, const Span &b, size_t ld_b, size_t cols, size_t E) {
  if (!a.overlaps(b)) return false;
  if (ld_a != ld_b) return true;
  const size_t row = ld_a * E, apart = a.lo < b.lo ? (b.lo - a.lo) % row : row - (a.lo - b.lo) % row, at = apart % row;
  return at < cols * E || at + cols * E > row;
}
inline bool aligned16(const void *ptr, size_t rows, size_t ld, size_t E) {
  return reinterpret_cast<uintptr_t>(ptr) % 16 == 0 && (rows <= 1 || ld * E % 16 == 0);
}

inline bool aligned32(const void *ptr, size_t rows, size_t ld, size_t E) {
  return reinterpret_cast<uintptr_t>(ptr) % 32 == 0 && (rows <= 1 || ld * E % 32 == 0);
}

}  // namespace rr
