// What the entry points check their arguments with: sizes, alignment, overlap.
#pragma once
#include <stdint.h>

#include "desc.h"
#include "muonh.h"

namespace muonh {

inline int64_t up(int64_t v, int64_t m) { return (v + m - 1) / m * m; }

struct Span {
  uintptr_t lo, hi;
};
inline Span span_of(const void* p, int64_t bytes) { return {(uintptr_t)p, (uintptr_t)p + (p ? (uintptr_t)bytes : 0)}; }
// Empty spans (a null pointer, no bytes) overlap nothing.
inline bool overlap(const Span& x, const Span& y) { return x.lo < x.hi && y.lo < y.hi && x.lo < y.hi && y.lo < x.hi; }

inline bool bad_dtype(int d) { return d != MUONH_F32 && d != MUONH_BF16; }
inline int64_t dtype_size(int d) { return d == MUONH_F32 ? 4 : 2; }
inline int internal_dtype(int d) { return d == MUONH_F32 ? DT_F32 : DT_BF16; }
inline bool misaligned(const void* p, int64_t a) { return (uintptr_t)p % a != 0; }

}  // namespace muonh
