// ckda_checks.hpp -- argument checks and error reporting shared by the C ABI's
// source files (host code).
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "ckda.h"

namespace ckda {

// Records the thread's error text and returns `status`; ok() clears the text.
int fail(int status, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
int ok();

inline bool supported_dim(int d) { return d == 16 || d == 32 || d == 64 || d == 128; }
inline bool supported_chunk(int c) { return c == 16 || c == 32 || c == 64; }
inline bool supported_dtype(int t) { return t == CKDA_DTYPE_F32 || t == CKDA_DTYPE_BF16; }
inline size_t dtype_bytes(int t) { return t == CKDA_DTYPE_BF16 ? 2 : 4; }

struct Range {
  const char* name;
  uintptr_t lo, hi;  // [lo, hi)
};

inline Range range(const char* name, const void* p, size_t bytes) {
  uintptr_t a = (uintptr_t)p;
  return Range{name, a, a + bytes};
}

inline bool overlap(const Range& a, const Range& b) {
  return a.lo < a.hi && b.lo < b.hi && a.lo < b.hi && b.lo < a.hi;
}

inline bool misaligned(const void* p) { return ((uintptr_t)p & 15u) != 0; }

}  // namespace ckda
