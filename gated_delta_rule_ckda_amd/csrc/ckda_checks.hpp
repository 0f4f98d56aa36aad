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

inline int check_workspace(const char* fn, const void* workspace, size_t have, size_t need) {
  if (!workspace) return fail(CKDA_ERR_WORKSPACE, "%s: workspace is NULL", fn);
  if (have < need) return fail(CKDA_ERR_WORKSPACE, "%s: workspace of %zu bytes, need %zu", fn, have, need);
  if (((uintptr_t)workspace & 255u) != 0) return fail(CKDA_ERR_WORKSPACE, "%s: workspace not 256-byte aligned", fn);
  return CKDA_OK;
}

inline int check_aligned(const char* fn, const Range* r, int n) {
  for (int i = 0; i < n; ++i)
    if (r[i].lo && misaligned((const void*)r[i].lo))
      return fail(CKDA_ERR_DIM, "%s: %s is not 16-byte aligned", fn, r[i].name);
  return CKDA_OK;
}

// no output overlaps an input or another output, and the workspace (among the
// inputs, or NULL) no input; `same` may equal `with` exactly
inline int check_alias(const char* fn, const Range* in, int nin, const Range* out, int nout, const Range* ws,
                       const Range* same = nullptr, const Range* with = nullptr) {
  for (int j = 0; ws && j < nin; ++j)
    if (&in[j] != ws && overlap(*ws, in[j])) return fail(CKDA_ERR_ALIAS, "%s: workspace overlaps %s", fn, in[j].name);
  for (int i = 0; i < nout; ++i) {
    for (int j = 0; j < nin; ++j) {
      if (&out[i] == same && &in[j] == with && same->lo == with->lo) continue;
      if (overlap(out[i], in[j])) return fail(CKDA_ERR_ALIAS, "%s: %s overlaps %s", fn, out[i].name, in[j].name);
    }
    for (int j = 0; j < nout; ++j)
      if (j != i && overlap(out[i], out[j]))
        return fail(CKDA_ERR_ALIAS, "%s: %s overlaps %s", fn, out[i].name, out[j].name);
  }
  return CKDA_OK;
}

}  // namespace ckda
