// Helpers of the host-side argument checks, shared by the API translation units.
#pragma once

#include <stdarg.h>
#include <stdint.h>
#include <stdio.h>

namespace tsm {

// Text of the check that made this thread's last call fail (tsm_last_error_detail).
inline thread_local char g_detail[256];

inline int fail(int code, const char *fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_detail, sizeof g_detail, fmt, ap);
  va_end(ap);
  return code;
}

inline bool mul_ok(int64_t a, int64_t b, int64_t *out) { return !__builtin_mul_overflow(a, b, out); }
inline bool add_ok(int64_t a, int64_t b, int64_t *out) { return !__builtin_add_overflow(a, b, out); }

// Number of elements spanned by `batch` matrices of rows x cols with leading
// dimension ld and batch stride s: (batch-1)*s + (rows-1)*ld + cols.
inline bool extent(int64_t batch, int64_t s, int64_t rows, int64_t ld, int64_t cols, int64_t *out) {
  int64_t a, b, c;
  if (!mul_ok(batch - 1, s, &a) || !mul_ok(rows - 1, ld, &b)) return false;
  if (!add_ok(a, b, &c) || !add_ok(c, cols, out)) return false;
  return true;
}

inline bool ranges_overlap(const void *p, int64_t pbytes, const void *q, int64_t qbytes) {
  const uintptr_t a = (uintptr_t)p, b = (uintptr_t)q;
  return a < b + (uintptr_t)qbytes && b < a + (uintptr_t)pbytes;
}

}  // namespace tsm
