// Host helpers shared by the C entry points (defined in api.hip).
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "ttt.h"

namespace ttt {

// Sets the thread's error text and returns `status`.
int fail(int status, const char *fmt, ...) __attribute__((format(printf, 2, 3)));
bool overlap(const void *a, size_t na, const void *b, size_t nb);
size_t align256(size_t x);
size_t esize(int dtype);
int check_ws(void *ws, size_t have, size_t need);

// Timing events around one kernel kind's launches (both null when timing is off).
struct Timing {
  hipEvent_t e0, e1;
};
Timing timing_begin(hipStream_t s);
void timing_end(int kind, const Timing &t, hipStream_t s);

template <class F> int run(int kind, const char *what, hipStream_t s, F &&f) {
  const Timing t = timing_begin(s);
  const hipError_t err = f();
  timing_end(kind, t, s);
  if (err != hipSuccess) return fail(TTT_EHIP, "%s: %s", what, hipGetErrorString(err));
  return TTT_OK;
}

// ------------------------------------------------------------------ rows
// A launch has at most 2^32 - 1 work-items in a direction: below 2^23 workgroups of 512.
constexpr int64_t kMaxGroups = (int64_t(1) << 23) - 1;
constexpr int64_t kMaxRows = 2147483647LL - 64;

// Rows [n][ld] of `width` elements of `es` bytes.
struct Rows {
  const void *p;
  int64_t ld, width;
  size_t es;
  const char *name;
};

inline int check_row(const Rows &r, int64_t n) {
  if (r.ld < r.width)
    return fail(TTT_EINVAL, "ld of %s (%lld) < its width (%lld)", r.name, (long long)r.ld, (long long)r.width);
  if (n == 0) return TTT_OK;
  if (!r.p) return fail(TTT_EINVAL, "%s is null", r.name);
  if (((uintptr_t)r.p) % 16 != 0 || (r.ld * (int64_t)r.es) % 16 != 0)
    return fail(TTT_EINVAL, "%s rows must be 16-byte aligned", r.name);
  return TTT_OK;
}

// Whether two sets of n rows share bytes.  Column slices of one buffer (equal strides) do not
// where their columns are apart.
inline bool rows_overlap(const Rows &a, const Rows &b, int64_t n) {
  if (n == 0 || !a.p || !b.p) return false;
  const int64_t sa = a.ld * (int64_t)a.es, sb = b.ld * (int64_t)b.es;
  const int64_t wa = a.width * (int64_t)a.es, wb = b.width * (int64_t)b.es;
  if (!overlap(a.p, (size_t)((n - 1) * sa + wa), b.p, (size_t)((n - 1) * sb + wb))) return false;
  if (sa != sb || n == 1) return true;
  int64_t d = (int64_t)((intptr_t)b.p - (intptr_t)a.p) % sa;
  if (d < 0) d += sa;
  return d < wa || d + wb > sa;
}
inline bool rows_overlap_span(const Rows &a, int64_t n, const void *p, size_t bytes) {
  return n > 0 && a.p && p &&
         overlap(a.p, (size_t)(((n - 1) * a.ld + a.width) * (int64_t)a.es), p, bytes);
}

inline int check_dtype(int dtype) {
  if (dtype != TTT_F32 && dtype != TTT_BF16) return fail(TTT_EUNSUPPORTED, "unknown dtype %d", dtype);
  return TTT_OK;
}
inline int check_aligned(const void *p, const char *name) {
  if (p && ((uintptr_t)p) % 16 != 0) return fail(TTT_EINVAL, "%s must be 16-byte aligned", name);
  return TTT_OK;
}

}  // namespace ttt
