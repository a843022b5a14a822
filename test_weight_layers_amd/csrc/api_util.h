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

}  // namespace ttt
