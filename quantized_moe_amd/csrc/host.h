// Host-side pieces shared by the translation units with C entry points: the
// thread-local error text, the device check and the last-plan text.  Defined
// in runtime.cpp.
#pragma once

#include "internal.h"

namespace chord {

// Records the error text of this thread and returns `s`.
chord_status fail(chord_status s, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
chord_status hip_fail(hipError_t e, const char* what);
void clear_last_error();
void set_last_plan(const char* text);
// CHORD_OK if the current device is a gfx950; its compute units in *cus.
chord_status check_device(int* cus);

#define CHORD_CHECK(expr)                    \
  do {                                       \
    chord_status _s = (expr);                \
    if (_s != CHORD_OK) return _s;           \
  } while (0)

#define HIP_TRY(expr, what)                       \
  do {                                            \
    hipError_t _e = (expr);                       \
    if (_e != hipSuccess) return hip_fail(_e, what); \
  } while (0)

}  // namespace chord
