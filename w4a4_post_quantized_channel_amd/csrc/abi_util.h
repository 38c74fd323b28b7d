// Helpers of the C entry points: the thread-local error message, alignment
// and launch status.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/w4a4.h"

namespace w4a4 {

// Sets the message w4a4_last_error() returns on this thread; returns status.
int fail(int status, const char* fmt, ...) __attribute__((format(printf, 2, 3)));

inline int ok() { return W4A4_OK; }

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

inline int launch_status(hipError_t e, const char* what) {
  if (e != hipSuccess) return fail(W4A4_ERR_LAUNCH_FAILED, "%s: %s", what, hipGetErrorString(e));
  return ok();
}

}  // namespace w4a4
