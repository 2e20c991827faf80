// What the C entry points share on the host: status text, pointer checks (not installed).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "replayssm.h"

namespace rs {

// Keeps the text for replayssm_last_error() of this thread and returns `code`.
int fail(int code, const char* fmt, ...);

namespace host {

using rs::fail;

inline int hip_result(hipError_t e, const char* what) {
  if (e == hipSuccess) return REPLAYSSM_OK;
  return fail(REPLAYSSM_EHIP, "%s: %s", what, hipGetErrorString(e));
}

inline bool aligned(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline hipStream_t as_stream(void* s) { return reinterpret_cast<hipStream_t>(s); }

// Pointer must be non-NULL and 16-byte aligned.
#define NEED(ptr)                                                                   \
  do {                                                                              \
    if ((ptr) == nullptr) return fail(REPLAYSSM_EINVAL, "%s is NULL", #ptr);        \
    if (!aligned(ptr)) return fail(REPLAYSSM_EINVAL, "%s is not 16-byte aligned", #ptr); \
  } while (0)

}  // namespace host
}  // namespace rs
