// What the C entry points share on the host: status text, checks of pointers, types and strides (not installed).
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

inline int element_bytes(int dtype) { return dtype == REPLAYSSM_F32 ? 4 : 2; }

inline int check_dtype(int dtype, const char* name) {
  if (dtype != REPLAYSSM_F32 && dtype != REPLAYSSM_BF16 && dtype != REPLAYSSM_F16)
    return fail(REPLAYSSM_EINVAL, "%s %d unknown", name, dtype);
  return REPLAYSSM_OK;
}

// Elements between tokens: at least the row, whole 16-byte units.
inline int check_stride(int64_t stride, int64_t row, int dtype, const char* name) {
  if (stride < row || stride > (int64_t)1 << 31)
    return fail(REPLAYSSM_EINVAL, "%s=%lld outside %lld..2^31", name, (long long)stride, (long long)row);
  if (stride * element_bytes(dtype) % 16 != 0)
    return fail(REPLAYSSM_EINVAL, "%s=%lld is not a multiple of 16 bytes", name, (long long)stride);
  return REPLAYSSM_OK;
}

}  // namespace host
}  // namespace rs
