// api_common.h -- what the C entry points share (internal to libnvfp4.so):
// the calling thread's error text, the size bound and the launch status.
#pragma once

#include <hip/hip_runtime_api.h>

#include <cstdarg>
#include <cstdint>
#include <cstdio>

#include "../../include/nvfp4.h"

namespace nvfp4 {
namespace api {

inline thread_local char g_last_error[256] = "";

// No tensor or buffer the library touches may exceed 2^40 elements or bytes
// (far beyond the 288 GB of one MI355X): with that bound every size, offset
// and grid computation in the entry points and in the launchers stays within
// int64 (and the grids within their 32-bit dimensions).
constexpr int64_t kMaxElems = int64_t(1) << 40;

inline int fail(int status, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_last_error, sizeof g_last_error, fmt, ap);
  va_end(ap);
  return status;
}

inline bool aligned(const void* p, uintptr_t a) {
  return (reinterpret_cast<uintptr_t>(p) % a) == 0;
}

inline int launched(hipError_t e) {
  if (e != hipSuccess) return fail(NVFP4_ERR_LAUNCH, "launch failed: %s", hipGetErrorString(e));
  g_last_error[0] = '\0';
  return NVFP4_OK;
}

inline hipStream_t as_stream(void* s) { return reinterpret_cast<hipStream_t>(s); }

}  // namespace api
}  // namespace nvfp4
