// Error reporting shared by libpe's C entry points: a status code is returned
// and a message kept for pe_last_error() on the calling thread.
#pragma once
#include <hip/hip_runtime.h>

#include "../../include/pe.h"

namespace pe {
int fail(int code, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
}  // namespace pe

#define PE_HIP(call)                                                                      \
  do {                                                                                    \
    hipError_t e_ = (call);                                                               \
    if (e_ != hipSuccess)                                                                 \
      return pe::fail(PE_ERR_HIP, "%s failed: %s (line %d)", #call, hipGetErrorString(e_), \
                      __LINE__);                                                          \
  } while (0)
