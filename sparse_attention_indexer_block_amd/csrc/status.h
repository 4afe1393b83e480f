// Error reporting shared by the C entry points.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/misa.h"

namespace misa {

// Records the calling thread's error text and returns st.
misa_status fail(misa_status st, const char* fmt, ...);
misa_status hip_fail(hipError_t e, const char* where);

inline bool aligned(const void* ptr, size_t a) { return (reinterpret_cast<uintptr_t>(ptr) % a) == 0; }

}  // namespace misa

#define MISA_TRY(expr)                   \
  do {                                   \
    misa_status _st = (expr);            \
    if (_st != MISA_OK) return _st;      \
  } while (0)

#define HIP_TRY(expr, where)                     \
  do {                                           \
    hipError_t _e = (expr);                      \
    if (_e != hipSuccess) return hip_fail(_e, where); \
  } while (0)
