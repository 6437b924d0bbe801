// Host-side helpers shared by the sources behind include/nvfp4_serving.h.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "nvfp4_serving.h"

namespace serving {

inline bool aligned(const void* p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

// rows * pitch * size bytes fits in int64 (all non-negative).
inline bool extent_ok(int64_t rows, int64_t pitch, int64_t size)
{
    return pitch == 0 || rows <= INT64_MAX / size / pitch;
}

inline nvfp4_status_t launched()
{
    return hipGetLastError() == hipSuccess ? NVFP4_SUCCESS : NVFP4_ERROR_LAUNCH;
}

template <class T>
constexpr T ceil_div(T a, T b) { return (a + b - 1) / b; }

}  // namespace serving
