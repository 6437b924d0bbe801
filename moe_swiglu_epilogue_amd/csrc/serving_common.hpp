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

// Whether [p, p + n) and [q, q + m) share a byte.
inline bool overlap(const void* p, int64_t n, const void* q, int64_t m)
{
    if (!p || !q || n <= 0 || m <= 0)
        return false;
    const uintptr_t a = (uintptr_t)p, b = (uintptr_t)q;
    return a <= b ? b - a < (uint64_t)n : a - b < (uint64_t)m;
}

inline nvfp4_status_t launched()
{
    return hipGetLastError() == hipSuccess ? NVFP4_SUCCESS : NVFP4_ERROR_LAUNCH;
}

template <class T>
constexpr T ceil_div(T a, T b) { return (a + b - 1) / b; }

}  // namespace serving
