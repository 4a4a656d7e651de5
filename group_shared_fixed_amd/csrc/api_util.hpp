// Host-side helpers of the C ABI's argument checks and workspace layouts.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "haste.h"

namespace haste {

inline size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }
inline int64_t round_up(int64_t x, int64_t m) { return (x + m - 1) / m * m; }
inline bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

inline int check_ws(void* ws, size_t ws_bytes, size_t need)
{
    if (need == 0) return HASTE_OK;
    if (ws == nullptr || ws_bytes < need || ((uintptr_t)ws & 255u) != 0) return HASTE_ERR_WORKSPACE;
    return HASTE_OK;
}

inline int hip_status()
{
    return hipGetLastError() == hipSuccess ? HASTE_OK : HASTE_ERR_HIP;
}

}  // namespace haste

#define HASTE_TRY(x)                 \
    do {                             \
        int _st = (x);               \
        if (_st != HASTE_OK) return _st; \
    } while (0)
