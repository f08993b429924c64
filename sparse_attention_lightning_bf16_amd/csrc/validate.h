// Host-side argument checks shared by the C entry points: alignment, element
// counts, the device of a pointer, and a launch's status.
#pragma once

#include <stdint.h>

#include <initializer_list>

#include <hip/hip_runtime_api.h>

#include "lix.h"

namespace lix {

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// Element counts must stay far inside int64 and the kernels' 32-bit grid limits.
inline bool fits(long long a, long long b, long long c = 1, long long d = 1) {
    const long long lim = 1LL << 40;
    long long x = a;
    for (long long f : {b, c, d}) {
        if (f <= 0 || x > lim / f) return false;
        x *= f;
    }
    return true;
}

// Every pointer must be device (or managed) memory of the current device.
inline int check_device(std::initializer_list<const void*> ptrs) {
    int dev = -1;
    if (hipGetDevice(&dev) != hipSuccess) return LIX_ERR_DEVICE;
    for (const void* p : ptrs) {
        if (p == nullptr) continue;
        hipPointerAttribute_t attr;
        if (hipPointerGetAttributes(&attr, p) != hipSuccess) {
            (void)hipGetLastError();
            return LIX_ERR_DEVICE;
        }
        if (attr.type != hipMemoryTypeDevice && attr.type != hipMemoryTypeManaged) return LIX_ERR_DEVICE;
        if (attr.device != dev) return LIX_ERR_DEVICE;
    }
    return LIX_OK;
}

inline int launch_status(hipError_t e) { return e == hipSuccess ? LIX_OK : LIX_ERR_LAUNCH; }

}  // namespace lix
