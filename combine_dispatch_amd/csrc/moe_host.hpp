// moe_host.hpp -- host-side helpers shared by the files that implement the C ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <string.h>

#include "../../include/moe.h"

namespace moe {

// gfx950 check, cached per device.
inline int device_ok() {
    static int cache[64];  // 0 unknown, 1 ok, 2 bad
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0) return 0;
    if (dev < 64 && cache[dev]) return cache[dev] == 1;
    hipDeviceProp_t prop;
    if (hipGetDeviceProperties(&prop, dev) != hipSuccess) return 0;
    const int ok = strncmp(prop.gcnArchName, "gfx950", 6) == 0;
    if (dev < 64) cache[dev] = ok ? 1 : 2;
    return ok;
}

// Compute units of the current device, cached per device (at least 8).
inline int device_cus() {
    static int cus[64];
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0) dev = 0;
    int n = dev < 64 ? cus[dev] : 0;
    if (n <= 0) {
        if (hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || n < 8)
            n = 8;
        if (dev < 64) cus[dev] = n;
    }
    return n;
}

inline int launch_status() { return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_DEVICE; }

inline bool aligned(const void* p, size_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

}  // namespace moe
