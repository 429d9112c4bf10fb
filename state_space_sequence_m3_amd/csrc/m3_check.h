// m3_check.h -- host-side checks shared by the C-ABI files (api.hip, block_api.hip): the calling
// thread's error text, the device check and overlap tests.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "m3scan.h"

namespace m3 {

// Sets the text m3_last_error() returns on this thread and returns `s`.
m3_status fail(m3_status s, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
// M3_OK when the current HIP device is a gfx950 GPU (cached per device).
m3_status check_device();
// Compute units of the current device (256 when there is none to ask), cached per device.
int device_cus();
m3_status launched(hipError_t e, const char* what);

inline bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

// [p, p + n) and [q, q + m) overlap (both non-empty)
inline bool overlap(const void* p, size_t n, const void* q, size_t m) {
    if (!p || !q || n == 0 || m == 0) return false;
    const uintptr_t a = (uintptr_t)p, b = (uintptr_t)q;
    return a < b + m && b < a + n;
}

}  // namespace m3
