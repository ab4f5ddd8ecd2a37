// Argument checks shared by the C-ABI translation units: plain host code that
// touches no HIP API, and the device check that runs once the arguments are
// known to be good.
#pragma once

#include <atomic>
#include <cstring>

#include "bg_internal.hpp"

namespace bg {

constexpr uint32_t kMaxDim = 0x7FFFFFFFu;   // kernels index rows and K with int32

struct Range {
    uintptr_t lo, hi;   // [lo, hi), empty when lo == hi
};

inline Range range_of(const void* p, uint64_t bytes) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(p);
    return Range{a, a + (uintptr_t)bytes};
}

inline bool overlap(Range x, Range y) {
    if (x.lo == x.hi || y.lo == y.hi) return false;
    return x.lo < y.hi && y.lo < x.hi;
}

inline bool misaligned(const void* p, uint64_t bytes) {
    return bytes != 0 && (reinterpret_cast<uintptr_t>(p) & 15u) != 0;
}

inline bool missing(const void* p, uint64_t bytes) { return bytes != 0 && p == nullptr; }

inline bool dims_ok(uint32_t M, uint32_t N, uint32_t K) {
    return M <= kMaxDim && N <= kMaxDim && K <= kMaxDim;
}

// Per-device cache: 0 unknown, 2 not gfx950, otherwise 2 + compute-unit count.
inline std::atomic<int> g_dev_info[64];

// Checks the current device and reports its compute-unit count.
inline bg_status check_device(uint32_t* cus) {
    int dev = -1;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0) return BG_ERR_DEVICE;
    if (dev < 64) {
        const int cached = g_dev_info[dev].load(std::memory_order_relaxed);
        if (cached == 2) return BG_ERR_DEVICE;
        if (cached > 2) {
            *cus = (uint32_t)(cached - 2);
            return BG_OK;
        }
    }
    hipDeviceProp_t prop;
    if (hipGetDeviceProperties(&prop, dev) != hipSuccess) return BG_ERR_DEVICE;
    const bool ok = std::strncmp(prop.gcnArchName, "gfx950", 6) == 0;
    const int n = prop.multiProcessorCount > 0 ? prop.multiProcessorCount : 256;
    if (dev < 64) g_dev_info[dev].store(ok ? 2 + n : 2, std::memory_order_relaxed);
    *cus = (uint32_t)n;
    return ok ? BG_OK : BG_ERR_DEVICE;
}

inline bg_status check_device() {
    uint32_t cus = 0;
    return check_device(&cus);
}

inline bg_status launched(hipError_t e) { return e == hipSuccess ? BG_OK : BG_ERR_LAUNCH; }

}  // namespace bg
