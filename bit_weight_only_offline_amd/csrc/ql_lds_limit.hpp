// A kernel's limit of dynamic LDS, raised once on each device that launches it.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <atomic>

namespace ql {

// One static object a kernel.  A failure is reported and tried again by the next call; a device
// number past the mask is raised by every call.
struct LdsLimit {
    std::atomic<uint64_t> raised{0};

    hipError_t raise(const void *kern, int bytes) {
        int device = 0;
        hipError_t e = hipGetDevice(&device);
        if (e != hipSuccess) return e;
        const uint64_t bit = device >= 0 && device < 64 ? uint64_t(1) << device : 0;
        if (raised.load(std::memory_order_relaxed) & bit) return hipSuccess;
        e = hipFuncSetAttribute(kern, hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e == hipSuccess) raised.fetch_or(bit, std::memory_order_relaxed);
        return e;
    }
};

}  // namespace ql
