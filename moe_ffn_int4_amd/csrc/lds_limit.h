// lds_limit.h -- dynamic LDS of more than 64 KB, which a kernel must be allowed on each
// device that runs it (internal to the library).
#pragma once

#include <atomic>
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace moe {

// Devices, a bit each, on which a kernel has been allowed its LDS.
using LdsDevices = std::atomic<uint64_t>;

// Allows `kernel` `bytes` on the current device; `done` is the kernel's own. Threads that come
// here at once may both make the call, to the same end.
inline hipError_t allow_lds(const void* kernel, int bytes, LdsDevices& done) {
    int device = 0;
    hipError_t e = hipGetDevice(&device);
    if (e != hipSuccess) return e;
    const uint64_t bit = uint64_t{1} << (device & 63);  // the entry points refuse ordinals past 63
    if (done.load(std::memory_order_acquire) & bit) return hipSuccess;
    e = hipFuncSetAttribute(kernel, hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == hipSuccess) done.fetch_or(bit, std::memory_order_release);
    return e;
}

}  // namespace moe
