// What has been asked of hipFuncAttributeMaxDynamicSharedMemorySize: the
// largest size per kernel and device. Host code only; the caller locks.
#pragma once

#include <stdint.h>

namespace moed {

// Fixed, so that entry points for callers that cannot allocate may use it. A
// slot per kernel (hashed by address) with one size per device, so that the
// number of devices does not fill it; the library has about 130 kernels that ask.
struct LdsLimits {
    static constexpr int kKernels = 256, kDevices = 64;

    // The size recorded for (func, dev); null when the table is full.
    int* find(const void* func, int dev)
    {
        const unsigned at = (unsigned)(((uint64_t)(uintptr_t)func * 0x9E3779B97F4A7C15ull) >> 56);
        for (int i = 0; i < kKernels; ++i) {
            Entry& e = kernels[(at + (unsigned)i) % kKernels];
            if (!e.func)
                e.func = func;
            if (e.func == func)
                return &e.bytes[dev];
        }
        return nullptr;
    }

private:
    struct Entry {
        const void* func;
        int bytes[kDevices];
    };
    Entry kernels[kKernels];
};

}  // namespace moed
