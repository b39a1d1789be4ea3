// Host-side helpers that the library's source files share.
#pragma once

#include <hip/hip_runtime.h>

#include <algorithm>
#include <initializer_list>

#include "common.hpp"

namespace moe {

// Records a start and a stop event around a launch while the launch trace has room
// (moe.hip holds the records).
struct __attribute__((visibility("hidden"))) TraceScope {
    int rec;
    hipStream_t stream;
    TraceScope(const char *name, hipStream_t s);
    ~TraceScope();
};

// Per-device compute-unit count (the persistent grids are sized to it).
inline __attribute__((visibility("hidden"))) int device_cus() {
    static int cache[64] = {0};
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64) return 256;
    if (cache[dev] == 0) {
        int n = 0;
        if (hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || n <= 0) n = 256;
        cache[dev] = n;
    }
    return cache[dev];
}

static inline bool aligned16(const void *p) { return ((uintptr_t)p & 15u) == 0; }
static inline bool aligned4(const void *p) { return ((uintptr_t)p & 3u) == 0; }
static inline int64_t align256(int64_t x) { return (x + 255) / 256 * 256; }

// NULL or 16-byte aligned, each of them.
static inline bool all_aligned(std::initializer_list<const void *> ps) {
    for (const void *p : ps)
        if (!aligned16(p)) return false;
    return true;
}

static inline int launch_status() { return hipGetLastError() == hipSuccess ? MOE_OK : MOE_EHIP; }

constexpr size_t kMaxLds = 160 * 1024;  // LDS of one gfx950 workgroup

}  // namespace moe
