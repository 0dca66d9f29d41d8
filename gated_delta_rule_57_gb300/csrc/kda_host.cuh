// Host-side helpers shared by the entry points: argument checks, the error
// string of the calling thread, and profiler ranges. Not part of the ABI.
#pragma once

#include <stdint.h>
#include <string.h>

#include <atomic>

#include <nvtx3/nvToolsExt.h>

#include "kda_internal.cuh"

namespace kda {

// Reason of the last failure on this host thread (kda_last_error_string).
extern thread_local char g_last_error[256];

inline void set_last_error(const char* msg) {
    strncpy(g_last_error, msg, sizeof(g_last_error) - 1);
    g_last_error[sizeof(g_last_error) - 1] = '\0';
}

// An NVTX range around each entry point (named after it), so a timeline
// profiler shows every library call; free when no tool is attached.
struct NvtxRange {
    explicit NvtxRange(const char* name) { nvtxRangePushA(name); }
    ~NvtxRange() { nvtxRangePop(); }
    NvtxRange(const NvtxRange&) = delete;
    NvtxRange& operator=(const NvtxRange&) = delete;
};

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// [p, p + n) and [q, q + m) overlap (both non-empty)?
inline bool overlaps(const void* p, size_t n, const void* q, size_t m) {
    if (!p || !q || n == 0 || m == 0) return false;
    uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
    return a < b + m && b < a + n;
}

// n = a * b * c * d with overflow detection (all factors >= 0).
inline bool mul_ok(size_t* out, size_t a, size_t b, size_t c = 1, size_t d = 1) {
    const size_t lim = (size_t)1 << 62;
    size_t r = a;
    for (size_t f : {b, c, d}) {
        if (f != 0 && r > lim / f) return false;
        r *= f;
    }
    *out = r;
    return true;
}

inline kda_status_t fail(kda_status_t s, const char* why) {
    set_last_error(why);
    return s;
}

// The status of a launch: KDA_OK, or KDA_ERR_CUDA with the error's name kept.
inline kda_status_t launched(cudaError_t e) {
    if (e == cudaSuccess) return KDA_OK;
    set_last_error(cudaGetErrorString(e));
    return KDA_ERR_CUDA;
}

// SMs of the current device, 0 if none is visible; *device (if not null): its
// number.
inline int device_sms(int* device = nullptr) {
    static std::atomic<int> known[64];
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) {
        cudaGetLastError();
        return 0;
    }
    if (device) *device = dev;
    if (dev < 64 && (n = known[dev].load(std::memory_order_relaxed)) > 0) return n;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) {
        cudaGetLastError();
        return 0;
    }
    if (dev < 64) known[dev].store(n, std::memory_order_relaxed);
    return n;
}

// Lets a kernel be launched with up to `bytes` of dynamic shared memory on the current
// device, once per device. One limit for all calls of a kernel: a limit of the call's
// own size could be lowered by another thread before the launch.
template <typename Kernel>
inline cudaError_t allow_shared(Kernel kernel, size_t bytes, std::atomic<uint64_t>& ready, int dev) {
    const uint64_t bit = dev >= 0 && dev < 64 ? 1ull << dev : 0;
    if (ready.load(std::memory_order_relaxed) & bit) return cudaSuccess;
    const cudaError_t e =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e == cudaSuccess) ready.fetch_or(bit, std::memory_order_relaxed);
    return e;
}

}  // namespace kda
