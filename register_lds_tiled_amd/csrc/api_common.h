// api_common.h -- what the C entry points of every family share: the text of
// a thread's last HIP error, the extents and overlaps of matrices, and the
// shape of the device a launch runs on.
#pragma once

#include <hip/hip_runtime.h>

#include <atomic>
#include <cstdint>
#include <cstdio>

#include "sgemm.h"

namespace sgemm {

inline thread_local char g_last_error[256] = "";

inline int hip_fail(hipError_t e) {
    std::snprintf(g_last_error, sizeof(g_last_error), "%s: %s", hipGetErrorName(e),
                  hipGetErrorString(e));
    return SGEMM_EHIP;
}

// Byte range [lo, hi) spanned by a rows x cols row-major matrix of esize-byte
// elements with leading dimension ld (rows, cols >= 1).  The extent is
// formed in 128 bits; ok is false when the range would pass the end of the
// address space (no such matrix can exist).
struct Range {
    uintptr_t lo, hi;
    bool ok;
};
inline Range span(const void* p, long long rows, long long cols, long long ld,
                  long long esize = 4) {
    const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
    const unsigned __int128 bytes =
        ((unsigned __int128)(rows - 1) * (unsigned __int128)ld + (unsigned __int128)cols) *
        (unsigned __int128)esize;
    const unsigned __int128 hi = (unsigned __int128)lo + bytes;
    if (hi > (unsigned __int128)UINTPTR_MAX) return {lo, UINTPTR_MAX, false};
    return {lo, (uintptr_t)hi, true};
}
inline bool overlaps(Range a, Range b) { return a.lo < b.hi && b.lo < a.hi; }
inline long long at_least_1(long long n) { return n > 1 ? n : 1; }

// Up to twelve byte ranges, outputs first: every output must keep clear of
// all others.
struct Ranges {
    Range r[12];
    int n = 0, outputs = 0;
    bool ok = true;
    void add(const void* p, long long rows, long long row_elements, long long ld, long long esize,
             bool output = false) {
        r[n] = span(p, rows, row_elements, ld, esize);
        ok = ok && r[n].ok;
        ++n;
        if (output) outputs = n;
    }
    int status() const {
        if (!ok) return SGEMM_EINVAL_DIM;
        for (int i = 0; i < outputs; ++i)
            for (int j = i + 1; j < n; ++j)
                if (overlaps(r[i], r[j])) return SGEMM_EALIAS;
        return SGEMM_OK;
    }
};

// Compute units and XCDs of the device a stream's launches run on, queried
// once per device (the first 64 device ids) and then read from the cache.
// The XCD count falls back to one XCD per 32 CUs (gfx950's XCD) where the
// runtime does not report it.
constexpr int kMaxDevices = 64;
inline std::atomic<int> g_cus[kMaxDevices], g_xcds[kMaxDevices];

inline hipError_t device_shape(hipStream_t stream, int& cus, int& xcds) {
    int dev = 0;
    hipError_t e = stream ? hipStreamGetDevice(stream, &dev) : hipGetDevice(&dev);
    if (e != hipSuccess) return e;
    const bool cached = dev >= 0 && dev < kMaxDevices;
    if (cached && g_cus[dev].load(std::memory_order_acquire) > 0) {
        xcds = g_xcds[dev].load(std::memory_order_relaxed);
        cus = g_cus[dev].load(std::memory_order_relaxed);
        return hipSuccess;
    }
    int c = 0, x = 0;
    e = hipDeviceGetAttribute(&c, hipDeviceAttributeMultiprocessorCount, dev);
    if (e != hipSuccess) return e;
    if (hipDeviceGetAttribute(&x, hipDeviceAttributeNumberOfXccs, dev) != hipSuccess || x < 1) {
        (void)hipGetLastError();   // not reported: clear it, use the fallback
        x = c >= 32 ? c / 32 : 1;
    }
    cus = c > 0 ? c : 1;
    xcds = x;
    if (cached) {
        g_xcds[dev].store(xcds, std::memory_order_relaxed);
        g_cus[dev].store(cus, std::memory_order_release);
    }
    return hipSuccess;
}

}  // namespace sgemm
