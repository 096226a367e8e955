// Host-side checks shared by the training-step entry points (ar_step_api.hip,
// ar_layer_norm_api.hip): error texts, buffer ranges and their overlaps, and
// where buffers live.  Everything is inline in an unnamed namespace.
#pragma once

#include <hip/hip_runtime_api.h>

#include <algorithm>
#include <atomic>
#include <cstdarg>
#include <cstdint>
#include <cstdio>
#include <exception>
#include <new>
#include <vector>

#include "ar.h"
#include "ar_internal.h"

namespace arimpl {
namespace {

__attribute__((format(printf, 2, 3))) inline ar_result_t fail_with(ar_result_t code, const char* fmt, ...) {
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    std::vsnprintf(buf, sizeof(buf), fmt, ap);
    va_end(ap);
    set_error_detail(buf);
    return code;
}

// Runs an entry point's body; a C++ exception (host memory running out) ends
// as an error code, never in the C caller.
template <class Body>
ar_result_t guarded(Body body) {
    try {
        set_error_detail("");
        return body();
    } catch (const std::bad_alloc&) {
        return AR_ERR_INTERNAL;
    } catch (const std::exception&) {
        return AR_ERR_INTERNAL;
    }
}

inline bool float_type(ar_dtype_t dt) { return dt == AR_FLOAT32 || dt == AR_BFLOAT16 || dt == AR_FLOAT16; }

// A positive setting that float32 takes for 0.
inline bool rounds_to_zero(double x) { return x > 0 && static_cast<float>(x) == 0.0f; }

// A buffer of `bytes` bytes (rows of `row` bytes, `stride` bytes apart, when
// stride is not 0).
struct Range {
    uintptr_t lo, hi;
    bool writable;
    const char* what;
    int index;
    uint64_t row, stride;
};

inline ar_result_t add_range(std::vector<Range>& v, const void* p, uint64_t bytes, size_t align, bool writable,
                             const char* what, int index, uint64_t row = 0, uint64_t stride = 0) {
    if (bytes == 0) return AR_SUCCESS;
    const uintptr_t at = reinterpret_cast<uintptr_t>(p);
    if (p == nullptr) return fail_with(AR_ERR_INVALID_ARGUMENT, "%s[%d] is null", what, index);
    if (at % align != 0)
        return fail_with(AR_ERR_INVALID_ARGUMENT, "%s[%d] not aligned to its %zu-byte element", what, index, align);
    if (bytes > UINTPTR_MAX - at) return fail_with(AR_ERR_INVALID_ARGUMENT, "%s[%d] is too large", what, index);
    v.push_back({at, at + bytes, writable, what, index, row, stride});
    return AR_SUCCESS;
}

// Rows of both ranges interleave without touching.
inline bool rows_apart(const Range& a, const Range& b) {
    if (a.stride == 0 || a.stride != b.stride) return false;
    const Range& f = a.lo <= b.lo ? a : b;
    const Range& s = a.lo <= b.lo ? b : a;
    const uint64_t d = (s.lo - f.lo) % f.stride;
    return d >= f.row && d + s.row <= f.stride;
}

// Refuse a writable range that overlaps any other.
inline ar_result_t check_ranges(std::vector<Range>& v) {
    std::sort(v.begin(), v.end(), [](const Range& a, const Range& b) { return a.lo < b.lo; });
    std::vector<const Range*> active;
    for (const Range& cur : v) {
        active.erase(std::remove_if(active.begin(), active.end(), [&](const Range* x) { return x->hi <= cur.lo; }),
                     active.end());
        for (const Range* x : active) {
            if ((!x->writable && !cur.writable) || rows_apart(*x, cur)) continue;
            return fail_with(AR_ERR_INVALID_ARGUMENT, "%s[%d] overlaps %s[%d]", x->what, x->index, cur.what, cur.index);
        }
        // read-only ranges of the same bytes, rows and gaps alike, say the same thing
        // once (many ranks reading one weight)
        bool same = false;
        for (const Range* x : active)
            same = same || (x->lo == cur.lo && x->hi == cur.hi && x->row == cur.row && x->stride == cur.stride &&
                            !cur.writable);
        if (!same) active.push_back(&cur);
    }
    return AR_SUCCESS;
}

// Device memory of the current device (or managed memory) that holds the
// whole range.
inline ar_result_t check_device_memory(const std::vector<Range>& v) {
    int dev = 0;
    hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess) return fail_with(AR_ERR_HIP, "hipGetDevice: %s", hipGetErrorString(e));
    for (const Range& b : v) {
        void* p = reinterpret_cast<void*>(b.lo);
        hipPointerAttribute_t at{};
        e = hipPointerGetAttributes(&at, p);
        if (e != hipSuccess) {
            (void)hipGetLastError();   // the launches read the last error: leave none behind
            return fail_with(AR_ERR_INVALID_ARGUMENT, "%s[%d]: the HIP runtime does not know this address (%s)", b.what,
                             b.index, hipGetErrorString(e));
        }
        if (at.type == hipMemoryTypeUnregistered || at.type == hipMemoryTypeHost)
            return fail_with(AR_ERR_INVALID_ARGUMENT, "%s[%d] is host memory, not device memory", b.what, b.index);
        if (at.type == hipMemoryTypeDevice && at.device != dev)
            return fail_with(AR_ERR_INVALID_ARGUMENT, "%s[%d] is memory of device %d, not of the current device %d",
                             b.what, b.index, at.device, dev);
        hipDeviceptr_t base = nullptr;
        size_t size = 0;
        e = hipMemGetAddressRange(&base, &size, p);
        if (e != hipSuccess) {
            (void)hipGetLastError();   // extent unknown to the runtime: not checked
            continue;
        }
        const uintptr_t end = reinterpret_cast<uintptr_t>(base) + size;
        if (b.hi > end)
            return fail_with(AR_ERR_INVALID_ARGUMENT, "%s[%d] runs %llu bytes past the end of its allocation", b.what,
                             b.index, static_cast<unsigned long long>(b.hi - end));
    }
    return AR_SUCCESS;
}

inline ar_result_t hip_result(hipError_t e, const char* what) {
    if (e == hipSuccess) return AR_SUCCESS;
    return fail_with(AR_ERR_HIP, "%s: %s", what, hipGetErrorString(e));
}

}  // namespace
}  // namespace arimpl
