// ctx.h -- the context behind ar_ctx and the host helpers that every C entry
// point shares: error reporting, the device guard and the device-memory check
// of one array.  Internal to the library.
#pragma once

#include <hip/hip_runtime_api.h>

#include <cstdarg>
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <string>
#include <vector>

#include "ar.h"
#include "launch.h"

// A pointer set that passed the device-memory checks, with the byte size it
// was checked for.
struct CheckedSet {
    std::vector<uintptr_t> ptrs;
    size_t bytes = 0;
    uint64_t stamp = 0;
};

// A recorded launch sequence.  `done` is recorded after every replay so the
// executable graph can be released only once its last replay has finished.
struct GraphEntry {
    std::vector<uint64_t> key;
    hipGraphExec_t exec = nullptr;
    hipEvent_t done = nullptr;
    uint64_t stamp = 0;
};

static constexpr size_t kGraphCacheSize = 64;

struct ar_ctx {
    int device = 0;
    hipStream_t stream = nullptr;
    std::string last_error;
    // Recently validated pointer sets (least recently used is replaced): a
    // training loop reduces the same few buckets every step, and checking 64
    // pointers with the runtime costs more than a small message's kernel.
    // Off unless the caller turns it on (ar_set_pointer_cache): a buffer freed
    // and re-allocated smaller at the same address would not be re-checked.
    bool ptr_cache = false;
    std::vector<CheckedSet> checked;
    // Residency caps of the fused kernels (ar_set_residency_caps): on unless
    // the caller turns them off or the device's LDS per CU is not the size
    // they are computed for
    bool caps = true;
    bool caps_supported = true;
    uint64_t clock = 0;
    // Graph replay of multi-launch collectives (ar_set_graphs): one
    // instantiated graph per (collective, algorithm, shape, pointer set),
    // recorded on a private stream and launched on `stream`.
    size_t graph_max_bytes = 0;   // replay collectives of at most this many bytes per rank
    hipStream_t capture = nullptr;
    std::vector<GraphEntry> graph_cache;
    // ar_check's per-block partial records (kCheckMaxBlocks of them),
    // allocated on the first ar_check
    arlib::CheckPartial* check_part = nullptr;
    // ar_check_noalloc's records: the device-resident array on this
    // context's device, looked up in ar_create (NULL if that failed)
    arlib::CheckPartial* check_static = nullptr;
    std::string check_static_error;
    // the operators' calls check their arrays with the runtime
    // (ar_set_operator_checks)
    bool operator_checks = true;
};

namespace arlib {

inline thread_local std::string g_create_error;

inline bool debug_enabled() {
    static const bool on = [] {
        const char* v = std::getenv("AR_DEBUG");
        return v && *v && std::strcmp(v, "0") != 0;
    }();
    return on;
}

inline ar_status fail(ar_ctx* ctx, ar_status st, const char* fmt, ...) {
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    std::vsnprintf(buf, sizeof buf, fmt, ap);
    va_end(ap);
    if (ctx) ctx->last_error = buf;
    else g_create_error = buf;
    if (debug_enabled()) std::fprintf(stderr, "[ar] error: %s\n", buf);
    return st;
}

// Makes ctx->device current for the lifetime of the guard.
struct DeviceGuard {
    int prev = -1;
    bool ok = false;
    explicit DeviceGuard(int dev) {
        if (hipGetDevice(&prev) != hipSuccess) {
            (void)hipGetLastError();
            return;
        }
        ok = prev == dev || hipSetDevice(dev) == hipSuccess;
        if (!ok) (void)hipGetLastError();
    }
    ~DeviceGuard() {
        int cur = -1;
        if (ok && hipGetDevice(&cur) == hipSuccess && cur != prev && prev >= 0)
            (void)hipSetDevice(prev);
    }
};

// A device array of `bytes` bytes at p: device memory of ctx->device, inside
// its allocation (fail closed, like the rank buffers).
inline ar_status check_device_span(ar_ctx* ctx, const void* p, size_t bytes, const char* what) {
    hipPointerAttribute_t at;
    std::memset(&at, 0, sizeof at);
    if (hipPointerGetAttributes(&at, p) != hipSuccess) {
        (void)hipGetLastError();
        return fail(ctx, AR_ERR_INVALID_ARG, "%s is not a device pointer", what);
    }
    if (at.type != hipMemoryTypeDevice && at.type != hipMemoryTypeManaged)
        return fail(ctx, AR_ERR_INVALID_ARG, "%s is not device memory", what);
    if (at.device != ctx->device)
        return fail(ctx, AR_ERR_INVALID_ARG, "%s lives on device %d, context on %d", what,
                    at.device, ctx->device);
    hipDeviceptr_t base = nullptr;
    size_t size = 0;
    if (hipMemGetAddressRange(&base, &size, const_cast<void*>(p)) != hipSuccess || !base) {
        (void)hipGetLastError();
        return fail(ctx, AR_ERR_INVALID_ARG, "%s: cannot determine its allocation", what);
    }
    const uintptr_t b = reinterpret_cast<uintptr_t>(base), q = reinterpret_cast<uintptr_t>(p);
    if (q < b || bytes > size || q - b > size - bytes)
        return fail(ctx, AR_ERR_INVALID_ARG, "%s: %zu bytes run past the end of its allocation",
                    what, bytes);
    return AR_OK;
}

}  // namespace arlib
