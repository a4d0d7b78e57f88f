// ops_args.h -- what the C entry points of the training operators (ops_api.cpp,
// model_api.cpp) share: argument validation and error reporting.
#pragma once

#include <hip/hip_runtime_api.h>

#include <cstdint>
#include <new>

#include "ar.h"
#include "ctx.h"

namespace arlib {

// bytes of an element, 0 for a dtype that the operators do not take
inline size_t float_bytes(int dtype) {
    return dtype == AR_BFLOAT16 ? 2 : dtype == AR_FLOAT32 ? 4 : 0;
}

// Widest row of a layer norm, of the experts and of the logits (byte offsets within a row stay
// below 2^32).
constexpr size_t kMostCols = size_t(1) << 28;

// *out = a * b, false on overflow.
inline bool times(size_t a, size_t b, size_t* out) { return !__builtin_mul_overflow(a, b, out); }

// Bytes from the first element of a row-strided array to its end.
inline bool strided_bytes(size_t rows, size_t cols, size_t stride, size_t eb, size_t* out) {
    size_t n;
    if (rows == 0 || cols == 0) {
        *out = 0;
        return true;
    }
    return times(rows - 1, stride, &n) && !__builtin_add_overflow(n, cols, &n) && times(n, eb, out);
}

// The arrays of one call, checked together: NULL, alignment, overlap of an
// output with anything else, and (unless the context leaves it to the caller)
// device memory and extent.  Empty arrays are not looked at.
class Arrays {
public:
    explicit Arrays(ar_ctx* ctx) : ctx_(ctx) {}

    void in(const void* p, size_t bytes, size_t align, const char* name) {
        add(p, bytes, align, name, false);
    }
    void out(const void* p, size_t bytes, size_t align, const char* name) {
        add(p, bytes, align, name, true);
    }

    ar_status check() const {
        for (int i = 0; i < n_; ++i) {
            const Array& a = a_[i];
            if (!a.p) return fail(ctx_, AR_ERR_INVALID_ARG, "%s is NULL", a.name);
            const uintptr_t p = reinterpret_cast<uintptr_t>(a.p);
            if (p % a.align)
                return fail(ctx_, AR_ERR_INVALID_ARG, "%s is not %zu-byte aligned", a.name, a.align);
            if (p > UINTPTR_MAX - a.bytes)
                return fail(ctx_, AR_ERR_INVALID_ARG, "%s + size wraps the address space", a.name);
        }
        for (int i = 0; i < n_; ++i)
            for (int j = 0; a_[i].out && j < n_; ++j) {
                if (j == i || (a_[j].out && j < i)) continue;
                const uintptr_t p = reinterpret_cast<uintptr_t>(a_[i].p);
                const uintptr_t q = reinterpret_cast<uintptr_t>(a_[j].p);
                if (p < q + a_[j].bytes && q < p + a_[i].bytes)
                    return fail(ctx_, AR_ERR_INVALID_ARG, "%s overlaps %s", a_[i].name, a_[j].name);
            }
        for (int i = 0; ctx_->operator_checks && i < n_; ++i) {
            const ar_status s = check_device_span(ctx_, a_[i].p, a_[i].bytes, a_[i].name);
            if (s != AR_OK) return s;
        }
        return AR_OK;
    }

private:
    struct Array {
        const void* p;
        size_t bytes, align;
        const char* name;
        bool out;
    };
    void add(const void* p, size_t bytes, size_t align, const char* name, bool out) {
        if (bytes) a_[n_++] = {p, bytes, align, name, out};
    }
    ar_ctx* ctx_;
    Array a_[12];
    int n_ = 0;
};

inline ar_status launched(ar_ctx* ctx, hipError_t e, const char* what) {
    if (e == hipSuccess) return AR_OK;
    (void)hipGetLastError();
    return fail(ctx, AR_ERR_RUNTIME, "%s launch failed: %s", what, hipGetErrorString(e));
}

inline ar_status bad_size(ar_ctx* ctx) {
    return fail(ctx, AR_ERR_INVALID_ARG, "the sizes overflow");
}

inline ar_status workspace(ar_ctx* ctx, Arrays& arrays, void* ws, size_t have, size_t need) {
    if (have < need)
        return fail(ctx, AR_ERR_INVALID_ARG, "workspace of %zu bytes, %zu needed", have, need);
    arrays.out(ws, need, 16, "workspace");
    return AR_OK;
}

// Runs `body` with ctx's device current; no exception leaves.
template <class F>
ar_status guarded(ar_ctx* ctx, F body) {
    if (!ctx) return fail(nullptr, AR_ERR_INVALID_ARG, "ctx is NULL");
    try {
        DeviceGuard g(ctx->device);
        if (!g.ok) return fail(ctx, AR_ERR_RUNTIME, "cannot select device %d", ctx->device);
        return body();
    } catch (const std::bad_alloc&) {
        return AR_ERR_NO_MEMORY;
    } catch (...) {
        return AR_ERR_RUNTIME;
    }
}

inline ar_status check_index_bytes(ar_ctx* ctx, int index_bytes) {
    if (index_bytes == 4 || index_bytes == 8) return AR_OK;
    return fail(ctx, AR_ERR_INVALID_ARG, "index_bytes %d is neither 4 nor 8", index_bytes);
}

}  // namespace arlib
