// ops_driver.cpp -- runs the training operators' C entry points (ops_api.cpp)
// against the fake HIP runtime under the host sanitizers, with launchers that
// record their arguments.  Test infrastructure only: prints "ALL OK" and exits
// 0 when every check passes.
#include <cmath>
#include <cstdint>
#include <cstdio>

#include "ar.h"
#include "fake_hip.h"
#include "ops.h"

namespace {

int g_fail = 0;
#define CHECK(c)                                                         \
    do {                                                                 \
        if (!(c)) {                                                      \
            std::fprintf(stderr, "FAIL %s:%d: %s\n", __FILE__, __LINE__, #c); \
            ++g_fail;                                                    \
        }                                                                \
    } while (0)

int g_launches = 0;
arlib::NormArgs g_norm;
arlib::NormGradArgs g_norm_grad;
arlib::DispatchArgs g_dispatch;
arlib::CombineArgs g_combine;
arlib::DistillArgs g_distill;

// arrays 1 GiB apart from here on; nothing is dereferenced
constexpr uintptr_t kBase = uintptr_t(1) << 44, kStep = uintptr_t(1) << 30;
template <class T = void>
T* at(int i, size_t shift = 0) {
    return reinterpret_cast<T*>(kBase + (uintptr_t)i * kStep + shift);
}

// The call is refused with `want` and launches nothing.
#define REFUSED(want, call)                  \
    do {                                     \
        const int before = g_launches;       \
        CHECK((call) == (want));             \
        CHECK(g_launches == before);         \
        CHECK(ar_last_error(ctx)[0] != 0);   \
    } while (0)
#define RUNS(call)                           \
    do {                                     \
        const int before = g_launches;       \
        CHECK((call) == AR_OK);              \
        CHECK(g_launches == before + 1);     \
    } while (0)

ar_ctx* ctx = nullptr;

void norm() {
    const auto f = [&](size_t rows, size_t cols, size_t xs, int dt, int pt, float eps, const void* x,
                       const void* w, void* y, float* m, float* r) {
        return ar_layer_norm(ctx, x, xs, w, nullptr, (ar_dtype)pt, y, m, r, rows, cols,
                             (ar_dtype)dt, eps);
    };
    RUNS(f(8, 100, 100, AR_BFLOAT16, AR_FLOAT32, 1e-5f, at(0), at(1), at(2), at<float>(3), at<float>(4)));
    CHECK(g_norm.rows == 8 && g_norm.cols == 100 && g_norm.eb == 2 && g_norm.pb == 4 && !g_norm.bias);
    RUNS(f(8, 100, 104, AR_FLOAT32, AR_FLOAT32, 0.0f, at(0, 4), at(1), at(2, 12), at<float>(3), at<float>(4)));
    RUNS(f(0, 100, 100, AR_FLOAT32, AR_FLOAT32, 0.0f, nullptr, nullptr, nullptr, nullptr, nullptr));
    RUNS(f(1, 100, 0, AR_FLOAT32, AR_FLOAT32, 0.0f, at(0), nullptr, at(2), at<float>(3), at<float>(4)));
    REFUSED(AR_ERR_INVALID_ARG, f(8, 0, 0, 1, 1, 0.f, at(0), at(1), at(2), at<float>(3), at<float>(4)));
    REFUSED(AR_ERR_INVALID_ARG, f(8, 100, 99, 1, 1, 0.f, at(0), at(1), at(2), at<float>(3), at<float>(4)));
    REFUSED(AR_ERR_INVALID_ARG, f(8, 100, 100, 0, 1, 0.f, at(0), at(1), at(2), at<float>(3), at<float>(4)));
    REFUSED(AR_ERR_INVALID_ARG, f(8, 100, 100, 1, 7, 0.f, at(0), at(1), at(2), at<float>(3), at<float>(4)));
    REFUSED(AR_ERR_INVALID_ARG, f(8, 100, 100, 1, 1, -1.f, at(0), at(1), at(2), at<float>(3), at<float>(4)));
    REFUSED(AR_ERR_INVALID_ARG, f(8, 100, 100, 1, 1, NAN, at(0), at(1), at(2), at<float>(3), at<float>(4)));
    REFUSED(AR_ERR_INVALID_ARG, f(8, 100, 100, 1, 1, 0.f, nullptr, at(1), at(2), at<float>(3), at<float>(4)));
    REFUSED(AR_ERR_INVALID_ARG, f(8, 100, 100, 1, 1, 0.f, at(0), at(1), at(2), nullptr, at<float>(4)));
    REFUSED(AR_ERR_INVALID_ARG, f(8, 100, 100, 1, 1, 0.f, at(0, 2), at(1), at(2), at<float>(3), at<float>(4)));
    // overlap: y with x, rstd with mean's end
    REFUSED(AR_ERR_INVALID_ARG, f(8, 100, 100, 1, 1, 0.f, at(0), at(1), at(0, 3196), at<float>(3), at<float>(4)));
    RUNS(f(8, 100, 100, 1, 1, 0.f, at(0), at(1), at(0, 3200), at<float>(3), at<float>(4)));
    REFUSED(AR_ERR_INVALID_ARG, f(8, 100, 100, 1, 1, 0.f, at(0), at(1), at(2), at<float>(3), at<float>(3, 28)));
    // past the allocation, and host memory
    REFUSED(AR_ERR_INVALID_ARG, f(1 << 20, 4096, 4096, 1, 1, 0.f, at(60), at(1), at(2), at<float>(3), at<float>(4)));
    float host[8];
    REFUSED(AR_ERR_INVALID_ARG, f(8, 100, 100, 1, 1, 0.f, at(0), at(1), at(2), host, at<float>(4)));
    CHECK(ar_set_operator_checks(ctx, 0) == AR_OK);
    RUNS(f(8, 100, 100, 1, 1, 0.f, at(0), at(1), at(2), host, at<float>(4)));
    CHECK(ar_set_operator_checks(ctx, 1) == AR_OK);
    REFUSED(AR_ERR_INVALID_ARG, f(8, 100, 100, 1, 1, 0.f, at(0), at(1), at(2), host, at<float>(4)));
    // sizes
    REFUSED(AR_ERR_INVALID_ARG, f(SIZE_MAX / 8, 100, 100, 1, 1, 0.f, at(0), at(1), at(2), at<float>(3), at<float>(4)));
    REFUSED(AR_ERR_INVALID_ARG, f(8, 100, SIZE_MAX / 4, 1, 1, 0.f, at(0), at(1), at(2), at<float>(3), at<float>(4)));
    REFUSED(AR_ERR_UNSUPPORTED, f(8, (size_t(1) << 28) + 1, size_t(1) << 29, 1, 1, 0.f, at(0), at(1), at(2), at<float>(3), at<float>(4)));

    size_t need = 0;
    CHECK(ar_layer_norm_backward_workspace(50, 64, AR_BFLOAT16, &need) == AR_OK && need > 0);
    CHECK(ar_layer_norm_backward_workspace(50, 0, AR_BFLOAT16, &need) == AR_ERR_INVALID_ARG);
    CHECK(ar_layer_norm_backward_workspace(50, 64, AR_INT32, &need) == AR_ERR_INVALID_ARG);
    CHECK(ar_layer_norm_backward_workspace(50, 64, AR_FLOAT32, nullptr) == AR_ERR_INVALID_ARG);
    CHECK(ar_layer_norm_backward_workspace(50, SIZE_MAX / 2, AR_FLOAT32, &need) == AR_ERR_UNSUPPORTED);
    CHECK(ar_layer_norm_backward_workspace(50, 64, AR_BFLOAT16, &need) == AR_OK);
    const auto b = [&](const void* dy, size_t gs, void* dx, void* dw, void* db, void* ws, size_t n) {
        return ar_layer_norm_backward(ctx, dy, gs, at(1), 64, at<float>(2), at<float>(3), at(4),
                                      AR_FLOAT32, dx, dw, db, 50, 64, AR_BFLOAT16, ws, n);
    };
    RUNS(b(at(0), 64, at(5), at(6), at(7), at(8), need));
    CHECK(g_norm_grad.part == at<float>(8) && g_norm_grad.dystride == 64);
    RUNS(b(at(0), 80, at(5), nullptr, nullptr, nullptr, 0));
    RUNS(b(at(0), 80, at(5), nullptr, at(7), at(8), need + 64));
    REFUSED(AR_ERR_INVALID_ARG, b(at(0), 63, at(5), at(6), at(7), at(8), need));
    REFUSED(AR_ERR_INVALID_ARG, b(at(0), 64, at(5), at(6), at(7), at(8), need - 1));
    REFUSED(AR_ERR_INVALID_ARG, b(at(0), 64, at(5), at(6), at(7), nullptr, need));
    REFUSED(AR_ERR_INVALID_ARG, b(at(0), 64, at(5), at(6), at(7), at(8, 8), need));
    REFUSED(AR_ERR_INVALID_ARG, b(at(0), 64, at(0), at(6), at(7), at(8), need));
    REFUSED(AR_ERR_INVALID_ARG, b(at(0), 64, at(5), at(6), at(6), at(8), need));
    REFUSED(AR_ERR_INVALID_ARG, b(at(0), 64, at(5), at(6), at(7), at(6), need));
}

void route() {
    size_t need = 0;
    CHECK(ar_expert_dispatch_workspace(10, 2, 5, &need) == AR_OK);
    CHECK(ar_expert_dispatch_workspace(10, 0, 5, &need) == AR_ERR_INVALID_ARG);
    CHECK(ar_expert_dispatch_workspace(10, 2, 0, &need) == AR_ERR_INVALID_ARG);
    CHECK(ar_expert_dispatch_workspace(10, 2, 5, nullptr) == AR_ERR_INVALID_ARG);
    CHECK(ar_expert_dispatch_workspace(10, 2, AR_MAX_EXPERTS + 1, &need) == AR_ERR_UNSUPPORTED);
    CHECK(ar_expert_dispatch_workspace(size_t(1) << 30, 2, 5, &need) == AR_ERR_UNSUPPORTED);
    CHECK(ar_expert_dispatch_workspace(SIZE_MAX / 2 + 1, 2, 5, &need) == AR_ERR_INVALID_ARG);
    CHECK(ar_expert_dispatch_workspace(10, 2, 5, &need) == AR_OK);
    const auto d = [&](const void* x, size_t xs, int ib, size_t tokens, int k, int e, size_t h, int dt,
                       int* slot, void* ws, size_t n) {
        return ar_expert_dispatch(ctx, x, xs, at(1), ib, tokens, k, e, h, (ar_dtype)dt, at(2),
                                  at<int>(3), slot, at<int>(5), ws, n);
    };
    RUNS(d(at(0), 16, 8, 10, 2, 5, 16, AR_FLOAT32, at<int>(4), at(6), need));
    CHECK(g_dispatch.tokens == 10 && g_dispatch.ib == 8 && g_dispatch.hidden == 16);
    RUNS(d(nullptr, 16, 4, 0, 2, 5, 16, AR_BFLOAT16, nullptr, at(6), need));
    REFUSED(AR_ERR_INVALID_ARG, d(at(0), 15, 8, 10, 2, 5, 16, AR_FLOAT32, at<int>(4), at(6), need));
    REFUSED(AR_ERR_INVALID_ARG, d(at(0), 16, 2, 10, 2, 5, 16, AR_FLOAT32, at<int>(4), at(6), need));
    REFUSED(AR_ERR_INVALID_ARG, d(at(0), 16, 8, 10, 0, 5, 16, AR_FLOAT32, at<int>(4), at(6), need));
    REFUSED(AR_ERR_INVALID_ARG, d(at(0), 16, 8, 10, 2, 0, 16, AR_FLOAT32, at<int>(4), at(6), need));
    REFUSED(AR_ERR_INVALID_ARG, d(at(0), 16, 8, 10, 2, 5, 0, AR_FLOAT32, at<int>(4), at(6), need));
    REFUSED(AR_ERR_INVALID_ARG, d(at(0), 16, 8, 10, 2, 5, 16, AR_INT32, at<int>(4), at(6), need));
    REFUSED(AR_ERR_INVALID_ARG, d(at(0), 16, 8, 10, 2, 5, 16, AR_FLOAT32, at<int>(3), at(6), need));
    REFUSED(AR_ERR_INVALID_ARG, d(at(0), 16, 8, 10, 2, 5, 16, AR_FLOAT32, at<int>(4), at(6), need - 1));
    REFUSED(AR_ERR_UNSUPPORTED, d(at(0), 16, 8, 10, 2, 1025, 16, AR_FLOAT32, at<int>(4), at(6), need));
    REFUSED(AR_ERR_UNSUPPORTED, d(at(0), size_t(1) << 29, 8, 1, 2, 5, (size_t(1) << 28) + 1, AR_FLOAT32, at<int>(4), at(6), need));
    REFUSED(AR_ERR_UNSUPPORTED, d(at(0), 1, 8, size_t(1) << 31, 1, 5, 1, AR_FLOAT32, at<int>(4), at(6), need));
    REFUSED(AR_ERR_INVALID_ARG, d(at(0), 16, 8, SIZE_MAX / 2, 2, 5, 16, AR_FLOAT32, at<int>(4), at(6), need));

    RUNS(ar_expert_combine(ctx, at(0), at<float>(1), at<int>(2), at<int>(3), 10, 2, 5, 16,
                           AR_BFLOAT16, at(4)));
    CHECK(g_combine.weights == at<float>(1) && !g_combine.dy);
    REFUSED(AR_ERR_INVALID_ARG, ar_expert_combine(ctx, at(0), nullptr, at<int>(2), at<int>(3), 10, 2,
                                                  5, 16, AR_BFLOAT16, at(4)));
    RUNS(ar_expert_dispatch_backward(ctx, at(0), at<int>(2), at<int>(3), 10, 2, 5, 16, AR_BFLOAT16,
                                     at(4)));
    CHECK(!g_combine.weights);
    REFUSED(AR_ERR_INVALID_ARG, ar_expert_dispatch_backward(ctx, at(0), at<int>(2), at<int>(3), 10, 2,
                                                            5, 16, AR_BFLOAT16, at(0)));
    RUNS(ar_expert_combine_backward(ctx, at(0), 20, at(1), at<float>(2), at<int>(3), at<int>(4), 10,
                                    2, 5, 16, AR_FLOAT32, at(5), at<float>(6)));
    CHECK(g_combine.dystride == 20);
    REFUSED(AR_ERR_INVALID_ARG,
            ar_expert_combine_backward(ctx, at(0), 12, at(1), at<float>(2), at<int>(3), at<int>(4),
                                       10, 2, 5, 16, AR_FLOAT32, at(5), at<float>(6)));
    REFUSED(AR_ERR_INVALID_ARG,
            ar_expert_combine_backward(ctx, at(0), 16, at(1), at<float>(2), at<int>(3), at<int>(4),
                                       10, 2, 5, 16, AR_FLOAT32, at(1), at<float>(6)));
}

void distill() {
    size_t need = 0;
    for (int grad = 0; grad < 2; ++grad) {
        CHECK(ar_distill_workspace(4, 1000, 16, AR_FLOAT32, grad, &need) == AR_OK);
        CHECK(ar_distill_workspace(4, 0, 16, AR_FLOAT32, grad, &need) == AR_ERR_INVALID_ARG);
        CHECK(ar_distill_workspace(4, 1000, 0, AR_FLOAT32, grad, &need) == AR_ERR_INVALID_ARG);
        CHECK(ar_distill_workspace(4, 1000, 1025, AR_FLOAT32, grad, &need) == AR_ERR_UNSUPPORTED);
        CHECK(ar_distill_workspace(4, 1000, 16, AR_INT32, grad, &need) == AR_ERR_INVALID_ARG);
        CHECK(ar_distill_workspace(SIZE_MAX, 1000, 16, AR_FLOAT32, grad, &need) == AR_ERR_INVALID_ARG);
        CHECK(ar_distill_workspace(4, 1000, 16, AR_FLOAT32, grad, nullptr) == AR_ERR_INVALID_ARG);
    }
    CHECK(ar_distill_workspace(4, 1000, 16, AR_FLOAT32, 0, &need) == AR_OK);
    const auto l = [&](size_t stride, int ib, size_t rows, size_t vocab, size_t top, int dt, float T,
                       float* lse, void* ws, size_t n) {
        return ar_distill_loss(ctx, at(0), stride, at(1), ib, at(2), rows, vocab, top, (ar_dtype)dt,
                               T, at<float>(3), lse, ws, n);
    };
    RUNS(l(1000, 8, 4, 1000, 16, AR_FLOAT32, 2.0f, at<float>(4), at(5), need));
    CHECK(g_distill.rows == 4 && g_distill.ib == 8 && g_distill.temperature == 2.0f);
    RUNS(l(1000, 8, 0, 1000, 16, AR_FLOAT32, 2.0f, nullptr, nullptr, 0));
    REFUSED(AR_ERR_INVALID_ARG, l(999, 8, 4, 1000, 16, AR_FLOAT32, 2.0f, at<float>(4), at(5), need));
    REFUSED(AR_ERR_INVALID_ARG, l(1000, 3, 4, 1000, 16, AR_FLOAT32, 2.0f, at<float>(4), at(5), need));
    REFUSED(AR_ERR_INVALID_ARG, l(1000, 8, 4, 0, 16, AR_FLOAT32, 2.0f, at<float>(4), at(5), need));
    REFUSED(AR_ERR_INVALID_ARG, l(1000, 8, 4, 1000, 0, AR_FLOAT32, 2.0f, at<float>(4), at(5), need));
    REFUSED(AR_ERR_INVALID_ARG, l(1000, 8, 4, 1000, 16, AR_INT32, 2.0f, at<float>(4), at(5), need));
    for (float T : {0.0f, -1.0f, (float)NAN, (float)INFINITY})
        REFUSED(AR_ERR_INVALID_ARG, l(1000, 8, 4, 1000, 16, AR_FLOAT32, T, at<float>(4), at(5), need));
    REFUSED(AR_ERR_INVALID_ARG, l(1000, 8, 4, 1000, 16, AR_FLOAT32, 2.0f, nullptr, at(5), need));
    if (need) {
        REFUSED(AR_ERR_INVALID_ARG, l(1000, 8, 4, 1000, 16, AR_FLOAT32, 2.0f, at<float>(4), at(5), need - 1));
        REFUSED(AR_ERR_INVALID_ARG, l(1000, 8, 4, 1000, 16, AR_FLOAT32, 2.0f, at<float>(4), nullptr, need));
    }
    REFUSED(AR_ERR_UNSUPPORTED, l(1000, 8, 4, 1000, 1025, AR_FLOAT32, 2.0f, at<float>(4), at(5), need));
    REFUSED(AR_ERR_UNSUPPORTED, l(size_t(1) << 31, 8, 1, size_t(1) << 31, 16, AR_FLOAT32, 2.0f, at<float>(4), at(5), need));
    REFUSED(AR_ERR_INVALID_ARG, l(SIZE_MAX / 4, 8, 4, 1000, 16, AR_FLOAT32, 2.0f, at<float>(4), at(5), need));

    RUNS(ar_distill_backward(ctx, at<float>(3), at(0), 1000, at(1), 4, at(2), at<float>(4), 4, 1000,
                             16, AR_BFLOAT16, 1.0f, at(5)));
    CHECK(g_distill.lse_in == at<float>(4) && g_distill.ib == 4);
    REFUSED(AR_ERR_INVALID_ARG, ar_distill_backward(ctx, at<float>(3), at(0), 1000, at(1), 4, at(2),
                                                    at<float>(4), 4, 1000, 16, AR_BFLOAT16, 1.0f, at(0)));
    REFUSED(AR_ERR_INVALID_ARG, ar_distill_backward(ctx, nullptr, at(0), 1000, at(1), 4, at(2),
                                                    at<float>(4), 4, 1000, 16, AR_BFLOAT16, 1.0f, at(5)));
    CHECK(ar_distill_workspace(4, 1000, 16, AR_BFLOAT16, 1, &need) == AR_OK);
    RUNS(ar_distill_step(ctx, at<float>(3), at(0), 1000, at(1), 4, at(2), 4, 1000, 16, AR_BFLOAT16,
                         1.0f, at<float>(4), at(5), at(6), need));
    REFUSED(AR_ERR_INVALID_ARG,
            ar_distill_step(ctx, at<float>(3), at(0), 1000, at(1), 4, at(2), 4, 1000, 16,
                            AR_BFLOAT16, 1.0f, at<float>(3), at(5), at(6), need));
}

void null_context() {
    CHECK(ar_set_operator_checks(nullptr, 1) == AR_ERR_INVALID_ARG);
    CHECK(ar_layer_norm(nullptr, at(0), 4, nullptr, nullptr, AR_FLOAT32, at(1), at<float>(2),
                        at<float>(3), 1, 4, AR_FLOAT32, 0.f) == AR_ERR_INVALID_ARG);
    CHECK(ar_layer_norm_backward(nullptr, at(0), 4, at(1), 4, at<float>(2), at<float>(3), nullptr,
                                 AR_FLOAT32, at(4), nullptr, nullptr, 1, 4, AR_FLOAT32, nullptr,
                                 0) == AR_ERR_INVALID_ARG);
    CHECK(ar_expert_dispatch(nullptr, at(0), 4, at(1), 4, 1, 1, 1, 4, AR_FLOAT32, at(2), at<int>(3),
                             at<int>(4), at<int>(5), at(6), 64) == AR_ERR_INVALID_ARG);
    CHECK(ar_distill_loss(nullptr, at(0), 4, at(1), 4, at(2), 1, 4, 1, AR_FLOAT32, 1.f, at<float>(3),
                          at<float>(4), at(5), 64) == AR_ERR_INVALID_ARG);
}

}  // namespace

namespace arlib {
// stand-ins for the kernels' launchers and their scratch sizes
size_t norm_grad_parts(size_t rows, size_t, int) { return rows < 100 ? (rows ? 1 : 0) : 1024; }
hipError_t launch_norm(const NormArgs& a, hipStream_t) {
    g_norm = a;
    ++g_launches;
    return hipSuccess;
}
hipError_t launch_norm_grad(const NormGradArgs& a, hipStream_t) {
    g_norm_grad = a;
    ++g_launches;
    return hipSuccess;
}
size_t dispatch_work_ints(size_t tokens, int topk, int experts) {
    return (tokens * topk / 2048 + 1) * (experts + 1);
}
hipError_t launch_dispatch(const DispatchArgs& a, hipStream_t) {
    g_dispatch = a;
    ++g_launches;
    return hipSuccess;
}
hipError_t launch_combine(const CombineArgs& a, hipStream_t) {
    g_combine = a;
    ++g_launches;
    return hipSuccess;
}
hipError_t launch_combine_grad(const CombineArgs& a, hipStream_t) {
    g_combine = a;
    ++g_launches;
    return hipSuccess;
}
size_t distill_work_floats(size_t rows, size_t, size_t, int, bool step) { return rows * (step ? 4 : 2); }
hipError_t launch_distill_loss(const DistillArgs& a, hipStream_t) {
    g_distill = a;
    ++g_launches;
    return hipSuccess;
}
hipError_t launch_distill_backward(const DistillArgs& a, hipStream_t) {
    g_distill = a;
    ++g_launches;
    return hipSuccess;
}
hipError_t launch_distill_step(const DistillArgs& a, hipStream_t) {
    g_distill = a;
    ++g_launches;
    return hipSuccess;
}
}  // namespace arlib

int main() {
    fake_register(reinterpret_cast<void*>(kBase), 61 * kStep, 0);
    null_context();
    if (ar_create(&ctx, 0, nullptr) != AR_OK) return 1;
    norm();
    route();
    distill();
    ar_destroy(ctx);
    if (g_fail) return 1;
    std::printf("ALL OK\n");
    return 0;
}
