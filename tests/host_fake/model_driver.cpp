// model_driver.cpp -- runs the C entry points of the embedding, the experts'
// products and the gated activation (model_api.cpp) against the fake HIP runtime
// under the host sanitizers, with launchers that record their arguments.  Test
// infrastructure only: prints "ALL OK" and exits 0 when every check passes.
#include <cmath>
#include <cstdint>
#include <cstdio>

#include "ar.h"
#include "fake_hip.h"
#include "model_ops.h"

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
arlib::EmbedArgs g_embed;
arlib::EmbedGradArgs g_embed_grad;
arlib::ProductArgs g_product;
arlib::ProductKind g_kind;
arlib::GateArgs g_gate;

// arrays 1 GiB apart from here on; nothing is dereferenced
constexpr uintptr_t kBase = uintptr_t(1) << 44, kStep = uintptr_t(1) << 30;
template <class T = void>
T* at(int i, size_t shift = 0) {
    return reinterpret_cast<T*>(kBase + (uintptr_t)i * kStep + shift);
}
typedef signed char code_t;
typedef unsigned char scale_t;

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
#define BAD(call) REFUSED(AR_ERR_INVALID_ARG, call)
#define PAST(call) REFUSED(AR_ERR_UNSUPPORTED, call)

ar_ctx* ctx = nullptr;
constexpr size_t kBig = size_t(1) << 28;

void embed() {
    const auto f = [&](const void* table, const void* ids, int ib, size_t tokens, size_t vocab,
                       size_t hidden, int dt, float scale, void* y) {
        return ar_embedding(ctx, table, ids, ib, tokens, vocab, hidden, (ar_dtype)dt, scale, y);
    };
    RUNS(f(at(0), at(1), 8, 10, 100, 16, AR_BFLOAT16, 2.0f, at(2)));
    CHECK(g_embed.tokens == 10 && g_embed.vocab == 100 && g_embed.hidden == 16 && g_embed.eb == 2 &&
          g_embed.ib == 8 && g_embed.scale == 2.0f);
    RUNS(f(at(0, 4), at(1, 4), 4, 10, 100, 17, AR_FLOAT32, 0.0f, at(2, 12)));
    RUNS(f(at(0), nullptr, 4, 0, 100, 17, AR_FLOAT32, -1.0f, nullptr));
    BAD(f(at(0), at(1), 2, 10, 100, 16, AR_BFLOAT16, 1.0f, at(2)));
    BAD(f(at(0), at(1), 8, 10, 0, 16, AR_BFLOAT16, 1.0f, at(2)));
    BAD(f(at(0), at(1), 8, 10, 100, 0, AR_BFLOAT16, 1.0f, at(2)));
    BAD(f(at(0), at(1), 8, 10, 100, 16, AR_INT32, 1.0f, at(2)));
    for (const float s : {(float)NAN, (float)INFINITY, -(float)INFINITY})
        BAD(f(at(0), at(1), 8, 10, 100, 16, AR_BFLOAT16, s, at(2)));
    BAD(f(nullptr, at(1), 8, 10, 100, 16, AR_BFLOAT16, 1.0f, at(2)));
    BAD(f(at(0), at(1), 8, 10, 100, 16, AR_BFLOAT16, 1.0f, nullptr));
    BAD(f(at(0, 1), at(1), 8, 10, 100, 16, AR_BFLOAT16, 1.0f, at(2)));
    BAD(f(at(0), at(1, 4), 8, 10, 100, 16, AR_BFLOAT16, 1.0f, at(2)));
    BAD(f(at(0), at(1), 8, 10, 100, 16, AR_BFLOAT16, 1.0f, at(0, 3198)));
    RUNS(f(at(0), at(1), 8, 10, 100, 16, AR_BFLOAT16, 1.0f, at(0, 3200)));
    BAD(f(at(60), at(1), 8, 10, 1 << 20, 4096, AR_FLOAT32, 1.0f, at(2)));       // past the allocation
    PAST(f(at(0), at(1), 8, 10, kBig + 1, 16, AR_BFLOAT16, 1.0f, at(2)));
    PAST(f(at(0), at(1), 8, 10, 100, kBig + 1, AR_BFLOAT16, 1.0f, at(2)));
    PAST(f(at(0), at(1), 8, size_t(1) << 31, 100, 16, AR_BFLOAT16, 1.0f, at(2)));

    size_t need = 0;
    CHECK(ar_embedding_backward_workspace(50, 100, 16, AR_BFLOAT16, nullptr) == AR_ERR_INVALID_ARG);
    CHECK(ar_embedding_backward_workspace(50, 0, 16, AR_BFLOAT16, &need) == AR_ERR_INVALID_ARG);
    CHECK(ar_embedding_backward_workspace(50, 100, 0, AR_BFLOAT16, &need) == AR_ERR_INVALID_ARG);
    CHECK(ar_embedding_backward_workspace(50, 100, 16, AR_INT32, &need) == AR_ERR_INVALID_ARG);
    CHECK(ar_embedding_backward_workspace(50, kBig + 1, 16, AR_FLOAT32, &need) == AR_ERR_UNSUPPORTED);
    CHECK(ar_embedding_backward_workspace(SIZE_MAX, 100, 16, AR_FLOAT32, &need) == AR_ERR_UNSUPPORTED);
    CHECK(ar_embedding_backward_workspace(50, 100, 16, AR_BFLOAT16, &need) == AR_OK && need > 0);
    const auto b = [&](size_t stride, void* d, void* ws, size_t n) {
        return ar_embedding_backward(ctx, at(0), stride, at(1), 4, 50, 100, 16, AR_BFLOAT16, 1.0f, d, ws, n);
    };
    RUNS(b(20, at(2), at(3), need));
    CHECK(g_embed_grad.dystride == 20 && g_embed_grad.work == at<int>(3) && g_embed_grad.tokens == 50);
    BAD(b(15, at(2), at(3), need));
    BAD(b(16, at(2), at(3), need - 1));
    BAD(b(16, at(2), nullptr, need));
    BAD(b(16, at(2), at(3, 8), need));
    BAD(b(16, at(0), at(3), need));
    BAD(b(16, at(2), at(2), need));
    BAD(b(16, nullptr, at(3), need));
    BAD(b(SIZE_MAX / 16, at(2), at(3), need));
}

void product() {
    size_t need = 0;
    const ar_expert_product kinds[] = {AR_EXPERT_FORWARD, AR_EXPERT_DROWS, AR_EXPERT_DWEIGHTS};
    for (const auto k : kinds) {
        CHECK(ar_expert_matmul_workspace(k, 50, 4, 24, 40, AR_FLOAT32, &need) == AR_OK && need == 64);
        CHECK(ar_expert_matmul_workspace(k, 50, 0, 24, 40, AR_FLOAT32, &need) == AR_ERR_INVALID_ARG);
        CHECK(ar_expert_matmul_workspace(k, 50, 4, 0, 40, AR_FLOAT32, &need) == AR_ERR_INVALID_ARG);
        CHECK(ar_expert_matmul_workspace(k, 50, 4, 24, 0, AR_FLOAT32, &need) == AR_ERR_INVALID_ARG);
        CHECK(ar_expert_matmul_workspace(k, 50, 4, 24, 40, AR_INT32, &need) == AR_ERR_INVALID_ARG);
        CHECK(ar_expert_matmul_workspace(k, 50, 4, 24, 40, AR_FLOAT32, nullptr) == AR_ERR_INVALID_ARG);
        CHECK(ar_expert_matmul_workspace(k, 50, 1025, 24, 40, AR_FLOAT32, &need) == AR_ERR_UNSUPPORTED);
        CHECK(ar_expert_matmul_workspace(k, 50, 4, (1 << 20) + 1, 40, AR_FLOAT32, &need) == AR_ERR_UNSUPPORTED);
        CHECK(ar_expert_matmul_workspace(k, size_t(1) << 31, 4, 24, 40, AR_FLOAT32, &need) == AR_ERR_UNSUPPORTED);
    }
    CHECK(ar_expert_matmul_workspace((ar_expert_product)3, 50, 4, 24, 40, AR_FLOAT32, &need) == AR_ERR_INVALID_ARG);
    const auto f = [&](const void* rows, size_t stride, const void* w, const int* off, size_t n, int e,
                       size_t hidden, size_t out, int dt, void* y, void* ws, size_t bytes) {
        return ar_expert_matmul(ctx, rows, stride, w, off, n, e, hidden, out, (ar_dtype)dt, y, ws, bytes);
    };
    RUNS(f(at(0), 30, at(1), at<int>(2), 50, 4, 24, 40, AR_BFLOAT16, at(3), at(4), 64));
    CHECK(g_kind == arlib::PRODUCT_FORWARD && g_product.astride == 30 && g_product.hidden == 24 &&
          g_product.out == 40 && g_product.experts == 4 && g_product.nrows == 50 && g_product.eb == 2);
    RUNS(f(nullptr, 0, at(1), at<int>(2), 0, 4, 24, 40, AR_FLOAT32, nullptr, at(4), 64));
    RUNS(f(at(0), SIZE_MAX, at(1), at<int>(2), 1, 4, 24, 40, AR_FLOAT32, at(3), at(4), 64));
    CHECK(g_product.astride == 24);      // (a single row's is of no meaning)
    BAD(f(at(0), 23, at(1), at<int>(2), 50, 4, 24, 40, AR_FLOAT32, at(3), at(4), 64));
    BAD(f(at(0), 24, at(1), at<int>(2), 50, 0, 24, 40, AR_FLOAT32, at(3), at(4), 64));
    BAD(f(at(0), 24, at(1), at<int>(2), 50, 4, 0, 40, AR_FLOAT32, at(3), at(4), 64));
    BAD(f(at(0), 24, at(1), at<int>(2), 50, 4, 24, 0, AR_FLOAT32, at(3), at(4), 64));
    BAD(f(at(0), 24, at(1), at<int>(2), 50, 4, 24, 40, AR_INT32, at(3), at(4), 64));
    BAD(f(nullptr, 24, at(1), at<int>(2), 50, 4, 24, 40, AR_FLOAT32, at(3), at(4), 64));
    BAD(f(at(0), 24, nullptr, at<int>(2), 50, 4, 24, 40, AR_FLOAT32, at(3), at(4), 64));
    BAD(f(at(0), 24, at(1), nullptr, 50, 4, 24, 40, AR_FLOAT32, at(3), at(4), 64));
    BAD(f(at(0), 24, at(1), at<int>(2), 50, 4, 24, 40, AR_FLOAT32, nullptr, at(4), 64));
    BAD(f(at(0, 2), 24, at(1), at<int>(2), 50, 4, 24, 40, AR_FLOAT32, at(3), at(4), 64));
    BAD(f(at(0), 24, at(1), at<int>(2, 2), 50, 4, 24, 40, AR_FLOAT32, at(3), at(4), 64));
    BAD(f(at(0), 24, at(1), at<int>(2), 50, 4, 24, 40, AR_FLOAT32, at(1, 100), at(4), 64));
    BAD(f(at(0), 24, at(1), at<int>(2), 50, 4, 24, 40, AR_FLOAT32, at(3), at(4), 63));
    BAD(f(at(0), 24, at(1), at<int>(2), 50, 4, 24, 40, AR_FLOAT32, at(3), at(3, 16), 64));
    PAST(f(at(0), 24, at(1), at<int>(2), 50, 1025, 24, 40, AR_FLOAT32, at(3), at(4), 64));
    PAST(f(at(0), size_t(1) << 21, at(1), at<int>(2), 1, 4, size_t(1) << 21, 40, AR_FLOAT32, at(3), at(4), 64));
    PAST(f(at(0), (1 << 20) + 1, at(1), at<int>(2), 50, 4, 24, 40, AR_FLOAT32, at(3), at(4), 64));
    PAST(f(at(0), 24, at(1), at<int>(2), size_t(1) << 31, 4, 24, 40, AR_FLOAT32, at(3), at(4), 64));
    RUNS(ar_expert_matmul_drows(ctx, at(0), 40, at(1), at<int>(2), 50, 4, 24, 40, AR_FLOAT32, at(3),
                                at(4), 64));
    CHECK(g_kind == arlib::PRODUCT_DROWS && g_product.astride == 40);
    BAD(ar_expert_matmul_drows(ctx, at(0), 39, at(1), at<int>(2), 50, 4, 24, 40, AR_FLOAT32, at(3),
                               at(4), 64));
    const auto w = [&](size_t gs, size_t rs, size_t n, const void* rows, void* d) {
        return ar_expert_matmul_dweights(ctx, at(0), gs, rows, rs, at<int>(2), n, 4, 24, 40,
                                         AR_BFLOAT16, d, at(4), 64);
    };
    RUNS(w(40, 30, 50, at(1), at(3)));
    CHECK(g_kind == arlib::PRODUCT_DWEIGHTS && g_product.astride == 40 && g_product.bstride == 30);
    RUNS(w(40, 30, 0, nullptr, at(3)));
    BAD(w(39, 30, 50, at(1), at(3)));
    BAD(w(40, 23, 50, at(1), at(3)));
    BAD(w(40, 24, 50, nullptr, at(3)));
    BAD(w(40, 24, 50, at(1), nullptr));
    BAD(w(40, 24, 50, at(1), at(1)));
    PAST(w(40, (1 << 20) + 1, 50, at(1), at(3)));
}

void gate() {
    const auto s = [&](const void* x, size_t stride, size_t rows, size_t cols, int dt, code_t* c,
                       scale_t* z) {
        return ar_save_8bit(ctx, x, stride, rows, cols, (ar_dtype)dt, c, z);
    };
    RUNS(s(at(0), 50, 10, 40, AR_BFLOAT16, at<code_t>(1, 3), at<scale_t>(2, 1)));
    CHECK(g_gate.rows == 10 && g_gate.cols == 40 && g_gate.stride == 50 && g_gate.eb == 2);
    RUNS(s(nullptr, 40, 0, 40, AR_FLOAT32, nullptr, nullptr));
    BAD(s(at(0), 39, 10, 40, AR_FLOAT32, at<code_t>(1), at<scale_t>(2)));
    BAD(s(at(0), 40, 10, 0, AR_FLOAT32, at<code_t>(1), at<scale_t>(2)));
    BAD(s(at(0), 40, 10, 40, AR_INT32, at<code_t>(1), at<scale_t>(2)));
    BAD(s(nullptr, 40, 10, 40, AR_FLOAT32, at<code_t>(1), at<scale_t>(2)));
    BAD(s(at(0), 40, 10, 40, AR_FLOAT32, nullptr, at<scale_t>(2)));
    BAD(s(at(0), 40, 10, 40, AR_FLOAT32, at<code_t>(1), nullptr));
    BAD(s(at(0), 40, 10, 40, AR_FLOAT32, at<code_t>(0, 1599), at<scale_t>(2)));
    BAD(s(at(0), 40, 10, 40, AR_FLOAT32, at<code_t>(1), at<scale_t>(1, 399)));
    RUNS(s(at(0), 40, 10, 40, AR_FLOAT32, at<code_t>(1), at<scale_t>(1, 400)));
    PAST(s(at(0), kBig + 1, 1, kBig + 1, AR_FLOAT32, at<code_t>(1), at<scale_t>(2)));
    BAD(s(at(0), 40, SIZE_MAX / 8, 40, AR_FLOAT32, at<code_t>(1), at<scale_t>(2)));
    RUNS(ar_restore_8bit(ctx, at<code_t>(0), at<scale_t>(1), 10, 40, AR_FLOAT32, at(2)));
    BAD(ar_restore_8bit(ctx, at<code_t>(0), at<scale_t>(1), 10, 40, AR_FLOAT32, at(0, 396)));
    BAD(ar_restore_8bit(ctx, nullptr, at<scale_t>(1), 10, 40, AR_FLOAT32, at(2)));
    BAD(ar_restore_8bit(ctx, at<code_t>(0), at<scale_t>(1), 10, 40, AR_INT32, at(2)));
    const auto g = [&](const void* h, size_t stride, size_t rows, size_t cols, void* acts, code_t* c,
                       scale_t* z) {
        return ar_silu_gate(ctx, h, stride, rows, cols, AR_BFLOAT16, acts, c, z);
    };
    RUNS(g(at(0), 80, 10, 40, at(1), at<code_t>(2), at<scale_t>(3)));
    BAD(g(at(0), 79, 10, 40, at(1), at<code_t>(2), at<scale_t>(3)));
    BAD(g(at(0), 80, 10, 40, at(0, 1598), at<code_t>(2), at<scale_t>(3)));
    BAD(g(at(0), 80, 10, 40, at(1), at<code_t>(2), at<scale_t>(2, 799)));
    RUNS(g(at(0), 80, 10, 40, at(1), at<code_t>(2), at<scale_t>(2, 800)));
    BAD(g(at(0), 80, 10, 0, at(1), at<code_t>(2), at<scale_t>(3)));
    const auto b = [&](const void* d, size_t stride, const code_t* c, void* dh, void* acts) {
        return ar_silu_gate_backward(ctx, d, stride, c, at<scale_t>(2), 10, 40, AR_FLOAT32, dh, acts);
    };
    RUNS(b(at(0), 44, at<code_t>(1), at(3), at(4)));
    CHECK(g_gate.stride == 44 && g_gate.dacts == at(0) && g_gate.acts == at(4));
    BAD(b(at(0), 39, at<code_t>(1), at(3), at(4)));
    BAD(b(nullptr, 40, at<code_t>(1), at(3), at(4)));
    BAD(b(at(0), 40, nullptr, at(3), at(4)));
    BAD(b(at(0), 40, at<code_t>(1), nullptr, at(4)));
    BAD(b(at(0), 40, at<code_t>(1), at(3), at(3, 3196)));
    BAD(b(at(0), 40, at<code_t>(1), at(0), at(4)));
}

void null_context() {
    CHECK(ar_embedding(nullptr, at(0), at(1), 4, 1, 1, 1, AR_FLOAT32, 1.f, at(2)) == AR_ERR_INVALID_ARG);
    CHECK(ar_embedding_backward(nullptr, at(0), 1, at(1), 4, 1, 1, 1, AR_FLOAT32, 1.f, at(2), at(3),
                                1 << 20) == AR_ERR_INVALID_ARG);
    CHECK(ar_expert_matmul(nullptr, at(0), 1, at(1), at<int>(2), 1, 1, 1, 1, AR_FLOAT32, at(3), at(4),
                           64) == AR_ERR_INVALID_ARG);
    CHECK(ar_expert_matmul_dweights(nullptr, at(0), 1, at(1), 1, at<int>(2), 1, 1, 1, 1, AR_FLOAT32,
                                    at(3), at(4), 64) == AR_ERR_INVALID_ARG);
    CHECK(ar_save_8bit(nullptr, at(0), 1, 1, 1, AR_FLOAT32, at<code_t>(1), at<scale_t>(2)) ==
          AR_ERR_INVALID_ARG);
    CHECK(ar_silu_gate(nullptr, at(0), 2, 1, 1, AR_FLOAT32, at(1), at<code_t>(2), at<scale_t>(3)) ==
          AR_ERR_INVALID_ARG);
}

}  // namespace

namespace arlib {
// stand-ins for the kernels' launchers and their scratch sizes
size_t embed_grad_work_bytes(size_t tokens, size_t, size_t, int) { return tokens * 16 + 16; }
hipError_t launch_embed(const EmbedArgs& a, hipStream_t) {
    g_embed = a;
    ++g_launches;
    return hipSuccess;
}
hipError_t launch_embed_grad(const EmbedGradArgs& a, hipStream_t) {
    g_embed_grad = a;
    ++g_launches;
    return hipSuccess;
}
size_t product_work_bytes(ProductKind, size_t, int, size_t, size_t, int) { return 64; }
hipError_t launch_product(ProductKind kind, const ProductArgs& a, hipStream_t) {
    g_kind = kind;
    g_product = a;
    ++g_launches;
    return hipSuccess;
}
#define GATE(name)                                     \
    hipError_t name(const GateArgs& a, hipStream_t) {  \
        g_gate = a;                                    \
        ++g_launches;                                  \
        return hipSuccess;                             \
    }
GATE(launch_save)
GATE(launch_restore)
GATE(launch_gate)
GATE(launch_gate_grad)
}  // namespace arlib

int main() {
    fake_register(reinterpret_cast<void*>(kBase), 61 * kStep, 0);
    null_context();
    if (ar_create(&ctx, 0, nullptr) != AR_OK) return 1;
    embed();
    product();
    gate();
    ar_destroy(ctx);
    if (g_fail) return 1;
    std::printf("ALL OK\n");
    return 0;
}
