// model_launch_driver.cpp -- runs the launchers of the embedding, the experts'
// products and the gated activation (embed.hip, product.hip, gate.hip, host side
// only) through their C entry points against the fake HIP runtime, recording
// each launch instead of running it.  Test infrastructure only: prints "ALL OK"
// and exits 0 when every check passes.
//
// Every launch has to be one that HIP accepts (blocks of 1 .. 1024 threads, fewer
// than 2^32 threads in each dimension of the grid), over sizes from a row of one
// element to the largest that the operators take, with exactly the scratch that
// they ask for.
#include <hip/hip_runtime_api.h>

#include <cstdint>
#include <cstdio>
#include <map>
#include <string>

#include "ar.h"
#include "fake_hip.h"

namespace {

std::map<const void*, std::string>& names() {
    static std::map<const void*, std::string> m;
    return m;
}
struct Call {
    dim3 grid, block;
};
Call g_call;
std::map<std::string, int> g_seen;    // launches by kernel
int g_fail = 0, g_launches = 0;
std::string g_what;

#define CHECK(c)                                                                                  \
    do {                                                                                          \
        if (!(c)) {                                                                               \
            std::fprintf(stderr, "FAIL %s:%d: %s (%s)\n", __FILE__, __LINE__, #c, g_what.c_str()); \
            ++g_fail;                                                                             \
        }                                                                                         \
    } while (0)

}  // namespace

extern "C" {
hipError_t __hipPushCallConfiguration(dim3 grid, dim3 block, size_t, hipStream_t) {
    g_call = {grid, block};
    return hipSuccess;
}
hipError_t __hipPopCallConfiguration(dim3* grid, dim3* block, size_t* lds, hipStream_t* s) {
    *grid = g_call.grid;
    *block = g_call.block;
    *lds = 0;
    *s = nullptr;
    return hipSuccess;
}
hipError_t hipLaunchKernel(const void* f, dim3 grid, dim3 block, void**, size_t, hipStream_t) {
    const uint64_t g[3] = {grid.x, grid.y, grid.z}, b[3] = {block.x, block.y, block.z};
    bool good = b[0] * b[1] * b[2] >= 1 && b[0] * b[1] * b[2] <= 1024;
    for (int i = 0; i < 3; ++i) good = good && g[i] >= 1 && g[i] * b[i] < (uint64_t(1) << 32);
    CHECK(good);
    ++g_launches;
    ++g_seen[names()[f]];
    return hipSuccess;
}
void** __hipRegisterFatBinary(const void*) {
    static void* handle;
    return &handle;
}
void __hipRegisterFunction(void**, const void* host, char*, const char* name, unsigned, void*, void*,
                           void*, void*, int*) {
    names()[host] = name;
}
void __hipRegisterVar(void**, void*, char*, char*, int, size_t, int, int) {}
void __hipUnregisterFatBinary(void**) {}
}

namespace {

ar_ctx* ctx = nullptr;
constexpr uintptr_t kBase = uintptr_t(1) << 44;
// Byte i x 16 TiB into the device's memory.
template <class T = void>
T* at(int i) {
    return reinterpret_cast<T*>(kBase * (1 + i));
}

// Launches of a call that succeeds.
template <class F>
int launches(F call) {
    g_launches = 0;
    CHECK(call() == AR_OK);
    return g_launches;
}

int seen(const char* part) {
    int n = 0;
    for (const auto& k : g_seen)
        if (k.first.find(part) != std::string::npos) n += k.second;
    return n;
}

void embed() {
    for (const ar_dtype t : {AR_BFLOAT16, AR_FLOAT32})
        for (const int ib : {4, 8})
            for (const size_t tokens : {size_t(0), size_t(1), size_t(16), size_t(17), size_t(1000),
                                        size_t(32768), size_t(32769), size_t(65537), size_t(1) << 24,
                                        (size_t(1) << 31) - 1})
                for (const size_t vocab : {size_t(1), size_t(255), size_t(50021), size_t(1) << 20,
                                           size_t(1) << 28})
                    for (const size_t hidden : {size_t(1), size_t(7), size_t(64), size_t(771),
                                                size_t(8192), size_t(1) << 20}) {
                        if ((double)vocab * hidden > 1e12 || (double)tokens * hidden > 1e12) continue;
                        g_what = "embedding " + std::to_string(tokens) + " of " + std::to_string(vocab) +
                                 " x " + std::to_string(hidden);
                        const int f = launches([&] {
                            return ar_embedding(ctx, at(0), at(1), ib, tokens, vocab, hidden, t, 1.f, at(2));
                        });
                        CHECK(f == (tokens ? 1 : 0));
                        size_t need = 0;
                        CHECK(ar_embedding_backward_workspace(tokens, vocab, hidden, t, &need) == AR_OK);
                        const int b = launches([&] {
                            return ar_embedding_backward(ctx, at(0), hidden, at(1), ib, tokens, vocab,
                                                         hidden, t, 1.f, at(2), at(3), need);
                        });
                        // the order (with the buckets' two launches), the pieces, the rows
                        const int want = tokens == 0 ? 1 : tokens <= 16 ? 2 : tokens <= 32768 ? 3 : 5;
                        CHECK(b == want);
                    }
    CHECK(seen("k_embed_bucket") > 0 && seen("k_embed_pieces") > 0);
}

void product() {
    for (const ar_dtype t : {AR_BFLOAT16, AR_FLOAT32})
        for (const int experts : {1, 7, 64, 1024})
            for (const size_t n : {size_t(0), size_t(1), size_t(33), size_t(1000), size_t(65536),
                                   size_t(10000000), (size_t(1) << 31) - 1})
                for (const size_t hidden : {size_t(1), size_t(65), size_t(2048), size_t(8191),
                                            size_t(1) << 20})
                    for (const size_t out : {size_t(1), size_t(130), size_t(4096), size_t(1) << 20}) {
                        if ((double)n * hidden > 1e12 || (double)n * out > 1e12 ||
                            (double)experts * hidden * out > 1e12)
                            continue;
                        g_what = std::to_string(experts) + " experts, " + std::to_string(n) + " rows, " +
                                 std::to_string(hidden) + " -> " + std::to_string(out);
                        for (int k = 0; k < 3; ++k) {
                            size_t need = 0;
                            CHECK(ar_expert_matmul_workspace((ar_expert_product)k, n, experts, hidden,
                                                             out, t, &need) == AR_OK);
                            const int c = launches([&] {
                                const auto f = k == 0 ? ar_expert_matmul : ar_expert_matmul_drows;
                                return k < 2 ? f(ctx, at(0), k ? out : hidden, at(1), at<int>(2), n,
                                                 experts, hidden, out, t, at(3), at(4), need)
                                             : ar_expert_matmul_dweights(
                                                   ctx, at(0), out, at(1), hidden, at<int>(2), n,
                                                   experts, hidden, out, t, at(3), at(4), need);
                            });
                            // (parts of the depth are joined by a launch of their own)
                            CHECK(c == (n == 0 && k < 2 ? 0 : need ? 2 : 1));
                        }
                    }
    CHECK(seen("k_product_join") > 0);
}

void gate() {
    for (const ar_dtype t : {AR_BFLOAT16, AR_FLOAT32})
        for (const size_t rows : {size_t(0), size_t(1), size_t(1000), size_t(1) << 24, size_t(1) << 33})
            for (const size_t cols : {size_t(1), size_t(32), size_t(771), size_t(16384), size_t(1) << 28}) {
                if ((double)rows * cols > 2e12) continue;
                g_what = "gate " + std::to_string(rows) + " x " + std::to_string(cols);
                signed char* codes = at<signed char>(1);
                unsigned char* scales = at<unsigned char>(2);
                const int want = rows ? 1 : 0;
                CHECK(want == launches([&] { return ar_save_8bit(ctx, at(0), cols, rows, cols, t, codes, scales); }));
                CHECK(want == launches([&] { return ar_restore_8bit(ctx, codes, scales, rows, cols, t, at(3)); }));
                CHECK(want == launches([&] { return ar_silu_gate(ctx, at(0), 2 * cols, rows, cols, t, at(3), codes, scales); }));
                CHECK(want == launches([&] { return ar_silu_gate_backward(ctx, at(0), cols, codes, scales, rows, cols, t, at(3), at(4)); }));
            }
}

}  // namespace

int main() {
    fake_register(at(0), 7 * kBase, 0);
    if (ar_create(&ctx, 0, nullptr) != AR_OK) return 1;
    embed();
    product();
    gate();
    ar_destroy(ctx);
    if (g_fail) return 1;
    std::printf("ALL OK\n");
    return 0;
}
