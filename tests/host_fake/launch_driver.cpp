// launch_driver.cpp -- runs the training operators' launchers (norm.hip,
// route.hip, distill.hip, host side only) and C entry points against the fake
// HIP runtime, recording each launch instead of running it.  Test
// infrastructure only: prints "ALL OK" and exits 0 when every check of the
// section named on the command line passes.
//
// Every launch of every section has to be one that HIP accepts: blocks of
// 1 .. 1024 threads, fewer than 2^32 threads in each dimension of the grid.
#include <hip/hip_runtime_api.h>

#include <cfloat>
#include <cstdint>
#include <cstdio>
#include <cstring>
#include <map>
#include <string>
#include <vector>

#include "ar.h"
#include "fake_hip.h"
#include "ops.h"

namespace {

struct Launch {
    std::string kernel;   // mangled
    dim3 grid, block;
    size_t lds;
    size_t parts;         // of the kernels that are told how many parts the scratch holds
    bool is(const char* name) const { return kernel.find(name) != std::string::npos; }
};
// kernels by their host address (the objects register them before main, in any order)
std::map<const void*, std::string>& names() {
    static std::map<const void*, std::string> m;
    return m;
}
std::vector<Launch> g_launches;
Launch g_call;
int g_fail = 0;

#define CHECK(c)                                                              \
    do {                                                                      \
        if (!(c)) {                                                           \
            std::fprintf(stderr, "FAIL %s:%d: %s\n", __FILE__, __LINE__, #c); \
            ++g_fail;                                                         \
        }                                                                     \
    } while (0)

}  // namespace

extern "C" {
hipError_t __hipPushCallConfiguration(dim3 grid, dim3 block, size_t lds, hipStream_t) {
    g_call = Launch{"", grid, block, lds, 0};
    return hipSuccess;
}
hipError_t __hipPopCallConfiguration(dim3* grid, dim3* block, size_t* lds, hipStream_t* s) {
    *grid = g_call.grid;
    *block = g_call.block;
    *lds = g_call.lds;
    *s = nullptr;
    return hipSuccess;
}
hipError_t hipLaunchKernel(const void* f, dim3 grid, dim3 block, void** args, size_t lds,
                           hipStream_t) {
    Launch l{names()[f], grid, block, lds, 0};
    if (l.is("k_norm_fold") || l.is("k_distill_part") || l.is("k_distill_lossI"))
        l.parts = *static_cast<size_t*>(args[1]);
    else if (l.is("k_distill_grad"))
        l.parts = *static_cast<size_t*>(args[2]);
    g_launches.push_back(l);
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
void __hipUnregisterFatBinary(void**) {}
}

namespace {

// What `call` launches, each of them one that HIP accepts.
template <class F>
std::vector<Launch> launches(const char* what, F call) {
    g_launches.clear();
    CHECK(call() == hipSuccess);
    for (const Launch& l : g_launches) {
        const uint64_t g[3] = {l.grid.x, l.grid.y, l.grid.z}, b[3] = {l.block.x, l.block.y, l.block.z};
        bool good = b[0] * b[1] * b[2] >= 1 && b[0] * b[1] * b[2] <= 1024;
        for (int i = 0; i < 3; ++i)
            good = good && g[i] >= 1 && g[i] * b[i] < (uint64_t(1) << 32);
        if (!good) {
            std::fprintf(stderr, "FAIL %s: %s, grid (%u, %u, %u) of (%u, %u, %u) threads\n", what,
                         l.kernel.c_str(), l.grid.x, l.grid.y, l.grid.z, l.block.x, l.block.y,
                         l.block.z);
            ++g_fail;
        }
    }
    return g_launches;
}

// Not dereferenced: a launcher only passes arrays on.
template <class T = void>
T* array() {
    return reinterpret_cast<T*>(uintptr_t(1) << 44);
}

arlib::NormArgs norm(size_t rows, size_t cols, int eb) {
    return {array(), array(), array(), array(), array<float>(), array<float>(), cols, rows, cols,
            1e-5f,   eb,      4};
}

arlib::NormGradArgs norm_grad(size_t rows, size_t cols, int eb, bool columns = true) {
    return {array(), array(), array<float>(), array<float>(), array(), array(),
            columns ? array() : nullptr, columns ? array() : nullptr, array<float>(), cols, cols,
            rows, cols, eb, 4};
}

// More rows than a grid's blocks: the kernels walk the rest.
void rows() {
    for (const int eb : {2, 4})
        for (const size_t cols : {1, 5, 64, 200, 771, 1024, 4096, 5001, 8192, 16384, 20000})
            for (const size_t n : {size_t(1), size_t(255), size_t(1) << 22, (size_t(1) << 24) + 5,
                                   (size_t(1) << 33) + 1}) {
                launches("norm", [&] { return arlib::launch_norm(norm(n, cols, eb), nullptr); });
                launches("norm gradient",
                         [&] { return arlib::launch_norm_grad(norm_grad(n, cols, eb), nullptr); });
            }
}

// Rows up to the widest that the operators take.
void widths() {
    for (const int eb : {2, 4})
        for (const size_t cols : {(size_t(1) << 27) - 1, size_t(1) << 27, (size_t(1) << 28) - 3,
                                  size_t(1) << 28})
            for (const size_t n : {size_t(1), size_t(70), size_t(100000)}) {
                launches("norm", [&] { return arlib::launch_norm(norm(n, cols, eb), nullptr); });
                launches("norm gradient",
                         [&] { return arlib::launch_norm_grad(norm_grad(n, cols, eb), nullptr); });
            }
}

// A context on the fake device, whose memory starts at array().
struct Device {
    ar_ctx* ctx = nullptr;
    Device() {
        fake_register(array(), size_t(1) << 42, 0);
        CHECK(ar_create(&ctx, 0, nullptr) == AR_OK);
    }
    ~Device() { ar_destroy(ctx); }
};
// Byte i GiB into the device's memory.
template <class T = void>
T* at(size_t i) {
    return reinterpret_cast<T*>(reinterpret_cast<uintptr_t>(array()) + (i << 30));
}

// 1 / T has to be a number that fp32 holds.
void temperatures() {
    Device d;
    for (const float t : {FLT_MIN, 1.0f, FLT_MAX, FLT_MIN / 2, FLT_MIN / 8388608}) {
        const ar_status want = t < FLT_MIN ? AR_ERR_INVALID_ARG : AR_OK;
        g_launches.clear();
        CHECK(ar_distill_loss(d.ctx, at(0), 100, at(1), 8, at(2), 4, 100, 3, AR_FLOAT32, t,
                              at<float>(3), at<float>(4), at(5), 1 << 20) == want);
        CHECK(ar_distill_backward(d.ctx, at<float>(3), at(0), 100, at(1), 8, at(2), at<float>(4), 4,
                                  100, 3, AR_FLOAT32, t, at(5)) == want);
        CHECK(ar_distill_step(d.ctx, at<float>(3), at(0), 100, at(1), 8, at(2), 4, 100, 3, AR_FLOAT32,
                              t, at<float>(4), at(5), at(6), 1 << 20) == want);
        CHECK(g_launches.empty() == (want != AR_OK));
    }
}

// Every kernel stays inside the scratch that its call asks for: the C calls
// with exactly that many bytes, over the sizes where the kernels' forms change.
void scratch() {
    Device d;
    const ar_dtype types[] = {AR_BFLOAT16, AR_FLOAT32};
    size_t need = 0, seen = 0;
    for (const ar_dtype t : types)
        for (const size_t cols : {1, 7, 63, 64, 200, 771, 946, 1024, 2056, 4096, 5001, 8192, 16384,
                                  16391, 70001})
            for (const size_t rows : {0, 1, 2, 8, 9, 64, 65, 133, 700, 1021, 6416, 16384, 70000}) {
                CHECK(ar_layer_norm_backward_workspace(rows, cols, t, &need) == AR_OK);
                const auto ls = launches("norm gradient", [&] {
                    return ar_layer_norm_backward(d.ctx, at(0), cols, at(100), cols, at<float>(200),
                                                  at<float>(201), at(202), AR_FLOAT32, at(300),
                                                  at(400), at(401), rows, cols, t, at(402), need) ==
                                   AR_OK ? hipSuccess : hipErrorUnknown;
                });
                size_t parts = 0;       // what the rows' kernels leave
                bool folded = false;
                for (const Launch& l : ls) {
                    if (l.is("k_norm_grad_rows") || l.is("k_norm_grad_narrow"))
                        parts = l.grid.x > 1 ? l.grid.x : 0;
                    if (l.is("k_norm_cols")) parts = l.grid.y;
                    if (l.is("k_norm_fold")) {
                        CHECK(l.parts == parts);
                        folded = true;
                    }
                }
                CHECK(parts * 2 * cols * sizeof(float) <= need);
                CHECK(folded == (parts > 0 || rows == 0));
                seen += folded;
                // (none of it where the columns' sums are not wanted)
                CHECK(ar_layer_norm_backward(d.ctx, at(0), cols, at(100), cols, at<float>(200),
                                             at<float>(201), at(202), AR_FLOAT32, at(300), nullptr,
                                             nullptr, rows, cols, t, nullptr, 0) == AR_OK);
            }
    CHECK(seen > 0);
    seen = 0;
    for (const int topk : {1, 2, 5, 8, 9, 100})
        for (const int experts : {1, 7, 64, AR_MAX_EXPERTS})
            for (const size_t tokens : {0, 1, 300, 1024, 1448, 2000, 16384, 70001, 1000000}) {
                CHECK(ar_expert_dispatch_workspace(tokens, topk, experts, &need) == AR_OK);
                const auto ls = launches("dispatch", [&] {
                    return ar_expert_dispatch(d.ctx, at(0), 8, at(100), 8, tokens, topk, experts, 8,
                                              AR_FLOAT32, at(200), at<int>(300), at<int>(301),
                                              at<int>(302), at(303), need) == AR_OK
                               ? hipSuccess : hipErrorUnknown;
                });
                unsigned blocks = 0;
                for (const Launch& l : ls) {
                    if (l.is("k_route_count")) blocks = l.grid.x;
                    if (l.is("k_route_place")) CHECK(l.grid.x == blocks && blocks > 0);
                }
                CHECK((size_t)blocks * (experts + 1) * sizeof(int) <= need);
                seen += blocks > 0;
            }
    CHECK(seen > 0);
    seen = 0;
    for (const ar_dtype t : types)
        for (const size_t vocab : {1, 5, 8, 300, 1003, 4099, 8191, 32000, 50021, 65536, 65540, 131072,
                                   131073, 200000})
            for (const size_t rows : {0, 1, 8, 64, 65, 300, 511, 512, 2047, 7000})
                for (const int step : {0, 1}) {
                    CHECK(ar_distill_workspace(rows, vocab, 30, t, step, &need) == AR_OK);
                    const auto ls = launches("distillation", [&] {
                        const ar_status s =
                            step ? ar_distill_step(d.ctx, at<float>(0), at(100), vocab, at(200), 8,
                                                   at(201), rows, vocab, 30, t, 1.0f, at<float>(202),
                                                   at(300), at(400), need)
                                 : ar_distill_loss(d.ctx, at(100), vocab, at(200), 8, at(201), rows,
                                                   vocab, 30, t, 1.0f, at<float>(202), at<float>(203),
                                                   at(400), need);
                        return s == AR_OK ? hipSuccess : hipErrorUnknown;
                    });
                    size_t parts = 0;
                    for (const Launch& l : ls) {
                        if (l.is("k_distill_part")) parts = l.parts;
                        else if (!l.is("k_distill_rows") && !l.is("k_distill_loss_rows"))
                            CHECK(l.parts == parts && parts > 0);
                    }
                    CHECK(rows * parts * 2 * sizeof(float) <= need);
                    seen += parts > 0;
                }
    CHECK(seen > 0);
}

struct Section {
    const char* name;
    void (*run)();
};
const Section kSections[] = {
    {"rows", rows}, {"widths", widths}, {"temperatures", temperatures}, {"scratch", scratch}};

}  // namespace

int main(int argc, char** argv) {
    for (const Section& s : kSections)
        if (argc == 2 && !std::strcmp(argv[1], s.name)) {
            s.run();
            if (g_fail) return 1;
            std::printf("ALL OK\n");
            return 0;
        }
    std::fprintf(stderr, "no such section\n");
    return 2;
}
