// product_plan_driver.cpp -- which kernel the experts' products launch: runs
// their launcher (product.hip, host side only) through the C entry points
// against the fake HIP runtime and prints the launches.  Test infrastructure
// only; nothing is computed.
//
// A line of standard input is a call, "kind dtype rows experts hidden out
// a_stride b_stride a_shift b_shift" (ar_expert_product and ar_dtype as numbers,
// shifts in elements from an aligned address, b_stride for the weights' gradient
// alone); a line of output is the names of the kernels that it launches, with
// ';' between them.  Ends with "ALL OK" and status 0 if every call succeeded.
#include <cxxabi.h>
#include <hip/hip_runtime_api.h>

#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <map>
#include <string>

#include "ar.h"
#include "fake_hip.h"

namespace {

std::map<const void*, std::string>& names() {
    static std::map<const void*, std::string> m;
    return m;
}
std::string g_launched;

}  // namespace

extern "C" {
hipError_t __hipPushCallConfiguration(dim3, dim3, size_t, hipStream_t) { return hipSuccess; }
hipError_t __hipPopCallConfiguration(dim3* grid, dim3* block, size_t* lds, hipStream_t* s) {
    *grid = *block = dim3(1);
    *lds = 0;
    *s = nullptr;
    return hipSuccess;
}
hipError_t hipLaunchKernel(const void* f, dim3, dim3, void**, size_t, hipStream_t) {
    int status = 0;
    char* text = abi::__cxa_demangle(names()[f].c_str(), nullptr, nullptr, &status);
    g_launched += (status == 0 ? text : names()[f]) + std::string(";");
    std::free(text);
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

int main() {
    // arrays 16 TiB apart; nothing is dereferenced
    constexpr uintptr_t kBase = uintptr_t(1) << 44;
    fake_register(reinterpret_cast<void*>(kBase), 7 * kBase, 0);
    const auto at = [&](int i, size_t bytes = 0) {
        return reinterpret_cast<void*>(kBase * (1 + i) + bytes);
    };
    ar_ctx* ctx = nullptr;
    if (ar_create(&ctx, 0, nullptr) != AR_OK) return 1;
    int kind, dtype, experts;
    size_t rows, hidden, out, as, bs, sa, sb;
    while (std::scanf("%d %d %zu %d %zu %zu %zu %zu %zu %zu", &kind, &dtype, &rows, &experts, &hidden,
                      &out, &as, &bs, &sa, &sb) == 10) {
        const ar_dtype t = (ar_dtype)dtype;
        const size_t eb = t == AR_BFLOAT16 ? 2 : 4;
        size_t need = 0;
        g_launched.clear();
        ar_status s = ar_expert_matmul_workspace((ar_expert_product)kind, rows, experts, hidden, out,
                                                 t, &need);
        int* offsets = static_cast<int*>(at(2));
        if (s == AR_OK && kind == AR_EXPERT_DWEIGHTS)
            s = ar_expert_matmul_dweights(ctx, at(0, sa * eb), as, at(1, sb * eb), bs, offsets, rows,
                                          experts, hidden, out, t, at(3), at(4), need);
        else if (s == AR_OK)
            s = (kind == AR_EXPERT_FORWARD ? ar_expert_matmul : ar_expert_matmul_drows)(
                ctx, at(0, sa * eb), as, at(1, sb * eb), offsets, rows, experts, hidden, out, t, at(3),
                at(4), need);
        if (s != AR_OK) {
            std::fprintf(stderr, "status %d: %s\n", (int)s, ar_last_error(ctx));
            return 1;
        }
        std::printf("%s\n", g_launched.c_str());
    }
    ar_destroy(ctx);
    std::printf("ALL OK\n");
    return 0;
}
