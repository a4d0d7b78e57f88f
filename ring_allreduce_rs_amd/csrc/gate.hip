// gate.hip -- the experts' gated activation, and checkpoints of activations in
// 8 bits.
//
// A checkpoint keeps each value as a whole number in [-127, 127] times a power
// of two that 32 values along the row share (a group; the last of a row may be
// shorter).  With m the group's largest magnitude, the scale is the least
// 2^(b - 127), b >= 1, with m <= 127 * 2^(b - 127): read off m's bits, so that
// scale, codes and the values read back are exact and the same everywhere.  A
// value is off by at most half a scale: by max(m / 127, 2^-127), as no scale is
// below 2^-126.  Where m is above 1.984375 * 2^127, codes end at 63, so that
// values read back stay finite, and a value is off by less than the scale, 2^122.
// The values have 7 significant bits, so reading them back as bf16 rounds
// nothing.  A group that holds an infinity or a NaN has b = 255 and codes 0, and
// reads back as NaN (0 * 2^128 as binary32 computes it).
//
// The gate takes rows h = (a, u) of two halves of `cols` values:
//   acts = a s u, s = sigmoid(a) = 1 / (1 + e^-a)
// and writes the checkpoint of h in the same pass.  Its backward pass reads the
// checkpoint (a', u') in place of h:
//   da = dacts u' s (1 + a' (1 - s)),  du = dacts a' s,  acts' = a' s u'
// the last for the gradient of the weights that the activations met.
//
// All of it is bound by memory: the bytes of h, acts, codes and scales once, and a
// dozen operations a value beside them.  A thread has 8 values in a row, so a
// group is 4 neighbouring lanes and its maximum two DPP steps; the halves' units
// at the same column belong to one thread.  Measured at 65536 x 2048 bf16: gate
// 175 - 182 us (1.05 GB moved, 5.9 TB/s), gradient 223 us (1.35 GB, 6.0 TB/s),
// values of the checkpoint read back 138 - 151 us (0.82 GB, 5.7 TB/s).
#include "model_ops.h"
#include "ops_device.h"

namespace arlib {
namespace {

constexpr int kThreads = 256;
constexpr int kV = 8;                          // values of a thread
constexpr int kLanes = kSaveGroup / kV;        // lanes of a group
constexpr int kLastScale = 249;                // of magnitudes above 1.984375 * 2^127
constexpr float kLog2e = 1.44269504088896341f;
constexpr float kLog2eLow = 1.92596299112661746e-8f;   // log2(e) - kLog2e
constexpr float kLn2 = 0.693147180559945309f;

// 8 values from column i of a row of n; zeros past its end.
template <int EB>
__device__ __forceinline__ void ld8(const char* row, size_t i, size_t n, float (&v)[kV]) {
    if constexpr (EB == 2) {
        Vec<2>::unpack(ld_unit_of<2, true>(row, i, n, 0u), v);
    } else {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const u32x4 u = ld_unit_of<4, true>(row, i + 4 * h, n, 0u);
#pragma unroll
            for (int j = 0; j < 4; ++j) v[4 * h + j] = as_f32(u[j]);
        }
    }
}
// (bf16 past the caches, unless NT is false; fp32 through them, which join the two halves
// of a thread's 32 bytes: the gate's gradient of 65536 x 2048 fp32 488 us, 835 past them,
// values read back 242 and 509)
template <int EB, bool NT = true>
__device__ __forceinline__ void st8(char* row, size_t i, size_t n, const float (&v)[kV]) {
    if constexpr (EB == 2) {
        st_unit_of<2, NT>(row, i, n, Vec<2>::pack(v));
    } else {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const float q[4] = {v[4 * h], v[4 * h + 1], v[4 * h + 2], v[4 * h + 3]};
            st_unit_of<4>(row, i + 4 * h, n, Vec<4>::pack(q));
        }
    }
}

// 8 codes at any address.
typedef uint32_t codes_t __attribute__((ext_vector_type(2), aligned(1)));
typedef uint32_t codes_reg __attribute__((ext_vector_type(2)));

__device__ __forceinline__ codes_reg ld_codes(const int8_t* row, size_t i, size_t n) {
    if (i + kV <= n) return __builtin_nontemporal_load(reinterpret_cast<const codes_t*>(row + i));
    codes_reg c = {0u, 0u};
#pragma unroll
    for (int j = 0; j < kV - 1; ++j)
        if (i + j < n) c[j / 4] |= (uint32_t)(uint8_t)row[i + j] << (8 * (j % 4));
    return c;
}
__device__ __forceinline__ void st_codes(int8_t* row, size_t i, size_t n, codes_reg c) {
    if (i + kV <= n) {
        __builtin_nontemporal_store(c, reinterpret_cast<codes_t*>(row + i));
        return;
    }
#pragma unroll
    for (int j = 0; j < kV - 1; ++j)
        if (i + j < n) row[i + j] = (int8_t)(c[j / 4] >> (8 * (j % 4)));
}

__device__ __forceinline__ int larger(int v, int o) { return v > o ? v : o; }

// The biased exponent of a group's scale: of this lane's 8 values and those of
// the group's other lanes (every lane of the group calls this together).
__device__ __forceinline__ int group_exponent(const float (&v)[kV]) {
    int m = 0;   // magnitudes order as whole numbers do, NaN above all
#pragma unroll
    for (int j = 0; j < kV; ++j) m = larger(m, (int)(as_u32(v[j]) & 0x7fffffffu));
    m = larger(m, __builtin_amdgcn_update_dpp(0, m, kDppSwap1, 0xf, 0xf, false));
    m = larger(m, __builtin_amdgcn_update_dpp(0, m, kDppSwap2, 0xf, 0xf, false));
    // 127 = 1.984375 * 2^6
    const int b = (m >> 23) - 6 + ((m & 0x7fffff) > 0x7e0000 ? 1 : 0);
    return m >= 0x7f800000 ? 255 : b < 1 ? 1 : b;
}

__device__ __forceinline__ codes_reg encode(const float (&v)[kV], int b) {
    const float inv = as_f32((uint32_t)(254 - b) << 23);
    codes_reg c = {0u, 0u};
    if (b >= kLastScale) {
        if (b == kLastScale) {   // 64 of this scale is past the numbers
#pragma unroll
            for (int j = 0; j < kV; ++j)
                c[j / 4] |= ((uint32_t)(int)__builtin_rintf(
                                 __builtin_amdgcn_fmed3f(v[j] * inv, -63.0f, 63.0f)) & 0xffu)
                            << (8 * (j % 4));
        }
        return c;
    }
#pragma unroll
    for (int j = 0; j < kV; ++j)
        c[j / 4] |= ((uint32_t)(int)__builtin_rintf(v[j] * inv) & 0xffu) << (8 * (j % 4));
    return c;
}
__device__ __forceinline__ void decode(codes_reg c, int b, float (&v)[kV]) {
    const float scale = as_f32((uint32_t)b << 23);
#pragma unroll
    for (int j = 0; j < kV; ++j)
        v[j] = (float)(int8_t)(c[j / 4] >> (8 * (j % 4))) * scale;
}

// 1 / (1 + e^-a) for |a| < 64.  The product a log2(e) is kept to more than 32 bits, so that
// e^-a is good to 2 ulp where it is large.
__device__ __forceinline__ float sigmoid(float a) {
    const float hi = a * -kLog2e;
    float e = __builtin_amdgcn_exp2f(hi);
    const float lo = __builtin_fmaf(a, -kLog2e, -hi) - a * kLog2eLow;
    e *= __builtin_fmaf(lo, kLn2, 1.0f);
    return __builtin_amdgcn_rcpf(1.0f + e);
}
// For any a, as e^a / (1 + e^a) where a < 0: it may lie below fp32's normal numbers and yet
// have ordinary products with a large u and dacts, so it and they are in 64 bits.  0 below
// -400, where the largest of them is below fp32's numbers.
__device__ __forceinline__ double far_sigmoid(float a) {
    // (an infinite a would make NaN of the rest; NaN itself comes in by a's other factors)
    const float x = __builtin_amdgcn_fmed3f(__builtin_fabsf(a), 0.0f, 400.0f);
    const float hi = x * -kLog2e, n = __builtin_rintf(hi);
    const float lo = __builtin_fmaf(x, -kLog2e, -hi) - x * kLog2eLow;
    const float e = __builtin_amdgcn_exp2f(hi - n) * __builtin_fmaf(lo, kLn2, 1.0f);
    const double z = x < 400.0f ? __builtin_ldexp((double)e, (int)n) : 0.0;   // e^-|a|
    const double r = __builtin_amdgcn_rcpf(1.0f + (float)z);
    return a < 0.0f ? z * r : r;
}
// The scale's exponent from which on a group may hold magnitudes of 64 and more, and 32 bits do
// not.  (65536 x 2048 bf16, gate and gradient: no such group 180 and 218 us, all of them 193
// and 223, lanes of both kinds in each wavefront 215 and 248)
constexpr int kFar = 127;
// That from which on 1.1 times a magnitude may be past the numbers.
constexpr int kVast = 248;

// Where a block's thread works: its row and column.  The units of all rows lie
// in one line, each row padded to whole groups.
struct Spot {
    size_t row, col;
    bool live;
};
__device__ __forceinline__ Spot spot(size_t block, size_t rows, unsigned units) {
    const size_t first = block * kThreads;
    const size_t row0 = first / units;                      // (uniform)
    const unsigned at = (unsigned)(first - row0 * units) + threadIdx.x;
    const unsigned down = at / units;
    Spot s;
    s.row = row0 + down;
    s.col = (size_t)(at - down * units) * kV;
    s.live = s.row < rows;
    return s;
}
unsigned units_of(size_t cols) { return (unsigned)(save_groups(cols) * kLanes); }

template <int EB>
__global__ __launch_bounds__(kThreads) void k_save(const GateArgs a, unsigned units, size_t blocks) {
    const size_t groups = units / kLanes;
    for (size_t b = blockIdx.x; b < blocks; b += gridDim.x) {
        const Spot s = spot(b, a.rows, units);
        float v[kV] = {};
        if (s.live && s.col < a.cols)
            ld8<EB>(static_cast<const char*>(a.x) + s.row * a.stride * EB, s.col, a.cols, v);
        const int e = group_exponent(v);
        if (!s.live) continue;
        st_codes(a.codes + s.row * a.cols, s.col, a.cols, encode(v, e));
        if ((s.col / kV) % kLanes == 0)
            a.scales[s.row * groups + s.col / kSaveGroup] = (uint8_t)e;
    }
}

template <int EB>
__global__ __launch_bounds__(kThreads) void k_restore(const GateArgs a, unsigned units,
                                                      size_t blocks) {
    const size_t groups = units / kLanes;
    for (size_t b = blockIdx.x; b < blocks; b += gridDim.x) {
        const Spot s = spot(b, a.rows, units);
        if (!s.live || s.col >= a.cols) continue;
        float v[kV];
        const int e = a.scales[s.row * groups + s.col / kSaveGroup];
        decode(ld_codes(a.codes + s.row * a.cols, s.col, a.cols), e, v);
        st8<EB>(static_cast<char*>(a.y) + s.row * a.cols * EB, s.col, a.cols, v);
    }
}

template <int EB, bool NT>
__global__ __launch_bounds__(kThreads) void k_gate(const GateArgs a, unsigned units, size_t blocks) {
    const size_t groups = units / kLanes;
    for (size_t b = blockIdx.x; b < blocks; b += gridDim.x) {
        const Spot s = spot(b, a.rows, units);
        float g[kV] = {}, u[kV] = {};
        if (s.live && s.col < a.cols) {
            const char* h = static_cast<const char*>(a.x) + s.row * a.stride * EB;
            ld8<EB>(h, s.col, a.cols, g);
            ld8<EB>(h + a.cols * EB, s.col, a.cols, u);
        }
        const int eg = group_exponent(g), eu = group_exponent(u);
        if (!s.live) continue;
        const size_t at = 2 * s.row;
        st_codes(a.codes + at * a.cols, s.col, a.cols, encode(g, eg));
        st_codes(a.codes + (at + 1) * a.cols, s.col, a.cols, encode(u, eu));
        if ((s.col / kV) % kLanes == 0) {
            a.scales[at * groups + s.col / kSaveGroup] = (uint8_t)eg;
            a.scales[(at + 1) * groups + s.col / kSaveGroup] = (uint8_t)eu;
        }
        if (__builtin_expect(eg < kFar, 1)) {
#pragma unroll
            for (int j = 0; j < kV; ++j) g[j] = g[j] * sigmoid(g[j]) * u[j];
        } else {
#pragma unroll
            for (int j = 0; j < kV; ++j)
                g[j] = (float)((double)g[j] * far_sigmoid(g[j]) * (double)u[j]);
        }
        st8<EB, NT>(static_cast<char*>(a.y) + s.row * a.cols * EB, s.col, a.cols, g);
    }
}

// (64 registers at most, for 8 wavefronts a SIMD)
template <int EB>
__global__ __launch_bounds__(kThreads, 8) void k_gate_grad(const GateArgs a, unsigned units,
                                                           size_t blocks) {
    const size_t groups = units / kLanes;
    for (size_t b = blockIdx.x; b < blocks; b += gridDim.x) {
        const Spot s = spot(b, a.rows, units);
        if (!s.live || s.col >= a.cols) continue;
        const size_t at = 2 * s.row, group = s.col / kSaveGroup;
        const codes_reg cg = ld_codes(a.codes + at * a.cols, s.col, a.cols);
        const codes_reg cu = ld_codes(a.codes + (at + 1) * a.cols, s.col, a.cols);
        const int eg = a.scales[at * groups + group], eu = a.scales[(at + 1) * groups + group];
        float g[kV], u[kV], d[kV];
        ld8<EB>(static_cast<const char*>(a.dacts) + s.row * a.stride * EB, s.col, a.cols, d);
        decode(cg, eg, g);
        decode(cu, eu, u);
        float da[kV], du[kV];
        if (__builtin_expect(eg < kFar && eu < kVast, 1)) {
#pragma unroll
            for (int j = 0; j < kV; ++j) {
                const float q = sigmoid(g[j]), gq = g[j] * q;
                du[j] = d[j] * gq;
                // (s f, f = 1 + a (1 - s), is 1.1 at most, and comes before the factors that are
                // as large as the type's lowest value in masked places: dacts u may be infinite
                // where the gradient is not)
                da[j] = d[j] * (u[j] * (q * (1.0f + g[j] * (1.0f - q))));
                g[j] = gq * u[j];
            }
        } else {
#pragma unroll
            for (int j = 0; j < kV; ++j) {
                settle(g[j]), settle(u[j]), settle(d[j]);   // (one value after another: few registers)
                const double q = far_sigmoid(g[j]), gq = (double)g[j] * q, v = u[j], x = d[j];
                du[j] = (float)(x * gq);
                da[j] = (float)(x * v * (q * (1.0 + (double)g[j] * (1.0 - q))));
                g[j] = (float)(gq * v);
                settle(du[j]), settle(da[j]), settle(g[j]);
            }
        }
        char* dh = static_cast<char*>(a.y) + at * a.cols * EB;
        st8<EB>(dh, s.col, a.cols, da);
        st8<EB>(dh + a.cols * EB, s.col, a.cols, du);
        st8<EB>(static_cast<char*>(a.acts) + s.row * a.cols * EB, s.col, a.cols, g);
    }
}

// Blocks of a launch (the kernels walk the rest).
constexpr size_t kMostBlocks = size_t(1) << 22;

}  // namespace

#define LAUNCH(KERNEL) LAUNCH_AS(KERNEL<2>, KERNEL<4>)
#define LAUNCH_AS(TWO, FOUR)                                                                      \
    do {                                                                                          \
        if (a.rows == 0) return hipSuccess;                                                       \
        const unsigned units = units_of(a.cols);                                                  \
        const size_t blocks = (a.rows * units + kThreads - 1) / kThreads;                         \
        const dim3 grid((unsigned)(blocks < kMostBlocks ? blocks : kMostBlocks));                 \
        if (a.eb == 2) hipLaunchKernelGGL((TWO), grid, dim3(kThreads), 0, s, a, units, blocks);   \
        else hipLaunchKernelGGL((FOUR), grid, dim3(kThreads), 0, s, a, units, blocks);            \
        return hipGetLastError();                                                                 \
    } while (0)

hipError_t launch_save(const GateArgs& a, hipStream_t s) { LAUNCH(k_save); }
hipError_t launch_restore(const GateArgs& a, hipStream_t s) { LAUNCH(k_restore); }
// Activations go past the caches, except in rows that share their ends' lines (bf16, past
// and through them: 65536 x 1001 119 and 97 us; 2000 x 4096 13.1 and 14.4, 8192 x 2048 24.9
// and 26.2; 65536 x 2048 179 and 166 alone, 322 and 324 with the checkpoint read back).
hipError_t launch_gate(const GateArgs& a, hipStream_t s) {
    if (a.cols % 8 == 0) LAUNCH_AS((k_gate<2, true>), (k_gate<4, true>));
    else LAUNCH_AS((k_gate<2, false>), (k_gate<4, true>));
}
hipError_t launch_gate_grad(const GateArgs& a, hipStream_t s) { LAUNCH(k_gate_grad); }

}  // namespace arlib
