// ops_device.h -- device-side building blocks of the training operators:
// 16-byte units of bf16 or fp32 at any element alignment, and reductions over
// a wavefront and a block.
#pragma once

#include "elem.h"

namespace arlib {

// A unit is 16 bytes: 8 bf16 or 4 fp32 values.  Rows may start at any element
// (odd widths, strided views), so the vector type promises no more than the
// element's own alignment; gfx950 loads and stores 16 bytes at such addresses
// in one instruction, and an aligned row costs nothing for it.
template <int EB>
struct Vec;

template <>
struct Vec<2> {
    static constexpr int E = 8;
    typedef uint32_t mem_t __attribute__((ext_vector_type(4), aligned(2)));
    __device__ __forceinline__ static void unpack(u32x4 u, float (&v)[8]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = bf16_lo(u[i]);
            v[2 * i + 1] = bf16_hi(u[i]);
        }
    }
    // one rounding to the nearest bf16, ties to even; a NaN stays one
    __device__ __forceinline__ static u32x4 pack(const float (&v)[8]) {
        u32x4 u;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const f32x2_t f = {v[2 * i], v[2 * i + 1]};
            u[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector(f, bf16x2_t));
        }
        return u;
    }
    __device__ __forceinline__ static float ld1(const char* p) {
        return bf16_widen(*reinterpret_cast<const uint16_t*>(p));
    }
    __device__ __forceinline__ static void st1(char* p, float f) {
        *reinterpret_cast<uint16_t*>(p) = __builtin_bit_cast(uint16_t, (__bf16)f);
    }
};

template <>
struct Vec<4> {
    static constexpr int E = 4;
    typedef uint32_t mem_t __attribute__((ext_vector_type(4), aligned(4)));
    __device__ __forceinline__ static void unpack(u32x4 u, float (&v)[4]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = as_f32(u[i]);
    }
    __device__ __forceinline__ static u32x4 pack(const float (&v)[4]) {
        u32x4 u;
#pragma unroll
        for (int i = 0; i < 4; ++i) u[i] = as_u32(v[i]);
        return u;
    }
    __device__ __forceinline__ static float ld1(const char* p) {
        return *reinterpret_cast<const float*>(p);
    }
    __device__ __forceinline__ static void st1(char* p, float f) {
        *reinterpret_cast<float*>(p) = f;
    }
};

template <int EB, bool NT = false>
__device__ __forceinline__ u32x4 ld_unit(const char* p) {
    const auto* q = reinterpret_cast<const typename Vec<EB>::mem_t*>(p);
    if constexpr (NT) return __builtin_nontemporal_load(q);
    else return *q;
}

template <int EB, bool NT = false>
__device__ __forceinline__ void st_unit(char* p, u32x4 u) {
    auto* q = reinterpret_cast<typename Vec<EB>::mem_t*>(p);
    if constexpr (NT) __builtin_nontemporal_store(u, q);
    else *q = u;
}

// The unit at element i of a row of n elements; past the row's end it holds
// `fill` (an element's bits, repeated).
template <int EB, bool NT = false>
__device__ __forceinline__ u32x4 ld_unit_of(const char* row, size_t i, size_t n, uint32_t fill) {
    constexpr int E = Vec<EB>::E;
    if (i + E <= n) return ld_unit<EB, NT>(row + i * EB);
    u32x4 u = {fill, fill, fill, fill};
    if (i < n) {
        const char* p = row + i * EB;
        const int m = (int)(n - i);
#pragma unroll
        for (int j = 0; j < E - 1; ++j)
            if (j < m) {
                const uint32_t e = ld_elem<EB>(p + j * EB);
                if constexpr (EB == 4) u[j] = e;
                else if (j & 1) u[j / 2] = (u[j / 2] & 0xffffu) | (e << 16);
                else u[j / 2] = (u[j / 2] & 0xffff0000u) | e;
            }
    }
    return u;
}

template <int EB, bool NT = false>
__device__ __forceinline__ void st_unit_of(char* row, size_t i, size_t n, u32x4 u) {
    constexpr int E = Vec<EB>::E;
    if (i + E <= n) {
        st_unit<EB, NT>(row + i * EB, u);
    } else if (i < n) {
        char* p = row + i * EB;
        const int m = (int)(n - i);
#pragma unroll
        for (int j = 0; j < E - 1; ++j)
            if (j < m) {
                if constexpr (EB == 4) st_elem<4>(p + j * 4, u[j]);
                else st_elem<2>(p + j * 2, (j & 1) ? u[j / 2] >> 16 : u[j / 2] & 0xffffu);
            }
    }
}

// E parameters (weight, bias) at column i of n, `pb` bytes each; past the end
// and for a NULL array they are `none`.
template <int E>
__device__ __forceinline__ void ld_params(const void* base, int pb, size_t i, size_t n, float none,
                                          float (&v)[E]) {
#pragma unroll
    for (int j = 0; j < E; ++j) v[j] = none;
    if (!base) return;
    const char* p = static_cast<const char*>(base);
    if (pb == 4) {
        if (i + E <= n) {
#pragma unroll
            for (int h = 0; h < E / 4; ++h) {
                const u32x4 u = ld_unit<4>(p + (i + 4 * h) * 4);
#pragma unroll
                for (int j = 0; j < 4; ++j) v[4 * h + j] = as_f32(u[j]);
            }
        } else {
#pragma unroll
            for (int j = 0; j < E; ++j)
                if (i + j < n) v[j] = Vec<4>::ld1(p + (i + j) * 4);
        }
    } else {
        if (E == 8 && i + E <= n) {
            const u32x4 u = ld_unit<2>(p + i * 2);
#pragma unroll
            for (int j = 0; j < E; ++j) v[j] = (j & 1) ? bf16_hi(u[j / 2]) : bf16_lo(u[j / 2]);
        } else {
#pragma unroll
            for (int j = 0; j < E; ++j)
                if (i + j < n) v[j] = Vec<2>::ld1(p + (i + j) * 2);
        }
    }
}

// Sum over the 64 lanes, on every lane.  A butterfly: every lane adds the same
// pairs, so the lanes agree to the last bit.
__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) v += __shfl_xor(v, d, 64);
    return v;
}

__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) v = fmaxf(v, __shfl_xor(v, d, 64));
    return v;
}

// Sum over a block of W wavefronts, on every thread.  `lds` holds W floats and
// may be used again after the next barrier.
template <int W>
__device__ __forceinline__ float block_sum(float v, float* lds) {
    v = wave_sum(v);
    if constexpr (W == 1) return v;
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
    __syncthreads();
    float t = lds[0];
#pragma unroll
    for (int w = 1; w < W; ++w) t += lds[w];
    return t;
}

}  // namespace arlib
