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

// A byte offset that the compiler takes as new here: added to a uniform
// pointer it stays the 32-bit offset of the load or store, where a 64-bit sum
// kept across a loop would take two registers for each access.
__device__ __forceinline__ unsigned offset_here(unsigned v) {
    asm volatile("" : "+v"(v));
    return v;
}

// Where a thread's unit lies in a row of n >= E elements when the unit at
// element i is its share: a share that runs past the end moves back to the
// row's last E elements, and its first `skip` ones are another thread's.  The
// load is then the same for every thread, without a branch; the last unit's
// owner alone drops what is not its own.
struct Place {
    unsigned at;   // first element of the 16 bytes
    int skip;      // elements that are not this thread's (E: none is)
};
template <int E>
__device__ __forceinline__ Place place_unit(unsigned i, unsigned n) {
    Place p;
    p.at = i + E <= n ? i : n - E;
    p.skip = (int)(i - p.at < (unsigned)E ? i - p.at : (unsigned)E);
    return p;
}
// u with its first `skip` > 0 elements 0.  Where rows end at a unit's end
// (RAGGED false), skip is all of them or none.
template <int EB, bool RAGGED>
__device__ __forceinline__ u32x4 drop_first(u32x4 u, int skip) {
    if constexpr (!RAGGED) return u32x4{0u, 0u, 0u, 0u};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (EB == 4) u[i] = i < skip ? 0u : u[i];
        else u[i] = 2 * i + 1 < skip ? 0u : 2 * i < skip ? u[i] & 0xffff0000u : u[i];
    }
    return u;
}
// u with its first `skip` elements replaced by those of the word `fill`
template <int EB>
__device__ __forceinline__ u32x4 fill_first(u32x4 u, int skip, uint32_t fill) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (EB == 4) u[i] = i < skip ? fill : u[i];
        else
            u[i] = 2 * i + 1 < skip ? fill
                   : 2 * i < skip   ? (u[i] & 0xffff0000u) | (fill & 0xffffu)
                                    : u[i];
    }
    return u;
}
// Stores this thread's elements of u to the row.
template <int EB, bool RAGGED, bool NT = false>
__device__ __forceinline__ void st_place(char* row, Place p, u32x4 u) {
    if (p.skip == 0) {
        st_unit<EB, NT>(row + offset_here(p.at * EB), u);
    } else if (RAGGED) {
#pragma unroll
        for (int j = 1; j < Vec<EB>::E; ++j)
            if (j >= p.skip) {
                char* q = row + offset_here((p.at + j) * EB);
                if constexpr (EB == 4) st_elem<4>(q, u[j]);
                else st_elem<2>(q, (j & 1) ? u[j / 2] >> 16 : u[j / 2] & 0xffffu);
            }
    }
}

// How the units of a row of n elements are loaded and stored: ROW_FULL where n
// is a multiple of a unit, ROW_RAGGED where the last unit is a Place that moved
// back, ROW_SHORT where a row is shorter than a unit.
enum RowMode { ROW_FULL, ROW_RAGGED, ROW_SHORT };
inline RowMode row_mode(size_t n, int eb) {
    const size_t e = 16 / (size_t)eb;
    return n % e == 0 ? ROW_FULL : n > e ? ROW_RAGGED : ROW_SHORT;
}
// NT: the loads bypass the caches, for rows that are read once and would only
// push other data out.
template <int EB, RowMode MODE, bool NT>
struct RowIO {
    static constexpr int E = Vec<EB>::E;
    __device__ __forceinline__ static Place place(unsigned unit, unsigned n) {
        if constexpr (MODE == ROW_RAGGED) return place_unit<E>(unit * E, n);
        else return Place{unit * E, 0};
    }
    __device__ __forceinline__ static u32x4 ld(const char* row, Place p, unsigned n) {
        if constexpr (MODE == ROW_SHORT) return ld_unit_of<EB>(row, 0, n, 0u);
        else return ld_unit<EB, NT>(row + offset_here(p.at * EB));
    }
    __device__ __forceinline__ static void st(char* row, Place p, unsigned n, u32x4 u) {
        if constexpr (MODE == ROW_SHORT) st_unit_of<EB>(row, 0, n, u);
        else st_place<EB, MODE == ROW_RAGGED, true>(row, p, u);
    }
};

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

// Ends the reuse of values computed from u: what is needed of them later is
// computed again from the 16 bytes, where the compiler would hold 4 times as
// many registers across a barrier.
__device__ __forceinline__ void refresh(u32x4& u) { asm volatile("" : "+v"(u)); }

// Has v computed by here (an accumulator's update would else be put off, and
// its operands kept, past a barrier).
__device__ __forceinline__ void settle(float& v) { asm volatile("" : "+v"(v)); }

// A value at a uniform address that no store of this kernel changes.
__device__ __forceinline__ float ld_uniform(const float* p) {
    typedef const float __attribute__((address_space(4))) * constant_t;
    return *(constant_t)(uintptr_t)p;
}

__device__ __forceinline__ int ld_uniform(const int* p) {
    typedef const int __attribute__((address_space(4))) * constant_t;
    return *(constant_t)(uintptr_t)p;
}

// Sum and maximum over the 64 lanes, the same on every lane.  Lanes are joined
// with DPP moves (inside rows of 16, then across them towards lane 63), which
// cost one instruction a step where a shuffle goes through LDS.
template <int CTRL, int ROWS>
__device__ __forceinline__ float dpp(float old, float v) {
    return as_f32((uint32_t)__builtin_amdgcn_update_dpp((int)as_u32(old), (int)as_u32(v), CTRL, ROWS,
                                                        0xf, false));
}
constexpr int kDppSwap1 = 0xb1;         // quad_perm [1, 0, 3, 2]
constexpr int kDppSwap2 = 0x4e;         // quad_perm [2, 3, 0, 1]
constexpr int kDppHalfMirror = 0x141;   // lane i of 8 from lane 7 - i
constexpr int kDppMirror = 0x140;       // lane i of 16 from lane 15 - i
constexpr int kDppLast15 = 0x142;       // lane 15 of the row before
constexpr int kDppLast31 = 0x143;       // lane 31

__device__ __forceinline__ float lane63(float v) {
    return as_f32((uint32_t)__builtin_amdgcn_readlane((int)as_u32(v), 63));
}

__device__ __forceinline__ float wave_sum(float v) {
    v += dpp<kDppSwap1, 0xf>(0.0f, v);
    v += dpp<kDppSwap2, 0xf>(0.0f, v);
    v += dpp<kDppHalfMirror, 0xf>(0.0f, v);
    v += dpp<kDppMirror, 0xf>(0.0f, v);
    v += dpp<kDppLast15, 0xa>(0.0f, v);   // rows 1 and 3
    v += dpp<kDppLast31, 0xc>(0.0f, v);   // rows 2 and 3
    return lane63(v);
}

__device__ __forceinline__ int wave_sum(int v) {
#define ADD(CTRL, ROWS) v += __builtin_amdgcn_update_dpp(0, v, CTRL, ROWS, 0xf, false)
    ADD(kDppSwap1, 0xf);
    ADD(kDppSwap2, 0xf);
    ADD(kDppHalfMirror, 0xf);
    ADD(kDppMirror, 0xf);
    ADD(kDppLast15, 0xa);
    ADD(kDppLast31, 0xc);
#undef ADD
    return __builtin_amdgcn_readlane(v, 63);
}

__device__ __forceinline__ float wave_max(float v) {
    v = fmaxf(v, dpp<kDppSwap1, 0xf>(v, v));
    v = fmaxf(v, dpp<kDppSwap2, 0xf>(v, v));
    v = fmaxf(v, dpp<kDppHalfMirror, 0xf>(v, v));
    v = fmaxf(v, dpp<kDppMirror, 0xf>(v, v));
    v = fmaxf(v, dpp<kDppLast15, 0xa>(v, v));
    v = fmaxf(v, dpp<kDppLast31, 0xc>(v, v));
    return lane63(v);
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

// V sums over a block's `waves` wavefronts at once (V a power of two), on every
// thread.  `lds` holds V floats a wavefront; the barrier inside is the only
// one, so a caller that comes back before another barrier takes another buffer.
template <int V>
__device__ __forceinline__ void block_sums(float (&v)[V], float* lds, int waves) {
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = wave_sum(v[i]);
    if (waves == 1) return;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    float mine = v[0];
#pragma unroll
    for (int i = 1; i < V; ++i) mine = lane == i ? v[i] : mine;
    if (lane < V) lds[wave * V + lane] = mine;
    __syncthreads();
    // lane l takes sum l % V of every (64 / V)th wavefront
    float t = 0.0f;
#pragma unroll
    for (int w = 0; w < 16; w += 64 / V)
        if (w + lane / V < waves) t += lds[w * V + lane];
#pragma unroll
    for (int d = V; d < 64; d <<= 1)
        if (d / V < 16) t += __shfl_xor(t, d, 64);
#pragma unroll
    for (int i = 0; i < V; ++i)
        v[i] = as_f32((uint32_t)__builtin_amdgcn_readlane((int)as_u32(t), i));
}

}  // namespace arlib
