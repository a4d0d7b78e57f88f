// norm.hip -- layer norm over the last dimension, forward and backward.
//
//   forward   mu = sum x / n,  var = sum (x - mu)^2 / n,  r = 1/sqrt(var + eps)
//             y = (x - mu) r w + b
//   backward  g = dy w,  xh = (x - mu) r
//             dx = r (g - sum(g)/n - xh sum(g xh)/n)
//             dw = sum over rows of dy xh,  db = sum over rows of dy
//
// All sums and statistics are fp32; each output is rounded once.  The variance
// is taken from the centred values (a second pass over the row), so a mean far
// larger than the spread costs no digits.
//
// Bound by HBM: 2 (3) bytes x element size an element against 8 (14) flops.  A
// row stays in the registers of a block between its sums and its output, so x
// (and dy) are read once.  A block rather than a wavefront a row: the parameters
// are loaded once for R rows of a short share each (one wavefront with 8 units a
// lane reads them for every row: 70 us at 16384 x 4096 bf16, against 47).
// MI355X: forward 16384 x 4096 bf16 47.7 us (5.6 TB/s; a copy of as many bytes
// 41.5), backward 8192 x 8192 bf16 with fp32 weights 79.6 us (5.1 TB/s; 62),
// 1021 x 771 fp32 9.2 us, one row of 4096 5.5 us, of which the kernel is 2.6.
#include <cmath>

#include "ops.h"
#include "ops_device.h"

namespace arlib {
namespace {

constexpr int kCUs = 256;
constexpr int kNormThreads = 256;
constexpr int kNormWaves = kNormThreads / 64;

__device__ __forceinline__ void st_param(void* base, int pb, size_t i, float v) {
    if (pb == 4) Vec<4>::st1(static_cast<char*>(base) + i * 4, v);
    else Vec<2>::st1(static_cast<char*>(base) + i * 2, v);
}

// Narrow rows: TPR lanes a row (a power of two below 64), so that a wavefront
// takes 64 / TPR rows at once, and kNarrowSteps such steps in flight.
constexpr int kNarrowSteps = 4;

// Sum over the TPR lanes of a row, on each of them.
template <int TPR>
__device__ __forceinline__ float row_sum(float v) {
    static_assert(TPR == 8 || TPR == 16 || TPR == 32, "lanes of a row");
    v += dpp<kDppSwap1, 0xf>(0.0f, v);
    v += dpp<kDppSwap2, 0xf>(0.0f, v);
    v += dpp<kDppHalfMirror, 0xf>(0.0f, v);
    if constexpr (TPR > 8) v += dpp<kDppMirror, 0xf>(0.0f, v);
    if constexpr (TPR > 16) v += __shfl_xor(v, 16, 64);
    return v;
}

template <int EB, int TPR, bool RAGGED>
__global__ __launch_bounds__(kNormThreads) void k_norm_narrow(const NormArgs a) {
    constexpr int E = Vec<EB>::E, RW = 64 / TPR, RB = kNormWaves * kNarrowSteps * RW;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const float n = (float)a.cols;
    const Place at = place_unit<E>((lane % TPR) * E, (unsigned)a.cols);
    float w[E], b[E];
    ld_params<E>(a.weight, a.pb, at.at, a.cols, 1.0f, w);
    ld_params<E>(a.bias, a.pb, at.at, a.cols, 0.0f, b);
    for (size_t r0 = (size_t)blockIdx.x * RB; r0 < a.rows; r0 += (size_t)gridDim.x * RB) {
        u32x4 raw[kNarrowSteps];
        const size_t first = r0 + (size_t)wave * (kNarrowSteps * RW) + lane / TPR;
#pragma unroll
        for (int k = 0; k < kNarrowSteps; ++k) {
            const size_t r = first + k * RW < a.rows ? first + k * RW : a.rows - 1;
            raw[k] = ld_unit<EB>(static_cast<const char*>(a.x) + (r * a.xstride + at.at) * EB);
        }
#pragma unroll
        for (int k = 0; k < kNarrowSteps; ++k) {
            const size_t r = first + k * RW;
            if (at.skip) raw[k] = drop_first<EB, RAGGED>(raw[k], at.skip);
            float v[E], s = 0.0f;
            Vec<EB>::unpack(raw[k], v);
#pragma unroll
            for (int j = 0; j < E; ++j) s += v[j];
            const float mean = row_sum<TPR>(s) / n;
            s = 0.0f;
#pragma unroll
            for (int j = 0; j < E; ++j) {
                const float d = (RAGGED ? j < at.skip : at.skip != 0) ? 0.0f : v[j] - mean;
                s = __builtin_fmaf(d, d, s);
            }
            const float rstd = 1.0f / sqrtf(row_sum<TPR>(s) / n + a.eps);
            if (r >= a.rows) continue;
#pragma unroll
            for (int j = 0; j < E; ++j) v[j] = __builtin_fmaf((v[j] - mean) * rstd, w[j], b[j]);
            st_place<EB, RAGGED, true>(static_cast<char*>(a.y) + r * a.cols * EB, at,
                                       Vec<EB>::pack(v));
            if (lane % TPR == 0) {
                a.mean[r] = mean;
                a.rstd[r] = rstd;
            }
        }
    }
}

// E values at columns c ... of an array of `pb`-byte elements, the first `skip`
// left out.
template <int E>
__device__ __forceinline__ void st_params(void* base, int pb, size_t c, int skip,
                                          const float (&v)[E]) {
    char* p = static_cast<char*>(base) + c * pb;
    if (skip == 0 && pb == 4) {
#pragma unroll
        for (int h = 0; h < E / 4; ++h)
            st_unit<4>(p + 16 * h, u32x4{as_u32(v[4 * h]), as_u32(v[4 * h + 1]),
                                         as_u32(v[4 * h + 2]), as_u32(v[4 * h + 3])});
        return;
    }
    if constexpr (E == 8)
        if (skip == 0) {
            st_unit<2>(p, Vec<2>::pack(v));
            return;
        }
#pragma unroll
    for (int j = 0; j < E; ++j)
        if (j >= skip) st_param(base, pb, c + j, v[j]);
}

// Column sums' last stop: a row of partial sums, or the gradients themselves
// where there is no other part.
template <int E>
__device__ __forceinline__ void put_columns(const NormGradArgs& a, Place at, const float (&dw)[E],
                                            const float (&db)[E]) {
    if (at.skip >= E) return;
    if (gridDim.x > 1) {
        float* out = a.part + (size_t)blockIdx.x * 2 * a.cols;
        st_params<E>(out, 4, at.at, at.skip, dw);
        st_params<E>(out + a.cols, 4, at.at, at.skip, db);
    } else {
        if (a.dweight) st_params<E>(a.dweight, a.pb, at.at, at.skip, dw);
        if (a.dbias) st_params<E>(a.dbias, a.pb, at.at, at.skip, db);
    }
}

template <int EB, int TPR, bool RAGGED>
__global__ __launch_bounds__(kNormThreads) void k_norm_grad_narrow(const NormGradArgs a) {
    constexpr int E = Vec<EB>::E, RW = 64 / TPR, RB = kNormWaves * kNarrowSteps * RW;
    __shared__ float lds[kNormWaves][2 * E][TPR];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const float inv = 1.0f / (float)a.cols;
    const Place at = place_unit<E>((lane % TPR) * E, (unsigned)a.cols);
    float w[E], dw[E], db[E];
    ld_params<E>(a.weight, a.pb, at.at, a.cols, 1.0f, w);
#pragma unroll
    for (int j = 0; j < E; ++j) dw[j] = db[j] = 0.0f;
    for (size_t r0 = (size_t)blockIdx.x * RB; r0 < a.rows; r0 += (size_t)gridDim.x * RB) {
        u32x4 rx[kNarrowSteps], rg[kNarrowSteps];
        float mean[kNarrowSteps], rstd[kNarrowSteps];
        const size_t first = r0 + (size_t)wave * (kNarrowSteps * RW) + lane / TPR;
#pragma unroll
        for (int k = 0; k < kNarrowSteps; ++k) {
            const size_t r = first + k * RW < a.rows ? first + k * RW : a.rows - 1;
            rx[k] = ld_unit<EB>(static_cast<const char*>(a.x) + (r * a.xstride + at.at) * EB);
            rg[k] = ld_unit<EB>(static_cast<const char*>(a.dy) + (r * a.dystride + at.at) * EB);
            mean[k] = a.mean[r];
            rstd[k] = a.rstd[r];
        }
#pragma unroll
        for (int k = 0; k < kNarrowSteps; ++k) {
            const size_t r = first + k * RW;
            const int skip = r < a.rows ? at.skip : E;
            if (skip) {
                rx[k] = drop_first<EB, RAGGED>(rx[k], skip);
                rg[k] = drop_first<EB, RAGGED>(rg[k], skip);
            }
            float v[E], g[E], s1 = 0.0f, s2 = 0.0f;
            Vec<EB>::unpack(rx[k], v);
            Vec<EB>::unpack(rg[k], g);
#pragma unroll
            for (int j = 0; j < E; ++j) {
                v[j] = (v[j] - mean[k]) * rstd[k];
                db[j] += g[j];
                // (past the last row nothing counts, whatever that row holds)
                dw[j] = skip == E ? dw[j] : __builtin_fmaf(g[j], v[j], dw[j]);
                g[j] *= w[j];
                s1 += g[j];
                s2 = __builtin_fmaf(g[j], v[j], s2);
            }
            const float c1 = row_sum<TPR>(s1) * inv, c2 = row_sum<TPR>(s2) * inv;
            if (r >= a.rows) continue;
#pragma unroll
            for (int j = 0; j < E; ++j)
                v[j] = rstd[k] * __builtin_fmaf(-v[j], c2, g[j] - c1);
            st_place<EB, RAGGED>(static_cast<char*>(a.dx) + r * a.cols * EB, at, Vec<EB>::pack(v));
        }
    }
    if (!a.dweight && !a.dbias) return;
    // the wavefront's rows, then the wavefronts
#pragma unroll
    for (int j = 0; j < E; ++j) {
#pragma unroll
        for (int d = TPR; d < 64; d <<= 1) {
            dw[j] += __shfl_xor(dw[j], d, 64);
            db[j] += __shfl_xor(db[j], d, 64);
        }
        if (lane < TPR) {
            lds[wave][j][lane] = dw[j];
            lds[wave][E + j][lane] = db[j];
        }
    }
    __syncthreads();
    if (threadIdx.x >= TPR) return;
#pragma unroll
    for (int j = 0; j < E; ++j) {
        dw[j] = db[j] = 0.0f;
#pragma unroll
        for (int k = 0; k < kNormWaves; ++k) {
            dw[j] += lds[k][j][lane];
            db[j] += lds[k][E + j][lane];
        }
    }
    put_columns<E>(a, at, dw, db);
}

// Rows that a block holds in registers: up to NT threads (FIXED: exactly) with
// UPT units each, R
// rows at a time, so that a block has R rows of loads in flight and one barrier
// serves R sums.  The parameters stay in registers from row to row.  Rows past
// the last are loaded as the last one again and left out of sums and stores.
template <int EB, int NT, int UPT, int R, bool RAGGED, bool FIXED>
__global__ __launch_bounds__(NT) void k_norm_rows(const NormArgs a) {
    constexpr int E = Vec<EB>::E;
    __shared__ float lds[2][NT / 64 * R];
    const int nt = FIXED ? NT : (int)blockDim.x, waves = nt >> 6;
    const float n = (float)a.cols;
    Place at[UPT];
    u32x4 raw[R][UPT];
    const auto load = [&](size_t r0) {
#pragma unroll
        for (int k = 0; k < R; ++k) {
            const size_t r = r0 + k < a.rows ? r0 + k : a.rows - 1;
            const char* x = static_cast<const char*>(a.x) + r * a.xstride * EB;
#pragma unroll
            for (int u = 0; u < UPT; ++u)
                raw[k][u] = ld_unit<EB, true>(x + offset_here(at[u].at * EB));
        }
    };
#pragma unroll
    for (int u = 0; u < UPT; ++u)
        at[u] = place_unit<E>((u * nt + threadIdx.x) * E, (unsigned)a.cols);
    size_t r0 = (size_t)blockIdx.x * R;
    load(r0);   // (ahead of the parameters: one round trip for both)
    float w[UPT][E], b[UPT][E];
#pragma unroll
    for (int u = 0; u < UPT; ++u) {
        ld_params<E>(a.weight, a.pb, at[u].at, a.cols, 1.0f, w[u]);
        ld_params<E>(a.bias, a.pb, at[u].at, a.cols, 0.0f, b[u]);
    }
    for (; r0 < a.rows; r0 += (size_t)gridDim.x * R) {
        if (r0 != (size_t)blockIdx.x * R) load(r0);
        float mean[R], s[R];
#pragma unroll
        for (int k = 0; k < R; ++k) {
            mean[k] = 0.0f;
#pragma unroll
            for (int u = 0; u < UPT; ++u) {
                if (at[u].skip) raw[k][u] = drop_first<EB, RAGGED>(raw[k][u], at[u].skip);
                float v[E];
                Vec<EB>::unpack(raw[k][u], v);
#pragma unroll
                for (int j = 0; j < E; ++j) mean[k] += v[j];
            }
        }
        block_sums<R>(mean, lds[0], waves);
#pragma unroll
        for (int k = 0; k < R; ++k) {
            mean[k] /= n;
            s[k] = 0.0f;
#pragma unroll
            for (int u = 0; u < UPT; ++u) {
                float v[E];
                refresh(raw[k][u]);
                Vec<EB>::unpack(raw[k][u], v);
                if (at[u].skip) {   // the dropped elements read as the mean
#pragma unroll
                    for (int j = 0; j < E; ++j) v[j] = !RAGGED || j < at[u].skip ? mean[k] : v[j];
                }
#pragma unroll
                for (int j = 0; j < E; ++j) {
                    const float d = v[j] - mean[k];
                    s[k] = __builtin_fmaf(d, d, s[k]);
                }
            }
        }
        block_sums<R>(s, lds[1], waves);
#pragma unroll
        for (int k = 0; k < R; ++k) {
            if (r0 + k >= a.rows) break;
            const float rstd = 1.0f / sqrtf(s[k] / n + a.eps);
            char* y = static_cast<char*>(a.y) + (r0 + k) * a.cols * EB;
#pragma unroll
            for (int u = 0; u < UPT; ++u) {
                float v[E];
                refresh(raw[k][u]);
                Vec<EB>::unpack(raw[k][u], v);
#pragma unroll
                for (int j = 0; j < E; ++j)
                    v[j] = __builtin_fmaf((v[j] - mean[k]) * rstd, w[u][j], b[u][j]);
                st_place<EB, RAGGED>(y, at[u], Vec<EB>::pack(v));
            }
            if (threadIdx.x == 0) {
                a.mean[r0 + k] = mean[k];
                a.rstd[r0 + k] = rstd;
            }
        }
    }
}

// Both gradients in one pass over x and dy (a second pass for the column sums
// took 164 us in all at 8192 x 8192 bf16, this form 79.6).  Each thread owns the same columns
// in every row that its block takes, so the column sums stay in its registers
// until the block's last row and leave as one row of partial sums.
template <int EB, int NT, int UPT, int R, bool RAGGED, bool FIXED>
__global__ __launch_bounds__(NT) void k_norm_grad_rows(const NormGradArgs a) {
    constexpr int E = Vec<EB>::E;
    __shared__ float lds[2][NT / 64 * 2 * R];
    const int nt = FIXED ? NT : (int)blockDim.x, waves = nt >> 6;
    const float inv = 1.0f / (float)a.cols;
    Place at[UPT];
    u32x4 rx[R][UPT], rg[R][UPT];
    float mean[R], rstd[R];
    const auto load = [&](size_t r0, int k) {
        const size_t r = r0 + k < a.rows ? r0 + k : a.rows - 1;
        const char* x = static_cast<const char*>(a.x) + r * a.xstride * EB;
        const char* dy = static_cast<const char*>(a.dy) + r * a.dystride * EB;
        mean[k] = ld_uniform(a.mean + r);
        rstd[k] = ld_uniform(a.rstd + r);
#pragma unroll
        for (int u = 0; u < UPT; ++u) {
            const unsigned off = offset_here(at[u].at * EB);
            rx[k][u] = ld_unit<EB, true>(x + off);
            rg[k][u] = ld_unit<EB, true>(dy + off);
        }
    };
#pragma unroll
    for (int u = 0; u < UPT; ++u)
        at[u] = place_unit<E>((u * nt + threadIdx.x) * E, (unsigned)a.cols);
    size_t r0 = (size_t)blockIdx.x * R;
#pragma unroll
    for (int k = 0; k < R; ++k) load(r0, k);
    float w[UPT][E], dw[UPT][E], db[UPT][E];
#pragma unroll
    for (int u = 0; u < UPT; ++u) {
        ld_params<E>(a.weight, a.pb, at[u].at, a.cols, 1.0f, w[u]);
#pragma unroll
        for (int j = 0; j < E; ++j) dw[u][j] = db[u][j] = 0.0f;
    }
    int buf = 0;
    for (; r0 < a.rows; r0 += (size_t)gridDim.x * R, buf ^= 1) {
        float s[2 * R];
        const size_t next = r0 + (size_t)gridDim.x * R;
#pragma unroll
        for (int k = 0; k < R; ++k) {
            float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
            for (int u = 0; u < UPT; ++u) {
                // (a row past the last: none of its elements counts)
                const int skip = r0 + k < a.rows ? at[u].skip : E;
                if (skip) {
                    rx[k][u] = drop_first<EB, RAGGED>(rx[k][u], skip);
                    rg[k][u] = drop_first<EB, RAGGED>(rg[k][u], skip);
                }
                float v[E], g[E];
                Vec<EB>::unpack(rx[k][u], v);
                Vec<EB>::unpack(rg[k][u], g);
#pragma unroll
                for (int j = 0; j < E; ++j) {
                    const float xh = (v[j] - mean[k]) * rstd[k];
                    const float gw = g[j] * w[u][j];    // 0 where dropped
                    s1 += gw;
                    s2 = __builtin_fmaf(gw, xh, s2);
                    dw[u][j] = __builtin_fmaf(g[j], xh, dw[u][j]);
                    db[u][j] += g[j];
                }
            }
            s[2 * k] = s1;
            s[2 * k + 1] = s2;
#pragma unroll
            for (int u = 0; u < UPT; ++u)
#pragma unroll
                for (int j = 0; j < E; ++j) {
                    settle(dw[u][j]);
                    settle(db[u][j]);
                }
            __builtin_amdgcn_sched_barrier(0);   // one row's temporaries at a time
        }
        block_sums<2 * R>(s, lds[buf], waves);
#pragma unroll
        for (int k = 0; k < R; ++k) {
            const float c1 = s[2 * k] * inv, c2 = s[2 * k + 1] * inv;
            char* dx = static_cast<char*>(a.dx) + (r0 + k) * a.cols * EB;
#pragma unroll
            for (int u = 0; u < UPT; ++u) {
                float v[E], g[E];
                refresh(rx[k][u]);
                refresh(rg[k][u]);
                Vec<EB>::unpack(rx[k][u], v);
                Vec<EB>::unpack(rg[k][u], g);
#pragma unroll
                for (int j = 0; j < E; ++j) {
                    const float xh = (v[j] - mean[k]) * rstd[k];
                    v[j] = rstd[k] * __builtin_fmaf(-xh, c2, __builtin_fmaf(g[j], w[u][j], -c1));
                }
                if (r0 + k < a.rows) st_place<EB, RAGGED>(dx, at[u], Vec<EB>::pack(v));
            }
            // the row's registers are free: the next step's row comes in while
            // this step goes on
            if (next < a.rows) load(next, k);
            __builtin_amdgcn_sched_barrier(0);
        }
    }
    if (!a.dweight && !a.dbias) return;
#pragma unroll
    for (int u = 0; u < UPT; ++u) put_columns<E>(a, at[u], dw[u], db[u]);
}

// Rows of any width: one block per row, three walks over it (the second and
// third find it in the cache).
template <int EB>
__global__ __launch_bounds__(kNormThreads) void k_norm_wide(const NormArgs a) {
    constexpr int E = Vec<EB>::E;
    __shared__ float lds[2][kNormWaves];
    for (size_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
        const char* x = static_cast<const char*>(a.x) + r * a.xstride * EB;
        char* y = static_cast<char*>(a.y) + r * a.cols * EB;
        const float n = (float)a.cols;

        float s = 0.0f;
        for (size_t i = (size_t)threadIdx.x * E; i < a.cols; i += (size_t)kNormThreads * E) {
            float v[E];
            Vec<EB>::unpack(ld_unit_of<EB>(x, i, a.cols, 0u), v);
    #pragma unroll
            for (int j = 0; j < E; ++j) s += v[j];
        }
        const float mean = block_sum<kNormWaves>(s, lds[0]) / n;
        s = 0.0f;
        for (size_t i = (size_t)threadIdx.x * E; i < a.cols; i += (size_t)kNormThreads * E) {
            float v[E];
            Vec<EB>::unpack(ld_unit_of<EB>(x, i, a.cols, 0u), v);
    #pragma unroll
            for (int j = 0; j < E; ++j) {
                const float d = i + j < a.cols ? v[j] - mean : 0.0f;
                s = __builtin_fmaf(d, d, s);
            }
        }
        const float var = block_sum<kNormWaves>(s, lds[1]) / n;
        const float rstd = 1.0f / sqrtf(var + a.eps);
        for (size_t i = (size_t)threadIdx.x * E; i < a.cols; i += (size_t)kNormThreads * E) {
            float v[E], w[E], b[E];
            Vec<EB>::unpack(ld_unit_of<EB>(x, i, a.cols, 0u), v);
            ld_params<E>(a.weight, a.pb, i, a.cols, 1.0f, w);
            ld_params<E>(a.bias, a.pb, i, a.cols, 0.0f, b);
    #pragma unroll
            for (int j = 0; j < E; ++j) v[j] = __builtin_fmaf((v[j] - mean) * rstd, w[j], b[j]);
            st_unit_of<EB>(y, i, a.cols, Vec<EB>::pack(v));
        }
        if (threadIdx.x == 0) {
            a.mean[r] = mean;
            a.rstd[r] = rstd;
        }
    }
}

// dx of rows of any width: one block per row, two walks.
template <int EB>
__global__ __launch_bounds__(kNormThreads) void k_norm_grad_wide(const NormGradArgs a) {
    constexpr int E = Vec<EB>::E;
    __shared__ float lds[2][kNormWaves];
    for (size_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
        const char* x = static_cast<const char*>(a.x) + r * a.xstride * EB;
        const char* dy = static_cast<const char*>(a.dy) + r * a.dystride * EB;
        char* dx = static_cast<char*>(a.dx) + r * a.cols * EB;
        const float n = (float)a.cols, mean = a.mean[r], rstd = a.rstd[r];

        float s1 = 0.0f, s2 = 0.0f;
        for (size_t i = (size_t)threadIdx.x * E; i < a.cols; i += (size_t)kNormThreads * E) {
            float v[E], g[E], w[E];
            Vec<EB>::unpack(ld_unit_of<EB>(x, i, a.cols, 0u), v);
            Vec<EB>::unpack(ld_unit_of<EB>(dy, i, a.cols, 0u), g);
            ld_params<E>(a.weight, a.pb, i, a.cols, 1.0f, w);
    #pragma unroll
            for (int j = 0; j < E; ++j) {
                const float gw = g[j] * w[j];   // 0 past the end
                const float xh = i + j < a.cols ? (v[j] - mean) * rstd : 0.0f;
                s1 += gw;
                s2 = __builtin_fmaf(gw, xh, s2);
            }
        }
        const float c1 = block_sum<kNormWaves>(s1, lds[0]) / n;
        const float c2 = block_sum<kNormWaves>(s2, lds[1]) / n;
        for (size_t i = (size_t)threadIdx.x * E; i < a.cols; i += (size_t)kNormThreads * E) {
            float v[E], g[E], w[E];
            Vec<EB>::unpack(ld_unit_of<EB>(x, i, a.cols, 0u), v);
            Vec<EB>::unpack(ld_unit_of<EB>(dy, i, a.cols, 0u), g);
            ld_params<E>(a.weight, a.pb, i, a.cols, 1.0f, w);
    #pragma unroll
            for (int j = 0; j < E; ++j) {
                const float xh = (v[j] - mean) * rstd;
                v[j] = rstd * (__builtin_fmaf(g[j], w[j], -c1) - xh * c2);
            }
            st_unit_of<EB>(dx, i, a.cols, Vec<EB>::pack(v));
        }
    }
}

// The column sums' split of the rows: parts of at least kColRows rows, at most
// kColParts of them.
constexpr size_t kColRows = 64, kColParts = 1024;

// Partial column sums over rows_per rows: part[p][0] = sum dy xh, part[p][1] = sum dy.
template <int EB>
__global__ __launch_bounds__(kNormThreads) void k_norm_cols(const NormGradArgs a, size_t rows_per) {
    constexpr int E = Vec<EB>::E;
    const size_t i = ((size_t)blockIdx.x * kNormThreads + threadIdx.x) * E;
    if (i >= a.cols) return;
    const size_t p = blockIdx.y;
    size_t r1 = (p + 1) * rows_per;
    if (r1 > a.rows) r1 = a.rows;
    float dw[E] = {}, db[E] = {};
    for (size_t r = p * rows_per; r < r1; ++r) {
        float v[E], g[E];
        Vec<EB>::unpack(ld_unit_of<EB>(static_cast<const char*>(a.x) + r * a.xstride * EB, i,
                                       a.cols, 0u), v);
        Vec<EB>::unpack(ld_unit_of<EB>(static_cast<const char*>(a.dy) + r * a.dystride * EB, i,
                                       a.cols, 0u), g);
        const float mean = a.mean[r], rstd = a.rstd[r];
#pragma unroll
        for (int j = 0; j < E; ++j) {
            dw[j] = __builtin_fmaf(g[j], (v[j] - mean) * rstd, dw[j]);
            db[j] += g[j];
        }
    }
    float* out = a.part + p * 2 * a.cols;
#pragma unroll
    for (int j = 0; j < E; ++j)
        if (i + j < a.cols) {
            out[i + j] = dw[j];
            out[a.cols + i + j] = db[j];
        }
}

// The last step: the partial rows of a column added in a fixed order, 64
// columns a block with its wavefronts side by side down the parts.  (Groups of
// columns past a grid's x go on in its y: blocks that walk them instead took 0.5
// us more at 6416 x 946.)
constexpr int kFoldThreads = 1024, kFoldWaves = kFoldThreads / 64;
__global__ __launch_bounds__(kFoldThreads) void k_norm_fold(const NormGradArgs a, size_t parts) {
    __shared__ float lds[kFoldWaves][64];
    const unsigned lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const size_t c = ((size_t)blockIdx.y * gridDim.x + blockIdx.x) * 64 + lane;   // of 2 * cols
    float s = 0.0f;
    if (c < 2 * a.cols) {
        constexpr int kAhead = 16;   // loads in flight
        const float* p = a.part + c;
        for (size_t k = wave; k < parts; k += kFoldWaves * kAhead) {
            float v[kAhead];
#pragma unroll
            for (int q = 0; q < kAhead; ++q)
                v[q] = k + q * kFoldWaves < parts ? p[(k + q * kFoldWaves) * 2 * a.cols] : 0.0f;
#pragma unroll
            for (int q = 0; q < kAhead; ++q) s += v[q];
        }
    }
    lds[wave][lane] = s;
    __syncthreads();
    if (wave != 0 || c >= 2 * a.cols) return;
#pragma unroll
    for (int w = 1; w < kFoldWaves; ++w) s += lds[w][lane];
    void* out = c < a.cols ? a.dweight : a.dbias;
    if (out) st_param(out, a.pb, c < a.cols ? c : c - a.cols, s);
}

}  // namespace

// Blocks of a launch in one dimension, of those that its rows (or groups of
// columns) would take: a grid holds fewer than 2^32 threads, a block up to 2^10
// of them.  The row kernels walk the rest.
static unsigned row_blocks(size_t blocks) {
    constexpr size_t kMost = size_t(1) << 21;
    return (unsigned)(blocks < kMost ? blocks : kMost);
}

// The shape of a row kernel: threads, units per thread and rows at a time;
// threads 0: rows too wide for registers, or narrower than a unit, are the wide
// kernels'; threads below 64: the narrow kernels', that many lanes a row.
struct RowShape {
    int threads, upt, r;
};
// A block has the wavefronts that a row's units need: 8192 x 5120 bf16 forwards
// takes 45 us with 640 threads and 57 with 1024.  (Two blocks of up to 12
// wavefronts fit a compute unit, one of more: 8192 x 6144 42 us, x 7168 64.)
static RowShape row_shape(size_t cols, int eb) {
    if (cols < 16u / eb) return {0, 0, 0};   // no 16 bytes in a row
    const size_t units = (cols * eb + 15) / 16;
    if (units <= 32) {
        const int tpr = units <= 8 ? 8 : units <= 16 ? 16 : 32;
        return {tpr, 1, kNormWaves * kNarrowSteps * 64 / tpr};
    }
    const auto threads = [&](size_t upt) {
        return (int)((units + 64 * upt - 1) / (64 * upt) * 64);
    };
    if (units <= 1024) return {threads(1), 1, 4};
    if (units <= 2048) return {threads(2), 2, 1};
    if (units <= 4096 && eb == 4) return {threads(4), 4, 1};
    return {0, 0, 0};
}

// Blocks of the backward row kernels, each of which leaves a row of partial
// sums.  More blocks share out the steps over the rows (about 3 us a step of R
// rows, mostly latency), and cost the last step more: 8 bytes a column and
// block at about 4 TB/s, or about 1/160 us a block where there are few columns
// and the additions follow one another.  With both costs c, P blocks of S steps
// in all take 3 S / P + c P, the least at P = sqrt(3 S / c).  Two steps of one
// block are cheaper than a second launch.
static size_t grad_blocks(size_t rows, size_t cols, RowShape sh) {
    const size_t steps = (rows + sh.r - 1) / sh.r;
    if (steps <= 2) return rows ? 1 : 0;
    // (whole rounds of the compute units: 16 wavefronts each, blocks not divided)
    const size_t most = sh.threads < 64 ? 1024 : kCUs * (1024 / sh.threads);
    const double c = cols * 2e-6 > 0.00625 ? cols * 2e-6 : 0.00625;
    const size_t best = (size_t)std::sqrt(3.0 * (double)steps / c) + 1;
    const size_t p = best < most ? best : most;
    return p < steps ? p : steps;
}

size_t norm_grad_parts(size_t rows, size_t cols, int eb) {
    const RowShape sh = row_shape(cols, eb);
    if (sh.threads) return grad_blocks(rows, cols, sh);
    const size_t p = (rows + kColRows - 1) / kColRows;
    return p < kColParts ? p : kColParts;
}

#define ROWS_BY_SHAPE(EB, RAGGED, CALL)                             \
    if (sh.upt == 2) { CALL(EB, 1024, 2, 1, RAGGED); }              \
    else if (sh.upt == 4) {                                         \
        if constexpr (EB == 4) { CALL(EB, 1024, 4, 1, RAGGED); }    \
    }                                                               \
    else if (sh.threads <= 64) { CALL(EB, 64, 1, 4, RAGGED); }      \
    else if (sh.threads <= 256) { CALL(EB, 256, 1, 4, RAGGED); }    \
    else if (sh.threads <= 512) { CALL(EB, 512, 1, 4, RAGGED); }    \
    else { CALL(EB, 1024, 1, 4, RAGGED); }
#define NARROW_BY_SHAPE(EB, RAGGED, CALL)                   \
    if (sh.threads == 8) { CALL(EB, 8, RAGGED); }           \
    else if (sh.threads == 16) { CALL(EB, 16, RAGGED); }    \
    else { CALL(EB, 32, RAGGED); }
// RAGGED: the row's end lies inside a unit (the other form spends no
// registers on that)
#define BY_TYPE(SHAPE, CALL)                                                            \
    if (a.cols % (16 / a.eb) == 0) {                                                    \
        if (a.eb == 2) { SHAPE(2, false, CALL) } else { SHAPE(4, false, CALL) }         \
    } else {                                                                            \
        if (a.eb == 2) { SHAPE(2, true, CALL) } else { SHAPE(4, true, CALL) }           \
    }

hipError_t launch_norm(const NormArgs& a, hipStream_t s) {
    if (a.rows == 0) return hipSuccess;
    const RowShape sh = row_shape(a.cols, a.eb);
    if (sh.threads == 0) {
        const dim3 grid(row_blocks(a.rows)), block(kNormThreads);
        if (a.eb == 2) hipLaunchKernelGGL(k_norm_wide<2>, grid, block, 0, s, a);
        else hipLaunchKernelGGL(k_norm_wide<4>, grid, block, 0, s, a);
        return hipGetLastError();
    }
    dim3 grid(row_blocks((a.rows + sh.r - 1) / sh.r));
    if (sh.threads < 64) {
#define CALL(EB, TPR, RAGGED) \
    hipLaunchKernelGGL((k_norm_narrow<EB, TPR, RAGGED>), grid, dim3(kNormThreads), 0, s, a)
        BY_TYPE(NARROW_BY_SHAPE, CALL)
#undef CALL
        return hipGetLastError();
    }
    // one row a block until every compute unit has rows at R a block
    const dim3 block(sh.threads);
    const bool few = a.rows <= (size_t)kCUs * sh.r;
    if (few) grid.x = (unsigned)a.rows;
#define LAUNCH(EB, NT, UPT, R, RAGGED, FIXED) \
    hipLaunchKernelGGL((k_norm_rows<EB, NT, UPT, R, RAGGED, FIXED>), grid, block, 0, s, a)
#define CALL(EB, NT, UPT, R, RAGGED)                                          \
    if (few) LAUNCH(EB, NT, UPT, 1, RAGGED, false);                           \
    else if (sh.threads == NT && !RAGGED) LAUNCH(EB, NT, UPT, R, RAGGED, !RAGGED); \
    else LAUNCH(EB, NT, UPT, R, RAGGED, false)
    BY_TYPE(ROWS_BY_SHAPE, CALL)
#undef CALL
#undef LAUNCH
    return hipGetLastError();
}

static hipError_t launch_grad_wide(const NormGradArgs& a, size_t parts, hipStream_t s) {
    const dim3 grid(row_blocks(a.rows)), block(kNormThreads);
    if (a.eb == 2) hipLaunchKernelGGL(k_norm_grad_wide<2>, grid, block, 0, s, a);
    else hipLaunchKernelGGL(k_norm_grad_wide<4>, grid, block, 0, s, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || (!a.dweight && !a.dbias)) return e;
    const size_t per = (size_t)kNormThreads * (16 / a.eb);
    const size_t rows_per = (a.rows + parts - 1) / parts;
    const dim3 g2((unsigned)((a.cols + per - 1) / per), (unsigned)parts);
    if (a.eb == 2) hipLaunchKernelGGL(k_norm_cols<2>, g2, block, 0, s, a, rows_per);
    else hipLaunchKernelGGL(k_norm_cols<4>, g2, block, 0, s, a, rows_per);
    return hipGetLastError();
}

hipError_t launch_norm_grad(const NormGradArgs& a, hipStream_t s) {
    const size_t parts = norm_grad_parts(a.rows, a.cols, a.eb);
    const RowShape sh = row_shape(a.cols, a.eb);
    if (a.rows > 0 && sh.threads) {
        const dim3 grid((unsigned)parts), block(sh.threads);
        if (sh.threads < 64) {
#define CALL(EB, TPR, RAGGED) \
    hipLaunchKernelGGL((k_norm_grad_narrow<EB, TPR, RAGGED>), grid, dim3(kNormThreads), 0, s, a)
            BY_TYPE(NARROW_BY_SHAPE, CALL)
#undef CALL
        } else {
#define LAUNCH(EB, NT, UPT, R, RAGGED, FIXED) \
    hipLaunchKernelGGL((k_norm_grad_rows<EB, NT, UPT, R, RAGGED, FIXED>), grid, block, 0, s, a)
#define CALL(EB, NT, UPT, R, RAGGED)                                                   \
    if (sh.threads == NT && !RAGGED) LAUNCH(EB, NT, UPT, R, RAGGED, !RAGGED);          \
    else LAUNCH(EB, NT, UPT, R, RAGGED, false)
            BY_TYPE(ROWS_BY_SHAPE, CALL)
#undef CALL
#undef LAUNCH
        }
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess || parts == 1) return e;
    } else if (a.rows > 0) {
        const hipError_t e = launch_grad_wide(a, parts, s);
        if (e != hipSuccess) return e;
    }
    if (!a.dweight && !a.dbias) return hipSuccess;
    const size_t groups = (2 * a.cols + 63) / 64;
    const unsigned gx = row_blocks(groups);
    hipLaunchKernelGGL(k_norm_fold, dim3(gx, (unsigned)((groups + gx - 1) / gx)),
                       dim3(kFoldThreads), 0, s, a, parts);
    return hipGetLastError();
}

}  // namespace arlib
