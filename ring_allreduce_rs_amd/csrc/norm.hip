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
#include "ops.h"
#include "ops_device.h"

namespace arlib {
namespace {

constexpr int kNormThreads = 256;
constexpr int kNormWaves = kNormThreads / 64;

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

// The last step: the partial rows of one column added in a fixed order.
__global__ __launch_bounds__(kNormThreads) void k_norm_fold(const NormGradArgs a, size_t parts) {
    __shared__ float lds[kNormWaves][64];
    const unsigned lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const size_t c = (size_t)blockIdx.x * 64 + lane;   // of 2 * cols
    float s = 0.0f;
    if (c < 2 * a.cols)
        for (size_t p = wave; p < parts; p += kNormWaves) s += a.part[p * 2 * a.cols + c];
    lds[wave][lane] = s;
    __syncthreads();
    if (wave != 0 || c >= 2 * a.cols) return;
#pragma unroll
    for (int w = 1; w < kNormWaves; ++w) s += lds[w][lane];
    void* out = c < a.cols ? a.dweight : a.dbias;
    const size_t i = c < a.cols ? c : c - a.cols;
    if (!out) return;
    if (a.pb == 4) Vec<4>::st1(static_cast<char*>(out) + i * 4, s);
    else Vec<2>::st1(static_cast<char*>(out) + i * 2, s);
}

}  // namespace

// Rows of a launch: the kernels walk the rest (a grid holds fewer than 2^32 threads).
static unsigned row_blocks(size_t rows) {
    constexpr size_t kMost = size_t(1) << 22;
    return (unsigned)(rows < kMost ? rows : kMost);
}

size_t norm_grad_parts(size_t rows, size_t cols, int eb) {
    (void)cols;
    (void)eb;
    const size_t p = (rows + kColRows - 1) / kColRows;
    return p < kColParts ? p : kColParts;
}

hipError_t launch_norm(const NormArgs& a, hipStream_t s) {
    if (a.rows == 0) return hipSuccess;
    const dim3 grid(row_blocks(a.rows)), block(kNormThreads);
    if (a.eb == 2) hipLaunchKernelGGL(k_norm_wide<2>, grid, block, 0, s, a);
    else hipLaunchKernelGGL(k_norm_wide<4>, grid, block, 0, s, a);
    return hipGetLastError();
}

hipError_t launch_norm_grad(const NormGradArgs& a, hipStream_t s) {
    const size_t parts = norm_grad_parts(a.rows, a.cols, a.eb);
    if (a.rows > 0) {
        const dim3 grid(row_blocks(a.rows)), block(kNormThreads);
        if (a.eb == 2) hipLaunchKernelGGL(k_norm_grad_wide<2>, grid, block, 0, s, a);
        else hipLaunchKernelGGL(k_norm_grad_wide<4>, grid, block, 0, s, a);
        hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        if (a.dweight || a.dbias) {
            const size_t per = (size_t)kNormThreads * (16 / a.eb);
            const size_t rows_per = (a.rows + parts - 1) / parts;
            const dim3 g2((unsigned)((a.cols + per - 1) / per), (unsigned)parts);
            if (a.eb == 2) hipLaunchKernelGGL(k_norm_cols<2>, g2, block, 0, s, a, rows_per);
            else hipLaunchKernelGGL(k_norm_cols<4>, g2, block, 0, s, a, rows_per);
            e = hipGetLastError();
            if (e != hipSuccess) return e;
        }
    }
    if (a.dweight || a.dbias) {
        hipLaunchKernelGGL(k_norm_fold, dim3((unsigned)((2 * a.cols + 63) / 64)),
                           dim3(kNormThreads), 0, s, a, parts);
        return hipGetLastError();
    }
    return hipSuccess;
}

}  // namespace arlib
