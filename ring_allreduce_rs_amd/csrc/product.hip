// product.hip -- the experts' matrix products over ragged groups of rows, and
// their gradients.
#include "model_ops.h"
#include "ops_device.h"

namespace arlib {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kStep = 128;    // bytes of the reduced dimension in a step
constexpr int kStepUnits = kStep / 16;

// A tile of one operand in LDS, of T rows (or columns) of the result by one
// step, in 16-byte units.  KC: the reduced dimension is the contiguous one in
// memory, and the tile is [T][step]; otherwise [step][T].  Units are swapped
// within a line so that the lanes of a wavefront read from all banks.
template <int EB, bool KC, int T>
struct Tile {
    static constexpr int E = 16 / EB;
    static constexpr int S = kStep / EB;                 // elements of a step
    static constexpr int ROWS = KC ? T : S;
    static constexpr int UNITS = KC ? kStepUnits : T / E;   // of a line
    static constexpr int BYTES = ROWS * UNITS * 16;

    __device__ __forceinline__ static int swap_of(int row) {
        if constexpr (KC) return row & 7;
        else if constexpr (EB == 2) return 2 * ((row & 3) | ((row >> 1) & 4));
        else return 4 * ((row >> 2) & 3);
    }
    __device__ __forceinline__ static int at(int row, int unit) {
        return (row * UNITS + (unit ^ swap_of(row))) * 16;
    }

    // What a lane gives a 16-row matrix instruction, for rows first .. first + 15
    // of the result and part s of the step: bf16, 8 elements of the reduced
    // dimension from 32 s + 8 (lane / 16); fp32, 4 of them from 16 s + 4 (lane / 16),
    // one for each of 4 instructions.
    __device__ __forceinline__ static auto frag(const char* lds, int first, int s, int lane) {
        const int i = first + (lane & 15), g = lane >> 4;
        if constexpr (EB == 2) {
            if constexpr (KC) {
                return *reinterpret_cast<const bf16x8*>(lds + at(i, 4 * s + g));
            } else {
                // (the transposing read: 16 lanes load 4 lines of 16 elements, and lane i gets
                // element i of each)
                typedef __attribute__((address_space(3))) s16x4* lds_t;
                const int k = 32 * s + 8 * g + ((lane & 15) >> 2), c = first + 4 * (lane & 3);
                struct { s16x4 a, b; } v;
                v.a = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                    (lds_t)(lds + at(k, c / 8) + (c & 4) * 2));
                v.b = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                    (lds_t)(lds + at(k + 4, c / 8) + (c & 4) * 2));
                return __builtin_bit_cast(bf16x8, v);
            }
        } else {
            if constexpr (KC) {
                return *reinterpret_cast<const f32x4*>(lds + at(i, 4 * s + g));
            } else {
                f32x4 v;
#pragma unroll
                for (int t = 0; t < 4; ++t)
                    v[t] = *reinterpret_cast<const float*>(
                        lds + at(16 * s + 4 * g + t, i / 4) + (i & 3) * 4);
                return v;
            }
        }
    }
};

__device__ __forceinline__ f32x4 mma(bf16x8 a, bf16x8 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x4 mma(f32x4 a, f32x4 b, f32x4 c) {
#pragma unroll
    for (int t = 0; t < 4; ++t) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[t], b[t], c, 0, 0, 0);
    return c;
}

// An operand in memory: `rows` lines of `cols` elements that may be read.
struct Operand {
    const char* base;
    size_t stride;      // bytes
    size_t rows, cols;
};

// A thread's share of a tile, on its way through registers.
template <class TILE, int NT>
struct Share {
    static constexpr int N = TILE::ROWS * TILE::UNITS / NT;
    static_assert(TILE::ROWS * TILE::UNITS % NT == 0, "");
    u32x4 u[N];
    template <int EB>
    __device__ __forceinline__ void load(const Operand& o, size_t row0, size_t col0) {
#pragma unroll
        for (int q = 0; q < N; ++q) {
            const int at = q * NT + (int)threadIdx.x;
            const size_t row = row0 + at / TILE::UNITS, col = col0 + at % TILE::UNITS * TILE::E;
            u[q] = u32x4{0u, 0u, 0u, 0u};
            if (row < o.rows) u[q] = ld_unit_of<EB>(o.base + row * o.stride, col, o.cols, 0u);
        }
    }
    __device__ __forceinline__ void store(char* lds) const {
#pragma unroll
        for (int q = 0; q < N; ++q) {
            const int at = q * NT + (int)threadIdx.x;
            *reinterpret_cast<u32x4*>(lds + TILE::at(at / TILE::UNITS, at % TILE::UNITS)) = u[q];
        }
    }
};

// The rows of a group: [begin, end), whatever the offsets hold inside [0, nrows].
// Group `experts` are the rows behind the last expert.
__device__ __forceinline__ void group_of(const ProductArgs& a, int e, int* begin, int* end) {
    const int n = (int)a.nrows;
    const int b = a.offsets[e], f = e < a.experts ? a.offsets[e + 1] : n;
    *begin = b < 0 ? 0 : b < n ? b : n;
    *end = f < *begin ? *begin : f < n ? f : n;
}

// Tile `index` of the rows: its group and first row, or false past the last
// one.  Every group begins a tile of its own.  (All lanes of a wavefront
// together.)
struct RowTile {
    int group, row, end;
};
__device__ __forceinline__ bool find_tile(const ProductArgs& a, size_t index, int height,
                                          RowTile* t) {
    const int lane = threadIdx.x & 63;
    size_t run = 0;
    for (int e0 = 0; e0 <= a.experts; e0 += 64) {
        int begin = 0, end = 0;
        if (e0 + lane <= a.experts) group_of(a, e0 + lane, &begin, &end);
        const int tiles = (end - begin + height - 1) / height;
        int inc = tiles;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int o = __shfl_up(inc, d, 64);
            if (lane >= d) inc += o;
        }
        const unsigned long long past = __ballot(run + inc > index);
        if (past) {
            const int at = __builtin_ctzll(past);
            const int skip = (int)(index - run) -
                             (__builtin_amdgcn_readlane(inc, at) - __builtin_amdgcn_readlane(tiles, at));
            t->group = e0 + at;
            t->row = __builtin_amdgcn_readlane(begin, at) + skip * height;
            t->end = __builtin_amdgcn_readlane(end, at);
            return true;
        }
        run += __builtin_amdgcn_readlane(inc, 63);
    }
    return false;
}

// Stores 4 elements of a row of n from column j on.
template <int EB>
__device__ __forceinline__ void st4(char* row, size_t j, size_t n, f32x4 v) {
    if constexpr (EB == 2) {
        typedef uint32_t two_t __attribute__((ext_vector_type(2), aligned(2)));
        typedef uint32_t two_r __attribute__((ext_vector_type(2)));
        const f32x2_t a = {v[0], v[1]}, b = {v[2], v[3]};
        const two_r u = {__builtin_bit_cast(uint32_t, __builtin_convertvector(a, bf16x2_t)),
                         __builtin_bit_cast(uint32_t, __builtin_convertvector(b, bf16x2_t))};
        if (j + 4 <= n) *reinterpret_cast<two_t*>(row + j * 2) = u;
        else
#pragma unroll
            for (int k = 0; k < 3; ++k)
                if (j + k < n) st_elem<2>(row + (j + k) * 2, (u[k / 2] >> (16 * (k & 1))) & 0xffffu);
    } else {
        typedef float four_t __attribute__((ext_vector_type(4), aligned(4)));
        if (j + 4 <= n) *reinterpret_cast<four_t*>(row + j * 4) = v;
        else
#pragma unroll
            for (int k = 0; k < 3; ++k)
                if (j + k < n) *reinterpret_cast<float*>(row + (j + k) * 4) = v[k];
    }
}

// c (TI x TJ, from its row i0 and column j0) += A B^T over `depth` elements of
// the reduced dimension.  AK, BK: it is the contiguous one of the operand.
template <int EB, bool AK, bool BK, int TI, int TJ, int WI, int WJ>
struct Block {
    static constexpr int NT = WI * WJ * 64;
    using A = Tile<EB, AK, TI>;
    using B = Tile<EB, BK, TJ>;
    static constexpr int FI = TI / WI / 16, FJ = TJ / WJ / 16;   // a wavefront's 16 x 16 pieces
    static constexpr int STAGE = A::BYTES + B::BYTES;

    f32x4 acc[FI][FJ];

    __device__ __forceinline__ void run(char* lds, const Operand& oa, const Operand& ob, size_t i0,
                                        size_t j0, size_t depth) {
        const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
        const int wi = wave / WJ * (TI / WI), wj = wave % WJ * (TJ / WJ);
#pragma unroll
        for (int i = 0; i < FI; ++i)
#pragma unroll
            for (int j = 0; j < FJ; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
        if (depth == 0) return;
        Share<A, NT> sa;
        Share<B, NT> sb;
        const auto load = [&](size_t k) {
            sa.template load<EB>(oa, AK ? i0 : k, AK ? k : i0);
            sb.template load<EB>(ob, BK ? j0 : k, BK ? k : j0);
        };
        load(0);
        int buf = 0;
        for (size_t k = 0; k < depth; k += A::S, buf ^= 1) {
            char* la = lds + buf * STAGE;
            char* lb = la + A::BYTES;
            sa.store(la);
            sb.store(lb);
            __syncthreads();
            if (k + A::S < depth) load(k + A::S);
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                decltype(A::frag(la, 0, 0, 0)) fa[FI], fb[FJ];
#pragma unroll
                for (int i = 0; i < FI; ++i) fa[i] = A::frag(la, wi + 16 * i, s, lane);
#pragma unroll
                for (int j = 0; j < FJ; ++j) fb[j] = B::frag(lb, wj + 16 * j, s, lane);
                // (the operands change places, so that a lane holds 4 neighbours of a row)
#pragma unroll
                for (int i = 0; i < FI; ++i)
#pragma unroll
                    for (int j = 0; j < FJ; ++j) acc[i][j] = mma(fb[j], fa[i], acc[i][j]);
            }
        }
        __syncthreads();
    }

    // To the rows [i0, rows) of c, `cols` elements wide.
    __device__ __forceinline__ void store(char* c, size_t i0, size_t rows, size_t j0,
                                          size_t cols) const {
        const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
        const int wi = wave / WJ * (TI / WI), wj = wave % WJ * (TJ / WJ);
#pragma unroll
        for (int i = 0; i < FI; ++i) {
            const size_t row = i0 + wi + 16 * i + (lane & 15);
            if (row >= rows) continue;
#pragma unroll
            for (int j = 0; j < FJ; ++j)
                st4<EB>(c + row * cols * EB, j0 + wj + 16 * j + 4 * (lane >> 4), cols, acc[i][j]);
        }
    }
};

// The products of the rows (KIND: forward or drows).
template <int EB, ProductKind KIND, int TI, int TJ, int WI, int WJ>
__global__ __launch_bounds__(WI * WJ * 64) void k_product_rows(const ProductArgs a) {
    using BLOCK = Block<EB, true, KIND == PRODUCT_FORWARD, TI, TJ, WI, WJ>;
    __shared__ __attribute__((aligned(16))) char lds[2 * BLOCK::STAGE];
    const size_t cols = KIND == PRODUCT_FORWARD ? a.out : a.hidden;
    const size_t depth = KIND == PRODUCT_FORWARD ? a.hidden : a.out;
    const size_t across = (cols + TJ - 1) / TJ;
    for (size_t at = blockIdx.x;; at += gridDim.x) {
        RowTile t;
        if (!find_tile(a, at / across, TI, &t)) break;
        const size_t j0 = at % across * TJ;
        const char* w = static_cast<const char*>(a.b) + (size_t)t.group * a.out * a.hidden * EB;
        const Operand oa = {static_cast<const char*>(a.a), a.astride * EB, (size_t)t.end, depth};
        const Operand ob = {w, a.hidden * EB, a.out, a.hidden};
        BLOCK b;
        b.run(lds, oa, ob, t.row, j0, t.group < a.experts ? depth : 0);
        b.store(static_cast<char*>(a.c), t.row, t.end, j0, cols);
    }
}

// The weights' gradient.
template <int EB, int TI, int TJ, int WI, int WJ>
__global__ __launch_bounds__(WI * WJ * 64) void k_product_weights(const ProductArgs a) {
    using BLOCK = Block<EB, false, false, TI, TJ, WI, WJ>;
    __shared__ __attribute__((aligned(16))) char lds[2 * BLOCK::STAGE];
    const size_t across = (a.hidden + TJ - 1) / TJ, down = (a.out + TI - 1) / TI;
    const size_t tiles = across * down * a.experts;
    for (size_t at = blockIdx.x; at < tiles; at += gridDim.x) {
        const int e = (int)(at / (across * down));
        const size_t i0 = at / across % down * TI, j0 = at % across * TJ;
        int begin, end;
        group_of(a, e, &begin, &end);
        const size_t n = (size_t)(end - begin);
        const Operand oa = {static_cast<const char*>(a.a) + (size_t)begin * a.astride * EB,
                            a.astride * EB, n, a.out};
        const Operand ob = {static_cast<const char*>(a.b) + (size_t)begin * a.bstride * EB,
                            a.bstride * EB, n, a.hidden};
        BLOCK b;
        b.run(lds, oa, ob, i0, j0, n);
        b.store(static_cast<char*>(a.c) + (size_t)e * a.out * a.hidden * EB, i0, a.out, j0,
                a.hidden);
    }
}

// Tiles of `height` rows that nrows rows in experts + 1 groups make at most.
size_t most_row_tiles(size_t nrows, int experts, size_t height) {
    const size_t full = (nrows + ((size_t)experts + 1) * (height - 1)) / height;
    return full < nrows ? full : nrows;
}

constexpr size_t kMostBlocks = size_t(1) << 22;
unsigned most(size_t blocks) { return (unsigned)(blocks < kMostBlocks ? blocks : kMostBlocks); }

}  // namespace

size_t product_work_bytes(ProductKind, size_t, int, size_t, size_t, int) { return 0; }

hipError_t launch_product(ProductKind kind, const ProductArgs& a, hipStream_t s) {
    constexpr int T = 128, NT = 256;
    if (kind == PRODUCT_DWEIGHTS) {
        const size_t tiles = (a.hidden + T - 1) / T * ((a.out + T - 1) / T) * a.experts;
        if (a.eb == 2)
            hipLaunchKernelGGL((k_product_weights<2, T, T, 2, 2>), dim3(most(tiles)), dim3(NT), 0, s, a);
        else
            hipLaunchKernelGGL((k_product_weights<4, T, T, 2, 2>), dim3(most(tiles)), dim3(NT), 0, s, a);
        return hipGetLastError();
    }
    if (a.nrows == 0) return hipSuccess;
    const size_t cols = kind == PRODUCT_FORWARD ? a.out : a.hidden;
    const dim3 grid(most(most_row_tiles(a.nrows, a.experts, T) * ((cols + T - 1) / T)));
#define CALL(EB, KIND) \
    hipLaunchKernelGGL((k_product_rows<EB, KIND, T, T, 2, 2>), grid, dim3(NT), 0, s, a)
    if (kind == PRODUCT_FORWARD) {
        if (a.eb == 2) CALL(2, PRODUCT_FORWARD);
        else CALL(4, PRODUCT_FORWARD);
    } else {
        if (a.eb == 2) CALL(2, PRODUCT_DROWS);
        else CALL(4, PRODUCT_DROWS);
    }
#undef CALL
    return hipGetLastError();
}

}  // namespace arlib
