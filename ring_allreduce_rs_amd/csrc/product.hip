// product.hip -- the experts' matrix products over ragged groups of rows, and
// their gradients.  Expert e has the rows [offsets[e], offsets[e + 1]):
//
//   forward    y[j] = W_e x[j]               W_e is (out, hidden), out's rows contiguous
//   drows      dx[j] = W_e^T dy[j]
//   dweights   dW_e = sum over its rows j of dy[j] x[j]^T
//
// Each is C = A B^T for an operand of lines along the reduced dimension or across
// it; the second kind is turned on the way from LDS into the matrix instructions
// (bf16 by the transposing read, fp32 element by element), so nothing is
// transposed in memory.  Sums are fp32 in the matrix accumulators and rounded
// once, at the store.
//
// Blocks stay and walk the tiles of all experts, so that a group's last, partly
// filled tile is next to others' work; the experts' tiles are counted on the
// device from the offsets.  Many rows: bound by the matrix units at a clock of
// 2.05 of 2.4 GHz (8192^3 bf16 forward 787 us, 1397 TFLOP/s; the three of 64
// experts of 1024 rows, 4096 -> 2048, 910, 952 and 1066 us, 1208 to 1031 TFLOP/s,
// the rest being stores of tiles that end together).  Ragged groups cost part
// tiles and a last round of few (65536 rows in 290 tiles of 256: ten rounds, 1040
// us) and, in the weights' gradient, dies with deeper tiles than others (131072
// rows over 128 experts, 2048 x 1024: 634 - 660 us, equal groups 555).
// Few rows: bound by reading the weights once (64 experts of 2 rows, 2048 -> 2048,
// 537 MB in 91 us forward, 5.9 TB/s, and 96 us for drows); one row of 26 experts out of
// the last-level cache 34 us.  Why there are several tiles, and in which order the depth is
// walked, stands at Shape, at kCosts and at RowJobs.
#include "model_ops.h"
#include "ops_device.h"

#include <climits>
#include <cmath>
#include <type_traits>

namespace arlib {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

// LDS by its own 32-bit addresses.
typedef __attribute__((address_space(3))) char* lds_t;
template <class T>
__device__ __forceinline__ T ld_lds(lds_t p) {
    return *(__attribute__((address_space(3))) const T*)p;
}


// A tile of one operand in LDS, of T rows (or columns) of the result by one
// step, in 16-byte units.  KC: the reduced dimension is the contiguous one in
// memory, and the tile is [T][step]; otherwise [step][T].  Units are swapped
// within a line so that the lanes of a wavefront read from all banks.
template <int EB, bool KC, int T, int STEP>
struct Tile {
    static constexpr int E = 16 / EB;
    static constexpr int S = STEP / EB;                  // elements of a step of STEP bytes
    static constexpr int ROWS = KC ? T : S;
    static constexpr int UNITS = KC ? STEP / 16 : T / E;   // of a line
    static constexpr int BYTES = ROWS * UNITS * 16;

    __device__ __forceinline__ static int swap_of(int row) {
        if constexpr (KC) return row & (UNITS - 1);
        else if constexpr (EB == 2) return 2 * ((row & 3) | ((row >> 1) & 4)) & (UNITS - 1);
        else return 4 * ((row >> 2) & 3) & (UNITS - 1);
    }
    __device__ __forceinline__ static int at(int row, int unit) {
        return (row * UNITS + (unit ^ swap_of(row))) * 16;
    }

    // What a lane gives a 16-row matrix instruction, for rows first .. first + 15
    // of the result and part s of the step: bf16, 8 elements of the reduced
    // dimension from 32 s + 8 (lane / 16); fp32, 4 of them from 16 s + 4 (lane / 16),
    // one for each of 4 instructions.
    //
    // origin() is the place of part 0 of the rows that begin at `first`, a multiple
    // of 16 that the wavefront adds to every piece's; frag() takes it, in one of
    // the buffers, and the piece's own `first` (a constant).  The swaps only change
    // bits that the lines' and buffers' addresses leave 0, so a piece's place is
    // the origin's with some bits turned over, plus a constant.
    static constexpr int kTurn = (KC ? 0 : EB == 2 ? 14 : 12) & (UNITS - 1);   // units that swaps reach
    __device__ __forceinline__ static unsigned origin(int lane, int first) {
        const int i = lane & 15, g = lane >> 4;
        if constexpr (KC) return at(first + i, g);
        else if constexpr (EB == 2) return at(8 * g + (i >> 2), first / 8 + ((i & 3) >> 1)) + (i & 1) * 8;
        else return at(4 * g, first / 4 + (i >> 2)) + (i & 3) * 4;
    }
    __device__ __forceinline__ static auto frag(lds_t from, int first, int s) {
        constexpr int kLine = UNITS * 16;
        if constexpr (KC) {
            using V = std::conditional_t<EB == 2, bf16x8, f32x4>;
            return ld_lds<V>((lds_t)((uintptr_t)from ^ (64 * s)) + first * kLine);
        } else {
            const int unit = first / E;
            const lds_t p = (lds_t)((uintptr_t)from ^ ((unit & kTurn) * 16)) + (unit & ~kTurn) * 16;
            if constexpr (EB == 2) {
                // (the transposing read: 16 lanes load 4 lines of 16 elements, and lane i gets
                // element i of each)
                typedef __attribute__((address_space(3))) s16x4* quad_t;
                struct { s16x4 a, b; } v;
                v.a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((quad_t)(p + 32 * s * kLine));
                v.b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((quad_t)(p + (32 * s + 4) * kLine));
                return __builtin_bit_cast(bf16x8, v);
            } else {
                f32x4 v;
#pragma unroll
                for (int t = 0; t < 4; ++t) v[t] = ld_lds<float>(p + (16 * s + t) * kLine);
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

// What is the same on every lane, in scalar registers.
__device__ __forceinline__ unsigned uniform(unsigned v) {
    return (unsigned)__builtin_amdgcn_readfirstlane((int)v);
}
__device__ __forceinline__ uint64_t uniform64(uint64_t v) {
    return (uint64_t)uniform((unsigned)(v >> 32)) << 32 | uniform((unsigned)v);
}
template <class T>
__device__ __forceinline__ T* uniform(T* p) {
    return (T*)(uintptr_t)uniform64((uint64_t)(uintptr_t)p);
}

// An operand in memory: `rows` lines of `cols` elements that may be read.
struct Operand {
    const char* base;
    size_t stride;      // bytes
    unsigned rows, cols;
};

// The last `live` elements of a line of n, first in a unit with zeros behind them.
template <int EB>
__device__ __forceinline__ u32x4 ld_end(const char* line, unsigned n, unsigned live) {
    constexpr unsigned E = 16 / EB;
    if (n < E) return ld_unit_of<EB>(line, n - live, n, 0u);
    const u32x4 u = ld_unit<EB>(line + (size_t)(n - E) * EB);
    uint64_t lo = (uint64_t)u[1] << 32 | u[0], hi = (uint64_t)u[3] << 32 | u[2];
    const unsigned away = (E - live) * EB * 8;    // bits, 1 .. 127
    if (away >= 64) {
        lo = hi >> (away - 64);
        hi = 0;
    } else {
        lo = lo >> away | hi << (64 - away);
        hi >>= away;
    }
    return u32x4{(uint32_t)lo, (uint32_t)(lo >> 32), (uint32_t)hi, (uint32_t)(hi >> 32)};
}

__device__ __forceinline__ void st_lds(lds_t p, u32x4 v) {
    *(__attribute__((address_space(3))) u32x4*)p = v;
}

// s_waitcnt's operand for vmcnt(0) alone.
constexpr int kVmcnt0 = 0x0f70;

// How a tile comes from memory into LDS, a step of the reduced dimension at a
// time, in 16-byte units, N a thread.  begin() says where, aim() which step;
// load() starts the thread's unit q, and arrive(), before the wavefronts meet,
// has the step that aim() had last on its way to LDS.
//
// A unit outside the operand is zeros.  So is one that a line's end cuts, where
// what lies behind it may not be read (behind the reduced dimension, and behind
// the operand's last line), but for the elements that belong to it.  Lines closer
// together than a unit (`narrow`) are cut every one: a unit would reach over
// several of them, and over the last from lines before it.
template <int EB, class TILE, bool KC, int NT>
struct Lines {
    static constexpr int N = TILE::ROWS * TILE::UNITS / NT;
    static_assert(TILE::ROWS * TILE::UNITS % NT == 0, "");
    static constexpr unsigned E = TILE::E;
    static constexpr unsigned kOutside = 0x80000000u;
    const char* base;       // the tile's first line (KC), its first column's
    unsigned off[N];        // bytes from the step's begin
    unsigned depth, wide, high, step;
    size_t stride;
    bool narrow;
    // Thread t's unit q, which goes to LDS unit q * NT + t: its line, and its unit in memory.
    __device__ __forceinline__ static unsigned line(int q, unsigned t) {
        return ((unsigned)(q * NT) + t) / TILE::UNITS;
    }
    __device__ __forceinline__ static unsigned unit(int q, unsigned t) {
        return ((unsigned)(q * NT) + t) % TILE::UNITS ^ (unsigned)TILE::swap_of((int)line(q, t));
    }
    __device__ __forceinline__ static lds_t slot(lds_t lds, int q, unsigned t) {
        return lds + (q * NT + (int)t) * 16;
    }
    __device__ __forceinline__ void begin(const Operand& o, unsigned first, unsigned depth_) {
        depth = uniform(depth_);
        stride = uniform64(o.stride);
        narrow = !KC && stride < 16;
        base = uniform(o.base + (KC ? first * o.stride : first * (size_t)EB));
        high = uniform(o.rows - first);   // (KC) lines from the tile's first on
        wide = uniform(o.cols - first);   // (otherwise) elements of a line from the tile's first on
        const unsigned t = offset_here(threadIdx.x);   // (nothing of it is kept over the steps)
#pragma unroll
        for (int q = 0; q < N; ++q) {
            const bool in = KC ? line(q, t) < high : unit(q, t) * E < wide && !narrow;
            off[q] = in ? line(q, t) * (unsigned)stride + unit(q, t) * 16 : kOutside;
        }
    }
    __device__ __forceinline__ void end() { depth = 0; }
    // Where the step begins; the units that are not whole go outside.
    __device__ __forceinline__ const char* at_step(unsigned k) {
        step = k;
        if (__builtin_expect(k + TILE::S >= depth, 0)) {   // (nor is a step after this one whole)
            const unsigned t = offset_here(threadIdx.x);
#pragma unroll
            for (int q = 0; q < N; ++q) {
                const unsigned u = unit(q, t) * E, l = line(q, t);
                const bool in = KC ? k + u + E <= depth
                                   : k + l + 1 < depth || (k + l + 1 == depth && u + E <= wide);
                off[q] = in ? off[q] : kOutside;
            }
        }
        return base + (KC ? k * (size_t)EB : k * stride);
    }
    // Whether the step has cut units, whether this one is, and what it holds.
    __device__ __forceinline__ bool cut() const {
        if constexpr (KC) return step < depth && step + TILE::S > depth && depth % E;
        else return step < depth && (narrow || (step + TILE::S >= depth && wide % E &&
                                                wide < TILE::UNITS * E));
    }
    __device__ __forceinline__ bool cut(int q, unsigned t) const {
        if constexpr (KC) return unit(q, t) == (depth - step) / E && line(q, t) < high;
        else return narrow ? unit(q, t) == 0 && line(q, t) < depth - step
                           : unit(q, t) == wide / E && line(q, t) == depth - 1 - step;
    }
    __device__ __forceinline__ u32x4 rest(int q, unsigned t) const {
        if constexpr (KC) return ld_end<EB>(base + line(q, t) * stride, depth, depth % E);
        else return ld_end<EB>(base + (step + line(q, t)) * stride, wide, wide % E);
    }
    // Writes the step's cut units over the zeros that this thread's loads left there.
    __device__ __forceinline__ void mend(lds_t lds) const {
        if (__builtin_expect(!cut(), 1)) return;
        __builtin_amdgcn_s_waitcnt(kVmcnt0);   // (loads straight into LDS, too)
        const unsigned t = offset_here(threadIdx.x);
#pragma unroll
        for (int q = 0; q < N; ++q)
            if (cut(q, t)) st_lds(slot(lds, q, t), rest(q, t));
        // (known to the compiler, which would wait for these loads among the next step's:
        // 64 experts of 1024 rows 1029 us, 906 so)
        __builtin_amdgcn_s_waitcnt(kVmcnt0);
    }
};

// Through registers, for lines at any address.  A unit outside comes from a unit of
// zeros, so that no load waits for a branch.
__device__ const u32x4 kZeros = {0u, 0u, 0u, 0u};

template <int EB, class TILE, bool KC, int NT>
struct Through : Lines<EB, TILE, KC, NT> {
    using L = Lines<EB, TILE, KC, NT>;
    u32x4 u[L::N];
    const char* from;
    __device__ __forceinline__ void aim(unsigned k) { from = this->at_step(k); }
    __device__ __forceinline__ void load(lds_t, int q) {
        typedef const typename Vec<EB>::mem_t __attribute__((address_space(1))) * unit_t;
        const unsigned f = this->off[q];
        const uintptr_t zeros = (uintptr_t)&kZeros;
        u[q] = *(unit_t)(f != L::kOutside ? (uintptr_t)from + f : zeros);
    }
    __device__ __forceinline__ void arrive(lds_t lds) const {
#pragma unroll
        for (int q = 0; q < L::N; ++q) st_lds(L::slot(lds, q, threadIdx.x), u[q]);
        this->mend(lds);
    }
};

// (m0 is a register that the compiler keeps for itself: it sets it where it needs it)
#pragma clang diagnostic ignored "-Winline-asm"

// Straight into LDS, for lines at 4-byte addresses.  A wavefront's load fills 1 KiB of LDS in lane order, so the swapping of
// units is in the addresses that the lanes read; an offset past the buffer loads
// zeros.
//
// The load is written out because the compiler takes a transposing read for one
// that may see the load's bytes, and waits for memory before it (the products of
// 8192^3 by dout and by rows 1150 and 1130 us with the builtin, 773 and 816 so).
// It has no register output, and meet() waits for it.
template <int EB, class TILE, bool KC, int NT>
struct Straight : Lines<EB, TILE, KC, NT> {
    using L = Lines<EB, TILE, KC, NT>;
    u32x4 buffer;
    __device__ __forceinline__ void aim(unsigned k) {
        const uint64_t at = uniform64((uint64_t)(uintptr_t)this->at_step(k));
        buffer = u32x4{(uint32_t)at, (uint32_t)(at >> 32), 0x7fffffffu, 0x00020000u};
    }
    __device__ __forceinline__ void load(lds_t lds, int q) {
        const uint32_t at = uniform((uint32_t)(uintptr_t)L::slot(lds, q, threadIdx.x & ~63u));
        asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
                     :: "s"(at), "v"(this->off[q]), "s"(buffer) : "m0", "memory");
    }
    __device__ __forceinline__ void arrive(lds_t lds) const { this->mend(lds); }
};

// Everything this wavefront has asked for has arrived, then the block's
// wavefronts meet.
__device__ __forceinline__ void meet() {
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
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

// One tile of the result: TI x TJ of c = A B^T from row i0 (of `rows`) and column
// j0 (of `cols`), over `depth` elements of the reduced dimension.
struct Job {
    Operand a, b;
    char* c;
    unsigned i0, rows, j0, cols, depth;
    unsigned turn;      // the step that comes first; those before it come last
};

// Takes part `p` of the job's depth where it is split, whole steps of `step`.
template <int EB, bool AK, bool BK>
__device__ __forceinline__ void take_part(Job* job, unsigned p, unsigned parts, unsigned step) {
    const unsigned each = ((job->depth + step - 1) / step + parts - 1) / parts * step;
    const unsigned from = p * each < job->depth ? p * each : job->depth;
    const auto cut = [&](Operand& o, bool contiguous, unsigned to) {
        o.base += contiguous ? from * (size_t)EB : from * o.stride;
        (contiguous ? o.cols : o.rows) = to - from;
    };
    const unsigned to = job->depth - from < each ? job->depth : from + each;
    cut(job->a, AK, to);
    cut(job->b, BK, to);
    job->depth = to - from;
}

// 4 elements of row i from column j on: of the result, or in 32 bits where it is
// one of several parts.
template <int EB>
__device__ __forceinline__ void store(const Job& job, bool part, unsigned i, unsigned j, f32x4 v) {
    const size_t at = (size_t)i * job.cols;
    if (EB == 4 || part) st4<4>(job.c + at * 4, j, job.cols, v);
    else st4<EB>(job.c + at * EB, j, job.cols, v);
}

// Two pieces side by side, as bf16: a lane has 4 neighbours of each, and the odd
// rows of 16 lanes give theirs of the first piece for the even rows' of the
// second, so that a lane has 8 neighbours of one row of one piece.
__device__ __forceinline__ u32x4 pair(f32x4 a, f32x4 b) {
    const f32x2_t v[4] = {{a[0], a[1]}, {a[2], a[3]}, {b[0], b[1]}, {b[2], b[3]}};
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        u[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector(v[i], bf16x2_t));
    const auto x = __builtin_amdgcn_permlane16_swap(u[0], u[2], false, false);
    const auto y = __builtin_amdgcn_permlane16_swap(u[1], u[3], false, false);
    return u32x4{x[0], y[0], x[1], y[1]};
}

// Fills a tile with zeros.
template <int EB, int TI, int TJ, int NT>
__device__ __forceinline__ void clear(const Job& job, bool part) {
    const unsigned high = job.rows - job.i0 < TI ? job.rows - job.i0 : TI;
    for (unsigned at = threadIdx.x; at < high * (TJ / 4); at += NT)
        store<EB>(job, part, job.i0 + at / (TJ / 4), job.j0 + at % (TJ / 4) * 4,
                  f32x4{0.f, 0.f, 0.f, 0.f});
}

// A block's tiles one after another.  AK, BK: the reduced dimension is the
// operand's contiguous one; AS, BS: its lines are for Straight.  JOBS::next gives
// the next job, if there is one.
//
// LDS holds two steps.  A step has parts, 64 bytes of its depth by half of the
// wavefront's rows: while one part's pieces are multiplied, the next part's come
// from LDS, one read after each matrix instruction, and before the last part the
// wavefronts meet.  What they wait for there was asked for a whole step ago, and
// nobody reads the other buffer any more, so the loads of the step after the
// next go between the last part's instructions.  The tiles follow one another in
// this without a gap: a tile's last two steps load the first two of the next,
// and its result is stored while these come.
template <int EB, bool AK, bool BK, bool AS, bool BS, int TI, int TJ, int WI, int WJ,
          int STEP>
struct Block {
    static constexpr int NT = WI * WJ * 64;
    using A = Tile<EB, AK, TI, STEP>;
    using B = Tile<EB, BK, TJ, STEP>;
    using FeedA = std::conditional_t<AS, Straight<EB, A, AK, NT>, Through<EB, A, AK, NT>>;
    using FeedB = std::conditional_t<BS, Straight<EB, B, BK, NT>, Through<EB, B, BK, NT>>;
    static constexpr int FI = TI / WI / 16, FJ = TJ / WJ / 16;   // a wavefront's 16 x 16 pieces
    static constexpr int H = FI / 2;
    static constexpr int STAGE = A::BYTES + B::BYTES;
    using Piece = decltype(A::frag(lds_t(), 0, 0));

    template <class JOBS>
    __device__ __forceinline__ static void run(lds_t lds, JOBS& jobs) {
        const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        // (the wavefronts' rows take turns, so that all of them have a share of a tile that
        // the group fills in part)
        const int wi = wave / WJ * 16, wj = wave % WJ * (TJ / WJ);
        FeedA feed_a;
        FeedB feed_b;
        f32x4 acc[FI][FJ];
        Piece pa[2][H], pb[2][FJ];
        const unsigned from_a = A::origin(lane, wi), from_b = A::BYTES + B::origin(lane, wj);
        // Part p: rows' half p % 2 of the depth's part p / 2.  Read r of those that it needs.
        const auto read = [&](lds_t at, int p, int r) {
            if (r < H) pa[p & 1][r] = A::frag(at + from_a, 16 * WI * (p % 2 * H + r), p / 2);
            else if (p % 2 == 0 && r < H + FJ)
                pb[p / 2 & 1][r - H] = B::frag(at + from_b, 16 * (r - H), p / 2);
        };
        const auto multiply = [&](int p, auto also) {
            __builtin_amdgcn_sched_barrier(0);
            // (the operands change places, so that a lane holds 4 neighbours of a row)
#pragma unroll
            for (int i = 0; i < H; ++i)
#pragma unroll
                for (int j = 0; j < FJ; ++j) {
                    f32x4& c = acc[p % 2 * H + i][j];
                    c = mma(pb[p / 2 & 1][j], pa[p & 1][i], c);
                    also(i * FJ + j);
                    __builtin_amdgcn_sched_barrier(0);
                }
        };
        const auto begin = [&](const Job& job) {
            feed_a.begin(job.a, job.i0, job.depth);
            feed_b.begin(job.b, job.j0, job.depth);
        };
        const auto aim = [&](unsigned k) {
            feed_a.aim(k);
            feed_b.aim(k);
        };
        const auto load = [&](lds_t at, int q) {
            if (q < FeedA::N) feed_a.load(at, q);
            else if (q < FeedA::N + FeedB::N) feed_b.load(at + A::BYTES, q - FeedA::N);
        };
        const auto arrive = [&](lds_t at) {
            feed_a.arrive(at);
            feed_b.arrive(at + A::BYTES);
        };
        constexpr int LOADS = FeedA::N + FeedB::N, READS = H + FJ, SLOTS = H * FJ;
        constexpr int PARTS = 2 * STEP / 64;
        static_assert(PARTS % 4 == 0, "a step ends with the registers that it began with");
        // The step that is loaded next, and where to begin anew for the steps before `turn`.
        constexpr unsigned kNever = ~0u;
        unsigned ahead, again;
        const auto start = [&](const Job& job) {
            begin(job);
            ahead = job.turn * A::S;
            again = job.turn ? job.depth : kNever;
        };
        const auto advance = [&](const Job& job) {
            if (__builtin_expect(ahead >= again, 0)) {
                begin(job);
                ahead = 0;
                again = kNever;
            }
            aim(ahead);
            ahead += A::S;
        };
        Job job, after;
        if (!jobs.next(&job)) return;
        start(job);
        advance(job);
        for (int q = 0; q < LOADS; ++q) load(lds, q);
        arrive(lds);
        meet();
        advance(job);
        for (int q = 0; q < LOADS; ++q) load(lds + STAGE, q);
#pragma unroll
        for (int r = 0; r < READS; ++r) read(lds, 0, r);
        int at = 0;
        for (bool more = true; more;) {
#pragma unroll
            for (int i = 0; i < FI; ++i)
#pragma unroll
                for (int j = 0; j < FJ; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
            // (two steps at least, so that the loads are never more than one tile ahead)
            unsigned left = uniform((job.depth + A::S - 1) / A::S);
            left = left < 2 ? 2 : left;
            for (; left; --left) {
                const lds_t now = lds + at, next = lds + (at ^= STAGE);
#pragma unroll
                for (int p = 0; p < PARTS - 1; ++p)
                    multiply(p, [&](int i) {   // (in the part's first half)
                        constexpr int HALF = SLOTS > 1 ? SLOTS / 2 : 1;
                        if (i < HALF)
#pragma unroll
                            for (int r = i * READS / HALF; r < (i + 1) * READS / HALF; ++r)
                                read(now, p + 1, r);
                    });
                arrive(next);
                meet();
                if (__builtin_expect(left == 2, 0)) {
                    more = jobs.next(&after);
                    if (more) {
                        start(after);
                    } else {
                        feed_a.end();
                        feed_b.end();
                        ahead = 0;
                        again = kNever;
                    }
                }
                advance(left > 2 ? job : after);
                multiply(PARTS - 1, [&](int i) {
#pragma unroll
                    for (int r = i * READS / SLOTS; r < (i + 1) * READS / SLOTS; ++r) read(next, 0, r);
#pragma unroll
                    for (int q = i * LOADS / SLOTS; q < (i + 1) * LOADS / SLOTS; ++q) load(now, q);
                });
            }
            const bool part = jobs.a.parts > 1;
#pragma unroll
            for (int i = 0; i < FI; ++i) {
                const unsigned row = job.i0 + wi + 16 * WI * i + (lane & 15);
                const unsigned col = job.j0 + wj;
                if constexpr (EB == 2 && FJ % 2 == 0) {
                    if (__builtin_expect(!part, 1)) {
#pragma unroll
                        for (int j = 0; j < FJ; j += 2) {
                            const u32x4 u = pair(acc[i][j], acc[i][j + 1]);
                            const unsigned at = col + 16 * j + 16 * (lane >> 4 & 1) + 8 * (lane >> 5);
                            if (row < job.rows)
                                st_unit_of<2>(job.c + (size_t)row * job.cols * 2, at, job.cols, u);
                        }
                        continue;
                    }
                }
                if (row < job.rows)
#pragma unroll
                    for (int j = 0; j < FJ; ++j)
                        store<EB>(job, part, row, col + 16 * j + 4 * (lane >> 4), acc[i][j]);
            }
            job = after;
        }
    }
};

// Consecutive blocks go to the 8 dies in turn, each with an L2 of its own: die
// d takes a run of the tiles, [d * per, (d + 1) * per).  Past the last: -1.
constexpr int kDies = 8;
__device__ __forceinline__ int tile_of(unsigned id, unsigned total) {
    const unsigned per = (total + kDies - 1) / kDies;
    const unsigned at = id % kDies * per + id / kDies;
    return id / kDies < per && at < total ? (int)at : -1;
}

// In a run, tiles next to each other make a patch of the result kPatch tiles
// high, so that those in flight on a die share lines of both operands.
constexpr unsigned kPatch = 4;
__device__ __forceinline__ void patch(unsigned at, unsigned down, unsigned across, unsigned* i,
                                      unsigned* j) {
    const unsigned g = at / (kPatch * across), rest = at - g * kPatch * across;
    const unsigned high = down - g * kPatch < kPatch ? down - g * kPatch : kPatch;
    *i = g * kPatch + rest % high;
    *j = rest / high;
}

// The groups of rows: expert e has [begin[e], end(e)), whatever the offsets hold
// inside [0, nrows] and with the first row in group 0; group `experts` is the rows behind the last expert.  tiles[e]
// are those of the groups up to e, each group beginning a tile of its own.
constexpr int kGroups = 1024 + 1;
struct Groups {
    int begin[kGroups + 1], tiles[kGroups];
    __device__ __forceinline__ int end(int e) const { return max(begin[e], begin[e + 1]); }
    // (called by the whole block; `height` rows a tile)
    __device__ __forceinline__ void fill(const ProductArgs& a, int height) {
        const int n = (int)a.nrows;
        for (int e = threadIdx.x; e <= a.experts + 1; e += blockDim.x) {
            const int o = e == 0 ? 0 : e <= a.experts ? a.offsets[e] : n;
            begin[e] = o < 0 ? 0 : o < n ? o : n;
        }
        __syncthreads();
        const int lane = threadIdx.x;
        if (lane < 64) {
            int run = 0;
            for (int e0 = 0; e0 <= a.experts; e0 += 64) {
                const int e = e0 + lane, rows = e <= a.experts ? end(e) - begin[e] : 0;
                int inc = rows / height + (rows % height ? 1 : 0);
#pragma unroll
                for (int d = 1; d < 64; d <<= 1) {
                    const int o = __shfl_up(inc, d, 64);
                    if (lane >= d) inc += o;
                }
                if (e <= a.experts) tiles[e] = run + inc;
                run += __builtin_amdgcn_readlane(inc, 63);
            }
        }
        __syncthreads();
    }
    // The group of tile `index` < tiles[experts].
    __device__ __forceinline__ int of(int index, int experts) const {
        const int lane = threadIdx.x & 63;
        for (int e0 = 0;; e0 += 64) {
            const bool past = e0 + lane > experts || tiles[e0 + lane] > index;
            const unsigned long long m = __ballot(past);
            if (m) return e0 + __builtin_ctzll(m);
        }
    }
};

// The arguments, and how many parts the reduced dimension has: more than one
// leave sums in 32 bits to `work`, one result after the other.  turned: whether
// tiles may begin inside their depth (RowJobs), by the sizes alone, so that
// the order of a sum does not depend on where the operands lie.
struct PartArgs : ProductArgs {
    unsigned parts;
    bool turned;
};

// The tiles of the rows' products (KIND: forward or drows) that this block has.
template <int EB, ProductKind KIND, int TI, int TJ, int NT, int STEP>
struct RowJobs {
    const PartArgs& a;
    const Groups& groups;
    unsigned id, across, tiles, total;
    __device__ __forceinline__ RowJobs(const PartArgs& args, const Groups& g)
        : a(args), groups(g), id(blockIdx.x) {
        across = (cols() + TJ - 1) / TJ;
        tiles = across * down();
        total = tiles * a.parts;
    }
    __device__ __forceinline__ unsigned cols() const {
        return (unsigned)(KIND == PRODUCT_FORWARD ? a.out : a.hidden);
    }
    __device__ __forceinline__ unsigned down() const {
        return (unsigned)__builtin_amdgcn_readfirstlane(groups.tiles[a.experts]);
    }
    __device__ __forceinline__ bool next(Job* job) {
        for (; id / kDies <= total / kDies; id += gridDim.x) {
            const int at = tile_of(id, total);
            if (at < 0) continue;
            const unsigned p = (unsigned)at / tiles;
            unsigned ti, tj;
            patch((unsigned)at - p * tiles, down(), across, &ti, &tj);
            const int e = groups.of((int)ti, a.experts);
            const int begin = __builtin_amdgcn_readfirstlane(groups.begin[e]);
            const int end = __builtin_amdgcn_readfirstlane(groups.end(e));
            const int before = e ? __builtin_amdgcn_readfirstlane(groups.tiles[e - 1]) : 0;
            const unsigned depth = (unsigned)(KIND == PRODUCT_FORWARD ? a.hidden : a.out);
            job->a = {static_cast<const char*>(a.a), a.astride * EB, (unsigned)end, depth};
            job->c = a.parts == 1 ? static_cast<char*>(a.c)
                                  : reinterpret_cast<char*>(a.work + p * a.nrows * cols());
            job->i0 = (unsigned)begin + (ti - before) * TI;
            job->rows = (unsigned)end;
            job->j0 = tj * TJ;
            job->cols = cols();
            job->depth = depth;
            job->b = {static_cast<const char*>(a.b) + (e < a.experts ? (size_t)e : 0) * a.out * a.hidden * EB,
                      a.hidden * EB, (unsigned)a.out, (unsigned)a.hidden};
            if (a.parts > 1) take_part<EB, true, KIND == PRODUCT_FORWARD>(job, p, a.parts, STEP / EB);
            if (e == a.experts || job->depth == 0) {
                clear<EB, TI, TJ, NT>(*job, a.parts > 1);
                continue;
            }
            // Weights whose lines are whole 2 KiB lie in few of the memory's channels at one
            // place of the depth: neighbours begin at different steps (64 experts of 2 rows,
            // 2048 x 2048 weights 123 us from the first step, 91 so; 40 rows 131 and 115).  Not
            // where lines are of other widths (60 experts of 2 rows, 771 x 1001 weights 23.2 us,
            // 24.9 so), where they read the same lines of many rows (8192^3 787 and 794 us), nor
            // where the neighbours' weights are the rest of the same lines (drows of the 2 rows
            // 125 and 130).
            if (KIND == PRODUCT_FORWARD && a.turned)
                job->turn = tj % ((job->depth + STEP / EB - 1) / (STEP / EB));
            else job->turn = 0;
            id += gridDim.x;
            return true;
        }
        return false;
    }
};

// The tiles of the weights' gradient.
template <int EB, int TI, int TJ, int NT, int STEP>
struct WeightJobs {
    const PartArgs& a;
    const Groups& groups;
    unsigned id, across, down, tiles, total;
    __device__ __forceinline__ WeightJobs(const PartArgs& args, const Groups& g)
        : a(args), groups(g), id(blockIdx.x) {
        across = (unsigned)((a.hidden + TJ - 1) / TJ);
        down = (unsigned)((a.out + TI - 1) / TI);
        tiles = across * down * (unsigned)a.experts;
        total = tiles * a.parts;
    }
    __device__ __forceinline__ bool next(Job* job) {
        for (; id / kDies <= total / kDies; id += gridDim.x) {
            const int at = tile_of(id, total);
            if (at < 0) continue;
            const unsigned p = (unsigned)at / tiles, t = (unsigned)at - p * tiles;
            const unsigned e = t / (across * down);
            unsigned ti, tj;
            patch(t - e * across * down, down, across, &ti, &tj);
            const int begin = __builtin_amdgcn_readfirstlane(groups.begin[e]);
            const int end = __builtin_amdgcn_readfirstlane(groups.end(e));
            const unsigned n = (unsigned)(end - begin);
            job->a = {static_cast<const char*>(a.a) + (size_t)begin * a.astride * EB,
                      a.astride * EB, n, (unsigned)a.out};
            job->b = {static_cast<const char*>(a.b) + (size_t)begin * a.bstride * EB,
                      a.bstride * EB, n, (unsigned)a.hidden};
            const size_t each = a.out * a.hidden;
            job->c = a.parts == 1 ? static_cast<char*>(a.c) + e * each * EB
                                  : reinterpret_cast<char*>(a.work + (p * a.experts + e) * each);
            job->i0 = ti * TI;
            job->rows = (unsigned)a.out;
            job->j0 = tj * TJ;
            job->cols = (unsigned)a.hidden;
            job->depth = n;
            if (a.parts > 1) take_part<EB, false, false>(job, p, a.parts, STEP / EB);
            if (job->depth == 0) {
                clear<EB, TI, TJ, NT>(*job, a.parts > 1);
                continue;
            }
            job->turn = 0;
            id += gridDim.x;
            return true;
        }
        return false;
    }
};

// The shapes of a block's tile: TI x TJ, WI x WJ wavefronts, steps of STEP bytes,
// EACH blocks a compute unit.
template <int TI_, int TJ_, int WI_, int WJ_, int STEP_, int EACH_>
struct Shape {
    static constexpr int TI = TI_, TJ = TJ_, WI = WI_, WJ = WJ_, STEP = STEP_, EACH = EACH_;
    static constexpr int NT = WI * WJ * 64;
};
using Large = Shape<256, 256, 2, 4, 128, 1>;
using Middle = Shape<128, 128, 2, 2, 128, 2>;
using Small = Shape<32, 64, 1, 4, 256, 2>;
// (drows of few rows reads 256 bytes of each line of weights, not 128: 64 experts of 2 rows,
// 2048 x 2048 weights 126 us by Small, 96 so; but for few tiles, 4 experts of 50 rows,
// 4096 x 4096 weights 27 us by Small, 40 so)
using Flat = Shape<32, 128, 1, 4, 128, 2>;

template <int EB, ProductKind KIND, bool AS, bool BS, class SHAPE>
__global__ __launch_bounds__(SHAPE::NT, SHAPE::EACH * SHAPE::NT / 256) void k_product(
    const PartArgs a) {
    using BLOCK = Block<EB, KIND != PRODUCT_DWEIGHTS, KIND == PRODUCT_FORWARD, AS, BS, SHAPE::TI,
                        SHAPE::TJ, SHAPE::WI, SHAPE::WJ, SHAPE::STEP>;
    __shared__ __attribute__((aligned(1024))) char lds[2 * BLOCK::STAGE];
    __shared__ Groups groups;
    groups.fill(a, SHAPE::TI);
    if constexpr (KIND == PRODUCT_DWEIGHTS) {
        WeightJobs<EB, SHAPE::TI, SHAPE::TJ, SHAPE::NT, SHAPE::STEP> jobs(a, groups);
        BLOCK::run((lds_t)lds, jobs);
    } else {
        RowJobs<EB, KIND, SHAPE::TI, SHAPE::TJ, SHAPE::NT, SHAPE::STEP> jobs(a, groups);
        BLOCK::run((lds_t)lds, jobs);
    }
}

// The sum of the parts, each n elements.
template <int EB>
__global__ __launch_bounds__(256) void k_product_join(const float* part, unsigned parts, size_t n,
                                                      char* c) {
    constexpr int E = Vec<EB>::E;
    for (size_t i = ((size_t)blockIdx.x * 256 + threadIdx.x) * E; i < n;
         i += (size_t)gridDim.x * 256 * E) {
        float sum[E] = {};
        for (unsigned p = 0; p < parts; ++p) {
            const char* from = reinterpret_cast<const char*>(part + p * n);
#pragma unroll
            for (int h = 0; h < E / 4; ++h) {
                const u32x4 u = ld_unit_of<4>(from, i + 4 * h, n, 0u);
#pragma unroll
                for (int j = 0; j < 4; ++j) sum[4 * h + j] += as_f32(u[j]);
            }
        }
        st_unit_of<EB>(c, i, n, Vec<EB>::pack(sum));
    }
}

// Tiles of `height` rows that nrows rows in experts + 1 groups make at most.
size_t most_row_tiles(size_t nrows, int experts, size_t height) {
    const size_t full = (nrows + ((size_t)experts + 1) * (height - 1)) / height;
    return full < nrows ? full : nrows;
}

// Blocks that walk `tiles` tiles, `each` of them on a compute unit at a time.
constexpr size_t kUnits = 256;
unsigned blocks_of(size_t tiles, size_t each) {
    const size_t b = (tiles + kDies - 1) / kDies * kDies;
    return (unsigned)(b < kUnits * each ? b : kUnits * each);
}

template <int EB, ProductKind KIND, bool AS, bool BS, class SHAPE>
hipError_t launch(const PartArgs& a, hipStream_t s) {
    const size_t cols = KIND == PRODUCT_FORWARD ? a.out : a.hidden;
    const size_t high = KIND == PRODUCT_DWEIGHTS
                            ? (a.out + SHAPE::TI - 1) / SHAPE::TI * a.experts
                            : most_row_tiles(a.nrows, a.experts, SHAPE::TI);
    const size_t tiles = high * ((cols + SHAPE::TJ - 1) / SHAPE::TJ) * a.parts;
    if (tiles > size_t(INT_MAX) - 64 * kUnits) return hipErrorInvalidValue;   // (no memory holds them)
    hipLaunchKernelGGL((k_product<EB, KIND, AS, BS, SHAPE>), dim3(blocks_of(tiles, SHAPE::EACH)),
                       dim3(SHAPE::NT), 0, s, a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || a.parts == 1) return e;
    const size_t n = (KIND == PRODUCT_DWEIGHTS ? a.out * a.experts : a.nrows) * cols;
    const size_t blocks = (n + 256 * (16 / EB) - 1) / (256 * (16 / EB));
    hipLaunchKernelGGL(k_product_join<EB>, dim3((unsigned)(blocks < 4096 ? blocks : 4096)), dim3(256), 0,
                       s, a.work, a.parts, n, static_cast<char*>(a.c));
    return hipGetLastError();
}

// Lines of fp32 are always for Straight; those of bf16 where they are an even
// number of elements apart, at 4-byte addresses.
template <int EB, ProductKind KIND, class SHAPE>
hipError_t by_lines(const PartArgs& a, hipStream_t s) {
    if constexpr (EB == 4) return launch<EB, KIND, true, true, SHAPE>(a, s);
    else {
        const auto even = [](const void* p, size_t stride) {
            return reinterpret_cast<uintptr_t>(p) % 4 == 0 && stride % 2 == 0;
        };
        const bool as = even(a.a, a.astride);
        const bool bs = even(a.b, KIND == PRODUCT_DWEIGHTS ? a.bstride : a.hidden);
        if (as && bs) return launch<EB, KIND, true, true, SHAPE>(a, s);
        if constexpr (SHAPE::TI == 256) return by_lines<EB, KIND, Middle>(a, s);
        else if (as) return launch<EB, KIND, true, false, SHAPE>(a, s);
        else if (bs) return launch<EB, KIND, false, true, SHAPE>(a, s);
        else return launch<EB, KIND, false, false, SHAPE>(a, s);
    }
}

// How a product is computed: the tile's shape and the parts of its depth, from the
// time that each would take.  A block's tile takes `each` us and `step` us for a
// step; `alone` where a compute unit has one block.
struct Cost {
    int ti, tj, step_bytes, blocks;
    double each, step, alone;
};
// (fitted on MI355X to times of each shape alone, between 1 tile and 8 a compute unit
// and between 8 and 128 steps, weights in the last-level cache where they fit.  The
// shapes' sides: 64 experts of 40 rows, 2048 -> 2048, drows 104 us in 128 x 128, 166 in
// 32 x 64; 4 experts of 50 rows, 4096 -> 4096, 45 and 27)
constexpr Cost kCosts[2][2][4] = {
    // bf16, lines for Straight; and through registers
    {{{256, 256, 128, 1, 6.0, 1.4, 1.4}, {128, 128, 128, 2, 4.0, 1.0, 0.62}, {32, 64, 256, 2, 3.5, 0.62, 0.6},
      {32, 128, 128, 2, 3.5, 0.5, 0.3}},
     {{256, 256, 128, 1, 6.0, 9.0, 9.0}, {128, 128, 128, 2, 4.0, 1.5, 1.0}, {32, 64, 256, 2, 3.5, 1.0, 0.9},
      {32, 128, 128, 2, 3.5, 0.6, 0.45}}},
    // fp32
    {{{256, 256, 128, 1, 6.0, 99.0, 99.0}, {128, 128, 128, 2, 4.0, 3.7, 1.95}, {32, 64, 256, 2, 3.5, 1.13, 0.7},
      {32, 128, 128, 2, 3.5, 1.18, 0.76}},
     {{256, 256, 128, 1, 6.0, 99.0, 99.0}, {128, 128, 128, 2, 4.0, 3.7, 1.95}, {32, 64, 256, 2, 3.5, 1.13, 0.7},
      {32, 128, 128, 2, 3.5, 1.18, 0.76}}}};

struct Plan {
    int shape;
    unsigned parts;
};

Plan plan_of(ProductKind kind, size_t nrows, int experts, size_t hidden, size_t out, int eb) {
    // (rows are taken as spread evenly over the experts that can have some)
    const size_t used = nrows < (size_t)experts ? (nrows ? nrows : 1) : (size_t)experts;
    const size_t rows = (nrows + used - 1) / used;
    const size_t cols = kind == PRODUCT_FORWARD ? out : hidden;
    const size_t depth = kind == PRODUCT_FORWARD ? hidden : kind == PRODUCT_DROWS ? out : rows;
    const size_t results = kind == PRODUCT_DWEIGHTS ? (size_t)experts * out * hidden : nrows * cols;
    const bool odd = eb == 2 && (hidden % 2 || (kind != PRODUCT_FORWARD && out % 2));
    Plan best{1, 1};
    double least = 1e300;
    for (int i = 0; i < (kind == PRODUCT_DROWS ? 4 : 3); ++i) {
        const Cost& c = kCosts[eb == 4][odd][i];
        const size_t down = kind == PRODUCT_DWEIGHTS ? (out + c.ti - 1) / c.ti * (size_t)experts
                                                     : (rows + c.ti - 1) / c.ti * used;
        const double tiles = (double)down * ((cols + c.tj - 1) / c.tj);
        const size_t steps = (depth * eb + c.step_bytes - 1) / c.step_bytes;
        for (unsigned parts = 1; parts <= 16; parts *= 2) {
            if (parts > 1 && steps < 4 * parts) break;
            const size_t n = (steps + parts - 1) / parts;
            const double all = tiles * parts;
            const double rounds = std::ceil(all / (kUnits * c.blocks));
            double t = rounds * (c.each + (n < 2 ? 2 : n) * (all <= kUnits ? c.alone : c.step));
            // (a launch, and the parts' traffic at 4 TB/s)
            if (parts > 1) t += 4.0 + results * (8.0 * parts) / 4e6;
            if (t < least * 0.97) {
                least = t;
                best = {i, parts};
            }
        }
    }
    return best;
}

template <int EB, ProductKind KIND>
hipError_t launch(const ProductArgs& a, hipStream_t s) {
    const Plan plan = plan_of(KIND, a.nrows, a.experts, a.hidden, a.out, EB);
    PartArgs p;
    static_cast<ProductArgs&>(p) = a;
    p.parts = plan.parts;
    p.turned = plan.shape != 0 && a.hidden * EB % 2048 == 0;
    if (plan.shape == 2) return by_lines<EB, KIND, Small>(p, s);
    if constexpr (KIND == PRODUCT_DROWS)
        if (plan.shape == 3) return by_lines<EB, KIND, Flat>(p, s);
    if constexpr (EB == 2)
        if (plan.shape == 0) return by_lines<EB, KIND, Large>(p, s);
    return by_lines<EB, KIND, Middle>(p, s);
}

}  // namespace

size_t product_work_bytes(ProductKind kind, size_t nrows, int experts, size_t hidden, size_t out,
                          int eb) {
    const unsigned parts = plan_of(kind, nrows, experts, hidden, out, eb).parts;
    if (parts == 1) return 0;
    const size_t rows = kind == PRODUCT_DWEIGHTS ? out * (size_t)experts : nrows;
    return rows * (kind == PRODUCT_FORWARD ? out : hidden) * parts * sizeof(float);
}

hipError_t launch_product(ProductKind kind, const ProductArgs& a, hipStream_t s) {
    if (kind == PRODUCT_DWEIGHTS)
        return a.eb == 2 ? launch<2, PRODUCT_DWEIGHTS>(a, s) : launch<4, PRODUCT_DWEIGHTS>(a, s);
    if (a.nrows == 0) return hipSuccess;
    if (kind == PRODUCT_DROWS)
        return a.eb == 2 ? launch<2, PRODUCT_DROWS>(a, s) : launch<4, PRODUCT_DROWS>(a, s);
    return a.eb == 2 ? launch<2, PRODUCT_FORWARD>(a, s) : launch<4, PRODUCT_FORWARD>(a, s);
}

}  // namespace arlib
