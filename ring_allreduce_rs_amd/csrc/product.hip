// product.hip -- the experts' matrix products over ragged groups of rows, and
// their gradients.
#include "model_ops.h"
#include "ops_device.h"

#include <climits>
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
    //
    // origin() is the place of part 0 of the rows that begin at `first`, a multiple
    // of 16 that the wavefront adds to every piece's; frag() takes it, in one of
    // the buffers, and the piece's own `first` (a constant).  The swaps only change
    // bits that the lines' and buffers' addresses leave 0, so a piece's place is
    // the origin's with some bits turned over, plus a constant.
    static constexpr int kTurn = KC ? 0 : EB == 2 ? 14 : 12;   // units that swaps reach
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

// An operand in memory: `rows` lines of `cols` elements that may be read.
struct Operand {
    const char* base;
    size_t stride;      // bytes
    unsigned rows, cols;
};

// How a tile comes from memory into LDS, a step of the reduced dimension at a
// time.  begin() says where, aim() which step; load() starts share q of N of its
// loads; arrive(), before the wavefronts meet, has them on their way to LDS.

// Through registers, for lines at any address.
template <int EB, class TILE, bool KC, int NT>
struct Through {
    static constexpr int N = TILE::ROWS * TILE::UNITS / NT;
    static_assert(TILE::ROWS * TILE::UNITS % NT == 0, "");
    u32x4 u[N];
    Operand o;
    unsigned first, k;
    __device__ __forceinline__ void begin(const Operand& op, unsigned at, unsigned) {
        o = op;
        first = at;
    }
    __device__ __forceinline__ void end() { o.rows = 0; }
    __device__ __forceinline__ void aim(unsigned step) { k = step; }
    __device__ __forceinline__ void load(lds_t, int q) {
        const int at = q * NT + (int)threadIdx.x;
        const unsigned row = (KC ? first : k) + at / TILE::UNITS;
        const unsigned col = (KC ? k : first) + at % TILE::UNITS * TILE::E;
        u[q] = u32x4{0u, 0u, 0u, 0u};
        if (row < o.rows) u[q] = ld_unit_of<EB>(o.base + row * o.stride, col, o.cols, 0u);
    }
    __device__ __forceinline__ void arrive(lds_t lds) const {
#pragma unroll
        for (int q = 0; q < N; ++q) {
            const int at = q * NT + (int)threadIdx.x;
            *(__attribute__((address_space(3))) u32x4*)(lds + TILE::at(at / TILE::UNITS,
                                                                       at % TILE::UNITS)) = u[q];
        }
    }
};

// (m0 is a register that the compiler keeps for itself: it sets it where it needs it)
#pragma clang diagnostic ignored "-Winline-asm"

// Straight into LDS, for lines of whole 16-byte units at 16-byte addresses whose
// tile spans less than 2 GiB.  A wavefront's load fills 1 KiB of LDS in lane
// order, so the swapping of units is in the addresses that the lanes read; a
// unit outside the operand has an offset past the buffer and loads as zeros.
//
// The load is written out because the compiler takes a transposing read for one
// that may see the load's bytes, and waits for memory before it (the products of
// 8192^3 by dout and by rows 1150 and 1130 us with the builtin, 773 and 816 so).
// It has no register output, and meet() waits for it.
template <int EB, class TILE, bool KC, int NT>
struct Straight {
    static constexpr int N = TILE::ROWS * TILE::UNITS / NT;
    static_assert(TILE::ROWS * TILE::UNITS % NT == 0, "");
    static constexpr unsigned kOutside = 0x80000000u;
    const char* base;
    unsigned off[N];
    unsigned depth;
    size_t stride;
    u32x4 buffer;
    __device__ __forceinline__ static int line(int q, int thread) {
        return (q * NT + thread) / TILE::UNITS;
    }
    __device__ __forceinline__ static int unit(int q, int thread) {   // in memory
        return (q * NT + thread) % TILE::UNITS ^ TILE::swap_of(line(q, thread));
    }
    __device__ __forceinline__ void begin(const Operand& o, unsigned first, unsigned depth_) {
        depth = depth_;
        stride = o.stride;
        base = o.base + (KC ? first * o.stride : first * (size_t)EB);
        const int t = (int)offset_here(threadIdx.x);   // (nothing of it is kept over the steps)
#pragma unroll
        for (int q = 0; q < N; ++q) {
            const bool in = KC ? first + line(q, t) < o.rows : first + unit(q, t) * TILE::E < o.cols;
            off[q] = in ? line(q, t) * (unsigned)o.stride + unit(q, t) * 16 : kOutside;
        }
    }
    __device__ __forceinline__ void end() { depth = 0; }
    __device__ __forceinline__ void aim(unsigned k) {
        const uint64_t at = (uint64_t)(uintptr_t)(base + (KC ? k * (size_t)EB : k * stride));
        buffer = u32x4{(uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)at),
                       (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)(at >> 32)),
                       0x7fffffffu, 0x00020000u};
        if (k + TILE::S > depth) {   // (no step after this one is whole either)
            const int t = (int)offset_here(threadIdx.x);
#pragma unroll
            for (int q = 0; q < N; ++q)
                off[q] = k + (KC ? unit(q, t) * TILE::E : line(q, t)) < depth ? off[q] : kOutside;
        }
    }
    __device__ __forceinline__ void load(lds_t lds, int q) {
        const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        const uint32_t at = (uint32_t)__builtin_amdgcn_readfirstlane(
            (int)((uint32_t)(uintptr_t)lds + (q * NT + wave * 64) * 16));
        asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
                     :: "s"(at), "v"(off[q]), "s"(buffer) : "m0", "memory");
    }
    __device__ __forceinline__ void arrive(lds_t) const {}
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
};

// Fills a tile with zeros.
template <int EB, int TI, int TJ, int NT>
__device__ __forceinline__ void clear(const Job& job) {
    const unsigned high = job.rows - job.i0 < TI ? job.rows - job.i0 : TI;
    for (unsigned at = threadIdx.x; at < high * (TJ / 4); at += NT)
        st4<EB>(job.c + (size_t)(job.i0 + at / (TJ / 4)) * job.cols * EB, job.j0 + at % (TJ / 4) * 4, job.cols,
                f32x4{0.f, 0.f, 0.f, 0.f});
}

// A block's tiles one after another.  AK, BK: the reduced dimension is the
// operand's contiguous one; AS, BS: its lines are for Straight.  JOBS::next gives
// the next job, if there is one.
//
// LDS holds two steps.  A step has four parts, two of its depth by two of the
// wavefront's rows: while one part's pieces are multiplied, the next part's come
// from LDS, one read after each matrix instruction, and before the last part the
// wavefronts meet.  What they wait for there was asked for a whole step ago, and
// nobody reads the other buffer any more, so the loads of the step after the
// next go between the last part's instructions.  The tiles follow one another in
// this without a gap: a tile's last two steps load the first two of the next,
// and its result is stored while these come.
template <int EB, bool AK, bool BK, bool AS, bool BS, int TI, int TJ, int WI, int WJ>
struct Block {
    static constexpr int NT = WI * WJ * 64;
    using A = Tile<EB, AK, TI>;
    using B = Tile<EB, BK, TJ>;
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
        Piece a0[H], a1[H], b0[FJ], b1[FJ];
        const unsigned from_a = A::origin(lane, wi), from_b = A::BYTES + B::origin(lane, wj);
        const auto read_a = [&](Piece (&p)[H], lds_t at, int s, int half, int i) {
            p[i] = A::frag(at + from_a, 16 * WI * (half * H + i), s);
        };
        const auto read_b = [&](Piece (&p)[FJ], lds_t at, int s, int j) {
            p[j] = B::frag(at + from_b, 16 * j, s);
        };
        const auto multiply = [&](const Piece (&pa)[H], const Piece (&pb)[FJ], int half, auto also) {
            __builtin_amdgcn_sched_barrier(0);
            // (the operands change places, so that a lane holds 4 neighbours of a row)
#pragma unroll
            for (int i = 0; i < H; ++i)
#pragma unroll
                for (int j = 0; j < FJ; ++j) {
                    acc[half * H + i][j] = mma(pb[j], pa[i], acc[half * H + i][j]);
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
        Job job, after;
        if (!jobs.next(&job)) return;
        begin(job);
        aim(0);
        for (int q = 0; q < LOADS; ++q) load(lds, q);
        arrive(lds);
        meet();
        aim(A::S);
        for (int q = 0; q < LOADS; ++q) load(lds + STAGE, q);
        for (int i = 0; i < H; ++i) read_a(a0, lds, 0, 0, i);
        for (int j = 0; j < FJ; ++j) read_b(b0, lds, 0, j);
        int at = 0;
        for (bool more = true; more;) {
#pragma unroll
            for (int i = 0; i < FI; ++i)
#pragma unroll
                for (int j = 0; j < FJ; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
            // (two steps at least, so that the loads are never more than one tile ahead)
            unsigned left = (job.depth + A::S - 1) / A::S, ahead = 2 * A::S;
            left = left < 2 ? 2 : left;
            for (; left; --left) {
                const lds_t now = lds + at, next = lds + (at ^= STAGE);
                multiply(a0, b0, 0, [&](int n) {
                    if (n < H) read_a(a1, now, 0, 1, n);
                });
                multiply(a1, b0, 1, [&](int n) {
                    if (n < H) read_a(a0, now, 1, 0, n);
                    else if (n < READS) read_b(b1, now, 1, n - H);
                });
                multiply(a0, b1, 0, [&](int n) {
                    if (n < H) read_a(a1, now, 1, 1, n);
                });
                arrive(next);
                meet();
                if (left == 2) {
                    more = jobs.next(&after);
                    ahead = 0;
                    if (more) {
                        begin(after);
                    } else {
                        feed_a.end();
                        feed_b.end();
                    }
                }
                aim(ahead);
                ahead += A::S;
                multiply(a1, b1, 1, [&](int n) {
                    // READS reads and LOADS loads over the part's SLOTS instructions
#pragma unroll
                    for (int r = n * READS / SLOTS; r < (n + 1) * READS / SLOTS; ++r) {
                        if (r < H) read_a(a0, next, 0, 0, r);
                        else read_b(b0, next, 0, r - H);
                    }
#pragma unroll
                    for (int q = n * LOADS / SLOTS; q < (n + 1) * LOADS / SLOTS; ++q) load(now, q);
                });
            }
#pragma unroll
            for (int i = 0; i < FI; ++i) {
                const unsigned row = job.i0 + wi + 16 * WI * i + (lane & 15);
                if (row < job.rows)
#pragma unroll
                    for (int j = 0; j < FJ; ++j)
                        st4<EB>(job.c + (size_t)row * job.cols * EB, job.j0 + wj + 16 * j + 4 * (lane >> 4),
                                job.cols, acc[i][j]);
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

// The groups of rows: expert e has [begin[e], end[e]), whatever the offsets hold
// inside [0, nrows]; group `experts` is the rows behind the last expert.  tiles[e]
// are those of the groups up to e, each group beginning a tile of its own.
constexpr int kGroups = 1024 + 1;
struct Groups {
    int begin[kGroups], end[kGroups], tiles[kGroups];
    // (called by the whole block; `height` rows a tile)
    __device__ __forceinline__ void fill(const ProductArgs& a, int height) {
        const int lane = threadIdx.x & 63, n = (int)a.nrows;
        if (threadIdx.x < 64) {
            int run = 0;
            for (int e0 = 0; e0 <= a.experts; e0 += 64) {
                const int e = e0 + lane;
                int b = 0, f = 0;
                if (e <= a.experts) {
                    b = a.offsets[e];
                    f = e < a.experts ? a.offsets[e + 1] : n;
                    b = b < 0 ? 0 : b < n ? b : n;
                    f = f < b ? b : f < n ? f : n;
                    begin[e] = b;
                    end[e] = f;
                }
                int inc = (f - b) / height + ((f - b) % height ? 1 : 0);
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

// The tiles of the rows' products (KIND: forward or drows) that this block has.
template <int EB, ProductKind KIND, int TI, int TJ, int NT>
struct RowJobs {
    const ProductArgs& a;
    const Groups& groups;
    unsigned id, across, total;
    __device__ __forceinline__ RowJobs(const ProductArgs& args, const Groups& g)
        : a(args), groups(g), id(blockIdx.x) {
        across = (cols() + TJ - 1) / TJ;
        total = across * down();
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
            unsigned ti, tj;
            patch((unsigned)at, down(), across, &ti, &tj);
            const int e = groups.of((int)ti, a.experts);
            const int begin = __builtin_amdgcn_readfirstlane(groups.begin[e]);
            const int end = __builtin_amdgcn_readfirstlane(groups.end[e]);
            const int before = e ? __builtin_amdgcn_readfirstlane(groups.tiles[e - 1]) : 0;
            const unsigned depth = (unsigned)(KIND == PRODUCT_FORWARD ? a.hidden : a.out);
            job->a = {static_cast<const char*>(a.a), a.astride * EB, (unsigned)end, depth};
            job->c = static_cast<char*>(a.c);
            job->i0 = (unsigned)begin + (ti - before) * TI;
            job->rows = (unsigned)end;
            job->j0 = tj * TJ;
            job->cols = cols();
            job->depth = depth;
            if (e == a.experts) {
                clear<EB, TI, TJ, NT>(*job);
                continue;
            }
            job->b = {static_cast<const char*>(a.b) + (size_t)e * a.out * a.hidden * EB,
                      a.hidden * EB, (unsigned)a.out, (unsigned)a.hidden};
            id += gridDim.x;
            return true;
        }
        return false;
    }
};

// The tiles of the weights' gradient.
template <int EB, int TI, int TJ, int NT>
struct WeightJobs {
    const ProductArgs& a;
    const Groups& groups;
    unsigned id, across, down, total;
    __device__ __forceinline__ WeightJobs(const ProductArgs& args, const Groups& g)
        : a(args), groups(g), id(blockIdx.x) {
        across = (unsigned)((a.hidden + TJ - 1) / TJ);
        down = (unsigned)((a.out + TI - 1) / TI);
        total = across * down * (unsigned)a.experts;
    }
    __device__ __forceinline__ bool next(Job* job) {
        for (; id / kDies <= total / kDies; id += gridDim.x) {
            const int at = tile_of(id, total);
            if (at < 0) continue;
            const unsigned e = (unsigned)at / (across * down);
            unsigned ti, tj;
            patch((unsigned)at - e * across * down, down, across, &ti, &tj);
            const int begin = __builtin_amdgcn_readfirstlane(groups.begin[e]);
            const int end = __builtin_amdgcn_readfirstlane(groups.end[e]);
            const unsigned n = (unsigned)(end - begin);
            job->a = {static_cast<const char*>(a.a) + (size_t)begin * a.astride * EB,
                      a.astride * EB, n, (unsigned)a.out};
            job->b = {static_cast<const char*>(a.b) + (size_t)begin * a.bstride * EB,
                      a.bstride * EB, n, (unsigned)a.hidden};
            job->c = static_cast<char*>(a.c) + (size_t)e * a.out * a.hidden * EB;
            job->i0 = ti * TI;
            job->rows = (unsigned)a.out;
            job->j0 = tj * TJ;
            job->cols = (unsigned)a.hidden;
            job->depth = n;
            if (n == 0) {
                clear<EB, TI, TJ, NT>(*job);
                continue;
            }
            id += gridDim.x;
            return true;
        }
        return false;
    }
};

template <int EB, ProductKind KIND, bool AS, bool BS, int TI, int TJ, int WI, int WJ>
__global__ __launch_bounds__(WI * WJ * 64, 2) void k_product(const ProductArgs a) {
    constexpr int NT = WI * WJ * 64;
    using BLOCK = Block<EB, KIND != PRODUCT_DWEIGHTS, KIND == PRODUCT_FORWARD, AS, BS, TI, TJ, WI, WJ>;
    __shared__ __attribute__((aligned(1024))) char lds[2 * BLOCK::STAGE];
    __shared__ Groups groups;
    groups.fill(a, TI);
    if constexpr (KIND == PRODUCT_DWEIGHTS) {
        WeightJobs<EB, TI, TJ, NT> jobs(a, groups);
        BLOCK::run((lds_t)lds, jobs);
    } else {
        RowJobs<EB, KIND, TI, TJ, NT> jobs(a, groups);
        BLOCK::run((lds_t)lds, jobs);
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

// Whether lines of n elements, `stride` elements apart from p on, are whole
// 16-byte units, and 512 of them span less than 2 GiB.
bool lines(const void* p, size_t n, size_t stride, int eb) {
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && n * eb % 16 == 0 && stride * eb % 16 == 0 &&
           stride * eb < (size_t(1) << 22);
}

template <int EB, ProductKind KIND, bool AS, bool BS, int T, int WI, int WJ>
hipError_t launch(const ProductArgs& a, hipStream_t s) {
    const size_t cols = KIND == PRODUCT_FORWARD ? a.out : a.hidden;
    const size_t high = KIND == PRODUCT_DWEIGHTS ? (a.out + T - 1) / T * a.experts
                                                 : most_row_tiles(a.nrows, a.experts, T);
    const size_t tiles = high * ((cols + T - 1) / T);
    if (tiles > size_t(INT_MAX) - 64 * kUnits) return hipErrorInvalidValue;   // (no memory holds them)
    const unsigned blocks = blocks_of(tiles, T == 256 ? 1 : 2);
    hipLaunchKernelGGL((k_product<EB, KIND, AS, BS, T, T, WI, WJ>), dim3(blocks), dim3(WI * WJ * 64),
                       0, s, a);
    return hipGetLastError();
}

template <int EB, ProductKind KIND>
hipError_t launch(const ProductArgs& a, hipStream_t s) {
    const size_t acols = KIND == PRODUCT_FORWARD ? a.hidden : a.out;
    const bool as = lines(a.a, acols, a.nrows > 1 ? a.astride : acols, a.eb);
    const bool bs = lines(a.b, a.hidden,
                          KIND == PRODUCT_DWEIGHTS && a.nrows > 1 ? a.bstride : a.hidden, a.eb);
    if (as && bs) {
        if constexpr (EB == 2) return launch<EB, KIND, true, true, 256, 2, 4>(a, s);
        else return launch<EB, KIND, true, true, 128, 2, 2>(a, s);
    }
    return launch<EB, KIND, false, false, 128, 2, 2>(a, s);
}

}  // namespace

size_t product_work_bytes(ProductKind, size_t, int, size_t, size_t, int) { return 0; }

hipError_t launch_product(ProductKind kind, const ProductArgs& a, hipStream_t s) {
    if (kind == PRODUCT_DWEIGHTS)
        return a.eb == 2 ? launch<2, PRODUCT_DWEIGHTS>(a, s) : launch<4, PRODUCT_DWEIGHTS>(a, s);
    if (a.nrows == 0) return hipSuccess;
    if (kind == PRODUCT_DROWS)
        return a.eb == 2 ? launch<2, PRODUCT_DROWS>(a, s) : launch<4, PRODUCT_DROWS>(a, s);
    return a.eb == 2 ? launch<2, PRODUCT_FORWARD>(a, s) : launch<4, PRODUCT_FORWARD>(a, s);
}

}  // namespace arlib
