// route.hip -- tokens sorted by expert and back, and the gradients.
//
// Slot i = t * topk + k is token t's k-th choice, with expert ids[i] (anything
// outside [0, experts) means none).  The slots are sorted by expert, stably,
// those without one last:
//   dest[i]     the sorted row that slot i goes to
//   slot[j]     the slot that sorted row j is (the inverse of dest)
//   offsets[e]  the first row of expert e; offsets[experts] = rows with an expert
//   rows[j]     = x[slot[j] / topk], zeros from offsets[experts] on
// and the way back, with weights:
//   y[t] = sum_k w[t,k] rows[dest[t,k]]          (k in order, fp32, rounded once)
//   drows[dest[t,k]] = w[t,k] dy[t],  dw[t,k] = rows[dest[t,k]] . dy[t]
//   dx[t] = sum_k drows[dest[t,k]]
// where a slot without an expert counts for nothing, whatever its row holds.
//
// The sort is a counting sort: its order comes from ballots and prefix sums,
// never from the order in which atomics land.  All traffic is in the rows, and
// every kernel that moves rows walks tokens, so that a token's row is read (or
// written) once and each sorted row is touched by exactly one token.  dest is
// checked against the rows' bounds before it is used as an address.
//
// MI355X: dispatch of 16384 x 8 rows of 2048 bf16 114 us (5.3 TB/s; a copy of as
// many bytes 94), 13 us of it the sort's two launches; both gradients of 8192 x
// 8 rows of 4096 bf16 314 us (5.6 TB/s; 270); combine of 4099 x 6 rows of 1000
// fp32 17.2 us (6.7 TB/s, partly from the last-level cache; 17.8); dispatch of 4
// tokens 6.3 us in one launch, the kernel 3.9.
#include "ops.h"
#include "ops_device.h"

namespace arlib {
namespace {

constexpr int kSortThreads = 1024;
constexpr int kSortWaves = kSortThreads / 64;
constexpr int kSortSteps = 1;                            // slots per thread
constexpr int kSortSlots = kSortThreads * kSortSteps;    // slots per block
constexpr size_t kSortBlocks = 128;                      // at most
constexpr int kMaxExperts = 1024;
constexpr int kBins = kMaxExperts + 1;                   // the last one: no expert

// The bin of slot i.
template <int IB>
__device__ __forceinline__ int bin_of(const void* ids, size_t i, int experts) {
    if constexpr (IB == 8) {
        const int64_t e = static_cast<const int64_t*>(ids)[i];
        return e >= 0 && e < experts ? (int)e : experts;
    } else {
        const int32_t e = static_cast<const int32_t*>(ids)[i];
        return e >= 0 && e < experts ? e : experts;
    }
}

// Lanes of the wavefront whose bin equals this lane's, among the lanes that
// take part.  `bits` ballots tell the bins apart.
__device__ __forceinline__ unsigned long long same_bin(int bin, int bits, bool live) {
    unsigned long long m = __ballot(live);
    for (int b = 0; b < bits; ++b) {
        const bool one = (bin >> b) & 1;
        const unsigned long long v = __ballot(one);
        m &= one ? v : ~v;
    }
    return m;
}

__device__ __forceinline__ int bin_bits(int experts) {
    return 32 - __clz(experts);   // bins 0 .. experts
}

// Orders LDS accesses among the lanes of one wavefront.
__device__ __forceinline__ void wave_lds_order() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// Block b of the sort takes the slots [b * share, (b + 1) * share), in rounds
// of kSortSlots; share is a multiple of that.

// Slots per bin of each block's share: work[bin][block].
template <int IB>
__global__ __launch_bounds__(kSortThreads) void k_route_count(const DispatchArgs a, size_t slots,
                                                              size_t share) {
    __shared__ int cnt[kBins];
    for (int b = threadIdx.x; b <= a.experts; b += kSortThreads) cnt[b] = 0;
    __syncthreads();
    const size_t begin = blockIdx.x * share;
    const size_t end = begin + share < slots ? begin + share : slots;
    for (size_t i = begin + threadIdx.x; i < end; i += kSortThreads)
        atomicAdd(&cnt[bin_of<IB>(a.ids, i, a.experts)], 1);
    __syncthreads();
    for (int b = threadIdx.x; b <= a.experts; b += kSortThreads)
        a.work[(size_t)b * gridDim.x + blockIdx.x] = cnt[b];
}

// v becomes the sum over the lanes up to this one.
__device__ __forceinline__ int wave_scan(int v, int lane) {
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int o = __shfl_up(v, d, 64);
        if (lane >= d) v += o;
    }
    return v;
}

// Where each slot goes.  A block needs, for every bin, the slots in smaller
// bins plus those of the same bin in earlier blocks (from the counts), then in
// earlier rounds and wavefronts of its own, then in earlier lanes.
template <int IB>
__global__ __launch_bounds__(kSortThreads) void k_route_place(const DispatchArgs a, size_t slots,
                                                              size_t share) {
    __shared__ int first[kBins];                       // next free row of each bin
    __shared__ int total[kBins];
    __shared__ unsigned short wcnt[kSortWaves][kBins]; // slots per wavefront and bin
    __shared__ int wsum[kSortWaves];
    const int bins = a.experts + 1, bits = bin_bits(a.experts);
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int nblk = gridDim.x, me = blockIdx.x;

    // the first round's slots (wavefront w takes 64 * kSortSteps in a row) are
    // loaded before the counts that they wait for
    const size_t begin = (size_t)me * share;
    const size_t own = (size_t)(wave * kSortSteps) * 64 + lane;
    int bin[kSortSteps];
    const auto load_bins = [&](size_t round) {
#pragma unroll
        for (int s = 0; s < kSortSteps; ++s) {
            const size_t i = round + own + s * 64;
            bin[s] = i < slots ? bin_of<IB>(a.ids, i, a.experts) : 0;
        }
    };
    load_bins(begin);

    // a wavefront per bin: its slots in all blocks, and in the earlier ones;
    // the loads of kAhead bins are in flight together
    constexpr int kAhead = 12;
    static_assert(kSortBlocks <= 128, "a lane holds two blocks' counts");
    for (int b0 = wave; b0 < bins; b0 += kSortWaves * kAhead) {
        int lo[kAhead], hi[kAhead];
#pragma unroll
        for (int q = 0; q < kAhead; ++q) {
            const int b = b0 + q * kSortWaves;
            const int* w = a.work + (size_t)b * nblk;
            lo[q] = b < bins && lane < nblk ? w[lane] : 0;
            hi[q] = b < bins && lane + 64 < nblk ? w[lane + 64] : 0;
        }
#pragma unroll
        for (int q = 0; q < kAhead; ++q) {
            const int all = wave_sum(lo[q] + hi[q]);
            const int before = wave_sum((lane < me ? lo[q] : 0) + (lane + 64 < me ? hi[q] : 0));
            const int b = b0 + q * kSortWaves;
            if (lane == 0 && b < bins) {
                total[b] = all;
                first[b] = before;
            }
        }
    }
    __syncthreads();
    int run = 0;
    for (int b0 = 0; b0 < bins; b0 += kSortThreads) {
        const int b = b0 + (int)threadIdx.x;
        const int mine = b < bins ? total[b] : 0;
        const int inc = wave_scan(mine, lane);
        if (lane == 63) wsum[wave] = inc;
        __syncthreads();
        int ahead = run;
        for (int w = 0; w < kSortWaves; ++w) {
            if (w < wave) ahead += wsum[w];
            run += wsum[w];
        }
        if (b < bins) {
            first[b] += ahead + inc - mine;
            if (me == 0) a.offsets[b] = ahead + inc - mine;   // bin `experts`: the last row in use
        }
        __syncthreads();
    }

    for (size_t round = begin; round < begin + share && round < slots; round += kSortSlots) {
        if (round != begin) load_bins(round);
        for (int b = lane; b < bins; b += 64) wcnt[wave][b] = 0;
        wave_lds_order();
        int rank[kSortSteps];
#pragma unroll
        for (int s = 0; s < kSortSteps; ++s) {
            const bool live = round + own + s * 64 < slots;
            const unsigned long long m = same_bin(bin[s], bits, live);
            const int below = __popcll(m & ((1ull << lane) - 1));
            const int had = wcnt[wave][bin[s]];
            rank[s] = had + below;
            wave_lds_order();   // all lanes have read before the bin's first lane writes
            if (live && below == 0) wcnt[wave][bin[s]] = (unsigned short)(had + __popcll(m));
            wave_lds_order();
        }
        __syncthreads();
        // per bin: slots of earlier wavefronts in place of each one's own
        int sum[(kBins + kSortThreads - 1) / kSortThreads];
#pragma unroll
        for (int q = 0; q < (kBins + kSortThreads - 1) / kSortThreads; ++q) {
            const int b = q * kSortThreads + (int)threadIdx.x;
            sum[q] = 0;
            if (b < bins) {
                int c[kSortWaves];
#pragma unroll
                for (int w = 0; w < kSortWaves; ++w) c[w] = wcnt[w][b];
#pragma unroll
                for (int w = 0; w < kSortWaves; ++w) {
                    wcnt[w][b] = (unsigned short)sum[q];
                    sum[q] += c[w];
                }
            }
        }
        __syncthreads();
#pragma unroll
        for (int s = 0; s < kSortSteps; ++s) {
            const size_t i = round + own + s * 64;
            if (i >= slots) continue;
            const int d = first[bin[s]] + wcnt[wave][bin[s]] + rank[s];
            a.dest[i] = d;
            a.slot[d] = (int)i;
        }
        __syncthreads();
        // the next round's rows come after this one's
#pragma unroll
        for (int q = 0; q < (kBins + kSortThreads - 1) / kSortThreads; ++q) {
            const int b = q * kSortThreads + (int)threadIdx.x;
            if (b < bins) first[b] += sum[q];
        }
    }
}

// ------------------------------------------------------------------- moving rows
//
// A block of NT threads per token, so that what belongs to the token (its
// sorted rows, its weights) is uniform: scalar registers hold the rows'
// addresses, and the loads of KB choices are in flight together.

// A token's row to each of its sorted rows.
template <int EB, int NT, RowMode MODE>
__global__ __launch_bounds__(NT) void k_route_rows(const DispatchArgs a) {
    const int live = ld_uniform(a.offsets + a.experts);
    for (size_t t = blockIdx.x; t < (size_t)a.tokens; t += gridDim.x) {
        const char* x = static_cast<const char*>(a.x) + t * a.xstride * EB;
        using IO = RowIO<EB, MODE, false>;
        const unsigned hidden = (unsigned)a.hidden, units = (hidden + IO::E - 1) / IO::E;
        const size_t n = (size_t)a.tokens * a.topk;
        for (unsigned i = threadIdx.x; i < units; i += NT) {
            const Place p = IO::place(i, hidden);
            const u32x4 u = IO::ld(x, p, hidden);
            const u32x4 z = {0u, 0u, 0u, 0u};
            for (int k = 0; k < a.topk; ++k) {
                const int d = ld_uniform(a.dest + t * a.topk + k);
                if ((size_t)d >= n) continue;
                IO::st(static_cast<char*>(a.rows) + (size_t)d * a.hidden * EB, p, hidden,
                       d < live ? u : z);
            }
        }
    }
}

// The whole dispatch in one launch, for few slots: the last block counts the
// experts' rows, every other block finds where its token's choices go by
// comparing them with every slot, then copies.
template <int EB, int IB, int NT, RowMode MODE>
__global__ __launch_bounds__(NT) void k_route_direct(const DispatchArgs a, int slots) {
    constexpr int W = NT / 64, KB = 8;
    __shared__ int lds[2][W * KB];
    __shared__ int cnt[kBins];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    if ((int)blockIdx.x == a.tokens) {
        for (int b = threadIdx.x; b <= a.experts; b += NT) cnt[b] = 0;
        __syncthreads();
        for (int i = threadIdx.x; i < slots; i += NT)
            atomicAdd(&cnt[bin_of<IB>(a.ids, i, a.experts)], 1);
        __syncthreads();
        if (wave == 0) {
            int run = 0;
            for (int b0 = 0; b0 <= a.experts; b0 += 64) {
                const int mine = b0 + lane <= a.experts ? cnt[b0 + lane] : 0;
                const int inc = wave_scan(mine, lane);
                if (b0 + lane <= a.experts) a.offsets[b0 + lane] = run + inc - mine;
                run += __builtin_amdgcn_readlane(inc, 63);
            }
        }
        return;
    }
    const size_t t = blockIdx.x;
    using IO = RowIO<EB, MODE, false>;
    const unsigned hidden = (unsigned)a.hidden, units = (hidden + IO::E - 1) / IO::E;
    const char* x = static_cast<const char*>(a.x) + t * a.xstride * EB;
    // the row's first units come while the slots are compared
    const Place mine = IO::place(threadIdx.x < units ? threadIdx.x : 0, hidden);
    const u32x4 held = IO::ld(x, mine, hidden);
    int buf = 0;
    for (int k0 = 0; k0 < a.topk; k0 += KB, buf ^= 1) {
        const int i0 = (int)t * a.topk + k0;
        int bin[KB], before[KB];
#pragma unroll
        for (int k = 0; k < KB; ++k) {
            bin[k] = k0 + k < a.topk ? bin_of<IB>(a.ids, i0 + k, a.experts) : -1;
            before[k] = 0;
        }
        for (int i = threadIdx.x; i < slots; i += NT) {
            const int e = bin_of<IB>(a.ids, i, a.experts);
#pragma unroll
            for (int k = 0; k < KB; ++k) before[k] += e < bin[k] || (e == bin[k] && i < i0 + k);
        }
#pragma unroll
        for (int k = 0; k < KB; ++k) {
            before[k] = wave_sum(before[k]);
            if (W > 1 && lane == 0) lds[buf][wave * KB + k] = before[k];
        }
        if constexpr (W > 1) {
            __syncthreads();
#pragma unroll
            for (int k = 0; k < KB; ++k) {
                before[k] = 0;
#pragma unroll
                for (int w = 0; w < W; ++w) before[k] += lds[buf][w * KB + k];
            }
        }
#pragma unroll
        for (int k = 0; k < KB; ++k)
            if (threadIdx.x == 0 && k0 + k < a.topk) {
                a.dest[i0 + k] = before[k];
                a.slot[before[k]] = i0 + k;
            }
        for (unsigned i = threadIdx.x; i < units; i += NT) {
            const Place p = IO::place(i, hidden);
            const u32x4 u = i < NT ? held : IO::ld(x, p, hidden), z = {0u, 0u, 0u, 0u};
#pragma unroll
            for (int k = 0; k < KB; ++k)
                if (k0 + k < a.topk)
                    IO::st(static_cast<char*>(a.rows) + (size_t)before[k] * a.hidden * EB, p, hidden,
                           bin[k] < a.experts ? u : z);
        }
    }
}

// y[t] = sum_k w[t,k] rows[dest[t,k]]
template <int EB, int NT, int KB, RowMode MODE, bool STREAM>
__global__ __launch_bounds__(NT) void k_route_combine(const CombineArgs a) {
    using IO = RowIO<EB, MODE, STREAM>;
    constexpr int E = IO::E;
    const unsigned hidden = (unsigned)a.hidden, units = (hidden + E - 1) / E;
    const int n = a.tokens * a.topk;
    const int live = min(ld_uniform(a.offsets + a.experts), n);
    for (size_t t = blockIdx.x; t < (size_t)a.tokens; t += gridDim.x) {
        char* y = static_cast<char*>(a.y) + t * a.hidden * EB;
        for (unsigned i = threadIdx.x; i < units; i += NT) {
            const Place p = IO::place(i, hidden);
            float acc[E] = {};
            for (int k0 = 0; k0 < a.topk; k0 += KB) {
                u32x4 raw[KB];
                float w[KB];
#pragma unroll
                for (int k = 0; k < KB; ++k) {
                    const size_t s = t * a.topk + k0 + k;
                    const int d = k0 + k < a.topk ? ld_uniform(a.dest + s) : -1;
                    raw[k] = u32x4{0u, 0u, 0u, 0u};
                    w[k] = 0.0f;
                    if (d >= 0 && d < live) {   // (the same for the whole block)
                        raw[k] = IO::ld(static_cast<const char*>(a.rows) +
                                            (size_t)d * a.hidden * EB, p, hidden);
                        w[k] = a.weights ? ld_uniform(a.weights + s) : 1.0f;
                    }
                }
#pragma unroll
                for (int k = 0; k < KB; ++k) {
                    float v[E];
                    Vec<EB>::unpack(raw[k], v);
#pragma unroll
                    for (int j = 0; j < E; ++j) acc[j] = __builtin_fmaf(v[j], w[k], acc[j]);
                }
            }
            IO::st(y, p, hidden, Vec<EB>::pack(acc));
        }
    }
}

// drows and dweights: the token's gradient is read once for KB choices.
template <int EB, int NT, int KB, RowMode MODE>
__global__ __launch_bounds__(NT) void k_route_combine_grad(const CombineArgs a) {
    using IO = RowIO<EB, MODE, true>;
    constexpr int E = IO::E, W = NT / 64;
    __shared__ float lds[2][W * KB];
    const unsigned hidden = (unsigned)a.hidden, units = (hidden + E - 1) / E;
    const int n = a.tokens * a.topk;
    const int live = min(ld_uniform(a.offsets + a.experts), n);
    int buf = 0;
    for (size_t t = blockIdx.x; t < (size_t)a.tokens; t += gridDim.x) {
        const char* dy = static_cast<const char*>(a.dy) + t * a.dystride * EB;
        for (int k0 = 0; k0 < a.topk; k0 += KB, buf ^= 1) {
            float dot[KB];
#pragma unroll
            for (int k = 0; k < KB; ++k) dot[k] = 0.0f;
            for (unsigned i = threadIdx.x; i < units; i += NT) {
                const Place p = IO::place(i, hidden);
                // (dy through the caches, the rows past them: both gradients of 8192 x 8
                // rows of 4096 bf16 314 us, 330 with dy past them too)
                u32x4 raw[KB], rg = RowIO<EB, MODE, false>::ld(dy, p, hidden);
#pragma unroll
                for (int k = 0; k < KB; ++k) {
                    const int d = k0 + k < a.topk ? ld_uniform(a.dest + t * a.topk + k0 + k) : -1;
                    raw[k] = u32x4{0u, 0u, 0u, 0u};
                    if (d >= 0 && d < live)
                        raw[k] = IO::ld(static_cast<const char*>(a.rows) +
                                            (size_t)d * a.hidden * EB, p, hidden);
                }
                if (MODE == ROW_RAGGED && p.skip) {
                    rg = drop_first<EB, true>(rg, p.skip);
                    // (an infinity there would make NaN of the dropped 0)
#pragma unroll
                    for (int k = 0; k < KB; ++k) raw[k] = drop_first<EB, true>(raw[k], p.skip);
                }
                float g[E];
                Vec<EB>::unpack(rg, g);
#pragma unroll
                for (int k = 0; k < KB; ++k) {
                    const size_t s = t * a.topk + k0 + k;
                    const int d = k0 + k < a.topk ? ld_uniform(a.dest + s) : -1;
                    if (d < 0 || d >= n) continue;
                    u32x4 out = {0u, 0u, 0u, 0u};
                    if (d < live) {
                        const float w = ld_uniform(a.weights + s);
                        float v[E];
                        Vec<EB>::unpack(raw[k], v);
#pragma unroll
                        for (int j = 0; j < E; ++j) {
                            dot[k] = __builtin_fmaf(g[j], v[j], dot[k]);
                            v[j] = g[j] * w;
                        }
                        out = Vec<EB>::pack(v);
                    }
                    IO::st(static_cast<char*>(a.drows) + (size_t)d * a.hidden * EB, p, hidden, out);
                }
            }
            block_sums<KB>(dot, lds[buf], W);
#pragma unroll
            for (int k = 0; k < KB; ++k)
                if (threadIdx.x == 0 && k0 + k < a.topk) {
                    const size_t s = t * a.topk + k0 + k;
                    const int d = a.dest[s];
                    a.dweights[s] = d >= 0 && d < live ? dot[k] : 0.0f;
                }
        }
    }
}

// Blocks of a launch over tokens (the kernels walk the rest).
unsigned token_blocks(int tokens) {
    constexpr int kMost = 1 << 22;
    return (unsigned)(tokens < kMost ? tokens : kMost);
}

// Threads of a token's block: a row's units, at most 512, or 1024 while there
// are fewer tokens than compute units (both gradients of 8192 x 8 rows of 4096
// bf16 323 us with 512 threads, 329 with 256; of 56 x 4 rows of 5742 fp32 11.7 us
// with 1024, 19.3 with 256).
int token_threads(size_t tokens, size_t hidden, int eb) {
    const size_t units = (hidden * eb + 15) / 16;
    return units <= 64 ? 64 : units <= 128 ? 128 : units <= 256 ? 256 : tokens > 256 ? 512 : 1024;
}

// The direct form's comparisons: every token with every slot, 8 choices at a
// time.  Up to kDirectWork of them it is one launch where the sort takes three
// (652 x 5 slots 9.2 us against 12.7, 859 x 2 6.6 against 11.1; past it 1024 x 8
// would take 19.5 against 16.5).
constexpr size_t kDirectWork = size_t(1) << 25;
bool direct_form(size_t tokens, size_t topk) {
    const size_t slots = tokens * topk;
    return slots <= 16384 && slots * tokens * ((topk + 7) / 8 * 8) <= kDirectWork;
}

// Combine (and dispatch's gradient) reads rows of more bytes than this past the
// caches: they would only push each other out of the 256 MB last-level cache
// (MI355X, rows of 537 MB: 98 us against 106; rows of 98 MB that are still in
// it: 19.5 us past it, 16.9 through it).  Combine's gradient, which writes as
// many rows as it reads, always reads past them; that was measured for rows of
// 537 MB alone.
constexpr size_t kStreamBytes = size_t(192) << 20;

// The sort's split: as many blocks as there are kSortSlots, at most kSortBlocks
// (each block adds up the counts of all of them).
size_t sort_share(size_t slots) {
    const size_t rounds = (slots + kSortSlots - 1) / kSortSlots;
    const size_t each = (rounds + kSortBlocks - 1) / kSortBlocks;
    return (each ? each : 1) * kSortSlots;
}
int sort_blocks(size_t slots) {
    const size_t share = sort_share(slots);
    const size_t b = (slots + share - 1) / share;
    return b ? (int)b : 1;
}

// CALL(EB, NT, MODE) with the types and sizes of `a`.
#define BY_MODE(EB, NT, CALL)                              \
    do {                                                   \
        if (mode == ROW_FULL) { CALL(EB, NT, ROW_FULL); }  \
        else if (mode == ROW_RAGGED) { CALL(EB, NT, ROW_RAGGED); } \
        else { CALL(EB, NT, ROW_SHORT); }                  \
    } while (0)
#define BY_WIDTH(EB, CALL)                  \
    do {                                    \
        if (nt == 64) BY_MODE(EB, 64, CALL); \
        else if (nt == 128) BY_MODE(EB, 128, CALL); \
        else if (nt == 256) BY_MODE(EB, 256, CALL); \
        else if (nt == 512) BY_MODE(EB, 512, CALL); \
        else BY_MODE(EB, 1024, CALL);       \
    } while (0)
#define BY_ROW(CALL)                                        \
    do {                                                    \
        const int nt = token_threads((size_t)a.tokens, a.hidden, a.eb); \
        const RowMode mode = row_mode(a.hidden, a.eb);      \
        if (a.eb == 2) BY_WIDTH(2, CALL);                   \
        else BY_WIDTH(4, CALL);                             \
    } while (0)

// The direct form's blocks walk all slots, so they have 256 threads at least.
#define BY_ROW_WIDE(CALL)                                                       \
    do {                                                                        \
        const int nt = token_threads((size_t)a.tokens, a.hidden, a.eb);         \
        const RowMode mode = row_mode(a.hidden, a.eb);                          \
        if (a.eb == 2 && nt <= 512) BY_MODE(2, 256, CALL);                      \
        else if (a.eb == 2) BY_MODE(2, 1024, CALL);                             \
        else if (nt <= 512) BY_MODE(4, 256, CALL);                              \
        else BY_MODE(4, 1024, CALL);                                            \
    } while (0)

}  // namespace

size_t dispatch_work_ints(size_t tokens, int topk, int experts) {
    const size_t slots = tokens * (size_t)topk;
    if (direct_form(tokens, (size_t)topk)) return 0;
    return (size_t)sort_blocks(slots) * (size_t)(experts + 1);
}

hipError_t launch_dispatch(const DispatchArgs& a, hipStream_t s) {
    const size_t slots = (size_t)a.tokens * a.topk;
    if (direct_form((size_t)a.tokens, (size_t)a.topk)) {
        const dim3 grid(a.tokens + 1);
#define CALL(EB, NT, MODE)                                                                    \
    if (a.ib == 8)                                                                            \
        hipLaunchKernelGGL((k_route_direct<EB, 8, NT, MODE>), grid, dim3(NT), 0, s, a, (int)slots); \
    else                                                                                      \
        hipLaunchKernelGGL((k_route_direct<EB, 4, NT, MODE>), grid, dim3(NT), 0, s, a, (int)slots)
        BY_ROW_WIDE(CALL);
#undef CALL
        return hipGetLastError();
    }
    const size_t share = sort_share(slots);
    const dim3 grid(sort_blocks(slots)), block(kSortThreads);
    if (a.ib == 8) hipLaunchKernelGGL(k_route_count<8>, grid, block, 0, s, a, slots, share);
    else hipLaunchKernelGGL(k_route_count<4>, grid, block, 0, s, a, slots, share);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    if (a.ib == 8) hipLaunchKernelGGL(k_route_place<8>, grid, block, 0, s, a, slots, share);
    else hipLaunchKernelGGL(k_route_place<4>, grid, block, 0, s, a, slots, share);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
#define CALL(EB, NT, MODE)                                                                  \
    hipLaunchKernelGGL((k_route_rows<EB, NT, MODE>), dim3(token_blocks(a.tokens)), dim3(NT), 0, s, a)
    BY_ROW(CALL);
#undef CALL
    return hipGetLastError();
}

hipError_t launch_combine(const CombineArgs& a, hipStream_t s) {
    if (a.tokens == 0) return hipSuccess;
    const dim3 grid(token_blocks(a.tokens));
    const bool stream = (size_t)a.tokens * a.topk * a.hidden * a.eb > kStreamBytes;
#define CALL2(EB, NT, KB, MODE)                                                                    \
    if (stream)                                                                                    \
        hipLaunchKernelGGL((k_route_combine<EB, NT, KB, MODE, true>), grid, dim3(NT), 0, s, a);    \
    else hipLaunchKernelGGL((k_route_combine<EB, NT, KB, MODE, false>), grid, dim3(NT), 0, s, a)
#define CALL(EB, NT, MODE)                              \
    if (a.topk <= 2) { CALL2(EB, NT, 2, MODE); }        \
    else if (a.topk <= 4) { CALL2(EB, NT, 4, MODE); }   \
    else { CALL2(EB, NT, 8, MODE); }
    BY_ROW(CALL);
#undef CALL
#undef CALL2
    return hipGetLastError();
}

hipError_t launch_combine_grad(const CombineArgs& a, hipStream_t s) {
    if (a.tokens == 0) return hipSuccess;
    const dim3 grid(token_blocks(a.tokens));
#define CALL(EB, NT, MODE)                                                                    \
    if (a.topk <= 2)                                                                          \
        hipLaunchKernelGGL((k_route_combine_grad<EB, NT, 2, MODE>), grid, dim3(NT), 0, s, a); \
    else if (a.topk <= 4)                                                                     \
        hipLaunchKernelGGL((k_route_combine_grad<EB, NT, 4, MODE>), grid, dim3(NT), 0, s, a); \
    else hipLaunchKernelGGL((k_route_combine_grad<EB, NT, 8, MODE>), grid, dim3(NT), 0, s, a)
    BY_ROW(CALL);
#undef CALL
    return hipGetLastError();
}

}  // namespace arlib
