// embed.hip -- embedding: rows of a table by token, and the table's gradient.
//
//   y[t] = scale * table[ids[t]]                   (zeros for an id outside [0, vocab))
//   dtable[v] = scale * sum over t with ids[t] = v of dy[t]
//
// The gradient is dense (it is a bucket of the AllReduce), so most of it is
// zeros and its floor is one store of vocab x hidden.  The tokens are sorted by
// id first, stably, so that a row's sum runs over its tokens in order, in fp32,
// and is stored once: no atomics on values, the same bits each time.
//   1. order: block b owns kRange ids.  It walks the tokens of a list (all of
//      them, or, past kWhole tokens, a bucket that two launches made by the
//      ids' high part), keeps those in its range, counts the smaller ones, and
//      writes first[v] and, sorted, the tokens themselves.
//   2. pieces: ids that come more than kPiece times (a text's few frequent
//      tokens have a large share of it) are summed kPiece sorted places at a
//      time into partial sums.
//   3. rows: one store of each row of dtable.
#include "model_ops.h"
#include "ops_device.h"

namespace arlib {
namespace {

// ------------------------------------------------------------------------ forward

__device__ __forceinline__ int64_t id_at(const void* ids, size_t i, int ib) {
    return ib == 8 ? static_cast<const int64_t*>(ids)[i]
                   : (int64_t)static_cast<const int32_t*>(ids)[i];
}

constexpr int kThreads = 256;

// Lanes that a row is given: the least power of two that holds its units, up to a block.
int row_lanes(size_t hidden, int eb) {
    const size_t units = (hidden * eb + 15) / 16;
    int l = 4;
    while (l < kThreads && (size_t)l < units) l *= 2;
    return l;
}

template <int EB>
__device__ __forceinline__ u32x4 scaled(u32x4 u, float scale) {
    float v[Vec<EB>::E];
    Vec<EB>::unpack(u, v);
#pragma unroll
    for (int j = 0; j < Vec<EB>::E; ++j) v[j] *= scale;
    return Vec<EB>::pack(v);
}

template <int EB, RowMode MODE>
__global__ __launch_bounds__(kThreads) void k_embed(const EmbedArgs a, int lanes) {
    using IO = RowIO<EB, MODE, false>;
    const unsigned hidden = (unsigned)a.hidden, units = (hidden + IO::E - 1) / IO::E;
    const unsigned lane = threadIdx.x & (lanes - 1), sub = threadIdx.x / lanes;
    const size_t each = kThreads / lanes;
    for (size_t t = blockIdx.x * each + sub; t < a.tokens; t += gridDim.x * each) {
        const int64_t id = id_at(a.ids, t, a.ib);
        const bool known = id >= 0 && id < (int64_t)a.vocab;
        const char* row = static_cast<const char*>(a.table) + (known ? (size_t)id : 0) * a.hidden * EB;
        char* y = static_cast<char*>(a.y) + t * a.hidden * EB;
        for (unsigned i = lane; i < units; i += lanes) {
            const Place p = IO::place(i, hidden);
            const u32x4 z = {0u, 0u, 0u, 0u};
            IO::st(y, p, hidden, known ? scaled<EB>(IO::ld(row, p, hidden), a.scale) : z);
        }
    }
}

// ----------------------------------------------------------------------- the order

constexpr int kOrderThreads = 1024;
constexpr int kOrderWaves = kOrderThreads / 64;
constexpr int kRange = 256;                     // ids of a block
constexpr size_t kWhole = 32768;                // tokens up to which each block walks them all
constexpr int kBuckets = 1024;                  // past it: at most, plus one for no id
constexpr size_t kBucketBlocks = 128;
constexpr int kPiece = 64;

__device__ __forceinline__ void wave_lds_order() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// Lanes whose bin equals this lane's, among the live ones.
__device__ __forceinline__ unsigned long long same_bin(unsigned bin, int bits, bool live) {
    unsigned long long m = __ballot(live);
    for (int b = 0; b < bits; ++b) {
        const bool one = (bin >> b) & 1;
        const unsigned long long v = __ballot(one);
        m &= one ? v : ~v;
    }
    return m;
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

// The bucket of a token: its id's high part, `buckets` where it has no id.
template <int IB>
__device__ __forceinline__ int bucket_of(const EmbedGradArgs& a, size_t t, int shift, int buckets) {
    const int64_t id = id_at(a.ids, t, IB);
    return id >= 0 && id < (int64_t)a.vocab ? (int)(id >> shift) : buckets;
}

// Tokens per bucket in each block's share: count[bucket][block].
template <int IB>
__global__ __launch_bounds__(kOrderThreads) void k_embed_count(const EmbedGradArgs a, int shift,
                                                               int buckets, size_t share, int* count) {
    __shared__ int cnt[kBuckets + 1];
    for (int b = threadIdx.x; b <= buckets; b += kOrderThreads) cnt[b] = 0;
    __syncthreads();
    const size_t begin = blockIdx.x * share;
    const size_t end = begin + share < a.tokens ? begin + share : a.tokens;
    for (size_t t = begin + threadIdx.x; t < end; t += kOrderThreads)
        atomicAdd(&cnt[bucket_of<IB>(a, t, shift, buckets)], 1);
    __syncthreads();
    for (int b = threadIdx.x; b <= buckets; b += kOrderThreads)
        count[(size_t)b * gridDim.x + blockIdx.x] = cnt[b];
}

// Exclusive prefix sums of n <= kOrderThreads values, one a thread; `sums` holds kOrderWaves.
__device__ __forceinline__ int block_scan(int v, int* sums, int* total) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int inc = wave_scan(v, lane);
    if (lane == 63) sums[wave] = inc;
    __syncthreads();
    int ahead = 0, all = 0;
    for (int w = 0; w < kOrderWaves; ++w) {
        if (w < wave) ahead += sums[w];
        all += sums[w];
    }
    __syncthreads();
    *total = all;
    return ahead + inc - v;
}

// The buckets' tokens in order: list, and each bucket's first place in it
// (start[buckets]: the tokens with an id).
template <int IB>
__global__ __launch_bounds__(kOrderThreads) void k_embed_bucket(const EmbedGradArgs a, int shift,
                                                                int buckets, size_t share,
                                                                const int* count, int* start,
                                                                int* list) {
    __shared__ int first[kBuckets + 1];
    __shared__ unsigned short wcnt[kOrderWaves][kBuckets + 1];
    __shared__ int sums[kOrderWaves];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int nblk = gridDim.x, me = blockIdx.x;
    const int bins = buckets + 1, bits = 32 - __clz(buckets);
    // this thread's buckets: threadIdx.x and the one for no id (thread 0)
    int carried = 0;
    for (int b0 = 0; b0 < bins; b0 += kOrderThreads) {
        const int b = b0 + (int)threadIdx.x;
        int all = 0, before = 0;
        if (b < bins)
            for (int k = 0; k < nblk; ++k) {
                const int c = count[(size_t)b * nblk + k];
                all += c;
                before += k < me ? c : 0;
            }
        int total;
        const int ahead = carried + block_scan(all, sums, &total);
        if (b < bins) {
            first[b] = ahead + before;
            if (me == 0) start[b] = ahead;
        }
        carried += total;
    }
    __syncthreads();
    const size_t begin = (size_t)me * share;
    for (size_t round = begin; round < begin + share && round < a.tokens; round += kOrderThreads) {
        const size_t t = round + threadIdx.x;
        const bool live = t < a.tokens;
        const int bin = live ? bucket_of<IB>(a, t, shift, buckets) : 0;
        for (int b = lane; b < bins; b += 64) wcnt[wave][b] = 0;
        wave_lds_order();
        const unsigned long long m = same_bin(bin, bits, live);
        const int below = __popcll(m & ((1ull << lane) - 1));
        if (live && below == 0) wcnt[wave][bin] = (unsigned short)__popcll(m);
        __syncthreads();
        int sum[(kBuckets + kOrderThreads) / kOrderThreads];
#pragma unroll
        for (int q = 0; q < (kBuckets + kOrderThreads) / kOrderThreads; ++q) {
            const int b = q * kOrderThreads + (int)threadIdx.x;
            sum[q] = 0;
            if (b < bins)
                for (int w = 0; w < kOrderWaves; ++w) {
                    const int c = wcnt[w][b];
                    wcnt[w][b] = (unsigned short)sum[q];
                    sum[q] += c;
                }
        }
        __syncthreads();
        if (live) list[first[bin] + wcnt[wave][bin] + below] = (int)t;
        __syncthreads();
#pragma unroll
        for (int q = 0; q < (kBuckets + kOrderThreads) / kOrderThreads; ++q) {
            const int b = q * kOrderThreads + (int)threadIdx.x;
            if (b < bins) first[b] += sum[q];
        }
        __syncthreads();
    }
}

// Block b sorts the tokens with ids in [b * kRange, (b + 1) * kRange).  LISTED:
// among those of its bucket; otherwise among all.  first[v] is the sorted place
// of id v's first token, first[vocab] the tokens with an id.
template <int IB, bool LISTED>
__global__ __launch_bounds__(kOrderThreads) void k_embed_order(const EmbedGradArgs a, int shift,
                                                               const int* start, const int* list,
                                                               int* first, int* order) {
    __shared__ int wcnt[kOrderWaves][kRange];   // tokens per wavefront and id; then where they go
    __shared__ int wless[kOrderWaves];
    __shared__ int sums[kOrderWaves];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    constexpr int bits = __builtin_ctz(kRange);
    static_assert(kRange <= kOrderThreads && (kRange & (kRange - 1)) == 0, "");
    for (size_t v0 = (size_t)blockIdx.x * kRange; v0 < a.vocab; v0 += (size_t)gridDim.x * kRange) {
        size_t from = 0, n = a.tokens;
        if constexpr (LISTED) {
            const int b = (int)(v0 >> shift);
            from = start[b];
            n = start[b + 1] - from;
        }
        // wavefront w takes a run of the list, in steps of 64
        const size_t run = (n + 64 * kOrderWaves - 1) / (64 * kOrderWaves) * 64;
        const size_t begin = wave * run < n ? wave * run : n;
        const size_t end = begin + run < n ? begin + run : n;
        for (int i = lane; i < kRange; i += 64) wcnt[wave][i] = 0;
        int less = 0;
        const auto token = [&](size_t i) { return LISTED ? (size_t)list[from + i] : i; };
        // calls body(id - v0, token) where the id lies in the range
        const auto walk = [&](auto body) {
            for (size_t i0 = begin; i0 < end; i0 += 64) {
                const size_t i = i0 + lane;
                const size_t t = i < end ? token(i) : 0;
                // (no id: past every vocabulary)
                const uint64_t id = i < end ? (uint64_t)id_at(a.ids, t, IB) : UINT64_MAX;
                const bool in = id >= v0 && id < a.vocab && id - v0 < kRange;
                if (__ballot(in)) body((unsigned)(id - v0), t, in);
                less += id < v0;
            }
        };
        wave_lds_order();
        walk([&](unsigned d, size_t, bool in) {
            const unsigned long long m = same_bin(d, bits, in);
            if (in && (m & ((1ull << lane) - 1)) == 0) wcnt[wave][d] += __popcll(m);
            wave_lds_order();
        });
        less = wave_sum(less);
        if (lane == 0) wless[wave] = less;
        __syncthreads();
        int mine = 0, ahead = (int)from;
        if (threadIdx.x < kRange)
            for (int w = 0; w < kOrderWaves; ++w) mine += wcnt[w][threadIdx.x];
        for (int w = 0; w < kOrderWaves; ++w) ahead += wless[w];
        int total;
        ahead += block_scan(mine, sums, &total);
        if (threadIdx.x < kRange) {
            const size_t v = v0 + threadIdx.x;
            if (v < a.vocab) first[v] = ahead;
            if (v + 1 == a.vocab) first[a.vocab] = ahead + mine;
            for (int w = 0; w < kOrderWaves; ++w) {
                const int c = wcnt[w][threadIdx.x];
                wcnt[w][threadIdx.x] = ahead;
                ahead += c;
            }
        }
        __syncthreads();
        walk([&](unsigned d, size_t t, bool in) {
            const unsigned long long m = same_bin(d, bits, in);
            const int below = __popcll(m & ((1ull << lane) - 1));
            const int at = in ? wcnt[wave][d] : 0;
            wave_lds_order();
            if (in) order[at + below] = (int)t;
            if (in && below == 0) wcnt[wave][d] = at + __popcll(m);
            wave_lds_order();
        });
        __syncthreads();
    }
}

// ------------------------------------------------------------------------- the sums

// acc += the rows dy[order[i]], i in [lo, hi), at place p
template <int EB, RowMode MODE>
__device__ __forceinline__ void add_rows(const EmbedGradArgs& a, const int* order, int lo, int hi,
                                         Place p, float (&acc)[Vec<EB>::E]) {
    using IO = RowIO<EB, MODE, true>;
    constexpr int KB = 4;   // rows in flight
    const unsigned hidden = (unsigned)a.hidden;
    for (int i = lo; i < hi; i += KB) {
        u32x4 raw[KB];
#pragma unroll
        for (int k = 0; k < KB; ++k) {
            raw[k] = u32x4{0u, 0u, 0u, 0u};
            if (i + k < hi)
                raw[k] = IO::ld(static_cast<const char*>(a.dy) +
                                    (size_t)order[i + k] * a.dystride * EB, p, hidden);
        }
#pragma unroll
        for (int k = 0; k < KB; ++k) {
            float v[Vec<EB>::E];
            Vec<EB>::unpack(raw[k], v);
#pragma unroll
            for (int j = 0; j < Vec<EB>::E; ++j) acc[j] += v[j];
        }
    }
}

// first[v] of the least v with first[v + 1] > i: whose row place i belongs to
__device__ __forceinline__ size_t row_of(const int* first, size_t vocab, int i) {
    size_t lo = 0, hi = vocab;   // first[lo] <= i < first[hi]
    while (hi - lo > 1) {
        const size_t mid = lo + (hi - lo) / 2;
        if (first[mid] <= i) lo = mid;
        else hi = mid;
    }
    return lo;
}

// Partial sums of the ids with more than kPiece tokens.  Piece q is the sorted
// places [q * kPiece, (q + 1) * kPiece); at most two such ids meet it, the first
// of them from before it (part 2 q) and one that begins in it (part 2 q + 1).
template <int EB, RowMode MODE>
__global__ __launch_bounds__(kThreads) void k_embed_pieces(const EmbedGradArgs a, const int* first,
                                                           const int* order, float* part,
                                                           size_t pitch) {
    using IO = RowIO<EB, MODE, true>;
    const unsigned hidden = (unsigned)a.hidden, units = (hidden + IO::E - 1) / IO::E;
    const int live = first[a.vocab];
    for (size_t q = blockIdx.x; q * kPiece < (size_t)live; q += gridDim.x) {
        const int lo = (int)(q * kPiece);
        const int hi = live - lo < kPiece ? live : lo + kPiece;
        const size_t ends[2] = {row_of(first, a.vocab, lo), row_of(first, a.vocab, hi - 1)};
        for (int e = 0; e < 2; ++e) {
            const size_t v = ends[e];
            if (e && v == ends[0]) break;
            const int b = first[v], c = first[v + 1];
            if (c - b <= kPiece) continue;
            const int from = b > lo ? b : lo, to = c < hi ? c : hi;
            float* out = part + (2 * q + (b > lo)) * pitch;
            for (unsigned i = blockIdx.y * kThreads + threadIdx.x; i < units;
                 i += gridDim.y * kThreads) {
                float acc[IO::E] = {};
                add_rows<EB, MODE>(a, order, from, to, IO::place(i, hidden), acc);
#pragma unroll
                for (int j = 0; j < IO::E; ++j) out[i * IO::E + j] = acc[j];
            }
        }
    }
}

template <int EB, RowMode MODE>
__global__ __launch_bounds__(kThreads) void k_embed_rows(const EmbedGradArgs a, const int* first,
                                                         const int* order, const float* part,
                                                         size_t pitch, int lanes) {
    using IO = RowIO<EB, MODE, true>;
    constexpr int E = IO::E;
    const unsigned hidden = (unsigned)a.hidden, units = (hidden + E - 1) / E;
    const unsigned lane = threadIdx.x & (lanes - 1), sub = threadIdx.x / lanes;
    const size_t each = kThreads / lanes;
    for (size_t v = blockIdx.x * each + sub; v < a.vocab; v += gridDim.x * each) {
        const int lo = first[v], hi = first[v + 1];
        char* out = static_cast<char*>(a.dtable) + v * a.hidden * EB;
        for (unsigned i = lane; i < units; i += lanes) {
            const Place p = IO::place(i, hidden);
            float acc[E] = {};
            if (hi - lo <= kPiece) {
                add_rows<EB, MODE>(a, order, lo, hi, p, acc);
            } else {
                for (int q = lo / kPiece; q <= (hi - 1) / kPiece; ++q) {
                    const float* from = part + (2 * (size_t)q + (lo > q * kPiece)) * pitch + i * E;
#pragma unroll
                    for (int j = 0; j < E; ++j) acc[j] += from[j];
                }
            }
#pragma unroll
            for (int j = 0; j < E; ++j) acc[j] *= a.scale;
            IO::st(out, p, hidden, Vec<EB>::pack(acc));
        }
    }
}

// ------------------------------------------------------------------------- launches

constexpr size_t kMostBlocks = size_t(1) << 22;
unsigned blocks_for(size_t n, size_t each) {
    const size_t b = (n + each - 1) / each;
    return (unsigned)(b < 1 ? 1 : b < kMostBlocks ? b : kMostBlocks);
}

// The scratch: first, order, and past kWhole tokens the buckets' counts, starts
// and list; then the partial sums, where an id can come more than kPiece times.
struct Layout {
    size_t first, order, count, start, list, part, bytes;   // bytes from the start
    size_t pitch;                                           // floats of a partial row
    int shift, buckets;
    size_t share;
    unsigned blocks;
};
Layout layout(size_t tokens, size_t vocab, size_t hidden, int eb) {
    Layout l{};
    size_t at = 0;
    const auto take = [&](size_t bytes) {
        const size_t was = at;
        at += (bytes + 15) / 16 * 16;
        return was;
    };
    l.first = take((vocab + 1) * sizeof(int));
    l.order = take(tokens * sizeof(int));
    if (tokens > kWhole) {
        l.shift = __builtin_ctz(kRange);
        while ((vocab - 1) >> l.shift >= (size_t)kBuckets) ++l.shift;
        l.buckets = (int)((vocab - 1) >> l.shift) + 1;
        const size_t rounds = (tokens + kOrderThreads - 1) / kOrderThreads;
        l.share = (rounds + kBucketBlocks - 1) / kBucketBlocks * kOrderThreads;
        l.blocks = (unsigned)((tokens + l.share - 1) / l.share);
        l.count = take((size_t)(l.buckets + 1) * l.blocks * sizeof(int));
        l.start = take((size_t)(l.buckets + 1) * sizeof(int));
        l.list = take(tokens * sizeof(int));
    }
    const size_t e = 16 / (size_t)eb;
    l.pitch = (hidden + e - 1) / e * e;
    if (tokens > kPiece) l.part = take((tokens + kPiece - 1) / kPiece * 2 * l.pitch * sizeof(float));
    l.bytes = at;
    return l;
}

#define BY_MODE(EB, CALL)                                \
    do {                                                 \
        if (mode == ROW_FULL) { CALL(EB, ROW_FULL); }    \
        else if (mode == ROW_RAGGED) { CALL(EB, ROW_RAGGED); } \
        else { CALL(EB, ROW_SHORT); }                    \
    } while (0)
#define BY_ROW(CALL)                                     \
    do {                                                 \
        const RowMode mode = row_mode(a.hidden, a.eb);   \
        if (a.eb == 2) BY_MODE(2, CALL);                 \
        else BY_MODE(4, CALL);                           \
    } while (0)

}  // namespace

size_t embed_grad_work_bytes(size_t tokens, size_t vocab, size_t hidden, int eb) {
    return layout(tokens, vocab, hidden, eb).bytes;
}

hipError_t launch_embed(const EmbedArgs& a, hipStream_t s) {
    if (a.tokens == 0) return hipSuccess;
    const int lanes = row_lanes(a.hidden, a.eb);
    const dim3 grid(blocks_for(a.tokens, kThreads / lanes));
#define CALL(EB, MODE) \
    hipLaunchKernelGGL((k_embed<EB, MODE>), grid, dim3(kThreads), 0, s, a, lanes)
    BY_ROW(CALL);
#undef CALL
    return hipGetLastError();
}

hipError_t launch_embed_grad(const EmbedGradArgs& a, hipStream_t s) {
    const Layout l = layout(a.tokens, a.vocab, a.hidden, a.eb);
    char* w = reinterpret_cast<char*>(a.work);
    int *first = reinterpret_cast<int*>(w + l.first), *order = reinterpret_cast<int*>(w + l.order);
    int *count = reinterpret_cast<int*>(w + l.count), *start = reinterpret_cast<int*>(w + l.start);
    int* list = reinterpret_cast<int*>(w + l.list);
    float* part = reinterpret_cast<float*>(w + l.part);
    const dim3 block(kOrderThreads), ranges(blocks_for(a.vocab, kRange));
    hipError_t e;
    if (a.tokens > kWhole) {
        const dim3 grid(l.blocks);
        if (a.ib == 8) hipLaunchKernelGGL(k_embed_count<8>, grid, block, 0, s, a, l.shift, l.buckets, l.share, count);
        else hipLaunchKernelGGL(k_embed_count<4>, grid, block, 0, s, a, l.shift, l.buckets, l.share, count);
        if ((e = hipGetLastError()) != hipSuccess) return e;
        if (a.ib == 8) hipLaunchKernelGGL(k_embed_bucket<8>, grid, block, 0, s, a, l.shift, l.buckets, l.share, count, start, list);
        else hipLaunchKernelGGL(k_embed_bucket<4>, grid, block, 0, s, a, l.shift, l.buckets, l.share, count, start, list);
        if ((e = hipGetLastError()) != hipSuccess) return e;
        if (a.ib == 8) hipLaunchKernelGGL((k_embed_order<8, true>), ranges, block, 0, s, a, l.shift, start, list, first, order);
        else hipLaunchKernelGGL((k_embed_order<4, true>), ranges, block, 0, s, a, l.shift, start, list, first, order);
    } else {
        if (a.ib == 8) hipLaunchKernelGGL((k_embed_order<8, false>), ranges, block, 0, s, a, 0, start, list, first, order);
        else hipLaunchKernelGGL((k_embed_order<4, false>), ranges, block, 0, s, a, 0, start, list, first, order);
    }
    if ((e = hipGetLastError()) != hipSuccess) return e;
    if (a.tokens > kPiece) {
        const size_t units = (a.hidden * a.eb + 15) / 16;
        const dim3 grid(blocks_for(a.tokens, kPiece), units < 64 * kThreads ? blocks_for(units, kThreads) : 64);
#define CALL(EB, MODE) \
        hipLaunchKernelGGL((k_embed_pieces<EB, MODE>), grid, dim3(kThreads), 0, s, a, first, order, part, l.pitch)
        BY_ROW(CALL);
#undef CALL
        if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    const int lanes = row_lanes(a.hidden, a.eb);
    const dim3 grid(blocks_for(a.vocab, kThreads / lanes));
#define CALL(EB, MODE)                                                                        \
    hipLaunchKernelGGL((k_embed_rows<EB, MODE>), grid, dim3(kThreads), 0, s, a, first, order, \
                       part, l.pitch, lanes)
    BY_ROW(CALL);
#undef CALL
    return hipGetLastError();
}

}  // namespace arlib
