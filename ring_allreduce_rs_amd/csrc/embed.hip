// embed.hip -- embedding: rows of a table by token, and the table's gradient.
//
//   y[t] = scale * table[ids[t]]                   (zeros for an id outside [0, vocab))
//   dtable[v] = scale * sum over t with ids[t] = v of dy[t]
//
// The gradient is dense (it is a bucket of the AllReduce), so most of it is
// zeros and its floor is one store of vocab x hidden.  The tokens are sorted by
// id first, stably, so that a row's sum runs over its tokens in order, in fp32,
// and is stored once: no atomics on values, the same bits each time.
//   1. order: a block owns a range of ids.  It walks the tokens of a list (all of
//      them, or, past kWhole tokens, a bucket that two launches made by the
//      ids' high part), keeps those in its range, counts the smaller ones, and
//      writes the tokens in their order and where each id's run of them begins.
//      Beside that it clears its share of dtable.
//   2. pieces: runs of more tokens than a piece (a text's few frequent tokens
//      have a large share of it) are summed a piece of sorted places at a time.
//   3. rows: the sum of each run, at the lanes of its first place, or of its
//      pieces.
// Measured: 16384 tokens of 4096 bf16 forward 33 us (84 MiB read and 128 written,
// 6.7 TB/s: frequent tokens' rows come from the caches); their gradient into a table of
// 131072 x 4096 247 us: order and clearing 162 - 177 us (1 GiB, 6.4 TB/s), pieces
// 16, rows 52.  One token forward is the launch, 2.2 us of kernel.
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
constexpr int kRange = 1024;                    // ids of a block, at most
constexpr size_t kWhole = 32768;                // tokens up to which each block walks them all
constexpr int kBuckets = 1024;                  // past it: at most, plus one for no id
constexpr size_t kBucketBlocks = 128;
constexpr size_t kUnits = 256;                  // compute units

// The sorted tokens with an id (`live` of them): order[j], the place start[j]
// where the run of its id begins, and there the run's length.
struct Sorted {
    int *order, *start, *length, *live;
};

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
#pragma unroll 8
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

// Clears dtable: 16 aligned bytes a thread, block `me` of `blocks`; the first also
// what lies before and behind whole ones.  (One store a thread and as many blocks
// as that takes: 1 GiB in 158 us; in loops over a grid that stays, 180 to 230.)
template <int EB>
__device__ __forceinline__ void clear(char* p, size_t bytes, size_t me, size_t blocks) {
    const size_t head = (16 - (uintptr_t)p % 16) % 16 < bytes ? (16 - (uintptr_t)p % 16) % 16 : bytes;
    const size_t units = (bytes - head) / 16, tail = head + units * 16;
    const u32x4 zero = {0u, 0u, 0u, 0u};
    for (size_t i = me * kOrderThreads + threadIdx.x; i < units; i += blocks * kOrderThreads)
        *reinterpret_cast<u32x4*>(p + head + i * 16) = zero;
    if (me == 0) {
        const size_t i = threadIdx.x * EB;
        if (i < head) st_elem<EB>(p + i, 0u);
        if (tail + i < bytes) st_elem<EB>(p + tail + i, 0u);
    }
}

// The first `sorters` blocks sort the tokens with ids in a range of 2^range_bits
// each.  LISTED: among those of its bucket; otherwise among all.  The others clear
// dtable meanwhile: a sorter is a few dependent loads, so there is one a compute
// unit at most, and the stores have the rest of it.
template <int IB, bool LISTED>
__global__ __launch_bounds__(kOrderThreads, 8) void k_embed_order(const EmbedGradArgs a, unsigned sorters, int range_bits,
                                                               int shift, const int* begins,
                                                               const int* list, const Sorted out) {
    __shared__ int wcnt[kOrderWaves][kRange];   // tokens per wavefront and id; then where they go
    __shared__ int begin_of[kRange];
    __shared__ int wless[kOrderWaves];
    __shared__ int sums[kOrderWaves];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const unsigned range = 1u << range_bits, vocab = (unsigned)a.vocab;
    static_assert(kRange <= kOrderThreads, "");
    if (blockIdx.x >= sorters) {
        char* p = static_cast<char*>(a.dtable);
        const size_t me = blockIdx.x - sorters, blocks = gridDim.x - sorters;
        if (a.eb == 2) clear<2>(p, a.vocab * a.hidden * 2, me, blocks);
        else clear<4>(p, a.vocab * a.hidden * 4, me, blocks);
        return;
    }
    for (size_t block = blockIdx.x; block << range_bits < a.vocab; block += sorters) {
        const unsigned v0 = (unsigned)(block << range_bits);
        const unsigned v1 = vocab - v0 < range ? vocab : v0 + range;
        size_t from = 0, n = a.tokens;
        if constexpr (LISTED) {
            const int b = (int)(v0 >> shift);
            from = begins[b];
            n = begins[b + 1] - from;
        }
        // wavefront w takes a run of the list, in steps of 64
        const size_t run = (n + 64 * kOrderWaves - 1) / (64 * kOrderWaves) * 64;
        const size_t begin = wave * run < n ? wave * run : n;
        const size_t end = begin + run < n ? begin + run : n;
        for (int i = lane; i < (int)range; i += 64) wcnt[wave][i] = 0;
        int less = 0;
        // calls body(id - v0, token, whether the id lies in the range) for every 64 tokens with
        // one in it; the loads of kAhead such steps are in flight together
        const auto walk = [&](auto body) {
            constexpr int kAhead = 4;   // (64 registers, for two blocks a compute unit)
            for (size_t i0 = begin; i0 < end; i0 += 64 * kAhead) {
                unsigned t[kAhead], id[kAhead];
#pragma unroll
                for (int k = 0; k < kAhead; ++k) {
                    const size_t i = i0 + k * 64 + lane;
                    t[k] = !LISTED ? (unsigned)i : i < end ? (unsigned)list[from + i] : 0u;
                }
#pragma unroll
                for (int k = 0; k < kAhead; ++k) {
                    const size_t i = i0 + k * 64 + lane;
                    const uint64_t v = i < end ? (uint64_t)id_at(a.ids, t[k], IB) : UINT64_MAX;
                    id[k] = v < vocab ? (unsigned)v : UINT32_MAX;   // (no id: past every vocabulary)
                }
#pragma unroll
                for (int k = 0; k < kAhead; ++k) {
                    const bool in = id[k] >= v0 && id[k] < v1;
                    if (__ballot(in)) body(id[k] - v0, t[k], in);
                    less += id[k] < v0;
                }
            }
        };
        wave_lds_order();
        walk([&](unsigned d, unsigned, bool in) {
            const unsigned long long m = same_bin(d, range_bits, in);
            if (in && (m & ((1ull << lane) - 1)) == 0) wcnt[wave][d] += __popcll(m);
            wave_lds_order();
        });
        less = wave_sum(less);
        if (lane == 0) wless[wave] = less;
        __syncthreads();
        int mine = 0, ahead = (int)from;
        if (threadIdx.x < range)
            for (int w = 0; w < kOrderWaves; ++w) mine += wcnt[w][threadIdx.x];
        for (int w = 0; w < kOrderWaves; ++w) ahead += wless[w];
        int total;
        const int before = ahead;
        ahead += block_scan(mine, sums, &total);
        if (threadIdx.x < range) {
            begin_of[threadIdx.x] = ahead;
            if (mine) out.length[ahead] = mine;
            for (int w = 0; w < kOrderWaves; ++w) {
                const int c = wcnt[w][threadIdx.x];
                wcnt[w][threadIdx.x] = ahead;
                ahead += c;
            }
        }
        if (threadIdx.x == 0 && v1 == vocab) *out.live = before + total;
        __syncthreads();
        if (total)
            walk([&](unsigned d, unsigned t, bool in) {
                const unsigned long long m = same_bin(d, range_bits, in);
                const int below = __popcll(m & ((1ull << lane) - 1));
                const int at = in ? wcnt[wave][d] : 0;
                wave_lds_order();
                if (in) {
                    out.order[at + below] = (int)t;
                    out.start[at + below] = begin_of[d];
                    if (below == 0) wcnt[wave][d] = at + __popcll(m);
                }
                wave_lds_order();
            });
        __syncthreads();
    }
}

// ------------------------------------------------------------------------- the sums

// Partial sums of the runs of more than `piece` tokens.  Piece q is the sorted
// places [q * piece, (q + 1) * piece); at most two such runs meet it, the first
// of them from before it (part 2 q) and one that begins in it (part 2 q + 1).
template <int EB, RowMode MODE>
__global__ __launch_bounds__(kThreads) void k_embed_pieces(const EmbedGradArgs a, const Sorted in,
                                                           int piece, float* part, size_t pitch) {
    using IO = RowIO<EB, MODE, true>;
    constexpr int E = IO::E, KB = 16;   // rows in flight
    const unsigned hidden = (unsigned)a.hidden, units = (hidden + E - 1) / E;
    const char* dy = static_cast<const char*>(a.dy);
    const int live = *in.live;
    for (size_t q = blockIdx.x; q * piece < (size_t)live; q += gridDim.x) {
        const int lo = (int)(q * piece);
        const int hi = live - lo < piece ? live : lo + piece;
        const int runs[2] = {in.start[lo], in.start[hi - 1]};
        const int lengths[2] = {in.length[runs[0]], in.length[runs[1]]};
        for (int e = 0; e < 2; ++e) {
            const int b = runs[e], c = b + lengths[e];
            if ((e && b == runs[0]) || lengths[e] <= piece) continue;
            const int from = b > lo ? b : lo, to = c < hi ? c : hi;
            float* out = part + (2 * q + (b > lo)) * pitch;
            // (every lane takes part, as the tokens are spread over the lanes)
            for (unsigned i0 = blockIdx.y * kThreads; i0 < units; i0 += gridDim.y * kThreads) {
                const unsigned i = i0 + threadIdx.x;
                const Place p = IO::place(i < units ? i : units - 1, hidden);
                float acc[E] = {};
                for (int r = from; r < to; r += KB) {
                    const int mine = r + (int)(threadIdx.x % KB);
                    const int tokens = mine < to ? in.order[mine] : -1;
                    u32x4 raw[KB];
#pragma unroll
                    for (int k = 0; k < KB; ++k) {
                        const int t = __builtin_amdgcn_readlane(tokens, k);
                        raw[k] = u32x4{0u, 0u, 0u, 0u};
                        if (t >= 0) raw[k] = IO::ld(dy + (size_t)t * a.dystride * EB, p, hidden);
                    }
#pragma unroll
                    for (int k = 0; k < KB; ++k) {
                        float v[E];
                        Vec<EB>::unpack(raw[k], v);
#pragma unroll
                        for (int j = 0; j < E; ++j) acc[j] += v[j];
                    }
                }
                if (i < units)
#pragma unroll
                    for (int j = 0; j < E; ++j) out[i * E + j] = acc[j];
            }
        }
    }
}

// out = scale * the rows dy[order[r]], r < n, by `lanes` lanes: U units and T rows
// at a time.
template <int EB, RowMode MODE, int U, int T>
__device__ __forceinline__ void add_run(const char* dy, const EmbedGradArgs& a, const int* order, int n,
                                        unsigned lane, unsigned lanes, unsigned units,
                                        unsigned hidden, char* out) {
    using IO = RowIO<EB, MODE, true>;
    constexpr int E = IO::E;
    for (unsigned i0 = lane; i0 < units; i0 += lanes * U) {
        float acc[U][E];
        Place p[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            p[u] = IO::place(i0 + u * lanes < units ? i0 + u * lanes : i0, hidden);
#pragma unroll
            for (int e = 0; e < E; ++e) acc[u][e] = 0.0f;
        }
        for (int r = 0; r < n; r += T) {
            u32x4 raw[T][U];
#pragma unroll
            for (int t = 0; t < T; ++t) {
                // (past the run: its last row again, counted for nothing)
                const char* row = dy + (size_t)order[r + t < n ? r + t : n - 1] * a.dystride * EB;
#pragma unroll
                for (int u = 0; u < U; ++u) raw[t][u] = IO::ld(row, p[u], hidden);
            }
#pragma unroll
            for (int t = 0; t < T; ++t)
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    float v[E];
                    Vec<EB>::unpack(raw[t][u], v);
#pragma unroll
                    for (int e = 0; e < E; ++e) acc[u][e] = r + t < n ? acc[u][e] + v[e] : acc[u][e];
                }
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (i0 + u * lanes < units) {
#pragma unroll
                for (int e = 0; e < E; ++e) acc[u][e] *= a.scale;
                IO::st(out, p[u], hidden, Vec<EB>::pack(acc[u]));
            }
    }
}

// The rows.  The first `joins` blocks have a piece and a share of the columns each
// (`across` of them a piece) and join the parts of the run that begins in it, if
// it is one of more than `piece` tokens: there is one at most.  In the others
// `lanes` lanes have a sorted place each, and sum the run that begins there.
template <int EB, RowMode MODE>
__global__ __launch_bounds__(kThreads, 8) void k_embed_rows(const EmbedGradArgs a, const Sorted in,
                                                         int piece, const float* part, size_t pitch,
                                                         unsigned joins, unsigned across, int lanes) {
    using IO = RowIO<EB, MODE, true>;
    constexpr int E = IO::E, KB = 4;
    const unsigned hidden = (unsigned)a.hidden, units = (hidden + E - 1) / E;
    const char* dy = static_cast<const char*>(a.dy);
    const int live = *in.live;
    const auto finish = [&](char* out, Place p, float (&acc)[E]) {
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] *= a.scale;
        IO::st(out, p, hidden, Vec<EB>::pack(acc));
    };
    const auto row_of = [&](int token) {
        return static_cast<char*>(a.dtable) + (size_t)id_at(a.ids, (size_t)token, a.ib) * a.hidden * EB;
    };
    for (size_t id = blockIdx.x; blockIdx.x < joins; id += joins) {
        const size_t q0 = id / across;
        if (q0 * piece >= (size_t)live) return;
        const int lo = (int)(q0 * piece);
        const int last = live - lo < piece ? live - 1 : lo + piece - 1;
        const int b = in.start[last], n = b >= lo ? in.length[b] : 0;
        if (n <= piece) continue;
        char* out = row_of(in.order[b]);
        const size_t q1 = (size_t)(b + n - 1) / piece;
        for (unsigned i = id % across * kThreads + threadIdx.x; i < units; i += across * kThreads) {
            float acc[E] = {};
            for (size_t q = q0; q <= q1; q += KB) {
                float x[KB][E];
#pragma unroll
                for (int k = 0; k < KB; ++k) {
                    const size_t at = 2 * (q + k) + ((size_t)b > (q + k) * piece);
#pragma unroll
                    for (int e = 0; e < E; ++e) x[k][e] = q + k <= q1 ? part[at * pitch + i * E + e] : 0.0f;
                }
#pragma unroll
                for (int k = 0; k < KB; ++k)
#pragma unroll
                    for (int e = 0; e < E; ++e) acc[e] += x[k][e];
            }
            finish(out, IO::place(i, hidden), acc);
        }
    }
    const unsigned lane = threadIdx.x & (lanes - 1), sub = threadIdx.x / lanes;
    const size_t each = kThreads / lanes, blocks = gridDim.x - joins;
    for (size_t j = (blockIdx.x - joins) * each + sub; j < a.tokens; j += blocks * each) {
        // (what a place needs is loaded together, before it is known whether a run begins there)
        const int start = in.start[j], n = in.length[j], token = in.order[j];
        if (j >= (size_t)live || start != (int)j || n > piece) continue;
        char* out = row_of(token);
        // many units of a row at a time for runs of one token, many rows of a unit for longer ones
        if (n == 1) add_run<EB, MODE, 2, 1>(dy, a, in.order + j, 1, lane, lanes, units, hidden, out);
        else if (n <= 4) add_run<EB, MODE, 2, 4>(dy, a, in.order + j, n, lane, lanes, units, hidden, out);
        else add_run<EB, MODE, 1, 8>(dy, a, in.order + j, n, lane, lanes, units, hidden, out);
    }
}

// ------------------------------------------------------------------------- launches

constexpr size_t kMostBlocks = size_t(1) << 21;   // (the kernels walk the rest)
unsigned blocks_for(size_t n, size_t each) {
    const size_t b = (n + each - 1) / each;
    return (unsigned)(b < 1 ? 1 : b < kMostBlocks ? b : kMostBlocks);
}

// The scratch: the sorted tokens, and past kWhole of them the buckets' counts,
// begins and list; then the partial sums, where an id can have more tokens than a
// piece.  Pieces are short while there are few tokens, so that a frequent one's
// sum is spread over the card (16384 tokens of 4096: 247 us with a piece of 16,
// 289 with 64), and long where the partial sums would take much memory.
struct Layout {
    size_t order, start, length, live, count, begins, list, part, bytes;   // bytes from the start
    size_t pitch;                                           // floats of a partial row
    int piece;
    int range_bits;     // ids of an order block: one block a compute unit, where that will do
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
    l.order = take(tokens * sizeof(int));
    l.start = take(tokens * sizeof(int));
    l.length = take(tokens * sizeof(int));
    l.live = take(sizeof(int));
    while (l.range_bits < __builtin_ctz(kRange) && (vocab - 1) >> l.range_bits >= kUnits) ++l.range_bits;
    if (tokens > kWhole) {
        l.shift = __builtin_ctz(kRange);
        while ((vocab - 1) >> l.shift >= (size_t)kBuckets) ++l.shift;
        l.buckets = (int)((vocab - 1) >> l.shift) + 1;
        const size_t rounds = (tokens + kOrderThreads - 1) / kOrderThreads;
        l.share = (rounds + kBucketBlocks - 1) / kBucketBlocks * kOrderThreads;
        l.blocks = (unsigned)((tokens + l.share - 1) / l.share);
        l.count = take((size_t)(l.buckets + 1) * l.blocks * sizeof(int));
        l.begins = take((size_t)(l.buckets + 1) * sizeof(int));
        l.list = take(tokens * sizeof(int));
    }
    const size_t e = 16 / (size_t)eb;
    l.pitch = (hidden + e - 1) / e * e;
    l.piece = tokens <= 65536 ? 16 : 64;
    if (tokens > (size_t)l.piece)
        l.part = take((tokens + l.piece - 1) / l.piece * 2 * l.pitch * sizeof(float));
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
    const auto ints = [&](size_t at) { return reinterpret_cast<int*>(w + at); };
    const Sorted sorted = {ints(l.order), ints(l.start), ints(l.length), ints(l.live)};
    int *count = ints(l.count), *begins = ints(l.begins), *list = ints(l.list);
    float* part = reinterpret_cast<float*>(w + l.part);
    const unsigned sorters = blocks_for(a.vocab, size_t(1) << l.range_bits);
    const dim3 block(kOrderThreads);
    const dim3 ranges(sorters + blocks_for(a.vocab * a.hidden * a.eb, 16 * kOrderThreads));
    hipError_t e;
#define CALL(IB)                                                                                  \
    do {                                                                                          \
        if (a.tokens <= kWhole) {                                                                 \
            hipLaunchKernelGGL((k_embed_order<IB, false>), ranges, block, 0, s, a, sorters, l.range_bits, 0, \
                               begins, list, sorted);                                             \
            break;                                                                                \
        }                                                                                         \
        hipLaunchKernelGGL(k_embed_count<IB>, dim3(l.blocks), block, 0, s, a, l.shift, l.buckets, \
                           l.share, count);                                                       \
        if ((e = hipGetLastError()) != hipSuccess) return e;                                      \
        hipLaunchKernelGGL(k_embed_bucket<IB>, dim3(l.blocks), block, 0, s, a, l.shift, l.buckets, \
                           l.share, count, begins, list);                                         \
        if ((e = hipGetLastError()) != hipSuccess) return e;                                      \
        hipLaunchKernelGGL((k_embed_order<IB, true>), ranges, block, 0, s, a, sorters, l.range_bits, l.shift, \
                           begins, list, sorted);                                                 \
    } while (0)
    if (a.ib == 8) CALL(8);
    else CALL(4);
#undef CALL
    if ((e = hipGetLastError()) != hipSuccess || a.tokens == 0) return e;
    const size_t units = (a.hidden * a.eb + 15) / 16;
    unsigned joins = 0;
    const unsigned across = units < 64 * kThreads ? blocks_for(units, kThreads) : 64;
    if (a.tokens > (size_t)l.piece) {
        const size_t pieces = (a.tokens + l.piece - 1) / l.piece;
        joins = blocks_for(pieces * across, 1);
        const dim3 grid(blocks_for(pieces, 1), across);
#define CALL(EB, MODE)                                                                           \
        hipLaunchKernelGGL((k_embed_pieces<EB, MODE>), grid, dim3(kThreads), 0, s, a, sorted, l.piece, \
                           part, l.pitch)
        BY_ROW(CALL);
#undef CALL
        if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    const int lanes = row_lanes(a.hidden, a.eb);
    const dim3 grid(joins + blocks_for(a.tokens, kThreads / lanes));
#define CALL(EB, MODE)                                                                              \
    hipLaunchKernelGGL((k_embed_rows<EB, MODE>), grid, dim3(kThreads), 0, s, a, sorted, l.piece, part, \
                       l.pitch, joins, across, lanes)
    BY_ROW(CALL);
#undef CALL
    return hipGetLastError();
}

}  // namespace arlib
