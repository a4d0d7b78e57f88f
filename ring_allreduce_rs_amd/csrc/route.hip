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
#include "ops.h"
#include "ops_device.h"

namespace arlib {
namespace {

constexpr int kSortThreads = 1024;
constexpr int kSortWaves = kSortThreads / 64;
constexpr int kSortSteps = 2;                            // slots per thread
constexpr int kSortSlots = kSortThreads * kSortSteps;    // slots per block
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

// Slots per bin of each block's share.
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
    int* out = a.work + (size_t)blockIdx.x * (a.experts + 1);
    for (int b = threadIdx.x; b <= a.experts; b += kSortThreads) out[b] = cnt[b];
}

// Where each slot goes.  A block needs, for every bin, the slots in smaller
// bins plus those of the same bin in earlier blocks (from the counts), then in
// earlier rounds and wavefronts of its own, then in earlier lanes.
template <int IB>
__global__ __launch_bounds__(kSortThreads) void k_route_place(const DispatchArgs a, size_t slots,
                                                              size_t share) {
    __shared__ int first[kBins];                       // next free row of each bin
    __shared__ unsigned short wcnt[kSortWaves][kBins]; // slots per wavefront and bin
    __shared__ int wsum[kSortWaves];
    const int bins = a.experts + 1, bits = bin_bits(a.experts);
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int nblk = slots ? (int)gridDim.x : 0;

    // totals, and the part that earlier blocks hold
    int run = 0;
    for (int b0 = 0; b0 < bins; b0 += kSortThreads) {
        const int b = b0 + (int)threadIdx.x;
        int total = 0, before = 0;
        if (b < bins)
            for (int k = 0; k < nblk; ++k) {
                const int c = a.work[(size_t)k * bins + b];
                total += c;
                if (k < (int)blockIdx.x) before += c;
            }
        int inc = total;   // inclusive sum over the wavefront
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int o = __shfl_up(inc, d, 64);
            if (lane >= d) inc += o;
        }
        if (lane == 63) wsum[wave] = inc;
        __syncthreads();
        int ahead = run;
        for (int w = 0; w < kSortWaves; ++w) {
            if (w < wave) ahead += wsum[w];
            run += wsum[w];
        }
        const int start = ahead + inc - total;
        if (b < bins) {
            first[b] = start + before;
            if (blockIdx.x == 0) a.offsets[b] = start;   // bin `experts`: the end of the last expert
        }
        __syncthreads();
    }

    const size_t begin = blockIdx.x * share;
    for (size_t round = begin; round < begin + share && round < slots; round += kSortSlots) {
        // wavefront w takes 64 * kSortSteps slots in a row
        const size_t base = round + wave * 64 * kSortSteps;
        for (int b = lane; b < bins; b += 64) wcnt[wave][b] = 0;
        wave_lds_order();
        int bin[kSortSteps], rank[kSortSteps];
#pragma unroll
        for (int s = 0; s < kSortSteps; ++s) {
            const size_t i = base + s * 64 + lane;
            const bool live = i < slots;
            bin[s] = live ? bin_of<IB>(a.ids, i, a.experts) : 0;
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
            if (b < bins)
                for (int w = 0; w < kSortWaves; ++w) {
                    const int c = wcnt[w][b];
                    wcnt[w][b] = (unsigned short)sum[q];
                    sum[q] += c;
                }
        }
        __syncthreads();
#pragma unroll
        for (int s = 0; s < kSortSteps; ++s) {
            const size_t i = base + s * 64 + lane;
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

constexpr int kRowThreads = 256;

// A token's row to each of its sorted rows: TPT threads per token.
template <int EB, int TPT>
__global__ __launch_bounds__(kRowThreads) void k_route_rows(const DispatchArgs a) {
    constexpr int E = Vec<EB>::E;
    const size_t n = (size_t)a.tokens * a.topk;
    const int live = a.offsets[a.experts];
    for (size_t t = (size_t)blockIdx.x * (kRowThreads / TPT) + threadIdx.x / TPT;
         t < (size_t)a.tokens; t += (size_t)gridDim.x * (kRowThreads / TPT)) {
        const char* x = static_cast<const char*>(a.x) + t * a.xstride * EB;
        const int* dest = a.dest + t * a.topk;
        for (size_t i = (size_t)(threadIdx.x % TPT) * E; i < a.hidden; i += (size_t)TPT * E) {
            const u32x4 u = ld_unit_of<EB>(x, i, a.hidden, 0u);
            for (int k = 0; k < a.topk; ++k) {
                const int d = dest[k];
                if ((size_t)d >= n) continue;
                const u32x4 z = {0u, 0u, 0u, 0u};
                st_unit_of<EB>(static_cast<char*>(a.rows) + (size_t)d * a.hidden * EB, i, a.hidden,
                               d < live ? u : z);
            }
        }
    }
}

// y[t] = sum_k w[t,k] rows[dest[t,k]]
template <int EB, int TPT>
__global__ __launch_bounds__(kRowThreads) void k_route_combine(const CombineArgs a) {
    constexpr int E = Vec<EB>::E;
    const int n = a.tokens * a.topk;
    const int live = min(a.offsets[a.experts], n);
    for (size_t t = (size_t)blockIdx.x * (kRowThreads / TPT) + threadIdx.x / TPT;
         t < (size_t)a.tokens; t += (size_t)gridDim.x * (kRowThreads / TPT)) {
        const int* dest = a.dest + t * a.topk;
        const float* w = a.weights ? a.weights + t * a.topk : nullptr;
        char* y = static_cast<char*>(a.y) + t * a.hidden * EB;
        for (size_t i = (size_t)(threadIdx.x % TPT) * E; i < a.hidden; i += (size_t)TPT * E) {
            float acc[E] = {};
            for (int k = 0; k < a.topk; ++k) {
                const int d = dest[k];
                if (d < 0 || d >= live) continue;
                const float wk = w ? w[k] : 1.0f;
                float v[E];
                Vec<EB>::unpack(ld_unit_of<EB>(static_cast<const char*>(a.rows) +
                                                   (size_t)d * a.hidden * EB, i, a.hidden, 0u), v);
#pragma unroll
                for (int j = 0; j < E; ++j) acc[j] = __builtin_fmaf(v[j], wk, acc[j]);
            }
            st_unit_of<EB>(y, i, a.hidden, Vec<EB>::pack(acc));
        }
    }
}

// drows and dweights: a wavefront per token, one choice at a time.
template <int EB>
__global__ __launch_bounds__(kRowThreads) void k_route_combine_grad(const CombineArgs a) {
    constexpr int E = Vec<EB>::E;
    const int n = a.tokens * a.topk;
    const int live = min(a.offsets[a.experts], n);
    const int lane = threadIdx.x & 63;
    for (size_t t = (size_t)blockIdx.x * (kRowThreads / 64) + threadIdx.x / 64;
         t < (size_t)a.tokens; t += (size_t)gridDim.x * (kRowThreads / 64)) {
        const char* dy = static_cast<const char*>(a.dy) + t * a.dystride * EB;
        for (int k = 0; k < a.topk; ++k) {
            const int d = a.dest[t * a.topk + k];
            const bool ok = d >= 0 && d < live;
            const float wk = a.weights[t * a.topk + k];
            float dot = 0.0f;
            if (d >= 0 && d < n) {
                const char* row = static_cast<const char*>(a.rows) + (size_t)d * a.hidden * EB;
                char* drow = static_cast<char*>(a.drows) + (size_t)d * a.hidden * EB;
                for (size_t i = (size_t)lane * E; i < a.hidden; i += 64 * E) {
                    u32x4 out = {0u, 0u, 0u, 0u};
                    if (ok) {
                        float g[E], v[E];
                        Vec<EB>::unpack(ld_unit_of<EB>(dy, i, a.hidden, 0u), g);
                        Vec<EB>::unpack(ld_unit_of<EB>(row, i, a.hidden, 0u), v);
#pragma unroll
                        for (int j = 0; j < E; ++j) {
                            dot = __builtin_fmaf(g[j], v[j], dot);
                            g[j] *= wk;
                        }
                        out = Vec<EB>::pack(g);
                    }
                    st_unit_of<EB>(drow, i, a.hidden, out);
                }
            }
            dot = wave_sum(dot);
            if (lane == 0) a.dweights[t * a.topk + k] = ok ? dot : 0.0f;
        }
    }
}

unsigned token_blocks(int tokens, int per) {
    constexpr int kMost = 1 << 22;
    const int b = tokens / per + (tokens % per != 0);
    return (unsigned)(b < 1 ? 1 : b < kMost ? b : kMost);
}

// The sort's split: as many blocks as there are kSortSlots, at most kSortBlocks
// (each block adds up the counts of all of them).
constexpr size_t kSortBlocks = 128;
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

template <int EB>
hipError_t rows_by_width(const DispatchArgs& a, hipStream_t s) {
    const size_t units = (a.hidden * EB + 15) / 16;
    if (units <= 64)
        hipLaunchKernelGGL((k_route_rows<EB, 64>), dim3(token_blocks(a.tokens, kRowThreads / 64)),
                           dim3(kRowThreads), 0, s, a);
    else
        hipLaunchKernelGGL((k_route_rows<EB, 256>), dim3(token_blocks(a.tokens, 1)),
                           dim3(kRowThreads), 0, s, a);
    return hipGetLastError();
}

template <int EB>
hipError_t combine_by_width(const CombineArgs& a, hipStream_t s) {
    const size_t units = (a.hidden * EB + 15) / 16;
    if (units <= 64)
        hipLaunchKernelGGL((k_route_combine<EB, 64>), dim3(token_blocks(a.tokens, kRowThreads / 64)),
                           dim3(kRowThreads), 0, s, a);
    else
        hipLaunchKernelGGL((k_route_combine<EB, 256>), dim3(token_blocks(a.tokens, 1)),
                           dim3(kRowThreads), 0, s, a);
    return hipGetLastError();
}

}  // namespace

size_t dispatch_work_ints(size_t slots, int experts) {
    return (size_t)sort_blocks(slots) * (size_t)(experts + 1);
}

hipError_t launch_dispatch(const DispatchArgs& a, hipStream_t s) {
    const size_t slots = (size_t)a.tokens * a.topk, share = sort_share(slots);
    const dim3 grid(sort_blocks(slots)), block(kSortThreads);
    if (slots > 0) {
        if (a.ib == 8) hipLaunchKernelGGL(k_route_count<8>, grid, block, 0, s, a, slots, share);
        else hipLaunchKernelGGL(k_route_count<4>, grid, block, 0, s, a, slots, share);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    if (a.ib == 8) hipLaunchKernelGGL(k_route_place<8>, grid, block, 0, s, a, slots, share);
    else hipLaunchKernelGGL(k_route_place<4>, grid, block, 0, s, a, slots, share);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || slots == 0) return e;
    return a.eb == 2 ? rows_by_width<2>(a, s) : rows_by_width<4>(a, s);
}

hipError_t launch_combine(const CombineArgs& a, hipStream_t s) {
    if (a.tokens == 0) return hipSuccess;
    return a.eb == 2 ? combine_by_width<2>(a, s) : combine_by_width<4>(a, s);
}

hipError_t launch_combine_grad(const CombineArgs& a, hipStream_t s) {
    if (a.tokens == 0) return hipSuccess;
    const dim3 grid(token_blocks(a.tokens, kRowThreads / 64)), block(kRowThreads);
    if (a.eb == 2) hipLaunchKernelGGL(k_route_combine_grad<2>, grid, block, 0, s, a);
    else hipLaunchKernelGGL(k_route_combine_grad<4>, grid, block, 0, s, a);
    return hipGetLastError();
}

}  // namespace arlib
