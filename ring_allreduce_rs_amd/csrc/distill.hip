// distill.hip -- distillation from a teacher's top logits, forward and backward.
//
// A row holds the student's logits z over the vocabulary, and the teacher's
// logits t at `top` places i_1 .. i_top.  With the temperature T:
//   p = softmax(t / T) over the entries kept (0 <= i_j < vocab)
//   q = softmax(z / T) over the vocabulary,  lse = log sum exp(z / T)
//   loss = T^2 sum_j p_j (log p_j - log q_{i_j})
//   d loss / d z_v = T (q_v - sum_{j: i_j = v} p_j)
// An entry with p_j = 0 adds nothing.  A row without a kept entry (or whose
// teacher logits are all -inf) has loss 0 and gradient 0, whatever z holds; a
// kept +inf or NaN among the teacher's makes every p_j of its row NaN.
//
// All sums are fp32 and are split the same way at every call, so results
// repeat bit for bit.  The traffic is the logits and their gradient; the
// teacher's entries are staged in LDS.
//
// MI355X: step of 4096 x 131072 bf16 408 us (5.3 TB/s; a copy of as many bytes
// 332), where two passes over the logits took 556; gradient of 2047 x 50021 fp32
// 155 us (5.3 TB/s; 127); loss of 1 x 131072 fp32 in two launches 7-9 us and
// step of 8 x 32000 bf16 7.9 us, both bound by launches and round trips.  A
// step's exponentials, two a logit at a quarter of the vector rate, take about
// 60 % of the time that its bytes take, which is why they have to overlap.
#include "ops.h"
#include "ops_device.h"

namespace arlib {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kMaxTop = 1024;
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

template <int IB>
__device__ __forceinline__ int place_of(const void* indices, size_t j, size_t vocab) {
    if constexpr (IB == 8) {
        const int64_t v = static_cast<const int64_t*>(indices)[j];
        return v >= 0 && v < (int64_t)vocab ? (int)v : -1;
    } else {
        const int32_t v = static_cast<const int32_t*>(indices)[j];
        return v >= 0 && (size_t)v < vocab ? v : -1;
    }
}

typedef int i32x4 __attribute__((ext_vector_type(4)));
// Entries of a row in LDS, rounded up so that four are read at a time; the
// places past the last are kNoPlace.
__host__ __device__ inline int padded(int top) { return (top + 3) & ~3; }
constexpr int kNoPlace = -2;

// How many of the row's entries name entry j's place, and how many of them
// before it.
__device__ __forceinline__ void count_same(const int* at, int pad, int j, int* same, int* before) {
    const i32x4* const quads = reinterpret_cast<const i32x4*>(at);
    const int mine = at[j];
    int s = 0, b = 0;
#pragma unroll 4
    for (int k = 0; k < pad; k += 4) {
        const i32x4 q = quads[k >> 2];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            s += q[i] == mine;
            b += q[i] == mine && k + i < j;
        }
    }
    *same = s;
    *before = b;
}

// The teacher of one row in LDS: places (-1: left out) and probabilities.
struct Teacher {
    alignas(16) int at[kMaxTop];
    float p[kMaxTop];
    float red[2][16];
};

template <int W>
__device__ __forceinline__ float block_max(float v, float* lds) {
    v = wave_max(v);
    if constexpr (W == 1) return v;
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
    __syncthreads();
    float t = lds[0];
#pragma unroll
    for (int w = 1; w < W; ++w) t = fmaxf(t, lds[w]);
    return t;
}

// Fills th for row r; returns whether the row has a teacher.  *zmax and *logs
// are what log p_j = t_j / T - zmax - logs takes.  A +inf logit less itself
// makes the sum, and so every p_j, NaN.  All threads call it.
template <int EB, int IB, int W>
__device__ bool load_teacher(const DistillArgs& a, size_t r, Teacher& th, float* zmax,
                             float* logs) {
    constexpr int NT = W * 64;
    const char* t = static_cast<const char*>(a.teacher) + r * a.top * EB;
    float m = -INFINITY;
    for (int j = threadIdx.x; j < (int)a.top; j += NT) {
        const int at = place_of<IB>(a.indices, r * a.top + j, a.vocab);
        const float z = at >= 0 ? Vec<EB>::ld1(t + (size_t)j * EB) / a.temperature : -INFINITY;
        th.at[j] = at;
        th.p[j] = z;
        m = z != z ? z : fmaxf(m, z);   // (a NaN reaches the sum below by itself)
    }
    if ((int)threadIdx.x < padded((int)a.top) - (int)a.top) th.at[a.top + threadIdx.x] = kNoPlace;
    m = block_max<W>(m == m ? m : -INFINITY, th.red[0]);
    const float base = m == -INFINITY ? 0.0f : m;
    float s = 0.0f;
    for (int j = threadIdx.x; j < (int)a.top; j += NT) {
        const float e = expf(th.p[j] - base);
        th.p[j] = e;
        s += e;
    }
    s = block_sum<W>(s, th.red[1]);
    *zmax = base;
    *logs = logf(s);
    const float inv = 1.0f / s;
    if (!(s == 0.0f))
        for (int j = threadIdx.x; j < (int)a.top; j += NT) th.p[j] *= inv;
    __syncthreads();
    return !(s == 0.0f);
}

// The row's loss, on every thread, with log q = (z - base) / T - logz.
template <int EB, int IB, int W>
__device__ float row_loss(const DistillArgs& a, size_t r, Teacher& th, float zmax, float logs,
                          float base, float logz) {
    const char* t = static_cast<const char*>(a.teacher) + r * a.top * EB;
    const char* z = static_cast<const char*>(a.logits) + r * a.lstride * EB;
    float s = 0.0f;
    for (int j = threadIdx.x; j < (int)a.top; j += W * 64) {
        const float p = th.p[j];
        if (th.at[j] < 0 || p == 0.0f) continue;
        const float logp = Vec<EB>::ld1(t + (size_t)j * EB) / a.temperature - zmax - logs;
        const float logq =
            (Vec<EB>::ld1(z + (size_t)th.at[j] * EB) - base) / a.temperature - logz;
        s = __builtin_fmaf(p, logp - logq, s);
    }
    __syncthreads();   // th.red is free again
    return block_sum<W>(s, th.red[0]) * (a.temperature * a.temperature);
}

// Running maximum and sum of exp((z - m) / T), c = log2(e) / T.
struct Soft {
    float m, s;
};
__device__ __forceinline__ Soft soft_zero() { return {-INFINITY, 0.0f}; }
// What the sum is relative to: an infinite maximum is left out, so that a row
// of -inf sums to 0 and a +inf makes the sum (and lse) infinite.
__device__ __forceinline__ float soft_base(float m) { return fabsf(m) < INFINITY ? m : 0.0f; }
// What q's exponentials are relative to: a +inf maximum, whose sum is infinite,
// stays, so that every finite value has exp(-inf) = 0 however large it is, and
// the infinite one NaN.
__device__ __forceinline__ float soft_top(float m) { return m > -INFINITY ? m : 0.0f; }
// The base that a sum of this maximum has, seen from another: -inf for an
// empty one, so that its 0 stays 0.
__device__ __forceinline__ float soft_from(float m) { return m < INFINITY ? m : 0.0f; }
__device__ __forceinline__ float soft_lse(Soft v, float temperature) {
    return soft_base(v.m) / temperature + logf(v.s);
}
__device__ __forceinline__ Soft soft_join(Soft a, Soft b, float c) {
    const float m = fmaxf(a.m, b.m);
    const float base = soft_base(m);
    // (a NaN in either sum stays in the sum)
    return {m, a.s * exp2_fast((soft_from(a.m) - base) * c) +
                   b.s * exp2_fast((soft_from(b.m) - base) * c)};
}
template <int E>
__device__ __forceinline__ void soft_add(Soft& a, const float (&v)[E], float c) {
    float m = a.m;
#pragma unroll
    for (int j = 0; j < E; ++j) m = fmaxf(m, v[j]);
    const float base = soft_base(m);
    float s = a.s * exp2_fast((soft_from(a.m) - base) * c);
#pragma unroll
    for (int j = 0; j < E; ++j) s += exp2_fast((v[j] - base) * c);
    a.m = m;
    a.s = s;
}
template <int W>
__device__ __forceinline__ Soft block_soft(Soft v, float c, Soft* lds) {
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) {
        const Soft o = {__shfl_xor(v.m, d, 64), __shfl_xor(v.s, d, 64)};
        v = soft_join(v, o, c);
    }
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
    __syncthreads();
    v = lds[0];
#pragma unroll
    for (int w = 1; w < W; ++w) v = soft_join(v, lds[w], c);
    return v;
}

// A wavefront's maximum and sum over its lanes'.
__device__ __forceinline__ Soft wave_soft(Soft v, float c) {
    const float m = wave_max(v.m);
    return {m, wave_sum(v.s * exp2_fast((soft_from(v.m) - soft_base(m)) * c))};
}
// G units added to a thread's share.  Values are taken from the maximum before
// they are scaled: scaled first (one fma less), a row of the type's lowest
// value would overflow.
template <int EB, int G>
__device__ __forceinline__ void soft_units(Soft& a, const u32x4* u, float c) {
    constexpr int E = Vec<EB>::E;
    float m = a.m;
#pragma unroll
    for (int g = 0; g < G; ++g) {
        float v[E];
        Vec<EB>::unpack(u[g], v);
#pragma unroll
        for (int j = 0; j < E; ++j) m = fmaxf(m, v[j]);
    }
    const float base = soft_base(m);
    float s = a.s * exp2_fast((soft_from(a.m) - base) * c);
#pragma unroll
    for (int g = 0; g < G; ++g) {
        float v[E];
        Vec<EB>::unpack(u[g], v);
#pragma unroll
        for (int j = 0; j < E; ++j) s += exp2_fast((v[j] - base) * c);
    }
    a.m = m;
    a.s = s;
}

// Units of a row's chunk in registers: thread x of NT holds units
// lo + u * NT + x for u < UPT, -inf where the chunk or the row ends.
template <int EB, int UPT, int NT>
struct Chunk {
    static constexpr int E = Vec<EB>::E;
    u32x4 raw[UPT];
    __device__ __forceinline__ static Place place(unsigned lo, int u, unsigned vocab) {
        return place_unit<E>((lo + u * NT + offset_here(threadIdx.x)) * E, vocab);
    }
    __device__ __forceinline__ void load(const char* z, unsigned lo, unsigned vocab) {
#pragma unroll
        for (int u = 0; u < UPT; ++u) raw[u] = ld_unit<EB, true>(z + place(lo, u, vocab).at * EB);
    }
    __device__ __forceinline__ void sum(Soft& acc, unsigned lo, unsigned vocab, float c) {
        constexpr uint32_t kNinf = EB == 2 ? 0xff80ff80u : 0xff800000u;
        constexpr int G = UPT < 4 ? UPT : 4;
#pragma unroll
        for (int u = 0; u < UPT; u += G) {
#pragma unroll
            for (int g = 0; g < G; ++g) {
                const int skip = place(lo, u + g, vocab).skip;
                if (skip) raw[u + g] = fill_first<EB>(raw[u + g], skip, kNinf);
            }
            soft_units<EB, G>(acc, raw + u, c);
        }
    }
};

// Maximum and sum of each chunk of each row; a row has `parts` of them.  Rows
// shorter than a unit (SHORT) are one chunk, a value a lane.
template <int EB, int UPT, bool SHORT>
__global__ __launch_bounds__(kThreads) void k_distill_part(const DistillArgs a, size_t parts) {
    __shared__ Soft lds[kWaves];
    const float c = kLog2e / a.temperature;
    for (size_t task = blockIdx.x; task < a.rows * parts; task += gridDim.x) {
        const size_t r = task / parts;
        const char* z = static_cast<const char*>(a.logits) + r * a.lstride * EB;
        Soft acc = soft_zero();
        if constexpr (SHORT) {
            const float one[1] = {threadIdx.x < a.vocab ? Vec<EB>::ld1(z + threadIdx.x * EB)
                                                        : -INFINITY};
            soft_add<1>(acc, one, c);
        } else {
            const unsigned lo = (unsigned)(task % parts) * (UPT * kThreads);
            Chunk<EB, UPT, kThreads> ch;
            ch.load(z, lo, (unsigned)a.vocab);
            ch.sum(acc, lo, (unsigned)a.vocab, c);
        }
        acc = block_soft<kWaves>(acc, c, lds);
        if (threadIdx.x == 0) {
            a.part[2 * task] = acc.m;
            a.part[2 * task + 1] = acc.s;
        }
        __syncthreads();
    }
}

// The row's maximum and sum from its parts, on every thread.
__device__ __forceinline__ Soft fold_parts(const DistillArgs& a, size_t r, size_t parts, float c) {
    Soft v = soft_zero();
    for (size_t k = threadIdx.x & 63; k < parts; k += 64)
        v = soft_join(v, Soft{a.part[2 * (r * parts + k)], a.part[2 * (r * parts + k) + 1]}, c);
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) {
        const Soft o = {__shfl_xor(v.m, d, 64), __shfl_xor(v.s, d, 64)};
        v = soft_join(v, o, c);
    }
    return v;
}

// Loss and lse of each row from its parts.
template <int EB, int IB>
__global__ __launch_bounds__(kThreads) void k_distill_loss(const DistillArgs a, size_t parts) {
    __shared__ Teacher th;
    const float c = kLog2e / a.temperature;
    for (size_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
        const Soft v = fold_parts(a, r, parts, c);
        const float lse = soft_lse(v, a.temperature);
        float zmax, logs;
        const bool some = load_teacher<EB, IB, kWaves>(a, r, th, &zmax, &logs);
        const float loss =
            row_loss<EB, IB, kWaves>(a, r, th, zmax, logs, soft_base(v.m), logf(v.s));
        if (threadIdx.x == 0) {
            a.loss[r] = some ? loss : 0.0f;
            a.lse[r] = lse;
        }
        __syncthreads();
    }
}

// Loss and lse in one launch, a block per row: the next chunk's units are
// loaded before this one's are added up.
template <int EB, int IB>
__global__ __launch_bounds__(kThreads) void k_distill_loss_rows(const DistillArgs a) {
    constexpr int UPT = 4;
    __shared__ Teacher th;
    __shared__ Soft lds[kWaves];
    const float c = kLog2e / a.temperature;
    const unsigned vocab = (unsigned)a.vocab, units = (vocab + Vec<EB>::E - 1) / Vec<EB>::E;
    for (size_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
        const char* z = static_cast<const char*>(a.logits) + r * a.lstride * EB;
        Chunk<EB, UPT, kThreads> now, next;
        now.load(z, 0, vocab);
        Soft acc = soft_zero();
        for (unsigned lo = 0; lo < units; lo += UPT * kThreads) {
            if (lo + UPT * kThreads < units) next.load(z, lo + UPT * kThreads, vocab);
            now.sum(acc, lo, vocab, c);
            now = next;
        }
        acc = block_soft<kWaves>(acc, c, lds);
        const float lse = soft_lse(acc, a.temperature);
        float zmax, logs;
        const bool some = load_teacher<EB, IB, kWaves>(a, r, th, &zmax, &logs);
        const float loss =
            row_loss<EB, IB, kWaves>(a, r, th, zmax, logs, soft_base(acc.m), logf(acc.s));
        if (threadIdx.x == 0) {
            a.loss[r] = some ? loss : 0.0f;
            a.lse[r] = lse;
        }
        __syncthreads();
    }
}

// The gradient of one chunk of a row, q from the parts (PARTS) or from lse_in.
// The chunk's loads are on their way while the teacher's entries are staged.
// The kept entries are written after the rest of the chunk, each place by the
// first entry that names it with the sum of its duplicates.
template <int EB, int IB, int UPT, bool PARTS>
__global__ __launch_bounds__(kThreads) void k_distill_grad(const DistillArgs a, size_t parts,
                                                           size_t soft_parts) {
    constexpr int E = Vec<EB>::E;
    __shared__ Teacher th;
    const float c = kLog2e / a.temperature, it = 1.0f / a.temperature;
    const unsigned vocab = (unsigned)a.vocab;
    for (size_t task = blockIdx.x; task < a.rows * parts; task += gridDim.x) {
        const size_t r = task / parts;
        const unsigned lo = (unsigned)(task % parts) * (UPT * kThreads);
        const char* z = static_cast<const char*>(a.logits) + r * a.lstride * EB;
        char* dz = static_cast<char*>(a.dlogits) + r * a.vocab * EB;
        Chunk<EB, UPT, kThreads> ch;
        const bool is_short = vocab < E;   // no 16 bytes in a row: a value a lane below
        if (!is_short) ch.load(z, lo, vocab);
        float zmax, logs;
        const bool some = load_teacher<EB, IB, kWaves>(a, r, th, &zmax, &logs);
        const float scale = a.dloss[r] * a.temperature;
        float base = 0.0f, lse = 0.0f, inv = 1.0f;
        if constexpr (PARTS) {
            const Soft v = fold_parts(a, r, soft_parts, c);
            base = soft_top(v.m);
            inv = 1.0f / v.s;
            if (lo == 0) {   // (uniform over the block)
                const float loss =
                    row_loss<EB, IB, kWaves>(a, r, th, zmax, logs, base, logf(v.s));
                if (threadIdx.x == 0) a.loss[r] = some ? loss : 0.0f;
            }
        } else {
            lse = a.lse_in[r];
        }
        const auto prob = [&](float v) -> float {
            if constexpr (PARTS) return exp2_fast((v - base) * c) * inv;
            // (fp32 results keep the digits that the scaled exponent would lose)
            const float x = __builtin_fmaf(v, it, -lse);
            return EB == 2 ? exp2_fast(x * kLog2e) : expf(x);
        };
        if (!is_short) {
#pragma unroll
            for (int u = 0; u < UPT; ++u) {
                u32x4 out = {0u, 0u, 0u, 0u};
                if (some) {
                    float v[E];
                    Vec<EB>::unpack(ch.raw[u], v);
#pragma unroll
                    for (int j = 0; j < E; ++j) v[j] = prob(v[j]) * scale;
                    out = Vec<EB>::pack(v);
                }
                st_place<EB, true, true>(dz, ch.place(lo, u, vocab), out);
            }
        } else if (threadIdx.x < vocab) {
            const float q = some ? prob(Vec<EB>::ld1(z + threadIdx.x * EB)) * scale : 0.0f;
            Vec<EB>::st1(dz + threadIdx.x * EB, q);
        }
        __syncthreads();
        const unsigned from = lo * E, to = from + UPT * kThreads * E;
        if (some)
            for (int j = threadIdx.x; j < (int)a.top; j += kThreads) {
                const int at = th.at[j];
                if (at < 0 || (unsigned)at < from || (unsigned)at >= to) continue;
                int same, before;
                count_same(th.at, padded((int)a.top), j, &same, &before);
                if (before) continue;
                float p = th.p[j];
                for (int k = j + 1; same > 1 && k < (int)a.top; ++k)
                    if (th.at[k] == at) p += th.p[k];
                const float q = prob(Vec<EB>::ld1(z + (size_t)at * EB));
                Vec<EB>::st1(dz + (size_t)at * EB, (q - p) * scale);
            }
        __syncthreads();
    }
}

// Loss and gradient of rows that a block holds in registers: UPT units a
// thread.  A block takes row after row, and while it turns one row's units into
// gradients it loads the next row's into the registers that become free, so
// that loads, exponentials and stores of one compute unit overlap although a
// row may fill most of its registers.
//
// Thread j keeps teacher entry j of the row (a block has a thread for each); the
// next row's entries are loaded among its units.  There is one barrier a row:
// before it every wavefront leaves its sums of this row, after it the entries'
// places of the row before are written again with q - p (its plain gradients
// were all stored before the barrier) and its loss is added up.  What one row
// leaves in LDS the next but one replaces.
struct RowSums {
    float m[16], s[16], tm[16], ts[16], loss[16];
};
// What a launch of the row kernel computes: loss and gradient, the gradient from
// a given lse, or loss and lse.
enum RowPass { PASS_STEP, PASS_BACKWARD, PASS_LOSS };

// FULL: every wavefront has lanes in each of its UPT units, and spends no branch
// on asking (4096 x 131072 bf16 407 us against 424).
template <int EB, int IB, int UPT, RowPass PASS, bool FULL>
__global__ __launch_bounds__(1024) void k_distill_rows(const DistillArgs a) {
    constexpr int E = Vec<EB>::E;
    constexpr uint32_t kNinf = EB == 2 ? 0xff80ff80u : 0xff800000u;
    constexpr bool kSums = PASS != PASS_BACKWARD, kGrad = PASS != PASS_LOSS;
    extern __shared__ i32x4 entries[];   // places, then teacher logits, of two rows
    __shared__ RowSums red[2];
    const int nt = blockDim.x, waves = nt >> 6, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int top = (int)a.top, tid = threadIdx.x, pad = padded(top);
    int* const at = reinterpret_cast<int*>(entries);
    float* const tz = reinterpret_cast<float*>(at + 2 * pad);
    const float c = kLog2e / a.temperature, it = 1.0f / a.temperature;
    u32x4 raw[UPT];
    // (worked out where it is used: kept, the masks of all units would take
    // more scalar registers than there are)
    const auto place = [&](int u) {
        return place_unit<E>((u * nt + offset_here(threadIdx.x)) * E, (unsigned)a.vocab);
    };
    // whether a unit is any lane's of this wavefront
    const int units = ((int)a.vocab + E - 1) / E;
    const int lane0 = __builtin_amdgcn_readfirstlane(tid);
    const auto live = [&](int u) { return FULL || u * nt + lane0 < units; };
    const auto logit = [&](size_t r, int v) {
        return Vec<EB>::ld1(static_cast<const char*>(a.logits) + (r * a.lstride + v) * EB);
    };
    const auto entry = [&](size_t r, int j, float* x) {
        const int v = place_of<IB>(a.indices, r * a.top + j, a.vocab);
        *x = Vec<EB>::ld1(static_cast<const char*>(a.teacher) + (r * a.top + j) * EB);
        return v;
    };

    size_t r = blockIdx.x;
    int my_at = -1;                 // this thread's entry of the row
    float my_t = -INFINITY, my_z = 0.0f;
    if (tid < top) my_at = entry(r, tid, &my_t);
    {
        const char* z = static_cast<const char*>(a.logits) + r * a.lstride * EB;
#pragma unroll
        for (int u = 0; u < UPT; ++u) {
            raw[u] = u32x4{0u, 0u, 0u, 0u};
            if (live(u)) raw[u] = ld_unit<EB, true>(z + place(u).at * EB);
        }
    }
    if (my_at >= 0) my_z = logit(r, my_at);   // (the row's loads are on their way)
    const auto stage = [&](int b) {
        if (tid < top) {
            my_t = my_at >= 0 ? my_t : -INFINITY;
            at[b * pad + tid] = my_at;
            tz[b * pad + tid] = my_t;
        }
        if (tid < pad - top) at[b * pad + top + tid] = kNoPlace;
    };
    stage(0);

    // the entry of the row before that is still to be written, and its loss
    bool owed = false;
    char* owed_at = nullptr;
    float owed_v = 0.0f;
    int b = 0;
    bool some_before = false;
    const auto settle_row = [&](size_t row, int rb) {
        if (kGrad && owed) Vec<EB>::st1(owed_at, owed_v);
        if (kSums && tid == 0) {
            float sum = 0.0f;
            for (int w = 0; w < waves; ++w) sum += red[rb].loss[w];
            a.loss[row] = some_before ? sum * (a.temperature * a.temperature) : 0.0f;
        }
    };

    for (; r < a.rows; r += gridDim.x, b ^= 1) {
        const int* const row_at = at + b * pad;
        const float* const row_tz = tz + b * pad;
        // this wavefront's share of both sums
        Soft zs = soft_zero(), ts = soft_zero();
        if constexpr (kSums) {
            constexpr int G = UPT < 4 ? UPT : 4;
#pragma unroll
            for (int u = 0; u < UPT; u += G) {
                if (!live(u)) continue;
#pragma unroll
                for (int g = 0; g < G; ++g) {
                    // (without a gradient to come back for, the compiler would
                    // unpack the next row's units as they arrive and spill)
                    if constexpr (!kGrad) refresh(raw[u + g]);
                    const int skip = place(u + g).skip;
                    if (skip) raw[u + g] = fill_first<EB>(raw[u + g], skip, kNinf);
                }
                soft_units<EB, G>(zs, raw + u, c);
                if constexpr (!kGrad) {
                    settle(zs.m);
                    settle(zs.s);
                }
            }
            zs = wave_soft(zs, c);
        }
        if (tid < top) {
            const float one[1] = {my_t};
            soft_add<1>(ts, one, c);
        }
        ts = wave_soft(ts, c);
        if (lane == 0) {
            red[b].m[wave] = zs.m;
            red[b].s[wave] = zs.s;
            red[b].tm[wave] = ts.m;
            red[b].ts[wave] = ts.s;
        }
        __syncthreads();
        if (r >= gridDim.x) settle_row(r - gridDim.x, b ^ 1);
        const bool has = lane < waves;
        const int w = lane & 15;
        if constexpr (kSums)
            zs = wave_soft({has ? red[b].m[w] : -INFINITY, has ? red[b].s[w] : 0.0f}, c);
        ts = wave_soft({has ? red[b].tm[w] : -INFINITY, has ? red[b].ts[w] : 0.0f}, c);
        if (ts.m == INFINITY) ts.s = NAN;   // (no softmax, as in load_teacher)
        const bool some = !(ts.s == 0.0f);
        const float scale = kGrad ? a.dloss[r] * a.temperature : 0.0f;
        const float base = soft_top(zs.m), logz = logf(zs.s), inv = 1.0f / zs.s;
        const float lse = kSums ? 0.0f : a.lse_in[r];
        const float tbase = soft_base(ts.m), logs = logf(ts.s), tinv = 1.0f / ts.s;
        char* dz = static_cast<char*>(a.dlogits) + r * a.vocab * EB;
        if (PASS == PASS_LOSS && tid == 0) a.lse[r] = soft_lse(zs, a.temperature);

        // loss terms, and the value that an entry's place gets
        const auto prob = [&](int j) { return exp2_fast((row_tz[j] - tbase) * c) * tinv; };
        const auto student = [&](float zj) {
            if constexpr (kSums) return exp2_fast((zj - base) * c) * inv;
            else return expf(__builtin_fmaf(zj, it, -lse));
        };
        float loss = 0.0f;
        owed = false;
        some_before = some;
        if (some && tid < top && my_at >= 0) {
            const float p = prob(tid);
            if (kSums && p != 0.0f)
                loss = p * ((my_t - tbase) / a.temperature - logs -
                            ((my_z - base) / a.temperature - logz));
            if constexpr (kGrad) {
                int same, before;
                count_same(row_at, pad, tid, &same, &before);
                float all = p;
                for (int k = tid + 1; same > 1 && k < top; ++k)
                    if (row_at[k] == my_at) all += prob(k);
                owed = before == 0;
                owed_at = dz + (size_t)my_at * EB;
                owed_v = (student(my_z) - all) * scale;
            }
        }
        if constexpr (kSums) {
            loss = wave_sum(loss);
            if (lane == 0) red[b].loss[wave] = loss;
        }

        // the row's gradient; the next row's units take the registers
        const bool more = r + gridDim.x < a.rows;
        const size_t next = r + gridDim.x;
        const char* zn = static_cast<const char*>(a.logits) + next * a.lstride * EB;
        if (more && tid < top) my_at = entry(next, tid, &my_t);
        const float gain = scale * inv, lift = log2f(fabsf(kSums ? gain : scale));
        const uint32_t sign = as_u32(scale) & 0x80000000u, sign2 = sign | (sign >> 16);
#pragma unroll
        for (int u = 0; u < UPT; ++u) {
            if (u == UPT / 2 && more && tid < top && my_at >= 0) my_z = logit(next, my_at);
            if (!live(u)) continue;
            const Place pl = place(u);
            if constexpr (kGrad) {
                u32x4 out = {0u, 0u, 0u, 0u};
                refresh(raw[u]);
                if (some) {
                    float v[E];
                    Vec<EB>::unpack(raw[u], v);
                    if constexpr (EB == 2) {
                        // the factor goes into the exponent, where fp32 still
                        // holds 2^-18 of a value: bf16 rounds at 2^-8
#pragma unroll
                        for (int j = 0; j < E; ++j)
                            v[j] = kSums ? exp2_fast(__builtin_fmaf(v[j] - base, c, lift))
                                         : exp2_fast(__builtin_fmaf(
                                               __builtin_fmaf(v[j], it, -lse), kLog2e, lift));
                        out = Vec<EB>::pack(v);
#pragma unroll
                        for (int i = 0; i < 4; ++i) out[i] ^= sign2;
                    } else {
#pragma unroll
                        for (int j = 0; j < E; ++j)
                            v[j] = kSums ? exp2_fast((v[j] - base) * c) * gain
                                         : expf(__builtin_fmaf(v[j], it, -lse)) * scale;
                        out = Vec<EB>::pack(v);
                    }
                }
                st_place<EB, true, true>(dz, pl, out);
            }
            if (more) raw[u] = ld_unit<EB, true>(zn + pl.at * EB);
        }
        if (more) stage(b ^ 1);
    }
    __syncthreads();
    if (r >= gridDim.x) settle_row(r - gridDim.x, b ^ 1);
}

// The split of rows into chunks of UPT units a thread: 8, or 2 where there are
// too few chunks of 8 for the card's compute units or rows fill less than half
// of one.
struct Split {
    int upt;
    size_t parts;
};
Split split_of(size_t rows, size_t vocab, int eb) {
    const size_t e = 16 / (size_t)eb, units = (vocab + e - 1) / e;
    const size_t parts = (units + 8 * kThreads - 1) / (8 * kThreads);
    if (rows * parts >= 1024 && units > 4 * kThreads) return {8, parts};
    return {2, (units + 2 * kThreads - 1) / (2 * kThreads)};
}

// The register form of a step: units per thread and threads; upt 0: the row
// does not fit (or is shorter than a unit), the two-pass form takes it.  Fewer
// units a thread give a row more threads, which pays while the rows are too few
// to fill the card's compute units.
constexpr int kCUs = 256;
struct RowFit {
    int upt, threads;
};
// (Above 256 threads in steps of 256, so that a compute unit's four SIMDs get
// the same number of wavefronts: 2047 x 50021 bf16 103 us, with the 13
// wavefronts that it takes instead of 16 126 us.)
RowFit row_fit(size_t rows, size_t vocab, size_t top, int eb) {
    const size_t e = 16 / (size_t)eb, units = (vocab + e - 1) / e;
    const auto threads = [&](size_t upt) {
        const size_t need = (units + upt - 1) / upt, nt = need > top ? need : top;
        const size_t step = nt > 256 ? 256 : 64;
        return (nt + step - 1) / step * step;
    };
    if (vocab < e || threads(16) > 1024) return {0, 0};
    int upt = 16;
    while (upt > 4 && threads(upt / 2) <= 1024 &&
           (rows * threads(upt) < (size_t)kCUs * 1024 || threads(upt / 2) == threads(upt)))
        upt /= 2;
    return {upt, (int)threads(upt)};
}
// Few long rows leave most compute units without one: two passes over chunks
// (1 x 131072 bf16 11.6 us against 17.3, 64 x 100000 18.3 against 19.5; 1 x
// 32000 is better off in one launch, 8.4 against 11.9).
RowFit step_fit(size_t rows, size_t vocab, size_t top, int eb) {
    const RowFit fit = row_fit(rows, vocab, top, eb);
    return rows <= 64 && fit.upt * fit.threads > 4096 ? RowFit{0, 0} : fit;
}

unsigned grid_of(size_t tasks) {
    constexpr size_t kMost = size_t(1) << 22;
    return (unsigned)(tasks < kMost ? tasks : kMost);
}

#define DISTILL_BY_TYPE(CALL)                     \
    do {                                          \
        if (a.eb == 2 && a.ib == 4) { CALL(2, 4); } \
        else if (a.eb == 2) { CALL(2, 8); }       \
        else if (a.ib == 4) { CALL(4, 4); }       \
        else { CALL(4, 8); }                      \
    } while (0)

hipError_t launch_part(const DistillArgs& a, Split sp, hipStream_t s) {
    const dim3 grid(grid_of(a.rows * sp.parts)), block(kThreads);
#define CALL(EB, UPT, SHORT) \
    hipLaunchKernelGGL((k_distill_part<EB, UPT, SHORT>), grid, block, 0, s, a, sp.parts)
    if (a.vocab < (size_t)(16 / a.eb)) {
        if (a.eb == 2) CALL(2, 2, true);
        else CALL(4, 2, true);
    } else if (sp.upt == 8) {
        if (a.eb == 2) CALL(2, 8, false);
        else CALL(4, 8, false);
    } else {
        if (a.eb == 2) CALL(2, 2, false);
        else CALL(4, 2, false);
    }
#undef CALL
    return hipGetLastError();
}

template <bool PARTS>
hipError_t launch_grad(const DistillArgs& a, Split sp, hipStream_t s) {
    const dim3 grid(grid_of(a.rows * sp.parts)), block(kThreads);
#define CALL(EB, IB)                                                                              \
    if (sp.upt == 8)                                                                              \
        hipLaunchKernelGGL((k_distill_grad<EB, IB, 8, PARTS>), grid, block, 0, s, a, sp.parts,    \
                           sp.parts);                                                             \
    else                                                                                          \
        hipLaunchKernelGGL((k_distill_grad<EB, IB, 2, PARTS>), grid, block, 0, s, a, sp.parts,    \
                           sp.parts)
    DISTILL_BY_TYPE(CALL);
#undef CALL
    return hipGetLastError();
}

template <RowPass PASS>
hipError_t launch_rows(const DistillArgs& a, RowFit fit, hipStream_t s) {
    // as many blocks as run at once: the registers of 4 units a thread leave
    // room for 24 wavefronts a compute unit, the others' for 16
    const size_t most = (size_t)kCUs * (fit.upt == 4 ? 1536 : 1024) / fit.threads;
    const dim3 grid((unsigned)(a.rows < most ? a.rows : most)), block(fit.threads);
    const size_t lds = (size_t)padded((int)a.top) * 4 * sizeof(float);
    const size_t e = 16 / (size_t)a.eb, units = (a.vocab + e - 1) / e;
    const bool full = PASS == PASS_STEP && units + 63 >= (size_t)fit.threads * 16;
#define LAUNCH(EB, IB, UPT, FULL) \
    hipLaunchKernelGGL((k_distill_rows<EB, IB, UPT, PASS, FULL>), grid, block, lds, s, a)
#define CALL(EB, IB)                                                                    \
    if (fit.upt == 4) LAUNCH(EB, IB, 4, false);                                         \
    else if (fit.upt == 8) LAUNCH(EB, IB, 8, false);                                    \
    else if (full) LAUNCH(EB, IB, 16, PASS == PASS_STEP);                               \
    else LAUNCH(EB, IB, 16, false)
    DISTILL_BY_TYPE(CALL);
#undef CALL
#undef LAUNCH
    return hipGetLastError();
}

// From this many rows on the loss takes a block per row and one launch.  Rows
// of up to kRowUnits units take the row kernel for the loss and for the
// gradient too (7698 x 1856 fp32 loss 19 us against 27, 2047 x 8001 bf16
// gradient 21 against 30); longer ones, whose pass has no use for the whole row
// at once, are faster in chunks (2047 x 50021 fp32 loss 73 against 100,
// gradient 164 against 176).
constexpr size_t kLossRows = 512;
constexpr int kRowUnits = 4096;
bool loss_by_rows(size_t rows, size_t vocab, int eb) {
    return rows >= kLossRows && vocab >= (size_t)(16 / eb);
}

}  // namespace

size_t distill_work_floats(size_t rows, size_t vocab, size_t top, int eb, bool step) {
    if (rows == 0 ||
        (step ? step_fit(rows, vocab, top, eb).upt != 0 : loss_by_rows(rows, vocab, eb)))
        return 0;
    return 2 * rows * split_of(rows, vocab, eb).parts;
}

hipError_t launch_distill_loss(const DistillArgs& a, hipStream_t s) {
    if (a.rows == 0) return hipSuccess;
    const dim3 grid(grid_of(a.rows)), block(kThreads);
    if (loss_by_rows(a.rows, a.vocab, a.eb)) {
        const RowFit fit = row_fit(a.rows, a.vocab, a.top, a.eb);
        if (fit.upt && fit.threads * fit.upt <= kRowUnits) return launch_rows<PASS_LOSS>(a, fit, s);
#define CALL(EB, IB) hipLaunchKernelGGL((k_distill_loss_rows<EB, IB>), grid, block, 0, s, a)
        DISTILL_BY_TYPE(CALL);
#undef CALL
        return hipGetLastError();
    }
    const Split sp = split_of(a.rows, a.vocab, a.eb);
    const hipError_t e = launch_part(a, sp, s);
    if (e != hipSuccess) return e;
#define CALL(EB, IB) hipLaunchKernelGGL((k_distill_loss<EB, IB>), grid, block, 0, s, a, sp.parts)
    DISTILL_BY_TYPE(CALL);
#undef CALL
    return hipGetLastError();
}

hipError_t launch_distill_backward(const DistillArgs& a, hipStream_t s) {
    if (a.rows == 0) return hipSuccess;
    const RowFit fit = row_fit(a.rows, a.vocab, a.top, a.eb);
    if (fit.upt && fit.threads * fit.upt <= kRowUnits && a.rows >= kLossRows)
        return launch_rows<PASS_BACKWARD>(a, fit, s);
    return launch_grad<false>(a, split_of(a.rows, a.vocab, a.eb), s);
}

hipError_t launch_distill_step(const DistillArgs& a, hipStream_t s) {
    if (a.rows == 0) return hipSuccess;
    const RowFit fit = step_fit(a.rows, a.vocab, a.top, a.eb);
    if (fit.upt) return launch_rows<PASS_STEP>(a, fit, s);
    const Split sp = split_of(a.rows, a.vocab, a.eb);
    const hipError_t e = launch_part(a, sp, s);
    return e != hipSuccess ? e : launch_grad<true>(a, sp, s);
}

}  // namespace arlib
