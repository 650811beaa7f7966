// Routing of tokens to experts, the order of their rows, and the weighted sum
// that puts a token's rows together again (see gemm_f16_experts.h).

#include <hip/hip_runtime.h>

#include <algorithm>
#include <stddef.h>
#include <stdint.h>

#include "gemm_f16_experts.h"

namespace gemm_f16_experts {

typedef _Float16 half8_t __attribute__((ext_vector_type(8)));
// 16 bytes at any 2-byte alignment (the target's unaligned-access mode)
typedef _Float16 half8_u_t __attribute__((ext_vector_type(8), aligned(2)));

constexpr int MOST_EXPERTS = 1024, MOST_TOP = 32, MOST_GROUPS = 64;

// The wave's index in its workgroup, in a scalar register.
__device__ __forceinline__ int wave_index() { return __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); }

// This workgroup's unit of work, where each XCD (workgroups mod 8) takes a
// contiguous range of them: neighbours share cache lines in its L2.
__device__ __forceinline__ int32_t xcd_unit()
{
    const int32_t q = gridDim.x >> 3, rem = gridDim.x & 7, x = blockIdx.x & 7;
    return x * q + (x < rem ? x : rem) + (blockIdx.x >> 3);
}

// Between a wave's LDS writes and its other lanes' reads of them: see that the
// compiler keeps their order (a wave's LDS operations are done in order).
__device__ __forceinline__ void wave_lds_fence()
{
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront", "local");
    __builtin_amdgcn_wave_barrier();
}

__device__ __forceinline__ double shfl_xor64(double v, int d)
{
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = __shfl_xor(static_cast<uint32_t>(b), d);
    const uint32_t hi = __shfl_xor(static_cast<uint32_t>(b >> 32), d);
    return __builtin_bit_cast(double, static_cast<uint64_t>(hi) << 32 | lo);
}

template <class T>
__device__ __forceinline__ T readlane64(T v, int lane)
{
    static_assert(sizeof(T) == 8, "two registers");
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = __builtin_amdgcn_readlane(static_cast<uint32_t>(b), lane);
    const uint32_t hi = __builtin_amdgcn_readlane(static_cast<uint32_t>(b >> 32), lane);
    return __builtin_bit_cast(T, static_cast<uint64_t>(hi) << 32 | lo);
}

// The largest of L neighbouring lanes' values (32 or 64), in each of them: rotations
// within rows of 16 lanes, then rows and halves of the wave exchanged.
template <int L>
__device__ __forceinline__ uint32_t lanes_max(uint32_t v)
{
    static_assert(L == 32 || L == 64, "lanes of a token");
#define STEP(CTRL) v = max(v, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, v, CTRL, 0xf, 0xf, true)))
    STEP(0x128);   // row_ror 8, 4, 2, 1
    STEP(0x124);
    STEP(0x122);
    STEP(0x121);
#undef STEP
    const auto rows = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    v = max(rows[0], rows[1]);
    if constexpr (L == 64) {
        const auto halves = __builtin_amdgcn_permlane32_swap(v, v, false, false);
        v = max(halves[0], halves[1]);
    }
    return v;
}

// Their sum, halves of the wave first: a token has the same sums in 32 lanes, which
// add experts l and l + 32 of each 64 (below), as in 64.
template <int L>
__device__ __forceinline__ double lanes_sum(double v)
{
#define STEP(CTRL)                                                                               \
    {                                                                                            \
        const uint64_t b = __builtin_bit_cast(uint64_t, v);                                      \
        const uint32_t lo = __builtin_amdgcn_update_dpp(0, static_cast<uint32_t>(b), CTRL, 0xf, 0xf, true); \
        const uint32_t hi = __builtin_amdgcn_update_dpp(0, static_cast<uint32_t>(b >> 32), CTRL, 0xf, 0xf, true); \
        v += __builtin_bit_cast(double, static_cast<uint64_t>(hi) << 32 | lo);                   \
    }
#define SWAP(HOW)                                                                                \
    {                                                                                            \
        const uint64_t b = __builtin_bit_cast(uint64_t, v);                                      \
        const auto lo = HOW(static_cast<uint32_t>(b), static_cast<uint32_t>(b), false, false);   \
        const auto hi = HOW(static_cast<uint32_t>(b >> 32), static_cast<uint32_t>(b >> 32), false, false); \
        v = __builtin_bit_cast(double, static_cast<uint64_t>(hi[0]) << 32 | lo[0]) +             \
            __builtin_bit_cast(double, static_cast<uint64_t>(hi[1]) << 32 | lo[1]);              \
    }
    if constexpr (L == 64) SWAP(__builtin_amdgcn_permlane32_swap)
    SWAP(__builtin_amdgcn_permlane16_swap)
    STEP(0x128);   // row_ror 8, 4, 2, 1
    STEP(0x124);
    STEP(0x122);
    STEP(0x121);
#undef STEP
#undef SWAP
    return v;
}

// Whether a condition holds in any of the lane's L lanes.
template <int L>
__device__ __forceinline__ bool lanes_any(bool v)
{
    const uint64_t b = __ballot(v);
    return L == 64 ? b != 0 : (threadIdx.x & 32 ? b >> 32 : b & 0xffffffffu) != 0;
}

// Numbers as integers in the same order (no NaN among them).
__device__ __forceinline__ uint32_t ordered(float v)
{
    const uint32_t b = __builtin_bit_cast(uint32_t, v);
    return b >> 31 ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float unordered(uint32_t b)
{
    return __builtin_bit_cast(float, b >> 31 ? b & 0x7fffffffu : ~b);
}
__device__ __forceinline__ uint64_t ordered(double v)
{
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    return b >> 63 ? ~b : b | 0x8000000000000000ull;
}

// ---------------------------------------------------------------------------
// The choice: one wave a token, or two tokens a wave
// ---------------------------------------------------------------------------
// Bound by the vector ALU: by its issue where tokens fill the card, below that by the
// chain of a token's 64-bit exponentials, quotients and the choices' reductions.
struct RouteParams {
    const void *logits;
    const float *bias;
    int32_t *experts;
    float *weights;
    double scale;
    int32_t T, E, top, groups, top_groups;
    bool f32, sigmoid, group_max, renormalize;
};

__device__ __forceinline__ double load_logit(const void *logits, bool f32, int64_t at)
{
    return f32 ? static_cast<double>(static_cast<const float *>(logits)[at])
               : static_cast<double>(static_cast<float>(static_cast<const _Float16 *>(logits)[at]));
}

// (The exchanges above need every lane: none stands behind a condition on the lane.)

// Of a token's L lanes lane l holds experts l, l + L, ...: their logits x to their
// scores s.  Absent experts have x = -inf.  False where the row has none (a NaN, or
// +inf with softmax).
template <int L, int V>
__device__ __forceinline__ bool scores_of(const double (&x)[V], bool sigmoid, double (&s)[V])
{
    constexpr double inf = __builtin_huge_val();
    bool bad = false;
#pragma unroll
    for (int i = 0; i < V; ++i) bad |= !(x[i] == x[i]) || (!sigmoid && x[i] == inf);
    const bool fine = !lanes_any<L>(bad);
    if (sigmoid) {
#pragma unroll
        for (int i = 0; i < V; ++i) s[i] = 1.0 / (1.0 + exp(-x[i]));
        return fine;
    }
    // the largest, exactly: logits are fp32 numbers
    uint32_t most = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) most = max(most, ordered(static_cast<float>(x[i])));
    const double m = static_cast<double>(unordered(lanes_max<L>(most)));
    double sums[2] = {0.0, 0.0};   // with 32 lanes, of the first and the second of each 64
#pragma unroll
    for (int i = 0; i < V; ++i) {
        s[i] = x[i] == -inf ? 0.0 : exp(x[i] - m);
        sums[L == 32 ? i % 2 : 0] += s[i];
    }
    const double sum = lanes_sum<L>(sums[0] + sums[1]);
    const double by = sum > 0.0 ? sum : 1.0;
#pragma unroll
    for (int i = 0; i < V; ++i) s[i] /= by;
    return fine;
}

template <int V>
__device__ __forceinline__ int32_t route_token(const RouteParams &p, int32_t t, int lane, double *cs)
{
    constexpr double inf = __builtin_huge_val();
    double x[V], s[V], c[V];
    float bias[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int32_t e = i * 64 + lane;
        x[i] = e < p.E ? load_logit(p.logits, p.f32, static_cast<int64_t>(t) * p.E + e) : -inf;
        bias[i] = p.bias && e < p.E ? p.bias[e] : 0.0f;
    }
    bool fine = scores_of<64>(x, p.sigmoid, s);
    if (fine) {
        bool bad = false;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            c[i] = s[i] + static_cast<double>(bias[i]);
            if (x[i] == -inf) c[i] = -inf;
            bad |= !(c[i] == c[i]);
        }
        fine = !__any(bad);
    }
    const int64_t out = static_cast<int64_t>(t) * p.top;
    if (!fine) {
        if (lane < p.top) {
            p.experts[out + lane] = -1;
            p.weights[out + lane] = __builtin_nanf("");
        }
        return -1;
    }
    if (p.groups > 1) {
        const int32_t per = p.E / p.groups;
        wave_lds_fence();
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (i * 64 + lane < p.E) cs[i * 64 + lane] = c[i];
        wave_lds_fence();
        // 64 / groups lanes a group (groups rounded up to a power of two)
        int shift = 6;
        while ((64 >> shift) < p.groups) --shift;
        const int g = lane >> shift;
        double first = -inf, second = -inf;
        if (g < p.groups)
            for (int32_t j = lane & ((1 << shift) - 1); j < per; j += 1 << shift) {
                const double v = cs[g * per + j];
                second = fmax(second, fmin(first, v));
                first = fmax(first, v);
            }
        for (int d = 1; d < 1 << shift; d *= 2) {
            const double f = shfl_xor64(first, d), o = shfl_xor64(second, d);
            second = fmax(fmax(second, o), fmin(first, f));
            first = fmax(first, f);
        }
        double score = first;
        if (!p.group_max && second > -inf) score += second;
        int rank = 0;
        for (int q = 0; q < p.groups; ++q) {
            const double o = readlane64(score, q << shift);
            rank += o > score || (o == score && q < g) ? 1 : 0;
        }
        const uint64_t kept = __ballot(g < p.groups && first > -inf && rank < p.top_groups);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int32_t e = i * 64 + lane;
            if (e < p.E && !(kept >> ((e / per) << shift) & 1)) c[i] = -inf;
        }
    }
    uint64_t key[V];
#pragma unroll
    for (int i = 0; i < V; ++i) key[i] = ordered(c[i]);
    const uint64_t none = ordered(-inf);
    int32_t mine = -1;
    double weight = 0.0;
    for (int j = 0; j < p.top; ++j) {
        // the lane's highest, its lowest index first
        uint64_t best = key[0];
        int at = 0;
#pragma unroll
        for (int i = 1; i < V; ++i)
            if (key[i] > best) {
                best = key[i];
                at = i;
            }
        const uint32_t hi = static_cast<uint32_t>(best >> 32);
        uint32_t e = static_cast<uint32_t>(at * 64 + lane);
        const uint32_t most = lanes_max<64>(hi);
        uint64_t has = __ballot(hi == most);
        if (has & (has - 1)) {
            // several lanes with the same upper halves: the lower ones, then the lowest
            // expert
            const uint32_t lo = lanes_max<64>(hi == most ? static_cast<uint32_t>(best) : 0u);
            const bool top = hi == most && static_cast<uint32_t>(best) == lo;
            const uint32_t first = ~lanes_max<64>(top ? ~e : 0u);
            has = __ballot(top && e == first);
        }
        const int from = __builtin_ctzll(has);
        if (readlane64(best, from) <= none) break;
        e = __builtin_amdgcn_readlane(e, from);
        double v = 0.0;
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (e == static_cast<uint32_t>(i * 64 + lane)) {
                key[i] = 0;
                v = s[i];
            }
        v = readlane64(v, from);
        if (lane == j) {
            mine = static_cast<int32_t>(e);
            weight = v;
        }
    }
    const double total = lanes_sum<64>(weight);
    if (lane < p.top) {
        weight *= p.scale;
        if (p.renormalize) weight /= total + 1e-20;
        p.experts[out + lane] = mine;
        p.weights[out + lane] = mine < 0 ? 0.0f : static_cast<float>(weight);
    }
    return mine;
}

template <int V>
__global__ __launch_bounds__(256) void route_kernel(RouteParams p)
{
    __shared__ double cs[4][64 * V];
    const int lane = threadIdx.x & 63, wave = wave_index();
    const int32_t t = blockIdx.x * 4 + wave;
    if (t < p.T) route_token<V>(p, t, lane, cs[wave]);
}

// Two tokens a wave, 32 lanes each: up to 128 experts in one group.  A choice is one
// reduction where the scores' upper halves tell all apart; the lane that has it
// notes its expert in LDS, and what belongs to the choices is looked up at the end.
// 8191 tokens of 128 experts, 6 chosen, 10.0 us (a wave a token 11.0; with the order
// 17.5 and 18.7, of 131072 tokens 81 and 115, of 64 experts 52 and 84).
template <int V>
__global__ __launch_bounds__(256) void route_pairs_kernel(RouteParams p)
{
    constexpr double inf = __builtin_huge_val();
    __shared__ double scores[4][64 * V];
    __shared__ int32_t chosen[4][64];
    const int lane = threadIdx.x & 63, wave = wave_index(), sub = lane & 31;
    const int32_t first = (blockIdx.x * 4 + wave) * 2;
    if (first >= p.T) return;
    // the last token twice where there is no second
    const int32_t t = min(first + lane / 32, p.T - 1);
    double x[V], s[V];
    float bias[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int32_t e = i * 32 + sub;
        x[i] = e < p.E ? load_logit(p.logits, p.f32, static_cast<int64_t>(t) * p.E + e) : -inf;
        bias[i] = p.bias && e < p.E ? p.bias[e] : 0.0f;
    }
    bool fine = scores_of<32>(x, p.sigmoid, s), bad = false;
    uint32_t hi[V], lo[V];   // of the ordered numbers of the choice's scores
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const double c = x[i] == -inf ? -inf : s[i] + static_cast<double>(bias[i]);
        bad |= !(c == c);
        const uint64_t key = ordered(c);
        hi[i] = static_cast<uint32_t>(key >> 32);
        lo[i] = static_cast<uint32_t>(key);
    }
    const bool any = lanes_any<32>(bad);
    fine = fine && !any;
    const uint32_t none = static_cast<uint32_t>(ordered(-inf) >> 32);   // no number's upper half
    chosen[wave][lane] = -1;
    wave_lds_fence();
    for (int32_t j = 0; j < p.top; ++j) {
        uint32_t most = hi[0], less = lo[0];
        int at = 0;
#pragma unroll
        for (int i = 1; i < V; ++i)
            if (hi[i] > most || (hi[i] == most && lo[i] > less)) {
                most = hi[i];
                less = lo[i];
                at = i;
            }
        const uint32_t top = lanes_max<32>(most);
        bool mine = most == top;
        const uint64_t has = __ballot(mine);   // one of each half at least
        if (has & (has - 0x0000000100000001ull)) {
            // several with the same upper halves: the lower ones, then the lowest expert
            const uint32_t l = lanes_max<32>(mine ? less : 0u);
            mine = mine && less == l;
            const uint32_t e = static_cast<uint32_t>(at * 32 + sub);
            const uint32_t lowest = ~lanes_max<32>(mine ? ~e : 0u);   // in all lanes
            mine = mine && e == lowest;
        }
        if (!__any(top > none)) break;
        if (mine && top > none) {
            chosen[wave][(lane & 32) + j] = at * 32 + sub;
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (at == i) hi[i] = 0;
        }
    }
#pragma unroll
    for (int i = 0; i < V; ++i) scores[wave][(lane / 32 * V + i) * 32 + sub] = s[i];
    wave_lds_fence();
    const int32_t e = chosen[wave][lane];
    double weight = e >= 0 ? scores[wave][lane / 32 * V * 32 + e] : 0.0;
    const double total = lanes_sum<32>(weight);
    if (sub >= p.top || first + lane / 32 >= p.T) return;
    weight *= p.scale;
    if (p.renormalize) weight /= total + 1e-20;
    const int64_t out = static_cast<int64_t>(t) * p.top + sub;
    p.experts[out] = fine ? e : -1;
    p.weights[out] = !fine ? __builtin_nanf("") : e < 0 ? 0.0f : static_cast<float>(weight);
}

// ---------------------------------------------------------------------------
// The order of the slots: a stable counting sort
// ---------------------------------------------------------------------------
// A workgroup orders a chunk of the slots, 1024 at a time: a wave finds for each
// slot how many of its lanes before it go to the same expert, the waves' counts
// and the chunk's first position of each expert give the rest.  Where there are
// several chunks their counts come from a kernel before.  49146 slots of 128
// experts: 5.5 to 6.5 us and 1.6 to 4 before it (one workgroup for all slots: 109 us).
struct OrderParams {
    const int32_t *experts;
    int32_t *rows, *places, *offsets;
    int32_t *counts;                 // [chunk][expert]; unused for one chunk
    int32_t S, E, chunks, chunk;     // slots of a chunk: a multiple of 1024
};

// The lanes of a wave with the same key below 2^bits, as a mask.
__device__ __forceinline__ uint64_t same_key(uint32_t key, int bits)
{
    uint64_t same = ~0ull;
    for (int b = 0; b < bits; ++b) {
        const uint64_t set = __ballot(key >> b & 1);
        same &= key >> b & 1 ? set : ~set;
    }
    return same;
}

// An expert's index, E for none.
__device__ __forceinline__ uint32_t expert_of(int32_t e, int32_t E)
{
    return min(static_cast<uint32_t>(e), static_cast<uint32_t>(E));
}

__global__ __launch_bounds__(1024) void count_kernel(OrderParams p)
{
    __shared__ int32_t count[MOST_EXPERTS + 1];
    const int tid = threadIdx.x;
    const int32_t from = blockIdx.x * p.chunk, to = from + min(p.S - from, p.chunk);
    if (tid < p.E) count[tid] = 0;
    __syncthreads();
    for (int32_t s = from + tid; s < to; s += 1024) {
        const uint32_t e = expert_of(p.experts[s], p.E);
        if (e < static_cast<uint32_t>(p.E)) atomicAdd(&count[e], 1);
    }
    __syncthreads();
    if (tid < p.E) p.counts[static_cast<int64_t>(blockIdx.x) * p.E + tid] = count[tid];
}

struct OrderMemory {
    int32_t base[MOST_EXPERTS + 1];      // next position of each expert
    int32_t parts[2][1024];
    uint16_t counts[16 * (MOST_EXPERTS + 1)];
    int32_t sums[16];
};

// Chunk `c`'s slots by a workgroup of 16 waves; ONE: the only one, and its slots'
// experts, at most 1024, are in `mine` by thread.
template <bool ONE>
__device__ __forceinline__ void order_chunk(const OrderParams &p, int32_t c, int32_t mine, OrderMemory &m)
{
    const int tid = threadIdx.x, lane = tid & 63, wave = wave_index();
    const int32_t E = p.E, from = c * p.chunk, to = from + min(p.S - from, p.chunk);
    int32_t count = 0, before = 0;       // of expert `tid`: all slots, those of the chunks before
    if (ONE || p.chunks == 1) {
        if (tid < E) m.base[tid] = 0;
        __syncthreads();
        for (int32_t s = from + tid; s < to; s += 1024) {
            const uint32_t e = expert_of(ONE ? mine : p.experts[s], E);
            if (e < static_cast<uint32_t>(E)) atomicAdd(&m.base[e], 1);
        }
        __syncthreads();
        if (tid < E) count = m.base[tid];
    } else {
        // 1024 / E threads an expert, each every so many chunks
        const int32_t share = 1024 / E, e = tid % E, part = tid / E;
        if (part < share)
#pragma unroll 8
            for (int32_t i = part; i < p.chunks; i += share) {
                const int32_t n = p.counts[static_cast<int64_t>(i) * E + e];
                count += n;
                before += i < c ? n : 0;
            }
        m.parts[0][tid] = count;
        m.parts[1][tid] = before;
        __syncthreads();
        count = before = 0;
        if (tid < E)
            for (int32_t i = 0; i < share; ++i) {
                count += m.parts[0][i * E + tid];
                before += m.parts[1][i * E + tid];
            }
    }
    int32_t upto = count;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const int32_t o = __shfl_up(upto, d);
        if (lane >= d) upto += o;
    }
    if (lane == 63) m.sums[wave] = upto;
    __syncthreads();
    int32_t all = 0;
#pragma unroll
    for (int w = 0; w < 16; ++w) {
        const int32_t n = m.sums[w];
        if (w < wave) upto += n;
        all += n;
    }
    if (tid < E) {
        m.base[tid] = upto - count + before;
        if (c == 0) p.offsets[tid] = upto - count;
    }
    if (c == 0 && tid == 0) p.offsets[E] = all;
    const int bits = 32 - __builtin_clz(E);
    for (int32_t s0 = from; s0 < to; s0 += 1024) {
        for (int32_t e = tid; e < 16 * (E + 1); e += 1024) m.counts[e] = 0;
        __syncthreads();
        const int32_t s = s0 + tid;
        uint32_t e = static_cast<uint32_t>(E);
        if (s < to) e = expert_of(ONE ? mine : p.experts[s], E);
        const uint64_t same = same_key(e, bits);
        const int rank = __popcll(same & ((1ull << lane) - 1));
        if (rank == 0) m.counts[wave * (E + 1) + e] = static_cast<uint16_t>(__popcll(same));
        __syncthreads();
        int32_t at = -1;
        if (e < static_cast<uint32_t>(E)) {
            at = m.base[e] + rank;
            for (int w = 0; w < wave; ++w) at += m.counts[w * (E + 1) + e];
            p.rows[at] = s;
        }
        if (s < to) {
            p.places[s] = at;
            if (s >= all) p.rows[s] = -1;
        }
        if (s0 + 1024 >= to) break;
        __syncthreads();
        if (tid < E)
            for (int w = 0; w < 16; ++w) m.base[tid] += m.counts[w * (E + 1) + tid];
        __syncthreads();
    }
}

__global__ __launch_bounds__(1024) void order_kernel(OrderParams p)
{
    __shared__ OrderMemory m;
    order_chunk<false>(p, blockIdx.x, 0, m);
}

// Up to 16 tokens: their choice, a wave each, and the order in one launch.  SMALL: up
// to 64 slots, which the first wave orders by comparing them all.
constexpr int FEW = 16;

template <int V, bool SMALL>
__global__ __launch_bounds__(1024) void route_few_kernel(RouteParams p, OrderParams o)
{
    __shared__ union {
        double cs[FEW][64 * V];
        OrderMemory m;
    } u;
    __shared__ int32_t chosen[FEW * MOST_TOP];
    const int tid = threadIdx.x, lane = tid & 63, wave = wave_index();
    if (wave < p.T) {
        const int32_t e = route_token<V>(p, wave, lane, u.cs[wave]);
        if (lane < p.top) chosen[wave * p.top + lane] = e;
    }
    __syncthreads();
    if constexpr (!SMALL) {
        order_chunk<true>(o, 0, tid < o.S ? chosen[tid] : -1, u.m);
        return;
    }
    if (wave > 0) return;
    const uint32_t E = static_cast<uint32_t>(o.E), mine = lane < o.S ? expert_of(chosen[lane], o.E) : E;
    int32_t at = 0, all = 0, before[V] = {};   // slots of the experts before l, l + 64, ...
    for (int32_t s = 0; s < o.S; ++s) {
        const uint32_t e = __builtin_amdgcn_readlane(mine, s);
        if (e == E) continue;
        ++all;
        if (e < mine || (e == mine && s < lane)) ++at;
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (e < static_cast<uint32_t>(i * 64 + lane)) ++before[i];
    }
    if (lane < o.S) {
        if (mine < E) o.rows[at] = lane;
        if (lane >= all) o.rows[lane] = -1;
        o.places[lane] = mine < E ? at : -1;
    }
#pragma unroll
    for (int i = 0; i < V; ++i)
        if (i * 64 + lane < o.E) o.offsets[i * 64 + lane] = before[i];
    if (lane == 0) o.offsets[E] = all;
}

// ---------------------------------------------------------------------------
// The logits' gradient: one wave a token, or two tokens a wave
// ---------------------------------------------------------------------------
struct RouteBackParams {
    const void *logits;
    const int32_t *experts;
    const float *weights, *dweights;
    void *dlogits;
    double scale;
    int32_t T, E, top;
    bool f32, sigmoid, renormalize;
};

// Scores go to LDS, where lane j takes that of choice j, and the choices' gradients
// come back the same way.  L lanes a token: 32, and two tokens a wave, up to 128
// experts.  8191 tokens of 128 experts, 6 chosen, 7.9 us (64 lanes: 8.3; of 131072
// tokens 55 and 70, of 64 experts 37 and 64).
template <int L, int V>
__global__ __launch_bounds__(256) void route_back_kernel(RouteBackParams p)
{
    constexpr double inf = __builtin_huge_val();
    constexpr int TOKENS = 64 / L;
    __shared__ double memory[4][64 * V];
    const int lane = threadIdx.x & 63, wave = wave_index(), sub = lane % L;
    const int32_t first = (blockIdx.x * 4 + wave) * TOKENS;
    if (first >= p.T) return;
    // the last token twice where there is no second
    const int32_t t = min(first + lane / L, p.T - 1);
    const bool there = first + lane / L < p.T;
    double *const ls = memory[wave] + lane / L * (L * V);
    double x[V], s[V], d[V];
    const int64_t row = static_cast<int64_t>(t) * p.E;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int32_t e = i * L + sub;
        x[i] = e < p.E ? load_logit(p.logits, p.f32, row + e) : -inf;
    }
    int32_t mine = -1;
    double dw = 0.0;
    bool bad = false;
    if (sub < p.top) {
        const int64_t at = static_cast<int64_t>(t) * p.top + sub;
        mine = p.experts[at];
        if (mine < 0 || mine >= p.E) mine = -1;
        const float w = p.weights[at], g = p.dweights[at];
        if (mine >= 0) dw = static_cast<double>(g);
        bad = !(w == w);
    }
    const bool scored = scores_of<L>(x, p.sigmoid, s), any = lanes_any<L>(bad), fine = scored && !any;
#pragma unroll
    for (int i = 0; i < V; ++i) ls[i * L + sub] = s[i];
    wave_lds_fence();
    const double own = mine >= 0 ? ls[mine] : 0.0;
    wave_lds_fence();
#pragma unroll
    for (int i = 0; i < V; ++i) ls[i * L + sub] = 0.0;
    wave_lds_fence();
    // sums over the choices: of their scores, and of those times dw
    double by = p.scale, less = 0.0;
    if (p.renormalize) {
        const double total = lanes_sum<L>(own) + 1e-20;
        by = p.scale / total;
        less = lanes_sum<L>(own * dw) / total;
    }
    const double g = by * (dw - less);
    if (mine >= 0) atomicAdd(&ls[mine], g);   // an expert is chosen once, unless the caller says so
    wave_lds_fence();
#pragma unroll
    for (int i = 0; i < V; ++i) d[i] = ls[i * L + sub];
    // sum of d s, which is where an expert was chosen
    double dot = 0.0;
    if (!p.sigmoid) dot = lanes_sum<L>(mine >= 0 ? g * own : 0.0);
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int32_t e = i * L + sub;
        if (e >= p.E || !there) continue;
        double g;
        if (!fine)
            g = __builtin_nan("");
        else if (x[i] == -inf)
            g = 0.0;
        else if (p.sigmoid)
            g = d[i] == 0.0 ? 0.0 : d[i] * s[i] * (1.0 / (1.0 + exp(x[i])));
        else
            g = s[i] * (d[i] - dot);
        if (p.f32)
            static_cast<float *>(p.dlogits)[row + e] = static_cast<float>(g);
        else
            static_cast<_Float16 *>(p.dlogits)[row + e] = static_cast<_Float16>(g);
    }
}

// ---------------------------------------------------------------------------
// A token's rows together
// ---------------------------------------------------------------------------
// What is written, and what is read for the last time (LAST), leaves the caches to
// the other rows: 4999 x 4160, 6 choices, with the gradients 159 us without, 142 so.
template <bool LAST = false>
__device__ __forceinline__ half8_t load8(const _Float16 *row, int32_t c, int32_t cols)
{
    if (c + 8 <= cols) {
        const half8_u_t *at = reinterpret_cast<const half8_u_t *>(row + c);
        return LAST ? __builtin_nontemporal_load(at) : *at;
    }
    half8_t v = {};
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (c + i < cols) v[i] = row[c + i];
    return v;
}

__device__ __forceinline__ void store8(_Float16 *row, int32_t c, int32_t cols, half8_t v)
{
    if (c + 8 <= cols) {
        __builtin_nontemporal_store(v, reinterpret_cast<half8_u_t *>(row + c));
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (c + i < cols) row[c + i] = v[i];
}

struct CombineParams {
    const _Float16 *y, *dout;
    const float *weights;
    const int32_t *rows, *places;
    _Float16 *out;             // or dy
    float *dweights;
    int32_t T, top, N, S;
    int32_t chunks;            // of 512 columns a row
};

// A wave takes 512 columns of a token: places and weights are scalars, and the
// rows of eight choices are on their way at once.  Bound by HBM and the last cache:
// 4999 x 4160, 6 choices, in 50 us (291 MB).
constexpr int AT_ONCE = 8;

__global__ __launch_bounds__(256) void combine_kernel(CombineParams p)
{
    const int32_t unit = blockIdx.x * 4 + wave_index();   // below 2^26
    const int64_t t = unit / p.chunks;
    if (t >= p.T) return;
    const int32_t c = (unit - static_cast<int32_t>(t) * p.chunks) * 512 + (threadIdx.x & 63) * 8;
    if (c >= p.N) return;
    const int32_t *places = p.places + t * p.top;
    const float *weights = p.weights + t * p.top;
    float sum[8] = {};
    for (int32_t j0 = 0; j0 < p.top; j0 += AT_ONCE) {
        half8_t v[AT_ONCE] = {};
#pragma unroll
        for (int j = 0; j < AT_ONCE; ++j) {
            if (j0 + j >= p.top) break;
            const int32_t place = places[j0 + j];
            if (static_cast<uint32_t>(place) < static_cast<uint32_t>(p.S))
                v[j] = load8(p.y + static_cast<int64_t>(place) * p.N, c, p.N);
        }
#pragma unroll
        for (int j = 0; j < AT_ONCE; ++j) {
            if (j0 + j >= p.top) break;
            const float w = p.weights ? weights[j0 + j] : 1.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i) sum[i] = __builtin_fmaf(w, static_cast<float>(v[j][i]), sum[i]);
        }
    }
    half8_t h;
#pragma unroll
    for (int i = 0; i < 8; ++i) h[i] = static_cast<_Float16>(sum[i]);
    store8(p.out + t * p.N, c, p.N, h);
}

// A wave a slot: its row of dy, its inner product, and zeros for the position of
// the slot's number where that is no slot's.  Four times 512 columns are on their
// way at once; the waves of a token read dout from its XCD's L2.  Bound by HBM: 4999 x
// 4160, 6 choices, in 93 us (541 MB, 5.8 TB/s).
__global__ __launch_bounds__(256) void combine_back_kernel(CombineParams p)
{
    constexpr int U = 4;
    const int32_t unit = xcd_unit() * 4 + wave_index();
    if (unit >= p.S) return;
    const int64_t slot = unit;
    const int lane = threadIdx.x & 63;
    const int32_t place = p.places[slot];
    const bool in = static_cast<uint32_t>(place) < static_cast<uint32_t>(p.S);
    const float w = p.weights ? p.weights[slot] : 1.0f;
    // columns are counted unsigned: the last step passes N, which may be 2^31 - 8
    const uint32_t N = static_cast<uint32_t>(p.N);
    float dot = 0.0f;
    if (in) {
        const _Float16 *dout = p.dout + static_cast<int64_t>(unit / p.top) * p.N;
        const _Float16 *y = p.y + static_cast<int64_t>(place) * p.N;
        _Float16 *dy = p.out + static_cast<int64_t>(place) * p.N;
        for (uint32_t c0 = lane * 8; c0 < N; c0 += U * 512) {
            half8_t d[U], v[U];
#pragma unroll
            for (int k = 0; k < U; ++k)
                if (c0 + k * 512 < N) {
                    d[k] = load8(dout, c0 + k * 512, p.N);
                    if (p.dweights) v[k] = load8<true>(y, c0 + k * 512, p.N);
                }
#pragma unroll
            for (int k = 0; k < U; ++k) {
                if (c0 + k * 512 >= N) break;
                half8_t h;
#pragma unroll
                for (int i = 0; i < 8; ++i) h[i] = static_cast<_Float16>(w * static_cast<float>(d[k][i]));
                store8(dy, c0 + k * 512, p.N, h);
                if (p.dweights)
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        dot = __builtin_fmaf(static_cast<float>(d[k][i]), static_cast<float>(v[k][i]), dot);
            }
        }
    }
    if (p.dweights) {
#pragma unroll
        for (int d = 1; d < 64; d *= 2) dot += __shfl_xor(dot, d);
        if (lane == 0) p.dweights[slot] = dot;
    }
    if (p.rows[slot] < 0)
        for (uint32_t c = lane * 8; c < N; c += 512) store8(p.out + slot * p.N, c, p.N, half8_t{});
}

// ---------------------------------------------------------------------------
// Host
// ---------------------------------------------------------------------------
static int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

struct Array {
    const void *p;
    int64_t bytes;
    int64_t align;
    bool written;
};

// NULL, alignment and overlap of a call's arrays (any with one that is written).
static int check_arrays(const Array *arrays, int count)
{
    for (int i = 0; i < count; ++i)
        if (arrays[i].bytes > 0 && !arrays[i].p) return GEMM_F16_INVALID_ARG;
    for (int i = 0; i < count; ++i)
        for (int j = 0; j < i; ++j) {
            if (!(arrays[i].written || arrays[j].written)) continue;
            if (arrays[i].bytes <= 0 || arrays[j].bytes <= 0) continue;
            const uintptr_t a = reinterpret_cast<uintptr_t>(arrays[i].p);
            const uintptr_t b = reinterpret_cast<uintptr_t>(arrays[j].p);
            if (a < b + static_cast<uintptr_t>(arrays[j].bytes) &&
                b < a + static_cast<uintptr_t>(arrays[i].bytes))
                return GEMM_F16_INVALID_ARG;
        }
    for (int i = 0; i < count; ++i)
        if (arrays[i].bytes > 0 && reinterpret_cast<uintptr_t>(arrays[i].p) % arrays[i].align != 0)
            return GEMM_F16_UNSUPPORTED;
    return GEMM_F16_OK;
}

static int launch(const void *fn, int64_t grid, int threads, void *params, hipStream_t stream,
                  void *more = nullptr)
{
    // the launch's own status only: the thread's sticky error state is neither
    // read nor cleared
    void *args[] = {params, more};
    const hipError_t err = hipLaunchKernel(fn, dim3(static_cast<uint32_t>(grid)),
                                           dim3(static_cast<uint32_t>(threads)), args, 0, stream);
    return err == hipSuccess ? GEMM_F16_OK : GEMM_F16_LAUNCH_FAILED;
}
template <class K>
static const void *address(K *kernel) { return reinterpret_cast<const void *>(kernel); }

constexpr int64_t MOST_THREADS = int64_t(1) << 32;

static int check_sizes(int64_t T, int64_t E, int32_t top)
{
    if (T < 0 || E < 1 || E > MOST_EXPERTS || top < 1 || top > MOST_TOP || top > E)
        return GEMM_F16_INVALID_ARG;
    return T > (INT32_MAX - 1023) / top ? GEMM_F16_INVALID_ARG : GEMM_F16_OK;
}

// The kernel for E experts: 64 V of them, V a power of two.
template <template <int> class Of>
static const void *by_experts(int64_t E)
{
    if (E <= 64) return Of<1>::get();
    if (E <= 128) return Of<2>::get();
    if (E <= 256) return Of<4>::get();
    if (E <= 512) return Of<8>::get();
    return Of<16>::get();
}
template <int V>
struct RouteFewOf { static const void *get() { return address(route_few_kernel<V, false>); } };
template <int V>
struct RouteSmallOf { static const void *get() { return address(route_few_kernel<V, true>); } };
template <int V>
struct RouteOf { static const void *get() { return address(route_kernel<V>); } };
// Lanes hold V experts each: two tokens a wave up to 128.
static const void *route_pairs(int64_t E)
{
    return E <= 32   ? address(route_pairs_kernel<1>)
           : E <= 64 ? address(route_pairs_kernel<2>)
                     : address(route_pairs_kernel<4>);
}

static const void *route_back(int64_t E)
{
    if (E <= 32) return address(route_back_kernel<32, 1>);
    if (E <= 64) return address(route_back_kernel<32, 2>);
    if (E <= 128) return address(route_back_kernel<32, 4>);
    if (E <= 256) return address(route_back_kernel<64, 4>);
    return E <= 512 ? address(route_back_kernel<64, 8>) : address(route_back_kernel<64, 16>);
}

// The chunks of S slots, and the bytes of their counts.  Up to 2048 slots in one:
// two passes of a workgroup cost less than a second launch.  No more than 256, whose
// counts every workgroup reads.
static int64_t order_chunks(int64_t S, int64_t E, OrderParams *o)
{
    const int64_t chunk = S <= 2048 ? 2048 : cdiv(cdiv(S, 256), 1024) * 1024;
    o->S = static_cast<int32_t>(S);
    o->E = static_cast<int32_t>(E);
    o->chunk = static_cast<int32_t>(chunk);
    o->chunks = static_cast<int32_t>(std::max<int64_t>(cdiv(S, chunk), 1));
    return o->chunks > 1 ? o->chunks * E * 4 : 0;
}

static int combine_sizes(int64_t T, int32_t top, int64_t N)
{
    if (T < 0 || N < 0 || top < 1 || top > MOST_TOP || T > (INT32_MAX - 1023) / top)
        return GEMM_F16_INVALID_ARG;
    return N > INT32_MAX - 7 ? GEMM_F16_UNSUPPORTED : GEMM_F16_OK;
}

}  // namespace gemm_f16_experts

using namespace gemm_f16_experts;

extern "C" int gemm_f16_route_workspace(int64_t T, int64_t E, int32_t top, int64_t *bytes)
{
    if (!bytes) return GEMM_F16_INVALID_ARG;
    const int v = check_sizes(T, E, top);
    if (v != GEMM_F16_OK) return v;
    OrderParams o;
    *bytes = order_chunks(T * top, E, &o);
    return GEMM_F16_OK;
}

extern "C" int gemm_f16_route(int64_t T, int64_t E, int32_t top, int32_t scores, int32_t groups,
                              int32_t top_groups, int32_t group_max, int32_t renormalize,
                              double scale, const void *logits, int32_t logits_f32,
                              const void *bias, void *experts, void *weights, void *rows,
                              void *places, void *offsets, void *workspace,
                              int64_t workspace_bytes, hipStream_t stream)
{
    int v = check_sizes(T, E, top);
    if (v != GEMM_F16_OK) return v;
    if ((scores != GEMM_F16_ROUTE_SOFTMAX && scores != GEMM_F16_ROUTE_SIGMOID) || groups < 1 ||
        groups > MOST_GROUPS || E % groups != 0 || top_groups < 1 || top_groups > groups ||
        workspace_bytes < 0)
        return GEMM_F16_INVALID_ARG;
    const int64_t S = T * top, width = logits_f32 ? 4 : 2;
    const Array arrays[8] = {{logits, T * E * width, width, false},
                             {bias, bias ? E * 4 : 0, 4, false},
                             {experts, S * 4, 4, true},
                             {weights, S * 4, 4, true},
                             {rows, S * 4, 4, true},
                             {places, S * 4, 4, true},
                             {offsets, (E + 1) * 4, 4, true},
                             {workspace, workspace ? workspace_bytes : 0, 256, true}};
    v = check_arrays(arrays, 8);
    if (v != GEMM_F16_OK) return v;
    OrderParams o;
    const int64_t need = order_chunks(S, E, &o);
    if (need > (workspace ? workspace_bytes : 0)) return GEMM_F16_INVALID_ARG;
    o.experts = static_cast<const int32_t *>(experts);
    o.rows = static_cast<int32_t *>(rows);
    o.places = static_cast<int32_t *>(places);
    o.offsets = static_cast<int32_t *>(offsets);
    o.counts = static_cast<int32_t *>(workspace);
    RouteParams p;
    p.logits = logits;
    p.bias = static_cast<const float *>(bias);
    p.experts = static_cast<int32_t *>(experts);
    p.weights = static_cast<float *>(weights);
    p.scale = scale;
    p.T = static_cast<int32_t>(T);
    p.E = static_cast<int32_t>(E);
    p.top = top;
    p.groups = groups;
    p.top_groups = top_groups;
    p.f32 = logits_f32 != 0;
    p.sigmoid = scores == GEMM_F16_ROUTE_SIGMOID;
    p.group_max = group_max != 0;
    p.renormalize = renormalize != 0;
    if (T <= FEW && S <= 64)
        return launch(by_experts<RouteSmallOf>(E), 1, static_cast<int>(std::max<int64_t>(T, 1)) * 64, &p, stream, &o);
    if (T <= FEW) return launch(by_experts<RouteFewOf>(E), 1, 1024, &p, stream, &o);
    const bool pairs = E <= 128 && groups == 1;
    const int64_t grid = cdiv(T, pairs ? 8 : 4);
    if (grid * 256 >= MOST_THREADS) return GEMM_F16_UNSUPPORTED;
    v = launch(pairs ? route_pairs(E) : by_experts<RouteOf>(E), grid, 256, &p, stream);
    if (v == GEMM_F16_OK && o.chunks > 1) v = launch(address(count_kernel), o.chunks, 1024, &o, stream);
    return v != GEMM_F16_OK ? v : launch(address(order_kernel), o.chunks, 1024, &o, stream);
}

extern "C" int gemm_f16_route_backward(int64_t T, int64_t E, int32_t top, int32_t scores,
                                       int32_t renormalize, double scale, const void *logits,
                                       int32_t logits_f32, const void *experts,
                                       const void *weights, const void *dweights, void *dlogits,
                                       hipStream_t stream)
{
    int v = check_sizes(T, E, top);
    if (v != GEMM_F16_OK) return v;
    if (scores != GEMM_F16_ROUTE_SOFTMAX && scores != GEMM_F16_ROUTE_SIGMOID)
        return GEMM_F16_INVALID_ARG;
    const int64_t S = T * top, width = logits_f32 ? 4 : 2;
    const Array arrays[5] = {{logits, T * E * width, width, false},
                             {experts, S * 4, 4, false},
                             {weights, S * 4, 4, false},
                             {dweights, S * 4, 4, false},
                             {dlogits, T * E * width, width, true}};
    v = check_arrays(arrays, 5);
    if (v != GEMM_F16_OK || T == 0) return v;
    RouteBackParams p;
    p.logits = logits;
    p.experts = static_cast<const int32_t *>(experts);
    p.weights = static_cast<const float *>(weights);
    p.dweights = static_cast<const float *>(dweights);
    p.dlogits = dlogits;
    p.scale = scale;
    p.T = static_cast<int32_t>(T);
    p.E = static_cast<int32_t>(E);
    p.top = top;
    p.f32 = logits_f32 != 0;
    p.sigmoid = scores == GEMM_F16_ROUTE_SIGMOID;
    p.renormalize = renormalize != 0;
    const int64_t grid = cdiv(T, E <= 128 ? 8 : 4);
    if (grid * 256 >= MOST_THREADS) return GEMM_F16_UNSUPPORTED;
    return launch(route_back(E), grid, 256, &p, stream);
}

extern "C" int gemm_f16_combine(int64_t T, int32_t top, int64_t N, const void *y,
                                const void *weights, const void *places, void *out,
                                hipStream_t stream)
{
    int v = combine_sizes(T, top, N);
    if (v != GEMM_F16_OK) return v;
    const int64_t S = T * top;
    const Array arrays[4] = {{y, S * N * 2, 2, false},
                             {weights, weights ? S * 4 : 0, 4, false},
                             {places, S * 4, 4, false},
                             {out, T * N * 2, 2, true}};
    v = check_arrays(arrays, 4);
    if (v != GEMM_F16_OK || T == 0 || N == 0) return v;
    CombineParams p{};
    p.y = static_cast<const _Float16 *>(y);
    p.weights = static_cast<const float *>(weights);
    p.places = static_cast<const int32_t *>(places);
    p.out = static_cast<_Float16 *>(out);
    p.T = static_cast<int32_t>(T);
    p.top = top;
    p.N = static_cast<int32_t>(N);
    p.S = static_cast<int32_t>(S);
    p.chunks = static_cast<int32_t>(cdiv(N, 512));
    if (T > MOST_THREADS / 64 / p.chunks - 4) return GEMM_F16_UNSUPPORTED;
    return launch(address(combine_kernel), cdiv(T * p.chunks, 4), 256, &p, stream);
}

extern "C" int gemm_f16_combine_backward(int64_t T, int32_t top, int64_t N, const void *dout,
                                         const void *y, const void *weights, const void *rows,
                                         const void *places, void *dy, void *dweights,
                                         hipStream_t stream)
{
    int v = combine_sizes(T, top, N);
    if (v != GEMM_F16_OK) return v;
    const int64_t S = T * top;
    const Array arrays[7] = {{dout, T * N * 2, 2, false},
                             {y, dweights ? S * N * 2 : 0, 2, false},
                             {weights, weights ? S * 4 : 0, 4, false},
                             {rows, S * 4, 4, false},
                             {places, S * 4, 4, false},
                             {dy, S * N * 2, 2, true},
                             {dweights, dweights ? S * 4 : 0, 4, true}};
    v = check_arrays(arrays, 7);
    if (v != GEMM_F16_OK || T == 0) return v;
    if (S + 3 >= MOST_THREADS / 64) return GEMM_F16_UNSUPPORTED;
    CombineParams p{};
    p.y = static_cast<const _Float16 *>(y);
    p.dout = static_cast<const _Float16 *>(dout);
    p.weights = static_cast<const float *>(weights);
    p.rows = static_cast<const int32_t *>(rows);
    p.places = static_cast<const int32_t *>(places);
    p.out = static_cast<_Float16 *>(dy);
    p.dweights = static_cast<float *>(dweights);
    p.T = static_cast<int32_t>(T);
    p.top = top;
    p.N = static_cast<int32_t>(N);
    p.S = static_cast<int32_t>(S);
    return launch(address(combine_back_kernel), cdiv(S, 4), 256, &p, stream);
}
