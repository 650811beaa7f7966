// Operands in 4 and 8 bits for MI355X (gfx950): quantising, reading back, and
// the products C = A W^T (4-bit weights) and C = A^T X (8-bit activations).
// The forms, and why every kernel here works on the same exact fp16 matrix,
// are described in gemm_f16_lowbit.h.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <stddef.h>
#include <stdint.h>

#include "gemm_f16_lowbit.h"

namespace gemm_f16_lowbit {

typedef _Float16 half2_t __attribute__((ext_vector_type(2)));
typedef _Float16 half4_t __attribute__((ext_vector_type(4)));
typedef _Float16 half8_t __attribute__((ext_vector_type(8)));
// 16 bytes at any 2-byte alignment (the target's unaligned-access mode)
typedef _Float16 half8_u_t __attribute__((ext_vector_type(8), aligned(2)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef int32_t i32x4_t __attribute__((ext_vector_type(4)));
typedef uint16_t u16x2_t __attribute__((ext_vector_type(2)));
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2_u_t __attribute__((ext_vector_type(2), aligned(1)));

constexpr int WAVES = 4;            // waves of a workgroup here
constexpr uint16_t FP16_NAN = 0x7e00;

template <class T, class S>
__device__ __forceinline__ T bits_as(S s)
{
    static_assert(sizeof(T) == sizeof(S), "same size");
    return __builtin_bit_cast(T, s);
}

// The wave's index in its workgroup, in a scalar register: what is computed from
// it alone (which tile, its addresses) then takes no vector operations.
__device__ __forceinline__ int wave_index() { return __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); }

// Between a wave's LDS writes and its other lanes' reads of them, and before the
// next writes: a wave's LDS operations are done in order, so no instruction is
// needed, but the compiler may move one lane's accesses past each other unless
// it is told that the lanes exchange them.
__device__ __forceinline__ void wave_lds_fence()
{
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront", "local");
    __builtin_amdgcn_wave_barrier();
}

// This workgroup's unit of work, where each XCD (workgroups mod 8) takes a
// contiguous range of them: neighbours share cache lines in its L2.
__device__ __forceinline__ int32_t xcd_unit()
{
    const int32_t q = gridDim.x >> 3, rem = gridDim.x & 7, x = blockIdx.x & 7;
    return x * q + (x < rem ? x : rem) + (blockIdx.x >> 3);
}

// Eight halves of a row at column c, as dwords; columns at or past `cols` are 0.
__device__ __forceinline__ u32x4_t load8(const uint16_t *row, int32_t c, int32_t cols)
{
    if (c + 8 <= cols) return bits_as<u32x4_t>(half8_t(*reinterpret_cast<const half8_u_t *>(row + c)));
    u32x4_t v = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (c + i < cols) v[i / 2] |= static_cast<uint32_t>(row[c + i]) << (16 * (i % 2));
    return v;
}

__device__ __forceinline__ void store8(uint16_t *row, int32_t c, int32_t cols, half8_t v)
{
    if (c + 8 <= cols) {
        *reinterpret_cast<half8_u_t *>(row + c) = v;
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (c + i < cols) row[c + i] = bits_as<uint16_t>(_Float16(v[i]));
}

// Largest of eight halves by magnitude, as fp16 bits: those of non-negative
// numbers, infinity and NaN order as integers.
__device__ __forceinline__ uint32_t largest8(u32x4_t v)
{
    u16x2_t m = bits_as<u16x2_t>(v[0] & 0x7fff7fffu);
#pragma unroll
    for (int i = 1; i < 4; ++i)
        m = __builtin_elementwise_max(m, bits_as<u16x2_t>(v[i] & 0x7fff7fffu));
    return m[0] > m[1] ? m[0] : m[1];
}

// The scale of a group whose largest magnitude has fp16 bits `big`: the
// smallest s of BITS significant bits, a multiple of 2^-24, with TOP s >= big.
// big / TOP is taken as a product with (1 - 2^-20) / TOP: big has 11
// significant bits and TOP s at most 11, so where they differ they do so by
// more than 2^-12 of their value, and where they are equal the product falls
// short of s and rounds up to it.  (Checked for every fp16 value.)
template <int BITS, int TOP>
__device__ __forceinline__ float group_scale(uint32_t big, float most)
{
    const float t = static_cast<float>(bits_as<_Float16>(static_cast<uint16_t>(big))) *
                    ((1.0f / TOP) * (1.0f - 0x1p-20f));
    constexpr uint32_t drop = (1u << (24 - BITS)) - 1;
    const float up = bits_as<float>((bits_as<uint32_t>(t) + drop) & ~drop);
    const float s = t < 0x1p-24f * (1 << (BITS - 1)) ? __builtin_ceilf(t * 0x1p24f) * 0x1p-24f : up;
    return fminf(fmaxf(s, 0x1p-24f), most);
}

// 1 / s as a sum of two numbers, to far below fp32's resolution.
struct Reciprocal {
    float hi, lo;
};

__device__ __forceinline__ Reciprocal reciprocal(float s)
{
    const float r = __builtin_amdgcn_rcpf(s);
    return Reciprocal{r, __builtin_fmaf(-s, r, 1.0f) * r};
}

// x / s rounded to nearest, ties to even, as the low bits of a float: below
// 2^22 in magnitude, adding 1.5 2^23 leaves the rounded integer in the low 22
// bits (two's complement).  A product with one fp32 reciprocal can miss a tie
// by an ulp; with the second part a tie comes out exact, and a quotient that
// is not a tie is further from one than fp32 resolves (checked for every fp16
// x and every scale, with hi an ulp off either way).
__device__ __forceinline__ uint32_t quotient(float x, Reciprocal r, float bias)
{
    return bits_as<uint32_t>(__builtin_fmaf(x, r.hi, x * r.lo) + (0x1.8p23f + bias));
}

// The eight halves of four dwords, as floats.
__device__ __forceinline__ float half_of(u32x4_t v, int i)
{
    return static_cast<float>(bits_as<half2_t>(v[i / 2])[i % 2]);
}

// ---------------------------------------------------------------------------
// W4: quantise or pack
// ---------------------------------------------------------------------------
// One wave per tile of 16 rows by 128 columns, each lane the 32 weights whose
// words it writes: four loads of 16 bytes (8 for int8 codes), the group's
// largest magnitude over the four lanes of a row, one 16-byte store.  Memory
// bounds quantising (8192 x 8192: 36.1 us, 4.7 TB/s); packing takes as long for 0.6
// of the bytes, with the vector ALU at its checks for 68% of the cycles.  Loads of
// 256 bytes of four rows, turned round in LDS, took 22 us for 28 where rows are not
// 16-byte aligned, and 1 to 2 us more where they are, as weights' rows mostly are.
struct W4EncodeParams {
    const uint16_t *W;       // fp16 [N, K], or
    const int8_t *codes;     // int8 [N, K] and
    const uint16_t *in_scales;  // fp16 [N, ceil(K / group)]
    u32x4_t *words;
    uint16_t *scales;
    int32_t N, K, kt, tiles;
    int32_t shift;           // log2 of the group
};

// Most significant 8 bits of a scale, to nearest with ties to even.  Infinities
// and NaN stay as they are: the carry out of a NaN's payload would make it zero.
__device__ __forceinline__ float round_scale(float s)
{
    const uint32_t u = bits_as<uint32_t>(s);
    if ((u & 0x7f800000u) == 0x7f800000u) return s;
    return bits_as<float>((u + 0x7fffu + ((u >> 16) & 1)) & 0xffff0000u);
}

template <bool PACK>
__global__ __launch_bounds__(64 * WAVES) void w4_encode_kernel(W4EncodeParams p)
{
    const int lane = threadIdx.x & 63;
    const int r = lane & 15, kq = lane >> 4;
    const int per_tile = 128 >> p.shift;
    const int64_t step = static_cast<int64_t>(gridDim.x) * WAVES;
    for (int64_t tile = static_cast<int64_t>(xcd_unit()) * WAVES + wave_index(); tile < p.tiles;
         tile += step) {
        const int32_t b = static_cast<int32_t>(tile) / p.kt;
        const int32_t t = static_cast<int32_t>(tile) - b * p.kt;
        const int64_t n = static_cast<int64_t>(b) * 16 + r;
        const int32_t cols = n < p.N ? p.K : 0;     // rows past N are zeros
        const int64_t row = n < p.N ? n : 0;
        const int64_t k0 = static_cast<int64_t>(t) * 128 + kq * 8;  // may pass 2^31 in a pad
        // A tile wholly inside the matrix takes the loads all at once; one at
        // its edge takes each under its own conditions (which make the loads
        // wait for each other: all tiles that way took 57.6 us at 8192 x 8192).
        const bool inside = (static_cast<int64_t>(t) + 1) * 128 <= p.K &&
                            (static_cast<int64_t>(b) + 1) * 16 <= p.N;
        u32x4_t v[4];
        u32x2_t d[4];
        int32_t q[4][8];
        uint32_t big[4];
        if constexpr (PACK) {
            const int8_t *src = p.codes + row * p.K + k0;
            if (inside) {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    d[j] = u32x2_t(*reinterpret_cast<const u32x2_u_t *>(src + 32 * j));
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    d[j] = u32x2_t{0, 0};
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        if (k0 + 32 * j + i < cols)
                            d[j][i / 4] |= static_cast<uint32_t>(static_cast<uint8_t>(src[32 * j + i]))
                                           << (8 * (i % 4));
                }
            }
        } else {
            const uint16_t *src = p.W + row * p.K;
            if (inside) {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    v[j] = bits_as<u32x4_t>(
                        half8_t(*reinterpret_cast<const half8_u_t *>(src + k0 + 32 * j)));
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    v[j] = k0 + 32 * j < cols ? load8(src, static_cast<int32_t>(k0 + 32 * j), cols)
                                              : u32x4_t{0, 0, 0, 0};
            }
        }
        // per 32 columns of this lane's row the largest magnitude, as fp16 bits
        // or of the codes
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if constexpr (PACK) {
                big[j] = 0;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    q[j][i] = static_cast<int8_t>(d[j][i / 4] >> (8 * (i % 4)));
                    // 9 marks a code that four bits do not hold
                    const uint32_t m = q[j][i] < -8 || q[j][i] > 7 ? 9 : q[j][i] < 0 ? -q[j][i] : q[j][i];
                    big[j] = m > big[j] ? m : big[j];
                }
            } else {
                big[j] = largest8(v[j]);
            }
            uint32_t o = __shfl_xor(big[j], 16);
            big[j] = o > big[j] ? o : big[j];
            o = __shfl_xor(big[j], 32);
            big[j] = o > big[j] ? o : big[j];
        }
        if (p.shift >= 6) {
            big[0] = big[1] = big[0] > big[1] ? big[0] : big[1];
            big[2] = big[3] = big[2] > big[3] ? big[2] : big[3];
        }
        if (p.shift == 7) big[0] = big[1] = big[2] = big[3] = big[0] > big[2] ? big[0] : big[2];
        u32x4_t out;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float s;
            bool bad;
            uint32_t word = 0;
            if constexpr (PACK) {
                const int64_t k = static_cast<int64_t>(t) * 128 + 32 * j;
                s = 0.0f;
                if (k < cols) {
                    const int64_t groups = (static_cast<int64_t>(p.K) + (1 << p.shift) - 1) >> p.shift;
                    s = round_scale(static_cast<float>(
                        bits_as<_Float16>(p.in_scales[row * groups + (k >> p.shift)])));
                }
                bad = !(__builtin_fabsf(s) <= 65504.0f) || big[j] > 8 ||
                      __builtin_fabsf(s) * static_cast<float>(big[j]) > 65504.0f;
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    word |= (static_cast<uint32_t>(q[j][i] + 8) & 15u) << (16 * (i % 2) + 4 * (i / 2));
            } else {
                s = group_scale<8, 7>(big[j], 9344.0f);
                bad = big[j] >= 0x7c00;
                const Reciprocal rcp = reciprocal(s);
                // a quotient is at most 7.01, also where s is capped; 8 more is
                // the code, alone in the low 16 bits
#pragma unroll
                for (int i = 0; i < 8; i += 2) {
                    const uint32_t pair = __builtin_amdgcn_perm(
                        quotient(half_of(v[j], i + 1), rcp, 8.0f),
                        quotient(half_of(v[j], i), rcp, 8.0f), 0x05040100u);
                    word |= pair << (2 * i);
                }
            }
            if (bad) word = 0x88888888u;
            out[j] = word;
            if (kq == 0 && ((32 * j) & ((1 << p.shift) - 1)) == 0) {
                const int64_t g = static_cast<int64_t>(t) * per_tile + ((32 * j) >> p.shift);
                uint16_t *to = p.scales + (static_cast<int64_t>(b) * p.kt * per_tile + g) * 16 + r;
                *to = bad ? FP16_NAN : bits_as<uint16_t>(static_cast<_Float16>(s));
            }
        }
        p.words[tile * 64 + lane] = out;
    }
}

// A word's mask and exponent, held in registers: as literals they cannot share
// the one instruction that does both (a third of the unpacking's operations).
struct W4Bits {
    uint32_t mask, exponent;
};

__device__ __forceinline__ W4Bits w4_bits(uint32_t mask, uint32_t exponent)
{
    asm("" : "+v"(mask));
    asm("" : "+s"(exponent));
    return W4Bits{mask, exponent};
}

// For w4_scaled: the low four bits of each half, under fp16's 1024.
__device__ __forceinline__ W4Bits w4_low_bits() { return w4_bits(0x000f000fu, 0x64006400u); }

// Weights 2 i and 2 i + 1 of a word times their scale: four bits u become the low
// bits of 1024 + u, less 1032 the code u - 8, times the scale, each exact in fp16.
__device__ __forceinline__ half2_t w4_pair(uint32_t word, int i, _Float16 s, W4Bits bits)
{
    const half2_t s2 = {s, s};
    const half2_t off = {_Float16(1032.0f), _Float16(1032.0f)};
    return (bits_as<half2_t>(((word >> (4 * i)) & bits.mask) | bits.exponent) - off) * s2;
}

__device__ __forceinline__ half8_t w4_scaled(uint32_t word, _Float16 s, W4Bits bits)
{
    half8_t h;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const half2_t x = w4_pair(word, i, s, bits);
        h[2 * i] = x[0];
        h[2 * i + 1] = x[1];
    }
    return h;
}

struct W4DecodeParams {
    const u32x4_t *words;
    const uint16_t *scales;
    uint16_t *W;
    int32_t N, K, ld, kt, tiles;   // W's rows start every ld values; up to ld they are written
    int32_t shift;
};

// W4 back to fp16, one wave per tile; memory bounds it (8192 x 8192: 39 to 43 us,
// 4.0 to 4.3 TB/s, and 25.8 where the words were written just before and come from
// the last cache; 28.3 there with neighbouring tiles on different XCDs).
__global__ __launch_bounds__(64 * WAVES) void w4_decode_kernel(W4DecodeParams p)
{
    const int lane = threadIdx.x & 63;
    const int r = lane & 15, kq = lane >> 4;
    const W4Bits bits = w4_low_bits();
    const int per_tile = 128 >> p.shift;
    const int64_t step = static_cast<int64_t>(gridDim.x) * WAVES;
    for (int64_t tile = static_cast<int64_t>(xcd_unit()) * WAVES + wave_index(); tile < p.tiles;
         tile += step) {
        const int32_t b = static_cast<int32_t>(tile) / p.kt;
        const int32_t t = static_cast<int32_t>(tile) - b * p.kt;
        const int64_t n = static_cast<int64_t>(b) * 16 + r;
        if (n >= p.N) continue;
        const u32x4_t w = p.words[tile * 64 + lane];
        const uint16_t *s = p.scales + tile * per_tile * 16 + r;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int64_t c = static_cast<int64_t>(t) * 128 + 32 * j + kq * 8;
            const _Float16 sj = bits_as<_Float16>(s[((32 * j) >> p.shift) * 16]);
            if (c < p.K) store8(p.W + n * p.ld, static_cast<int32_t>(c), p.ld,
                               w4_scaled(w[j], sj, bits));
        }
    }
}

// ---------------------------------------------------------------------------
// C = A W^T for at most 48 rows of A: the words streamed through registers
// ---------------------------------------------------------------------------
// One workgroup computes NB blocks of 16 columns of C (rows of W).  Its waves
// take the blocks' tiles in turn (wave w the tiles w, w + W, ..: together they
// read each block's words front to back) and add up their sums in LDS at the
// end, so a small N still puts W waves' loads in flight on each CU, and no sum
// crosses a workgroup.  The MFMA's rows are rows of W, straight from the words;
// its 16 columns are rows of A.  HBM bounds it (a tile's KB is one load for
// each lane), and next the loads of A, a KB of lanes' data for four rows of a
// tile: the two kernels differ in how they keep those few.
struct W4Params {
    const uint16_t *A;
    const u32x4_t *words;
    const uint16_t *scales;
    uint16_t *C;
    int32_t M, N, K, kt, nb;   // kt: tiles of 128 columns, nb: blocks of 16 rows of W
};

// Sums of the waves (W x JC sets of them) in order, rounded once.
template <int NB, int W, int JC>
__device__ __forceinline__ void w4_join_waves(const W4Params &p, int32_t b0, int32_t m0,
                                              const float (*red)[NB][16][20])
{
    constexpr int MC = 16 / JC;
    __syncthreads();
    for (int o = threadIdx.x; o < NB * MC * 16; o += 64 * W) {
        const int n = o & 15, m = (o >> 4) & (MC - 1), nb = o / (16 * MC);
        float sum = 0.0f;
#pragma unroll
        for (int w = 0; w < W; ++w)
#pragma unroll
            for (int j = 0; j < JC; ++j) sum += red[w][nb][j * MC + m][n];
        const int64_t col = static_cast<int64_t>(b0 + nb) * 16 + n;
        if (m0 + m < p.M && col < p.N)
            reinterpret_cast<_Float16 *>(p.C)[static_cast<int64_t>(m0 + m) * p.N + col] =
                static_cast<_Float16>(sum);
    }
}

// Zeros for the scales of groups past K, in the tile `t` that K ends in: they belong
// to no weight and may hold anything, and a NaN times a zero of A would be one.
template <int SH, int NB, int NS>
__device__ __forceinline__ void w4_clear_pads(_Float16 (&sc)[NB][NS], int32_t t, int32_t K)
{
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int s = 1; s < NS; ++s)
            if (t * 128 + (s << SH) >= K) sc[nb][s] = _Float16(0.0f);
}

// Runs a wave's whole tiles in two buffers of D: one's loads fly while the
// other's are multiplied.  Loads are unconditional (past the end the last tile
// again), so that the waits on one buffer leave the other's in flight.
template <int W, int D, class Load, class Mma>
__device__ __forceinline__ void w4_run_tiles(int32_t full, int wave, Load load, Mma mma)
{
    const int32_t count = full > wave ? (full - wave + W - 1) / W : 0;
    auto at = [&](int32_t i) {
        return static_cast<int64_t>(wave) + static_cast<int64_t>(i < count ? i : count - 1) * W;
    };
    if (count == 0) return;
#pragma unroll
    for (int d = 0; d < D; ++d) load(0, d, at(d));
    int32_t i = 0;
    for (; i + 2 * D <= count; i += 2 * D) {
#pragma unroll
        for (int d = 0; d < D; ++d) load(1, d, at(i + D + d));
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int d = 0; d < D; ++d) mma(0, d);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int d = 0; d < D; ++d) load(0, d, at(i + 2 * D + d));
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int d = 0; d < D; ++d) mma(1, d);
        __builtin_amdgcn_sched_barrier(0);
    }
    // fewer than 2 D left: those of buffer 0 first
    if (i + D < count) {
#pragma unroll
        for (int d = 0; d < D; ++d) load(1, d, at(i + D + d));
    }
#pragma unroll
    for (int d = 0; d < D; ++d)
        if (i + d < count) mma(0, d);
#pragma unroll
    for (int d = 0; d < D; ++d)
        if (i + D + d < count) mma(1, d);
}

// At most 16 / JC rows of A.  With so few the MFMA's columns would stand empty
// while the loads of A cost four times the words' own.  So MC = 16 / JC
// columns are rows of A, and JC sets of them hold the fragments of JC
// different steps j of the tile: one load brings them all.  Each of the JC
// accumulators multiplies the words of its own step with the whole register,
// and of its results only the columns of that step are used.
//
// JC = 4, eight waves with two tiles a buffer: 1 x 4096 x 14336 takes 7.9 us in the
// median of a trace (7.6 at best; 2.3 of it an empty kernel's), 1 x 16384 x 16384
// 25.2 us (5.3 TB/s).  One tile a buffer took 9.1 (and 27.1), four 9.8 (35.6).
template <int SH, int JC, int NB, int W, int D>
__global__ __launch_bounds__(64 * W) void w4_stream_kernel(W4Params p)
{
    constexpr int MC = 16 / JC;      // rows of A
    constexpr int AL = 4 / JC;       // loads of A a tile
    constexpr int NS = 128 >> SH;    // scales a tile and row
    __shared__ float red[W][NB][16][20];   // 20: rows of 16 sums apart in the banks
    const int lane = threadIdx.x & 63;
    const int wave = wave_index();
    const int r = lane & 15, kq = lane >> 4;
    const int m = r & (MC - 1), jj = r / MC;
    const int32_t b0 = blockIdx.x * NB;
    const uint16_t *row = p.A + static_cast<int64_t>(m < p.M ? m : 0) * p.K;
    const uint16_t *arow = row + 32 * jj + 8 * kq;
    const u32x4_t *words[NB];
    const uint16_t *scales[NB];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
        const int64_t b = b0 + nb < p.nb ? b0 + nb : p.nb - 1;   // the last again: not stored
        words[nb] = p.words + b * p.kt * 64 + lane;
        scales[nb] = p.scales + b * p.kt * NS * 16 + r;
    }
    const W4Bits bits = w4_low_bits();
    f32x4_t acc[NB][JC] = {};
    u32x4_t wv[2][D][NB];
    half8_t af[2][D][AL];
    _Float16 sc[2][D][NB][NS];
    auto load_w = [&](int buf, int d, int64_t t) {
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
            wv[buf][d][nb] = __builtin_nontemporal_load(words[nb] + t * 64);
#pragma unroll
            for (int s = 0; s < NS; ++s)
                sc[buf][d][nb][s] = bits_as<_Float16>(scales[nb][(t * NS + s) * 16]);
        }
    };
    auto load = [&](int buf, int d, int64_t t) {
        load_w(buf, d, t);
#pragma unroll
        for (int i = 0; i < AL; ++i)
            af[buf][d][i] = *reinterpret_cast<const half8_u_t *>(arow + t * 128 + 32 * JC * i);
    };
    auto mma = [&](int buf, int d) {
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                acc[nb][j % JC] = __builtin_amdgcn_mfma_f32_16x16x32_f16(
                    w4_scaled(wv[buf][d][nb][j], sc[buf][d][nb][(32 * j) >> SH], bits),
                    af[buf][d][j / JC], acc[nb][j % JC], 0, 0, 0);
    };
    const int32_t full = p.K / 128;
    w4_run_tiles<W, D>(full, wave, load, mma);
    // the tile that K ends in: columns past K are zeros
    if (full < p.kt && full % W == wave) {
        load_w(0, 0, full);
        w4_clear_pads<SH>(sc[0][0], full, p.K);
#pragma unroll
        for (int i = 0; i < AL; ++i) {
            const int64_t c = static_cast<int64_t>(full) * 128 + 32 * (jj + JC * i) + 8 * kq;
            af[0][0][i] = half8_t{};
            if (c < p.K) af[0][0][i] = bits_as<half8_t>(load8(row, static_cast<int32_t>(c), p.K));
        }
        mma(0, 0);
    }
    // lane l holds rows 4 (l / 16) .. + 3 of the block and column l % 16
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
        f32x4_t v = acc[nb][0];
#pragma unroll
        for (int j = 1; j < JC; ++j)
            if (jj == j) v = acc[nb][j];
        *reinterpret_cast<f32x4_t *>(&red[wave][nb][r][kq * 4]) = v;
    }
    w4_join_waves<NB, W, JC>(p, b0, 0, red);
}

// At most 4 RL rows of A.  Loads of A in the MFMA's own layout touch 64 bytes
// of each of 16 rows, and at 16 rows they, not the words, bound the kernel (16
// x 4096 x 14336: 16.4 us).  Here each load covers 256 bytes of four rows, and
// the wave turns the tile round in LDS of its own, with the 16-byte chunks of
// row r XORed with r to spread the reads over the banks: 12.3 us, and 5.4 us
// against 6.9 at K = 4096.  Several blocks a workgroup use the rows of A more
// than once, where N still gives nearly every CU a workgroup (16 x 16384 x
// 16384: 45 us with one, 33 with two, 29.2 with four; 16 x 4096 x 14336: 12.5,
// 14.9, 22.5).  For 17 to 48 rows, two or three tiles of 16 share a word's
// unpacking, and no sum goes through memory as it does where tiles split K (32 x
// 4096 x 4096: 7.5 us, 9.8 in tiles; 48 x 4096 x 4096 9.5 and 11.8).
template <int SH, int RL, int NB, int W>
__global__ __launch_bounds__(64 * W) void w4_rows_kernel(W4Params p)
{
    constexpr int NS = 128 >> SH;
    constexpr int MT = (RL + 3) / 4;   // tiles of 16 rows of A
    union Lds {
        float red[W][NB][16][20];
        half8_t abuf[W][RL * 4][16];
    };
    __shared__ Lds lds;
    const int lane = threadIdx.x & 63;
    const int wave = wave_index();
    const int r = lane & 15, kq = lane >> 4;
    const int32_t b0 = blockIdx.x * NB;
    const uint16_t *arow[RL];
#pragma unroll
    for (int i = 0; i < RL; ++i)
        arow[i] = p.A + static_cast<int64_t>(min(4 * i + kq, p.M - 1)) * p.K;
    half8_t *ab = lds.abuf[wave][0];
    const u32x4_t *words[NB];
    const uint16_t *scales[NB];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
        const int64_t b = b0 + nb < p.nb ? b0 + nb : p.nb - 1;
        words[nb] = p.words + b * p.kt * 64 + lane;
        scales[nb] = p.scales + b * p.kt * NS * 16 + r;
    }
    const W4Bits bits = w4_low_bits();
    f32x4_t acc[NB][MT] = {};
    u32x4_t wv[2][NB];
    half8_t af[2][RL];
    _Float16 sc[2][NB][NS];
    auto load_w = [&](int buf, int64_t t) {
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
            wv[buf][nb] = __builtin_nontemporal_load(words[nb] + t * 64);
#pragma unroll
            for (int s = 0; s < NS; ++s)
                sc[buf][nb][s] = bits_as<_Float16>(scales[nb][(t * NS + s) * 16]);
        }
    };
    auto load = [&](int buf, int, int64_t t) {
        load_w(buf, t);
#pragma unroll
        for (int i = 0; i < RL; ++i)
            af[buf][i] = *reinterpret_cast<const half8_u_t *>(arow[i] + t * 128 + 8 * r);
    };
    // columns past 4 RL repeat the last row, like rows past M: not stored
    const int rr = r < RL * 4 ? r : RL * 4 - 1;
    auto mma = [&](int buf, int) {
        half8_t a[4][MT];
        auto read_a = [&](int j, int mt) {
            a[j][mt] = ab[(16 * mt + rr) * 16 + ((4 * j + kq) ^ rr)];
        };
        // the wave alone uses these 4 RL rows; the reads that the first MFMAs wait
        // for start between the writes (after all of them: 48 x 14336 x 4096 takes
        // 16.4 us for 15.0)
        wave_lds_fence();
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
            for (int i = 4 * mt; i < 4 * mt + 4 && i < RL; ++i)
                ab[(4 * i + kq) * 16 + (r ^ ((4 * i + kq) & 15))] = af[buf][i];
            wave_lds_fence();
            read_a(0, mt);
        }
#pragma unroll
        for (int j = 1; j < 4; ++j)
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) read_a(j, mt);
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const half8_t w = w4_scaled(wv[buf][nb][j], sc[buf][nb][(32 * j) >> SH], bits);
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
                    acc[nb][mt] = __builtin_amdgcn_mfma_f32_16x16x32_f16(w, a[j][mt], acc[nb][mt], 0,
                                                                         0, 0);
            }
    };
    const int32_t full = p.K / 128;
    w4_run_tiles<W, 1>(full, wave, load, mma);
    if (full < p.kt && full % W == wave) {
        load_w(0, full);
        w4_clear_pads<SH>(sc[0], full, p.K);
#pragma unroll
        for (int i = 0; i < RL; ++i) {
            const int64_t c = static_cast<int64_t>(full) * 128 + 8 * r;
            af[0][i] = half8_t{};
            if (c < p.K) af[0][i] = bits_as<half8_t>(load8(arow[i], static_cast<int32_t>(c), p.K));
        }
        mma(0, 0);
    }
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
        __syncthreads();   // the sums' LDS is that of the rows, or of the last sums
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
            *reinterpret_cast<f32x4_t *>(&lds.red[wave][nb][r][kq * 4]) = acc[nb][mt];
        w4_join_waves<NB, W, 1>(p, b0, mt * 16, lds.red);
    }
}

// ---------------------------------------------------------------------------
// C = A W^T for more rows of A: tiles through LDS
// ---------------------------------------------------------------------------
// A workgroup computes 16 MT rows of A by WC NB blocks of 16 rows of W over a
// range of K.  Each step is one tile of 128 columns, or with KH = 2 sets of WC
// waves two, whose sums meet in LDS at the end: direct-to-LDS loads keep S - 1
// steps in flight (A's rows, which a set's waves share; each wave's own words
// and scales), one barrier a step says that a step's data is there and that the
// stage before it is free.  Every wave unpacks its own words, so no weight is
// unpacked twice in a workgroup.
//
// What bounds it is the vector ALU beside the matrix units: unpacking a word
// of eight weights takes 12 operations of 4 cycles, while its MFMAs take 16 MT
// cycles.  At 48 x 16384 x 16384 the two keep a SIMD busy for 50% and 35% of the
// cycles, and the waves stand at waits for 42% of theirs; the LDS is busy for
// 22% (19 to 29% at all sizes traced), so it is not what holds them up.
// w4_tile_pair scales and centres in one fused operation to save three of 15
// (333 x 4096 x 14336: 51.7 to 48.1 us, 48 x 16384 x 16384: 47.1 to 43.0), and a
// word is unpacked between the MFMAs of the word before it.  333 x 4096 x 14336
// now keeps the matrix units busy for 52% of the cycles, at a clock that the
// power limit holds near 1.75 GHz; 512 x 16384 x 16384 runs at 1.2 PFLOP/s.
//
// Few tiles leave CUs idle: K is then split, each range's fp32 sums go to the
// workspace in the order in which lanes hold them (every store and load a
// whole KB), and w4_join_kernel adds them up in order.  Two sets of waves make a
// tile half as wide for the same work a step, so twice as many tiles and half
// the ranges (512 x 4096 x 4096: 26.0 to 22.1 us, unsplit in both; 64 x 8192 x
// 8192: 20.4 to 18.9, four ranges of half the tile's sums).
struct W4TileParams {
    const uint16_t *A;
    const u32x4_t *words;
    const uint16_t *scales;
    uint16_t *C;
    float *partial;            // [splits][tiles][WC][NB][MT][64] of 4 values
    int32_t M, N, K, lda;      // lda a multiple of 8, A 16-byte aligned
    int32_t kt, nb;            // tiles of 128 columns, blocks of 16 rows of W
    int32_t tiles_m, tiles_n, splits;
    int32_t kt_split;          // tiles of 128 columns a range
};

constexpr uint32_t OOB_OFFSET = 0x80000000u;   // past every resource: reads 0

// Buffer resource for raw byte addressing of `bytes` bytes at `base`.
__device__ __forceinline__ i32x4_t make_rsrc(const void *base, uint32_t bytes)
{
    const uint64_t a = reinterpret_cast<uint64_t>(base);
    i32x4_t r;
    r.x = __builtin_amdgcn_readfirstlane(static_cast<int32_t>(a & 0xffffffffu));
    r.y = __builtin_amdgcn_readfirstlane(static_cast<int32_t>((a >> 32) & 0xffffu));
    r.z = __builtin_amdgcn_readfirstlane(static_cast<int32_t>(bytes));
    r.w = 0x00020000;
    return r;
}

// Direct-to-LDS loads: lane l copies 16 (4) bytes from rsrc + voff to LDS byte
// address lds + 16 l (4 l).  M0 carries the wave-uniform LDS base; the s_nop
// covers the M0-write hazard, which the compiler cannot see inside an asm.
__device__ __forceinline__ void dma16(i32x4_t rsrc, uint32_t voff, uint32_t lds)
{
    asm volatile("s_nop 0\n\tbuffer_load_dwordx4 %0, %1, 0 offen lds"
                 :
                 : "v"(voff), "s"(rsrc), "{m0}"(lds));
}

__device__ __forceinline__ void dma4(i32x4_t rsrc, uint32_t voff, uint32_t lds)
{
    asm volatile("s_nop 0\n\tbuffer_load_dword %0, %1, 0 offen lds"
                 :
                 : "v"(voff), "s"(rsrc), "{m0}"(lds));
}

// Weights 2 i and 2 i + 1 of a word times their scale, as w4_pair, for s up to 2720:
// the four bits u at the top of the significand of 16 + u, which times s less
// 24 s is s (u - 8).  24 s is exact (3 times a number of 8 significant bits)
// and the fused operation rounds once, a number that fp16 holds: no rounding.
__device__ __forceinline__ half2_t w4_tile_pair(uint32_t w, int i, _Float16 s, W4Bits bits)
{
    const half2_t s2 = {s, s};
    const half2_t c2 = s2 * _Float16(-24.0f);
    const uint32_t t = i < 2 ? w << (6 - 4 * i) : w >> (4 * i - 6);
    return __builtin_elementwise_fma(bits_as<half2_t>((t & bits.mask) | bits.exponent), s2, c2);
}
__device__ __forceinline__ W4Bits w4_high_bits() { return w4_bits(0x03c003c0u, 0x4c004c00u); }
constexpr float W4_TILE_WORD_MOST = 2720.0f;   // 24 * 2720 < 65504

// Four neighbouring columns of a row of C.
__device__ __forceinline__ void store4(uint16_t *C, int32_t M, int32_t N, int32_t m, int32_t n,
                                       f32x4_t v)
{
    if (m >= M) return;
    const half4_t h = __builtin_convertvector(v, half4_t);
    uint16_t *c = C + static_cast<int64_t>(m) * N + n;
    if (n + 4 <= N) {
        __builtin_memcpy(c, &h, 8);   // any 2-byte alignment
        return;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e)
        if (n + e < N) reinterpret_cast<_Float16 *>(c)[e] = h[e];
}

template <int SH, int MT, int NB, int W, int S, int KH>
__global__ __launch_bounds__(64 * W, 2) void w4_tile_kernel(W4TileParams p)
{
    static_assert((KH == 1 || KH == 2) && W % KH == 0, "sets of waves");
    constexpr int WC = W / KH;                     // waves of a set, side by side
    constexpr int NS = 128 >> SH;                  // scales a tile and row of W
    constexpr int AF = (4 * MT + WC - 1) / WC;     // loads of A a wave and step: 4 rows each
    constexpr int SC = (NB * NS * 8 + 63) / 64;    // loads of scales
    constexpr int LOADS = AF + NB + SC;
    constexpr int SET_BYTES = AF * WC * 1024;      // of A, for a set's tile
    constexpr int A_BYTES = KH * SET_BYTES, W_BYTES = W * NB * 1024, S_BYTES = W * SC * 256;
    constexpr int STAGE = A_BYTES + W_BYTES + S_BYTES;
    static_assert(S >= 2 && (S - 2) * LOADS <= 63, "vmcnt counts at most 63 loads");
    static_assert(S * STAGE <= 160 * 1024, "LDS");
    __shared__ __attribute__((aligned(1024))) uint8_t smem[S * STAGE];
    const int lane = threadIdx.x & 63;
    const int wave = wave_index(), set = wave / WC, wc = wave % WC;
    const int r = lane & 15, kq = lane >> 4;
    // units run over the rows of A first, so that a word's users are neighbours
    int32_t u = xcd_unit();
    const int32_t tm = u % p.tiles_m;
    const int32_t un = u / p.tiles_m;
    const int32_t tn = un % p.tiles_n;
    const int32_t t0 = un / p.tiles_n * p.kt_split;
    const int32_t T = min(p.kt_split, p.kt - t0), steps = (T + KH - 1) / KH;
    const int32_t m0 = tm * 16 * MT;
    const int32_t b0 = (tn * WC + wc) * NB;
    const uint32_t klen = static_cast<uint32_t>(p.K - t0 * 128);
    const int32_t rows = min(16 * MT, p.M - m0);
    // rows past M and blocks past N start past their resources: zeros
    const i32x4_t ra = make_rsrc(p.A + static_cast<int64_t>(m0) * p.lda + t0 * 128,
                                 static_cast<uint32_t>(rows * p.lda - t0 * 128) * 2u);
    i32x4_t rw[NB];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
        const bool in = b0 + nb < p.nb;
        rw[nb] = make_rsrc(p.words + (static_cast<int64_t>(in ? b0 + nb : 0) * p.kt + t0) * 64,
                           in ? static_cast<uint32_t>(T) * 1024u : 0u);
    }
    const i32x4_t rs = make_rsrc(
        p.scales + (static_cast<int64_t>(b0 < p.nb ? b0 : 0) * p.kt + t0) * NS * 16,
        b0 < p.nb ? static_cast<uint32_t>((min(NB, p.nb - b0) - 1) * p.kt + T) * (NS * 32u) : 0u);
    // A in LDS: rows of 256 bytes, the 16-byte chunks of row i XORed with i to
    // spread the fragments' reads over the banks; applied where they are fetched
    uint32_t va[AF], ka[AF], vs[SC], vp[SC];
    const int32_t t_end = p.kt - 1 - t0;   // K's last tile: past this range, if not the last
#pragma unroll
    for (int i = 0; i < AF; ++i) {
        const int row = (i * WC + wc) * 4 + kq;
        ka[i] = 8 * (r ^ (row & 15));
        va[i] = row < 16 * MT
                    ? (static_cast<uint32_t>(row) * static_cast<uint32_t>(p.lda) + ka[i]) * 2u
                    : OOB_OFFSET;
    }
#pragma unroll
    for (int i = 0; i < SC; ++i) {
        const int d = i * 64 + lane, blk = d / (NS * 8), rem = d % (NS * 8);
        vs[i] = blk < NB ? static_cast<uint32_t>(blk) * p.kt * (NS * 32u) + rem * 4u : OOB_OFFSET;
        // in the tile that K ends in, without the scales of groups past K, which may
        // hold anything (chosen by a scalar condition, which costs up to 1.5% with
        // groups of 64 and nothing with 128; compared for each step, group against K,
        // 20 x 4096 x 14336 took 1 to 2% longer throughout)
        vp[i] = static_cast<uint32_t>(t_end) * 128u + ((rem / 8) << SH) < klen ? vs[i] : OOB_OFFSET;
    }
    int aoff[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) aoff[j] = r * 256 + ((4 * j + kq) ^ r) * 16;
    const uint32_t lds0 = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(smem));
    // step i's loads; past the range's end they fetch zeros, so that every
    // step waits for the same count
    auto fetch = [&](int stage, int32_t i) {
        const uint32_t base = lds0 + stage * STAGE;
        const int32_t t = i * KH + set;
        const bool in = t < T;
        const uint32_t ut = static_cast<uint32_t>(t);
        // past the range half of OOB_OFFSET: past the resource, also after OOB_OFFSET
        const uint32_t scales_at = in ? ut * (NS * 32u) : OOB_OFFSET / 2;
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
            dma16(rw[nb], in ? lane * 16u + ut * 1024u : OOB_OFFSET,
                  base + A_BYTES + (wave * NB + nb) * 1024);
#pragma unroll
        for (int s = 0; s < SC; ++s)
            dma4(rs, (NS > 1 && t == t_end ? vp[s] : vs[s]) + scales_at,
                 base + A_BYTES + W_BYTES + (wave * SC + s) * 256);
#pragma unroll
        for (int f = 0; f < AF; ++f)
            dma16(ra, in && va[f] != OOB_OFFSET && ka[f] + ut * 128u < klen ? va[f] + ut * 256u
                                                                         : OOB_OFFSET,
                  base + set * SET_BYTES + (f * WC + wc) * 1024);
    };
    f32x4_t acc[MT][NB] = {};
#pragma unroll
    for (int s = 0; s < S - 1; ++s) fetch(s, s);
    int stage = 0;
    u32x4_t wv[NB];
    _Float16 sc[NB][NS];
    // Waits until step i has landed (its loads are the oldest) and every wave
    // has read step i - 1 to the end, and sends for step i + S - 1.
    auto begin = [&](int32_t i) {
        asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier"
                     :
                     : "n"((S - 2) * LOADS)
                     : "memory");
        fetch(stage == 0 ? S - 1 : stage - 1, i + S - 1);
        const uint8_t *sw = smem + stage * STAGE + A_BYTES + wave * NB * 1024 + lane * 16;
        const uint8_t *ss = smem + stage * STAGE + A_BYTES + W_BYTES + wave * SC * 256 + r * 2;
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
            wv[nb] = *reinterpret_cast<const u32x4_t *>(sw + nb * 1024);
#pragma unroll
            for (int s = 0; s < NS; ++s)
                sc[nb][s] = *reinterpret_cast<const _Float16 *>(ss + (nb * NS + s) * 32);
        }
    };
    auto compute = [&](auto pair) {
        const uint8_t *st = smem + stage * STAGE + set * SET_BYTES;
        half8_t a[2][MT];
        auto read_a = [&](int j) {
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
                a[j & 1][mt] = *reinterpret_cast<const half8_t *>(st + mt * 4096 + aoff[j]);
        };
        // The order is fixed by hand: after each MFMA a share of the next
        // word's unpacking and of the next fragments' reads.  The compiler puts
        // the two kinds of work one after the other (333 x 4096 x 14336: 50.3
        // us, so 48.1, and 46.2 with a third buffer, S = 3).
        read_a(0);
        half8_t w[2];
        auto unpack = [&](int v, int i) {
            const half2_t x = pair(wv[v % NB][v / NB], i, sc[v % NB][(32 * (v / NB)) >> SH]);
            w[v & 1][2 * i] = x[0];
            w[v & 1][2 * i + 1] = x[1];
        };
#pragma unroll
        for (int i = 0; i < 4; ++i) unpack(0, i);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int u = 0; u < 4 * NB; ++u) {
            const int j = u / NB, nb = u % NB;
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                acc[mt][nb] = __builtin_amdgcn_mfma_f32_16x16x32_f16(w[u & 1], a[j & 1][mt],
                                                                     acc[mt][nb], 0, 0, 0);
                if (nb == 0 && j < 3)
                    a[(j + 1) & 1][mt] =
                        *reinterpret_cast<const half8_t *>(st + mt * 4096 + aoff[j + 1]);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (i * MT / 4 == mt && u + 1 < 4 * NB) unpack(u + 1, i);
                __builtin_amdgcn_sched_barrier(0);
            }
        }
        stage = stage == S - 1 ? 0 : stage + 1;
    };
    // The loop stops at a step with a scale too large for w4_tile_pair; a
    // second one then goes on from there.  (Both in one loop cost registers:
    // 48 x 16384 x 16384 took 45.3 us.)  The waves of a workgroup may be in
    // different loops, with the same barriers.
    const W4Bits bits = w4_high_bits();
    int32_t i = 0;
    bool large = false;
    for (; i < steps; ++i) {
        begin(i);
        float most = 0.0f;
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int s = 0; s < NS; ++s)
                most = fmaxf(most, __builtin_fabsf(static_cast<float>(sc[nb][s])));
        large = __any(most > W4_TILE_WORD_MOST);
        if (large) break;
        compute([&](uint32_t w, int i, _Float16 s) { return w4_tile_pair(w, i, s, bits); });
    }
    if (large) {
        const W4Bits low = w4_low_bits();
        for (;;) {
            compute([&](uint32_t w, int i, _Float16 s) { return w4_pair(w, i, s, low); });
            if (++i == steps) break;
            begin(i);
        }
    }
    // no load may still be on its way to this LDS when the workgroup ends
    asm volatile("s_waitcnt vmcnt(0)" : : : "memory");
    if constexpr (KH == 2) {
        static_assert(WC * NB * MT * 1024 <= S * STAGE, "LDS");
        f32x4_t *other = reinterpret_cast<f32x4_t *>(smem) + wc * (NB * MT * 64) + lane;
        __syncthreads();
        if (set == 1) {
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) other[(nb * MT + mt) * 64] = acc[mt][nb];
        }
        __syncthreads();
        if (set == 0) {
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) acc[mt][nb] += other[(nb * MT + mt) * 64];
        }
    }
    // lane l holds columns 4 (l / 16) .. + 3 of the block, row l % 16 of A
    if (p.splits > 1) {
        if (set > 0) return;
        float *to = p.partial + (static_cast<int64_t>(u) * WC + wc) * (NB * MT * 256) + lane * 4;
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
                *reinterpret_cast<f32x4_t *>(to + (nb * MT + mt) * 256) = acc[mt][nb];
        return;
    }
    // C through LDS, so that a row's columns leave in one run (stored as lanes
    // hold them, 32 bytes of a row at a time, 3936 x 15296 x 64 took 56.3 us; 42.8)
    constexpr int COLS = 16 * NB * WC, PITCH = COLS + 8;
    static_assert(16 * MT * PITCH * 2 <= S * STAGE, "LDS");
    _Float16 *rows_c = reinterpret_cast<_Float16 *>(smem);
    __syncthreads();
    if (set == 0) {
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
                *reinterpret_cast<half4_t *>(
                    &rows_c[(mt * 16 + r) * PITCH + (wc * NB + nb) * 16 + kq * 4]) =
                    __builtin_convertvector(acc[mt][nb], half4_t);
    }
    __syncthreads();
    for (int o = threadIdx.x; o < 2 * MT * COLS; o += 64 * W) {
        const int row = o / (COLS / 8), c = o % (COLS / 8) * 8;
        const int32_t n = tn * COLS + c;
        if (row >= rows || n >= p.N) continue;
        store8(p.C + static_cast<int64_t>(m0 + row) * p.N, n, p.N,
               *reinterpret_cast<const half8_t *>(&rows_c[row * PITCH + c]));
    }
}

// C from the ranges' sums, in order; one lane's four values a thread.
struct W4JoinParams {
    const float *partial;
    uint16_t *C;
    int64_t stride;            // values between two ranges' sums
    int32_t M, N, tiles_m, splits, mt, nb_wg;   // nb_wg: blocks of 16 columns a workgroup
};

__global__ __launch_bounds__(256) void w4_join_kernel(W4JoinParams p)
{
    const int64_t idx = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    if (idx * 4 >= p.stride) return;
    const int64_t frag = idx >> 6;
    const int lane = threadIdx.x & 63, r = lane & 15, kq = lane >> 4;
    const int32_t mt = static_cast<int32_t>(frag % p.mt);
    const int64_t block = frag / p.mt;
    const int32_t nb = static_cast<int32_t>(block % p.nb_wg);
    const int32_t tile = static_cast<int32_t>(block / p.nb_wg);
    const int32_t tm = tile % p.tiles_m, tn = tile / p.tiles_m;
    const int32_t m = (tm * p.mt + mt) * 16 + r, n = (tn * p.nb_wg + nb) * 16 + kq * 4;
    if (m >= p.M || n >= p.N) return;
    const float *from = p.partial + idx * 4;
    f32x4_t sum = *reinterpret_cast<const f32x4_t *>(from);
#pragma unroll 4
    for (int32_t s = 1; s < p.splits; ++s)
        sum += *reinterpret_cast<const f32x4_t *>(from + s * p.stride);
    store4(p.C, p.M, p.N, m, n, sum);
}

// Rows of `cols` values from one pitch to another; those from `cols` up to
// `limit` become zeros.  For a matrix whose rows are not all 16-byte aligned,
// which direct-to-LDS loads need, and back.
struct CopyRowsParams {
    const uint16_t *from;
    uint16_t *to;
    int64_t rows;
    int32_t ld_from, ld_to, cols, limit;
};

__global__ __launch_bounds__(256) void copy_rows_kernel(CopyRowsParams p)
{
    const int32_t chunks = (p.limit + 7) / 8;
    const int64_t count = p.rows * chunks;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < count;
         i += static_cast<int64_t>(gridDim.x) * 256) {
        const int64_t row = i / chunks;
        const int32_t c = static_cast<int32_t>(i - row * chunks) * 8;
        store8(p.to + row * p.ld_to, c, p.limit,
               bits_as<half8_t>(load8(p.from + row * p.ld_from, c, p.cols)));
    }
}

// ---------------------------------------------------------------------------
// Q8: quantise and read back
// ---------------------------------------------------------------------------
// A thread handles eight neighbouring columns, four neighbouring threads the
// 32 of a group, 2^tx_shift threads (at most a wave: 512 columns) a row, and
// each thread ROWS rows, so that several loads are in flight.  Memory bounds
// both kernels: 4999 x 7001 takes 18.5 us to codes and 16.6 back (5.8 and 6.4
// TB/s, part of it from the last cache).  Rows of codes and scales end inside
// cache lines, so neighbouring workgroups belong on one XCD: in launch order
// they read up to 1.4 times as much and took 21.7 and 20.3 us.
constexpr int Q8_ROWS = 4;

struct Q8Params {
    const uint16_t *X;        // quantise: from X to codes and scales
    uint16_t *out;            // dequantise: from codes and scales to out
    u32x2_t *codes;           // 8 codes each, 4 Ng a row
    uint16_t *scales;
    int32_t R, N, chunks;     // chunks of 8 columns a row: 4 Ng
    int32_t ld;               // out's rows start every ld values; up to ld they are written
    int32_t tx_shift, col_blocks;
};

__device__ __forceinline__ uint32_t quad_max(uint32_t v)
{
    uint32_t o = __builtin_amdgcn_update_dpp(0, v, 0xb1, 0xf, 0xf, true);   // lane ^ 1
    v = o > v ? o : v;
    o = __builtin_amdgcn_update_dpp(0, v, 0x4e, 0xf, 0xf, true);            // lane ^ 2
    return o > v ? o : v;
}

__global__ __launch_bounds__(64 * WAVES) void q8_encode_kernel(Q8Params p)
{
    const int32_t u = xcd_unit(), rb = u / p.col_blocks, cb = u - rb * p.col_blocks;
    const int32_t chunk = (cb << p.tx_shift) + (threadIdx.x & ((1 << p.tx_shift) - 1));
    const int32_t ty = (64 * WAVES) >> p.tx_shift;
    const int64_t row0 = static_cast<int64_t>(rb) * ty * Q8_ROWS + (threadIdx.x >> p.tx_shift);
    if (chunk >= p.chunks) return;    // whole groups: chunks is a multiple of 4
    const int64_t c = static_cast<int64_t>(chunk) * 8;
    u32x4_t v[Q8_ROWS];
    // a workgroup wholly inside the matrix takes the loads all at once
    if ((static_cast<int64_t>(cb + 1) << p.tx_shift) * 8 <= p.N &&
        (static_cast<int64_t>(rb) + 1) * ty * Q8_ROWS <= p.R) {
#pragma unroll
        for (int i = 0; i < Q8_ROWS; ++i)
            v[i] = bits_as<u32x4_t>(
                half8_t(*reinterpret_cast<const half8_u_t *>(p.X + (row0 + i * ty) * p.N + c)));
    } else {
#pragma unroll
        for (int i = 0; i < Q8_ROWS; ++i) {
            const int64_t row = row0 + i * ty;
            v[i] = u32x4_t{0, 0, 0, 0};
            if (row < p.R && c < p.N) v[i] = load8(p.X + row * p.N, static_cast<int32_t>(c), p.N);
        }
    }
#pragma unroll
    for (int i = 0; i < Q8_ROWS; ++i) {
        const int64_t row = row0 + i * ty;
        const uint32_t big = quad_max(largest8(v[i]));
        const bool bad = big >= 0x7c00;
        const float s = group_scale<4, 127>(big, 576.0f);
        const Reciprocal rcp = reciprocal(s);
        uint32_t k[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) k[e] = quotient(half_of(v[i], e), rcp, 0.0f);
        // 576 (the only scale past 512) times 114 would pass fp16's largest
        if (__builtin_expect(s > 512.0f, 0)) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float f = bits_as<float>(k[e]) - 0x1.8p23f;
                k[e] = bits_as<uint32_t>(fminf(fmaxf(f, -113.0f), 113.0f) + 0x1.8p23f);
            }
        }
        u32x2_t q;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint32_t lo = __builtin_amdgcn_perm(k[4 * h + 1], k[4 * h], 0x0c0c0400u);
            const uint32_t hi = __builtin_amdgcn_perm(k[4 * h + 3], k[4 * h + 2], 0x04000c0cu);
            q[h] = bad ? 0 : lo | hi;
        }
        if (row < p.R) {
            p.codes[row * p.chunks + chunk] = q;
            if ((chunk & 3) == 0)
                p.scales[row * (p.chunks >> 2) + (chunk >> 2)] =
                    bad ? FP16_NAN : bits_as<uint16_t>(static_cast<_Float16>(s));
        }
    }
}

// Four int8 codes of a dword times their scale: a byte b biased by 128 becomes
// the low bits of 1024 + (b + 128), which is exact in fp16.
__device__ __forceinline__ void q8_scaled(uint32_t codes, half2_t s2, half2_t *lo, half2_t *hi)
{
    const uint32_t u = codes ^ 0x80808080u;
    const half2_t off = {_Float16(1152.0f), _Float16(1152.0f)};
    // v_perm_b32: bytes of u spread to the low bytes of two halves, 0x64 above
    const uint32_t a = __builtin_amdgcn_perm(0x64646464u, u, 0x04010400u);
    const uint32_t b = __builtin_amdgcn_perm(0x64646464u, u, 0x04030402u);
    *lo = (bits_as<half2_t>(a) - off) * s2;
    *hi = (bits_as<half2_t>(b) - off) * s2;
}

__global__ __launch_bounds__(64 * WAVES) void q8_decode_kernel(Q8Params p)
{
    const int32_t u = xcd_unit(), rb = u / p.col_blocks, cb = u - rb * p.col_blocks;
    const int32_t chunk = (cb << p.tx_shift) + (threadIdx.x & ((1 << p.tx_shift) - 1));
    const int32_t ty = (64 * WAVES) >> p.tx_shift;
    const int64_t row0 = static_cast<int64_t>(rb) * ty * Q8_ROWS + (threadIdx.x >> p.tx_shift);
    const int64_t c = static_cast<int64_t>(chunk) * 8;
    if (chunk >= p.chunks || c >= p.N) return;
    u32x2_t q[Q8_ROWS];
    uint16_t s[Q8_ROWS];
#pragma unroll
    for (int i = 0; i < Q8_ROWS; ++i) {
        const int64_t row = row0 + i * ty < p.R ? row0 + i * ty : 0;
        q[i] = p.codes[row * p.chunks + chunk];
        s[i] = p.scales[row * (p.chunks >> 2) + (chunk >> 2)];
    }
#pragma unroll
    for (int i = 0; i < Q8_ROWS; ++i) {
        const int64_t row = row0 + i * ty;
        if (row >= p.R) continue;
        const half2_t s2 = {bits_as<_Float16>(s[i]), bits_as<_Float16>(s[i])};
        half2_t x[4];
        q8_scaled(q[i][0], s2, &x[0], &x[1]);
        q8_scaled(q[i][1], s2, &x[2], &x[3]);
        half8_t h;
#pragma unroll
        for (int e = 0; e < 8; ++e) h[e] = x[e / 2][e % 2];
        store8(p.out + row * p.ld, static_cast<int32_t>(c), p.ld, h);
    }
}

// ---------------------------------------------------------------------------
// C = A^T X for few columns of A (rows of C): the codes streamed once
// ---------------------------------------------------------------------------
// A workgroup computes 16 MT rows of C by 16 CB columns over a range of the
// rows of X.  Its waves take steps of 32 rows in turn, and lane l of a wave CB
// neighbouring columns of rows 8 (l / 16) .. + 7: byte e of its eight rows is,
// as it lies in its registers, what the MFMA wants from one lane for the
// column (l % 16) CB + e, so the codes need no turning round.  A byte becomes
// an fp16 number by v_perm_b32, one XOR (its bias and the magic exponent), one
// subtraction and the product with its scale: exact, two operations a value.
// A's rows and the scales of a step go through LDS of the wave's own, which
// turns them round.  The waves' sums meet in LDS, those of several ranges in the
// workspace, where q8_join_kernel adds them up in order.
//
// HBM bounds it, after the launches' 5 us.  CB = 16 reads the most a step
// (268 MB of codes at 4.8 TB/s, with CB = 8 4.1), CB = 8 makes fewer ranges of
// a small matrix (16 x 4096 over 8192 rows: 14.1 us, 15.4).  One workgroup a
// CU is best; eight waves instead of four cost 1 us, three or four buffers
// instead of two as much.  Neighbouring blocks of columns share cache lines of
// scales, so each XCD takes a contiguous range of units (8192 columns over
// 32768 rows: 68.6 to 56.8 us).
struct Q8TnParams {
    const uint16_t *A;         // [T, M]
    const uint8_t *codes;      // [T, 32 ng]
    const uint16_t *scales;    // [T, ng]
    uint16_t *C;               // [M, N]: written here where there is one range,
    float *partial;            // which is nullptr then
    int64_t stride;            // values between two ranges' sums
    int32_t T, M, N, ng;
    int32_t blocks, m_tiles;   // blocks of 16 CB columns, tiles of 16 MT rows of C
    int32_t t_split;           // rows of X a range, a multiple of 32
};

// 16-bit elements turned round in LDS: within 16 lanes, lane i addresses 4
// elements of row i / 4 at columns 4 (i % 4) .., and gets column i of the 4 rows.
__device__ __forceinline__ half4_t lds_read_tr16(const _Float16 *p)
{
    typedef short s4_t __attribute__((ext_vector_type(4)));
    typedef __attribute__((address_space(3))) s4_t lds_s4_t;
    return bits_as<half4_t>(__builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4_t *)(p)));
}

template <int MT, int CB, int W>
__global__ __launch_bounds__(64 * W, 2) void q8_tn_kernel(Q8TnParams p)
{
    constexpr int D = CB / 4;               // dwords of codes a lane and row
    constexpr int G = CB / 2;               // groups of 32 columns a block
    constexpr int AC = 2 * MT;              // 8-column chunks of A's rows
    constexpr int AP = 16 * MT + 8;         // pitch of A's rows in LDS
    // sums of a wave: [mt][e][reg] of 64 lanes; the waves' are joined in rounds
    constexpr int SUMS = MT * CB * 4, ROUND = SUMS < 64 ? SUMS : 64;
    struct Wave {
        _Float16 a[32 * AP];
        _Float16 s[G][32 + 8];
    };
    union Lds {
        Wave wave[W];
        float red[W][ROUND][64 + 4];   // 4: the sums of a row apart in the banks
    };
    __shared__ __attribute__((aligned(16))) Lds lds;
    const int lane = threadIdx.x & 63;
    const int wave = wave_index();
    const int r = lane & 15, kq = lane >> 4;
    int32_t u = xcd_unit();
    const int32_t mtile = u % p.m_tiles;
    u /= p.m_tiles;
    const int32_t block = u % p.blocks, sp = u / p.blocks;
    const int32_t m0 = mtile * 16 * MT;
    const int32_t t0 = sp * p.t_split;
    const int32_t t1 = min(p.T - t0, p.t_split) + t0;
    const int64_t np = 32 * static_cast<int64_t>(p.ng);
    const int64_t col = (static_cast<int64_t>(block) * 16 + r) * CB;   // this lane's columns of X
    const uint8_t *cp = p.codes + (col < np ? col : 0);   // past the end: sums not stored
    // scales: lane l fetches groups (l % 2) G / 2 .. of row l / 2
    const int32_t g0 = block * G + (lane & 1) * (G / 2);
    Wave &my = lds.wave[wave];
    uint32_t q[2][8][D];
    u32x4_t av[2][MT];
    uint16_t sv[2][G / 2];
    // whole steps of 32 rows that lie so far from X's last row that 8-column
    // loads of A stay inside it: unconditional loads
    const int32_t steps = (t1 - t0 + 31) / 32;
    const int32_t safe = min((t1 - t0) / 32, max(p.T - 8 - t0, 0) / 32);
    const int32_t count = safe > wave ? (safe - wave + W - 1) / W : 0;
    auto load_codes = [&](int buf, int k, int64_t row) {
        const uint8_t *c = cp + row * np;
        if constexpr (D == 4) {
            const u32x4_t v = __builtin_nontemporal_load(reinterpret_cast<const u32x4_t *>(c));
#pragma unroll
            for (int d = 0; d < 4; ++d) q[buf][k][d] = v[d];
        } else {
            const u32x2_t v = __builtin_nontemporal_load(reinterpret_cast<const u32x2_t *>(c));
            q[buf][k][0] = v[0];
            q[buf][k][1] = v[1];
        }
    };
    auto load = [&](int buf, int32_t i) {
        const int64_t t = t0 + (wave + static_cast<int64_t>(min(i, count - 1)) * W) * 32;
#pragma unroll
        for (int k = 0; k < 8; ++k) load_codes(buf, k, t + kq * 8 + k);
        const uint16_t *srow = p.scales + (t + (lane >> 1)) * p.ng;
#pragma unroll
        for (int g = 0; g < G / 2; ++g) sv[buf][g] = srow[min(g0 + g, p.ng - 1)];
#pragma unroll
        for (int j = 0; j < MT; ++j) {
            const int c = j * 64 + lane, m = m0 + c % AC * 8;
            av[buf][j] = bits_as<u32x4_t>(half8_t(*reinterpret_cast<const half8_u_t *>(
                p.A + (t + c / AC) * p.M + (m < p.M ? m : 0))));
        }
    };
    // any step: rows past the range are zeros
    auto load_guarded = [&](int32_t step) {
        const int32_t t = t0 + step * 32;
#pragma unroll
        for (int k = 0; k < 8; ++k) load_codes(0, k, min(t + kq * 8 + k, t1 - 1));
        const int32_t ts = t + (lane >> 1);
#pragma unroll
        for (int g = 0; g < G / 2; ++g)
            sv[0][g] = ts < t1 ? p.scales[static_cast<int64_t>(ts) * p.ng + min(g0 + g, p.ng - 1)] : 0;
#pragma unroll
        for (int j = 0; j < MT; ++j) {
            const int c = j * 64 + lane, ta = t + c / AC, m = m0 + c % AC * 8;
            av[0][j] = u32x4_t{0, 0, 0, 0};
            if (ta < t1 && m < p.M) av[0][j] = load8(p.A + static_cast<int64_t>(ta) * p.M, m, p.M);
        }
    };
    f32x4_t acc[MT][CB] = {};
    auto mma = [&](int buf) {
        wave_lds_fence();
#pragma unroll
        for (int j = 0; j < MT; ++j) {
            const int c = j * 64 + lane;
            *reinterpret_cast<u32x4_t *>(&my.a[c / AC * AP + c % AC * 8]) = av[buf][j];
        }
#pragma unroll
        for (int g = 0; g < G / 2; ++g)
            my.s[(lane & 1) * (G / 2) + g][lane >> 1] = bits_as<_Float16>(sv[buf][g]);
        wave_lds_fence();
        half8_t a[MT];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            const _Float16 *src = &my.a[(kq * 8 + (r >> 2)) * AP + mt * 16 + 4 * (r & 3)];
            const half4_t lo = lds_read_tr16(src), hi = lds_read_tr16(src + 4 * AP);
            a[mt] = half8_t{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
        }
        const half8_t s = *reinterpret_cast<const half8_t *>(&my.s[r * CB / 32][kq * 8]);
        const half2_t off = {_Float16(1152.0f), _Float16(1152.0f)};
#pragma unroll
        for (int e = 0; e < CB; ++e) {
            half8_t x;
            constexpr uint32_t sel[4] = {0x0c040c00u, 0x0c050c01u, 0x0c060c02u, 0x0c070c03u};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                // bytes e of rows 2 i and 2 i + 1, biased by 128, under 0x64
                const uint32_t b = __builtin_amdgcn_perm(q[buf][2 * i + 1][e / 4],
                                                         q[buf][2 * i][e / 4], sel[e % 4]) ^ 0x64806480u;
                const half2_t v = (bits_as<half2_t>(b) - off) * half2_t{s[2 * i], s[2 * i + 1]};
                x[2 * i] = v[0];
                x[2 * i + 1] = v[1];
            }
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
                acc[mt][e] = __builtin_amdgcn_mfma_f32_16x16x32_f16(x, a[mt], acc[mt][e], 0, 0, 0);
        }
    };
    // one buffer's loads fly while the other's are multiplied; past the end
    // the last step's again
    if (count > 0) {
        load(0, 0);
        int32_t i = 0;
        for (; i + 2 <= count; i += 2) {
            load(1, i + 1);
            __builtin_amdgcn_sched_barrier(0);
            mma(0);
            __builtin_amdgcn_sched_barrier(0);
            load(0, i + 2);
            __builtin_amdgcn_sched_barrier(0);
            mma(1);
            __builtin_amdgcn_sched_barrier(0);
        }
        if (i < count) mma(0);
    }
    for (int32_t step = safe; step < steps; ++step)
        if (step % W == wave) {
            load_guarded(step);
            mma(0);
        }
    // sum idx = (mt, e, reg) of lane l: row m0 + 16 mt + r of C, column (block 16 + 4 kq + reg) CB + e
    constexpr int ROUNDS = SUMS / ROUND, PER = ROUND / W, RM = ROUND / (4 * CB);
    static_assert(SUMS % ROUND == 0 && ROUND % W == 0 && ROUND % (4 * CB) == 0, "rounds");
    const int64_t unit = static_cast<int64_t>(block) * p.m_tiles + mtile;
#pragma unroll
    for (int rd = 0; rd < ROUNDS; ++rd) {
        __syncthreads();
#pragma unroll
        for (int k = 0; k < ROUND; ++k) {
            const int idx = rd * ROUND + k;
            lds.red[wave][k][lane] = acc[idx / (4 * CB)][idx / 4 % CB][idx % 4];
        }
        __syncthreads();
        if (p.partial) {   // a range's sums, in the order in which lanes hold them
            float *to = p.partial + sp * p.stride + (unit * SUMS + rd * ROUND) * 64 + lane;
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                const int k = wave * PER + i;
                float sum = 0.0f;
#pragma unroll
                for (int w = 0; w < W; ++w) sum += lds.red[w][k][lane];
                to[k * 64] = sum;
            }
            continue;
        }
        // the whole sum, eight neighbouring columns a thread
#pragma unroll
        for (int o = threadIdx.x; o < RM * 16 * 2 * CB; o += 64 * W) {
            const int row = o / (2 * CB), c = o % (2 * CB) * 8;
            const int l = c / (4 * CB) * 16 + row % 16;
            const int32_t m = m0 + (rd * RM + row / 16) * 16 + row % 16;
            const int64_t n = static_cast<int64_t>(block) * 16 * CB + c;
            if (m >= p.M || n >= p.N) continue;
            half8_t h;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int k = (row / 16 * CB + c % CB + i) * 4 + c / CB % 4;
                float sum = 0.0f;
#pragma unroll
                for (int w = 0; w < W; ++w) sum += lds.red[w][k][l];
                h[i] = static_cast<_Float16>(sum);
            }
            store8(p.C + static_cast<int64_t>(m) * p.N, static_cast<int32_t>(n), p.N, h);
        }
    }
}

// C from the ranges' sums, in order: a thread the four columns e .. e + 3 of one
// (block, tile of rows, mt, e / 4, reg, lane).
struct Q8JoinParams {
    const float *partial;
    uint16_t *C;
    int64_t stride;
    int32_t M, N, m_tiles, splits, mt, cb;
};

__global__ __launch_bounds__(256) void q8_join_kernel(Q8JoinParams p)
{
    const int64_t idx = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    if (idx * 4 >= p.stride) return;
    const int lane = threadIdx.x & 63, r = lane & 15, kq = lane >> 4;
    int64_t k = idx >> 6;
    const int reg = static_cast<int>(k & 3);
    k >>= 2;
    const int e4 = static_cast<int>(k % (p.cb / 4));
    k /= p.cb / 4;
    const int mt = static_cast<int>(k % p.mt);
    k /= p.mt;
    const int32_t mtile = static_cast<int32_t>(k % p.m_tiles);
    const int64_t block = k / p.m_tiles;
    const int32_t m = (mtile * p.mt + mt) * 16 + r;
    const int64_t n = (block * 16 + 4 * kq + reg) * p.cb + 4 * e4;
    if (m >= p.M || n >= p.N) return;
    const float *from = p.partial + (block * p.m_tiles + mtile) * (static_cast<int64_t>(p.mt) * p.cb * 256) +
                        ((mt * p.cb + 4 * e4) * 4 + reg) * 64 + lane;
    f32x4_t sum = {0, 0, 0, 0};
#pragma unroll 4
    for (int32_t s = 0; s < p.splits; ++s) {
#pragma unroll
        for (int e = 0; e < 4; ++e) sum[e] += from[s * p.stride + e * 256];
    }
    store4(p.C, p.M, p.N, m, static_cast<int32_t>(n), sum);
}

// ---------------------------------------------------------------------------
// Host
// ---------------------------------------------------------------------------
static int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }
static int64_t round_up(int64_t a, int64_t b) { return cdiv(a, b) * b; }

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

static int launch(const void *fn, int64_t grid, int threads, void *params, hipStream_t stream)
{
    // the launch's own status only: the thread's sticky error state is neither
    // read nor cleared
    void *args[] = {params};
    const hipError_t err = hipLaunchKernel(fn, dim3(static_cast<uint32_t>(grid)),
                                           dim3(static_cast<uint32_t>(threads)), args, 0, stream);
    return err == hipSuccess ? GEMM_F16_OK : GEMM_F16_LAUNCH_FAILED;
}

struct W4Shape {
    int64_t nb, kt, tiles, words, scales;   // blocks, tiles a block, all tiles, bytes
    int32_t shift;
};

static int w4_shape(int64_t N, int64_t K, int32_t group, W4Shape *s)
{
    if (N < 0 || K < 0) return GEMM_F16_INVALID_ARG;
    if (group != 32 && group != 64 && group != 128) return GEMM_F16_INVALID_ARG;
    // the kernels count in whole tiles past the end in 32 bits
    if (N > INT32_MAX - 127 || K > INT32_MAX - 127) return GEMM_F16_UNSUPPORTED;
    s->nb = cdiv(N, 16);
    s->kt = cdiv(K, 128);
    s->tiles = s->nb * s->kt;
    if (s->tiles > INT32_MAX) return GEMM_F16_UNSUPPORTED;
    s->words = s->tiles * 1024;
    s->scales = s->tiles * (128 / group) * 32;
    s->shift = group == 32 ? 5 : group == 64 ? 6 : 7;
    return GEMM_F16_OK;
}

// workgroups for `tiles` waves of work: the loops take the rest
static int64_t wave_grid(int64_t tiles) { return std::min<int64_t>(cdiv(tiles, WAVES), 1 << 20); }

static int w4_encode(int64_t N, int64_t K, int32_t group, const void *W, const void *codes,
                     const void *in_scales, void *words, void *scales, hipStream_t stream)
{
    W4Shape s;
    const int v = w4_shape(N, K, group, &s);
    if (v != GEMM_F16_OK) return v;
    const bool pack = W == nullptr && codes != nullptr;
    const Array in[2] = {pack ? Array{codes, N * K, 1, false} : Array{W, N * K * 2, 2, false},
                         Array{in_scales, pack ? N * cdiv(K, group) * 2 : 0, 2, false}};
    const Array arrays[4] = {in[0], in[1], {words, s.words, 16, true}, {scales, s.scales, 8, true}};
    const int a = check_arrays(arrays, 4);
    if (a != GEMM_F16_OK || s.tiles == 0) return a;
    W4EncodeParams p;
    p.W = static_cast<const uint16_t *>(W);
    p.codes = static_cast<const int8_t *>(codes);
    p.in_scales = static_cast<const uint16_t *>(in_scales);
    p.words = static_cast<u32x4_t *>(words);
    p.scales = static_cast<uint16_t *>(scales);
    p.N = static_cast<int32_t>(N);
    p.K = static_cast<int32_t>(K);
    p.kt = static_cast<int32_t>(s.kt);
    p.tiles = static_cast<int32_t>(s.tiles);
    p.shift = s.shift;
    const void *fn = pack ? reinterpret_cast<const void *>(&w4_encode_kernel<true>)
                          : reinterpret_cast<const void *>(&w4_encode_kernel<false>);
    return launch(fn, wave_grid(s.tiles), 64 * WAVES, &p, stream);
}

static int w4_decode(int64_t N, int64_t K, const W4Shape &s, const void *words,
                     const void *scales, void *W, int64_t ld, hipStream_t stream)
{
    W4DecodeParams p;
    p.words = static_cast<const u32x4_t *>(words);
    p.scales = static_cast<const uint16_t *>(scales);
    p.W = static_cast<uint16_t *>(W);
    p.N = static_cast<int32_t>(N);
    p.K = static_cast<int32_t>(K);
    p.ld = static_cast<int32_t>(ld);
    p.kt = static_cast<int32_t>(s.kt);
    p.tiles = static_cast<int32_t>(s.tiles);
    p.shift = s.shift;
    return launch(reinterpret_cast<const void *>(&w4_decode_kernel), wave_grid(s.tiles), 64 * WAVES,
                  &p, stream);
}

struct Q8Shape {
    int64_t groups, codes, scales;   // groups a row, bytes
};

static int q8_shape(int64_t R, int64_t N, Q8Shape *s)
{
    if (R < 0 || N < 0) return GEMM_F16_INVALID_ARG;
    if (R > INT32_MAX - 31 || N > INT32_MAX - 31) return GEMM_F16_UNSUPPORTED;
    s->groups = cdiv(N, GEMM_F16_Q8_GROUP);
    s->codes = R * s->groups * GEMM_F16_Q8_GROUP;
    s->scales = R * s->groups * 2;
    // A workgroup of 256 takes 8192 values, in matrices a little wider than its
    // 512 columns 4352: 2^36 keep a launch's threads within 32 bits.
    if (s->codes > (int64_t(1) << 36)) return GEMM_F16_UNSUPPORTED;
    return GEMM_F16_OK;
}

static int q8_launch(const void *fn, int64_t R, int64_t N, const Q8Shape &s, const void *X,
                     void *out, int64_t ld, const void *codes, const void *scales,
                     hipStream_t stream)
{
    Q8Params p;
    p.X = static_cast<const uint16_t *>(X);
    p.out = static_cast<uint16_t *>(out);
    p.codes = static_cast<u32x2_t *>(const_cast<void *>(codes));
    p.scales = static_cast<uint16_t *>(const_cast<void *>(scales));
    p.R = static_cast<int32_t>(R);
    p.N = static_cast<int32_t>(N);
    p.chunks = static_cast<int32_t>(s.groups * 4);
    p.ld = static_cast<int32_t>(ld);
    p.tx_shift = 2;
    while (p.tx_shift < 6 && (1 << p.tx_shift) < p.chunks) ++p.tx_shift;
    const int64_t col_blocks = cdiv(p.chunks, int64_t(1) << p.tx_shift);
    p.col_blocks = static_cast<int32_t>(col_blocks);
    const int64_t grid = col_blocks * cdiv(R, int64_t((64 * WAVES) >> p.tx_shift) * Q8_ROWS);
    return launch(fn, grid, 64 * WAVES, &p, stream);
}

// ---- products ---------------------------------------------------------------
static int copy_rows(const void *from, int64_t ld_from, void *to, int64_t ld_to, int64_t rows,
                     int64_t cols, int64_t limit, hipStream_t stream)
{
    CopyRowsParams p;
    p.from = static_cast<const uint16_t *>(from);
    p.to = static_cast<uint16_t *>(to);
    p.rows = rows;
    p.ld_from = static_cast<int32_t>(ld_from);
    p.ld_to = static_cast<int32_t>(ld_to);
    p.cols = static_cast<int32_t>(cols);
    p.limit = static_cast<int32_t>(limit);
    return launch(reinterpret_cast<const void *>(&copy_rows_kernel),
                  std::min<int64_t>(cdiv(rows * cdiv(limit, 8), 256), 1 << 16), 256, &p, stream);
}

// Decode: the low-bit operand in fp16, then the library's fp16 GEMM.  The
// GEMM's fast kernels need rows of a multiple of 8 values, so the fp16 operand
// gets such rows, A a copy where it has none, and C a padded one where its
// columns (A^T X: or rows) are not a multiple of 8.  (The GEMM's kernels for
// other rows run at a fraction of the rate: C = A^T X of 1069 x 463 over 2357
// rows took 160 us.)  An A whose address is not 16-byte aligned takes those all
// the same.
struct Decode {
    int64_t M, N, K;                  // the GEMM's sizes
    int64_t b, a, c, split;           // offsets in the workspace: operand, A, C, partial sums
    int64_t bytes;
    int32_t splits;
    gemm_f16_nt_plan_t plan;
};

static int decode_layout(int64_t M, int64_t N, int64_t K, int32_t num_cus, bool tn, Decode *d)
{
    d->M = tn ? round_up(M, 8) : M;
    d->N = tn ? round_up(N, 8) : N;
    d->K = tn ? K : round_up(K, 8);
    // the workspace's offsets in 64 bits
    const int64_t most = int64_t(1) << 60;
    if (d->M * d->K > most || d->N * d->K > most || d->M * d->N > most) return GEMM_F16_UNSUPPORTED;
    int64_t ws = 0;
    const int v = tn ? gemm_f16_tn_splitk_plan(d->M, d->N, d->K, num_cus, 0, &d->plan, &d->splits, &ws)
                     : gemm_f16_nt_splitk_plan(d->M, d->N, d->K, num_cus, 0, &d->plan, &d->splits, &ws);
    if (v != GEMM_F16_OK) return v;
    d->b = 0;
    d->a = round_up(d->N * d->K * 2, 256);
    d->c = d->a + ((tn ? d->M != M : d->K != K) ? round_up(d->M * d->K * 2, 256) : 0);
    d->split = d->c + (d->M != M || d->N != N ? round_up(d->M * d->N * 2, 256) : 0);
    d->bytes = d->split + ws;
    return GEMM_F16_OK;
}

static int decode_plan(int64_t M, int64_t N, int64_t K, int32_t num_cus, bool tn,
                       gemm_f16_lowbit_plan_t *plan)
{
    Decode d;
    const int v = decode_layout(M, N, K, num_cus, tn, &d);
    if (v != GEMM_F16_OK) return v;
    plan->kernel = GEMM_F16_LOWBIT_DECODE;
    plan->block_m = d.plan.block_m;
    plan->block_n = d.plan.block_n;
    plan->waves = d.plan.waves;
    plan->splits = d.splits;
    plan->grid = d.plan.grid;
    plan->workspace_bytes = d.bytes;
    return GEMM_F16_OK;
}

// The GEMM, after the operand is written to the workspace's start.
static int decode_gemm(const Decode &d, int64_t M, int64_t N, int64_t K, bool tn, const void *A,
                       void *C, char *ws, hipStream_t stream)
{
    const int64_t cols = tn ? M : K, ld = tn ? d.M : d.K, rows = tn ? K : M;
    int v = GEMM_F16_OK;
    if (ld != cols) {
        v = copy_rows(A, cols, ws + d.a, ld, rows, cols, ld, stream);
        A = ws + d.a;
    }
    if (v != GEMM_F16_OK) return v;
    const bool padded = d.M != M || d.N != N;
    void *out = padded ? ws + d.c : C;
    v = tn ? gemm_f16_tn_splitk(d.M, d.N, d.K, A, ws, out, 0, ws + d.split, d.bytes - d.split, stream)
           : gemm_f16_nt_splitk(d.M, d.N, d.K, A, ws, out, 0, ws + d.split, d.bytes - d.split, stream);
    if (v != GEMM_F16_OK || !padded) return v;
    return copy_rows(out, d.N, C, N, M, N, N, stream);
}

// The kernels of the product with 4-bit weights that read the words directly,
// for each group size.
struct W4Kernel {
    int32_t kernel, rows, blocks, waves;   // rows of A, blocks of 16 rows of W a workgroup
    int32_t tiles_step;                    // tiles of 128 columns that its waves take at once
    // Where a model of times chooses: us before the first step, and a step with
    // one workgroup on a CU and with two (0: they do not fit).
    double start, step1, step2;
    const void *fn[3];                     // group 32, 64, 128
};
#define W4_KERNEL(KIND, ROWS, BLOCKS, W, STEP, T0, T1, T2, K5, K6, K7)                \
    W4Kernel{KIND, ROWS, BLOCKS, W, STEP, T0, T1, T2,                                 \
             {reinterpret_cast<const void *>(&K5), reinterpret_cast<const void *>(&K6), \
              reinterpret_cast<const void *>(&K7)}}
#define W4_STREAM(JC, NB, W, D)                                                       \
    W4_KERNEL(GEMM_F16_LOWBIT_STREAM, 16 / JC, NB, W, W, 0, 0, 0, (w4_stream_kernel<5, JC, NB, W, D>), \
              (w4_stream_kernel<6, JC, NB, W, D>), (w4_stream_kernel<7, JC, NB, W, D>))
#define W4_ROWS(RL, NB, W, T0, T1, T2)                                                \
    W4_KERNEL(GEMM_F16_LOWBIT_STREAM, 4 * RL, NB, W, W, T0, T1, T2, (w4_rows_kernel<5, RL, NB, W>), \
              (w4_rows_kernel<6, RL, NB, W>), (w4_rows_kernel<7, RL, NB, W>))
#define W4_TILE(MT, NB, W, S, KH, T1, T2)                                             \
    W4_KERNEL(GEMM_F16_LOWBIT_TILE, 16 * MT, NB * W / KH, W, KH, 3.35, T1, T2,        \
              (w4_tile_kernel<5, MT, NB, W, S, KH>), (w4_tile_kernel<6, MT, NB, W, S, KH>), \
              (w4_tile_kernel<7, MT, NB, W, S, KH>))
static const W4Kernel kW4Kernels[] = {
    W4_STREAM(4, 1, 8, 2),
    W4_ROWS(2, 1, 8, 0, 0, 0), W4_ROWS(2, 2, 8, 0, 0, 0),
    W4_ROWS(4, 1, 8, 0, 0, 0), W4_ROWS(4, 2, 8, 0, 0, 0), W4_ROWS(4, 4, 8, 0, 0, 0),
    W4_ROWS(8, 1, 8, 2.63, 1.043, 0),      W4_ROWS(8, 2, 4, 3.33, 0.625, 1.290),
    W4_ROWS(8, 4, 8, 3.44, 2.101, 0),      W4_ROWS(12, 1, 8, 2.83, 1.452, 0),
    W4_ROWS(12, 2, 4, 3.96, 0.806, 1.629), W4_ROWS(12, 4, 4, 4.45, 1.382, 0),
    W4_TILE(2, 2, 4, 4, 1, 0.500, 0.790), W4_TILE(3, 2, 8, 2, 1, 0.869, 1.417),
    W4_TILE(4, 2, 8, 2, 2, 1.170, 0),     W4_TILE(4, 2, 8, 3, 1, 0.962, 0),
    W4_TILE(6, 2, 8, 2, 2, 1.446, 0),     W4_TILE(6, 2, 8, 3, 1, 1.173, 0),
    W4_TILE(7, 2, 8, 3, 1, 1.312, 0),     W4_TILE(8, 2, 8, 3, 1, 1.452, 0),
};
constexpr int kNumW4Kernels = sizeof(kW4Kernels) / sizeof(kW4Kernels[0]);

// What a product runs: an index into kW4Kernels (-1: decode) and the ranges
// that K is split into.
struct W4Choice {
    int32_t id, splits;
};

// A launch counts its threads in 32 bits: of workgroups of 512, fewer than 2^23.
// Matrices of more blocks (67 million rows of W) are decoded for the GEMM, whose
// grid does not grow with them.
constexpr int64_t W4_MOST_WORKGROUPS = 1 << 22;

// Kernel `e`'s time in us by the model, its K in `ranges` ranges of `kt` tiles.
static double w4_model(const W4Kernel &e, int64_t workgroups, int64_t kt, int64_t ranges, int32_t cus)
{
    const int64_t steps = cdiv(kt, e.tiles_step);
    const bool two = e.step2 > 0;
    const int64_t slots = static_cast<int64_t>(cus) * (two ? 2 : 1);
    const int64_t full = workgroups / slots, rest = workgroups % slots;
    double us = e.start + full * (two ? e.step2 : e.step1) * steps;
    if (rest > 0) us += (rest <= cus || !two ? e.step1 : e.step2) * steps;
    if (ranges > 1)
        us += 2.27 + 0.111 * ranges +
              3.55e-7 * static_cast<double>(workgroups) * (e.rows / 16) * e.blocks * 1024;
    return us;
}

// The stream kernel for at most 48 rows, and its time (16 rows and fewer: none).
static int32_t w4_choose_stream(int64_t M, const W4Shape &s, int32_t cus, double *best_us)
{
    if (M <= 4) return 0;
    // the most blocks a workgroup that still give three CUs in four one
    const int64_t most = s.nb / std::max<int64_t>(1, 3 * static_cast<int64_t>(cus) / 4);
    if (M <= 8) return most >= 2 ? 2 : 1;
    if (M <= 16) return most >= 4 ? 5 : most >= 2 ? 4 : 3;
    int32_t best = -1;
    for (int32_t id = 0; id < kNumW4Kernels; ++id) {
        const W4Kernel &e = kW4Kernels[id];
        if (e.kernel != GEMM_F16_LOWBIT_STREAM || e.start == 0 || e.rows < M) continue;
        const double us = w4_model(e, cdiv(s.nb, e.blocks), s.kt, 1, cus);
        if (best < 0 || us < *best_us) {
            *best_us = us;
            best = id;
        }
    }
    return best;
}
constexpr int64_t W4_STREAM_ROWS = 48;

// The stream kernels up to 48 rows, the tile kernels and splits, and the
// decoding path, by a model of their times in us, fitted to 8,000 timings of
// 160 shapes (20 to 2048 rows, N and K of 512 to 32768, words from HBM): rounds
// of workgroups over the CUs times the steps of a range, the clock that long
// products lose to the power limit, and for a split the partial sums' way
// through memory and the join.  (Those timings are not kept with the source.)  Its
// error is 6%; what it chose took 1 to 2% longer than the best of each shape in
// the mean, 16 to 17% in the worst (333 x 4096 x 4096: 96 x 128 in two ranges,
// 24.3 us, where 64 x 128 unsplit took 20.7).  (Of 17 to 48 rows, the tile kernels
// alone took 25% longer: 32 x 4096 x 4096 9.8 us, streamed 7.5.)
static W4Choice w4_search(int64_t M, int64_t K, const W4Shape &s, int32_t cus)
{
    const double nk = static_cast<double>(s.nb) * 16 * K;
    // words to fp16 and back from memory, and the GEMM at its rate for large M
    W4Choice best = {-1, 1};
    double best_us = 12.2 + (7.0e-7 + 1.10e-9 * std::max<double>(M, 423)) * std::max(nk, 8.4e6);
    if (M <= W4_STREAM_ROWS) {
        double us = 0;
        const int32_t id = w4_choose_stream(M, s, cus, &us);
        if (us < best_us) {
            best_us = us;
            best.id = id;
        }
    }
    // 32-bit offsets of the tile kernel's resources
    if (M > 8192 || K > (1 << 21)) return best;
    for (int32_t id = 0; id < kNumW4Kernels; ++id) {
        const W4Kernel &e = kW4Kernels[id];
        if (e.kernel != GEMM_F16_LOWBIT_TILE) continue;
        const int64_t tiles = cdiv(M, e.rows) * cdiv(s.nb, e.blocks);
        if (tiles > W4_MOST_WORKGROUPS) continue;
        const int64_t slots = static_cast<int64_t>(cus) * (e.step2 > 0 ? 2 : 1);
        int64_t last = 0;
        for (int64_t sp = 1; sp <= 64 && sp <= s.kt && (sp == 1 || tiles * sp <= 4 * slots); ++sp) {
            const int64_t per = cdiv(s.kt, sp);
            if (per == last) continue;   // the same ranges
            last = per;
            const int64_t ranges = cdiv(s.kt, per);
            const double us = w4_model(e, tiles * ranges, per, ranges, cus) +
                              2.81e-10 * std::max(0.0, nk * static_cast<double>(M) - 1.05e10);
            if (us < best_us) {
                best_us = us;
                best = {id, static_cast<int32_t>(ranges)};
            }
        }
    }
    return best;
}

static W4Choice w4_choose(int64_t M, int64_t K, const W4Shape &s, int32_t cus)
{
    if (s.nb > W4_MOST_WORKGROUPS) return {-1, 1};
    // Streamed and never split, which is right where the blocks of 16 columns fill
    // the CUs.  Few columns of a long K leave them empty: 16 x 64 x 2^20 takes 723 us
    // and 17 rows, which a search splits, 81; 16 x 1024 x 16384 12.4 and 10.9.
    if (M <= 16) return {w4_choose_stream(M, s, cus, nullptr), 1};
    // the search takes microseconds: each thread keeps its last few choices
    struct Entry {
        int64_t M, K, nb;
        int32_t cus;
        W4Choice choice;
    };
    static thread_local Entry cache[8] = {};
    static thread_local int next = 0;
    for (const Entry &c : cache)
        if (c.cus == cus && c.M == M && c.K == K && c.nb == s.nb) return c.choice;
    const W4Choice choice = w4_search(M, K, s, cus);
    cache[next] = Entry{M, K, s.nb, cus, choice};
    next = (next + 1) % 8;
    return choice;
}

// The tile kernel's split of `kt` tiles of K: tiles a range, and how many
// ranges that makes.
static void w4_ranges(int64_t kt, int32_t splits, int64_t *per_range, int32_t *ranges)
{
    *per_range = cdiv(kt, splits);
    *ranges = static_cast<int32_t>(cdiv(kt, *per_range));
}

static int64_t w4_partial_bytes(const W4Kernel &e, int64_t M, const W4Shape &s)
{
    return cdiv(M, e.rows) * cdiv(s.nb, e.blocks) * (e.rows / 16) * e.blocks * 1024;
}

static int w4_plan_choice(const W4Choice &c, int64_t M, int64_t N, int64_t K, const W4Shape &s,
                          int32_t num_cus, gemm_f16_lowbit_plan_t *plan)
{
    if (c.id < 0) return decode_plan(M, N, K, num_cus, false, plan);
    const W4Kernel &e = kW4Kernels[c.id];
    plan->kernel = e.kernel;
    plan->block_m = e.rows;
    plan->block_n = 16 * e.blocks;
    plan->waves = e.waves;
    int64_t grid = cdiv(s.nb, e.blocks);
    if (e.kernel == GEMM_F16_LOWBIT_TILE) {
        int64_t per_range;
        w4_ranges(s.kt, c.splits, &per_range, &plan->splits);
        grid *= cdiv(M, e.rows) * plan->splits;
        if (plan->splits > 1) plan->workspace_bytes = plan->splits * w4_partial_bytes(e, M, s);
        if (K % 8 != 0) plan->workspace_bytes += round_up(M * round_up(K, 8) * 2, 256);   // A's copy
    }
    plan->grid = static_cast<int32_t>(grid);
    return GEMM_F16_OK;
}

static int w4_plan(int64_t M, int64_t N, int64_t K, int32_t group, int32_t num_cus,
                   gemm_f16_lowbit_plan_t *plan)
{
    W4Shape s;
    const int v = w4_shape(N, K, group, &s);
    if (v != GEMM_F16_OK) return v;
    if (M < 0 || num_cus <= 0) return GEMM_F16_INVALID_ARG;
    if (M > INT32_MAX) return GEMM_F16_UNSUPPORTED;
    *plan = gemm_f16_lowbit_plan_t{};
    plan->splits = 1;
    if (M == 0 || N == 0 || K == 0) return GEMM_F16_OK;
    return w4_plan_choice(w4_choose(M, K, s, num_cus), M, N, K, s, num_cus, plan);
}

static int w4_stream(int32_t id, int64_t M, int64_t N, int64_t K, const W4Shape &s, const void *A,
                     const void *words, const void *scales, void *C, hipStream_t stream)
{
    const W4Kernel &e = kW4Kernels[id];
    W4Params p;
    p.A = static_cast<const uint16_t *>(A);
    p.words = static_cast<const u32x4_t *>(words);
    p.scales = static_cast<const uint16_t *>(scales);
    p.C = static_cast<uint16_t *>(C);
    p.M = static_cast<int32_t>(M);
    p.N = static_cast<int32_t>(N);
    p.K = static_cast<int32_t>(K);
    p.kt = static_cast<int32_t>(s.kt);
    p.nb = static_cast<int32_t>(s.nb);
    return launch(e.fn[s.shift - 5], cdiv(s.nb, e.blocks), 64 * e.waves, &p, stream);
}

static int w4_run(const W4Choice &c, const gemm_f16_lowbit_plan_t &plan, int64_t M, int64_t N,
                  int64_t K, const W4Shape &s, const void *A, const void *words,
                  const void *scales, void *C, void *workspace, int32_t cus, hipStream_t stream)
{
    char *ws = static_cast<char *>(workspace);
    if (c.id < 0) {
        Decode d;
        int v = decode_layout(M, N, K, cus, false, &d);
        if (v == GEMM_F16_OK) v = w4_decode(N, K, s, words, scales, ws + d.b, d.K, stream);
        if (v == GEMM_F16_OK) v = decode_gemm(d, M, N, K, false, A, C, ws, stream);
        return v;
    }
    const W4Kernel &e = kW4Kernels[c.id];
    if (e.kernel == GEMM_F16_LOWBIT_STREAM)
        return w4_stream(c.id, M, N, K, s, A, words, scales, C, stream);
    if (K % 8 == 0 && reinterpret_cast<uintptr_t>(A) % 16 != 0) {
        // the tile kernels' loads need 16-byte aligned rows, and the workspace
        // is planned by sizes alone: 48 rows at a time by the kernels that take
        // any alignment (64 x 4096 x 14336: 68 us for 18; 512 x 4096 x 4096: 186 for 24)
        for (int64_t m = 0; m < M; m += W4_STREAM_ROWS) {
            const int64_t rows = std::min(W4_STREAM_ROWS, M - m);
            double us = 0;
            const int v = w4_stream(w4_choose_stream(rows, s, cus, &us), rows, N, K, s,
                                    static_cast<const uint16_t *>(A) + m * K, words, scales,
                                    static_cast<uint16_t *>(C) + m * N, stream);
            if (v != GEMM_F16_OK) return v;
        }
        return GEMM_F16_OK;
    }
    W4TileParams p;
    int64_t per_range;
    w4_ranges(s.kt, c.splits, &per_range, &p.splits);
    const int64_t partial = w4_partial_bytes(e, M, s);
    p.A = static_cast<const uint16_t *>(A);
    p.lda = static_cast<int32_t>(K);
    p.partial = static_cast<float *>(workspace);
    if (K % 8 != 0) {
        uint16_t *to =
            reinterpret_cast<uint16_t *>(ws + (p.splits > 1 ? p.splits * partial : 0));
        p.lda = static_cast<int32_t>(round_up(K, 8));
        const int v = copy_rows(A, K, to, p.lda, M, K, p.lda, stream);
        if (v != GEMM_F16_OK) return v;
        p.A = to;
    }
    p.words = static_cast<const u32x4_t *>(words);
    p.scales = static_cast<const uint16_t *>(scales);
    p.C = static_cast<uint16_t *>(C);
    p.M = static_cast<int32_t>(M);
    p.N = static_cast<int32_t>(N);
    p.K = static_cast<int32_t>(K);
    p.kt = static_cast<int32_t>(s.kt);
    p.nb = static_cast<int32_t>(s.nb);
    p.tiles_m = static_cast<int32_t>(cdiv(M, e.rows));
    p.tiles_n = static_cast<int32_t>(cdiv(s.nb, e.blocks));
    p.kt_split = static_cast<int32_t>(per_range);
    const int v = launch(e.fn[s.shift - 5], plan.grid, 64 * e.waves, &p, stream);
    if (v != GEMM_F16_OK || p.splits == 1) return v;
    W4JoinParams q;
    q.partial = p.partial;
    q.C = p.C;
    q.stride = partial / 4;
    q.M = p.M;
    q.N = p.N;
    q.tiles_m = p.tiles_m;
    q.splits = p.splits;
    q.mt = e.rows / 16;
    q.nb_wg = e.blocks;
    return launch(reinterpret_cast<const void *>(&w4_join_kernel), cdiv(partial, 4096), 256, &q,
                  stream);
}

// The kernels of the product with 8-bit activations that read the codes.
struct Q8Kernel {
    int32_t mt, cb, waves;
    double step;           // us a step of 32 rows of X for each wave
    const void *fn;
};
#define Q8_TN(MT, CB, W, STEP) \
    Q8Kernel{MT, CB, W, STEP, reinterpret_cast<const void *>(&q8_tn_kernel<MT, CB, W>)}
static const Q8Kernel kQ8Kernels[] = {
    Q8_TN(1, 8, 4, 0.651), Q8_TN(1, 16, 4, 1.11), Q8_TN(2, 8, 4, 0.810), Q8_TN(4, 8, 4, 1.06),
};
#undef Q8_TN
constexpr int kNumQ8Kernels = sizeof(kQ8Kernels) / sizeof(kQ8Kernels[0]);

// What a product runs: an index into kQ8Kernels (-1: decode), tiles and ranges.
struct Q8Choice {
    int32_t id;
    int64_t blocks, m_tiles, t_split, splits;
};

static Q8Choice q8_layout(int32_t id, int64_t M, int64_t K, const Q8Shape &s, int32_t cus,
                          bool split)
{
    const Q8Kernel &e = kQ8Kernels[id];
    Q8Choice c;
    c.id = id;
    c.blocks = cdiv(s.groups * GEMM_F16_Q8_GROUP, 16 * e.cb);
    c.m_tiles = cdiv(M, 16 * e.mt);
    // one workgroup a CU, where the rows suffice for a step for each wave
    const int64_t steps = cdiv(K, 32);
    const int64_t want = split ? std::max<int64_t>(1, cus / (c.blocks * c.m_tiles)) : 1;
    const int64_t per = cdiv(steps, std::min(want, cdiv(steps, e.waves)));
    c.t_split = per * 32;
    c.splits = cdiv(steps, per);
    return c;
}

// Streaming the codes (in one range, or in as many as fill the CUs), or
// decoding them for the GEMM, by models of their times in us, fitted to 2,900
// timings of 870 shapes (8 to 7668 rows of C, 64 to 14336 columns, 3 to 8192
// rows of X, sizes that are multiples of 8 and not; not kept with the source).
// Streaming reads the codes
// again for each tile of rows of C; it wins up to some 64 rows everywhere (1.1
// to 3.2 times), with hundreds of rows where the columns are few, and with
// thousands where the rows of X are (3300 x 3613 over 54 rows: 31.4 us decoded,
// 19.8 streamed).  What the models chose took 1.6% longer than the best of each
// shape in the mean, 37% in the worst.
static Q8Choice q8_choose(int64_t M, int64_t N, int64_t K, const Q8Shape &s, int32_t cus)
{
    const double m = static_cast<double>(M), n = static_cast<double>(N), k = static_cast<double>(K);
    Q8Choice best = {-1, 0, 0, 0, 0};
    // 32-bit counts of tiles and values in the kernels
    if (s.groups > (1 << 20) || M > (1 << 20) || M * s.groups > (1 << 26)) return best;
    // 1 us of each workspace is the caller's, who has to get one
    double best_us = 12.0 + 6.56e-7 * n * k + 1.62e-9 * std::max(m, 128.0) * std::max(n, 128.0) * k +
                     7.8e-4 * k + 2.07e-7 * m * n;
    if (M % 8 != 0) best_us += 3.02 + 7.49e-7 * m * k;                // A's copy
    if (M % 8 != 0 || N % 8 != 0) best_us += 3.02 + 7.93e-7 * m * n;   // and C's
    for (int32_t id = 0; id < 2 * kNumQ8Kernels; ++id) {
        const Q8Kernel &e = kQ8Kernels[id / 2];
        const Q8Choice c = q8_layout(id / 2, M, K, s, cus, id % 2 != 0);
        const int64_t wgs = c.blocks * c.m_tiles * c.splits;
        const double values = static_cast<double>(wgs) * e.mt * e.cb * 256;
        double us = 3.95 + static_cast<double>(cdiv(wgs, cus) * cdiv(c.t_split / 32, e.waves)) * e.step;
        us += c.splits > 1 ? 2.55 + 2.47e-6 * values + 0.0623 * static_cast<double>(c.splits)
                           : 6.53e-7 * values;
        if (us < best_us) {
            best_us = us;
            best = c;
        }
    }
    return best;
}

static int q8_plan_choice(const Q8Choice &c, int64_t M, int64_t N, int64_t K, int32_t num_cus,
                          gemm_f16_lowbit_plan_t *plan)
{
    if (c.id < 0) return decode_plan(M, N, K, num_cus, true, plan);
    const Q8Kernel &e = kQ8Kernels[c.id];
    plan->kernel = GEMM_F16_LOWBIT_STREAM;
    plan->block_m = 16 * e.mt;
    plan->block_n = 16 * e.cb;
    plan->waves = e.waves;
    plan->splits = static_cast<int32_t>(c.splits);
    plan->grid = static_cast<int32_t>(c.blocks * c.m_tiles * c.splits);
    if (c.splits > 1)
        plan->workspace_bytes = c.blocks * c.m_tiles * c.splits * e.mt * e.cb * 1024;
    return GEMM_F16_OK;
}

static int q8_plan(int64_t M, int64_t N, int64_t K, int32_t num_cus, gemm_f16_lowbit_plan_t *plan)
{
    Q8Shape s;
    const int v = q8_shape(K, N, &s);
    if (v != GEMM_F16_OK) return v;
    if (M < 0 || num_cus <= 0) return GEMM_F16_INVALID_ARG;
    if (M > INT32_MAX) return GEMM_F16_UNSUPPORTED;
    *plan = gemm_f16_lowbit_plan_t{};
    plan->splits = 1;
    if (M == 0 || N == 0 || K == 0) return GEMM_F16_OK;
    return q8_plan_choice(q8_choose(M, N, K, s, num_cus), M, N, K, num_cus, plan);
}

static int q8_run(const Q8Choice &c, int64_t M, int64_t N, int64_t K, const Q8Shape &s,
                  const void *A, const void *codes, const void *scales, void *C, void *workspace,
                  int32_t cus, hipStream_t stream)
{
    if (c.id < 0) {
        char *ws = static_cast<char *>(workspace);
        Decode d;
        int v = decode_layout(M, N, K, cus, true, &d);
        if (v == GEMM_F16_OK)
            v = q8_launch(reinterpret_cast<const void *>(&q8_decode_kernel), K, N, s, nullptr,
                          ws + d.b, d.N, codes, scales, stream);
        if (v == GEMM_F16_OK) v = decode_gemm(d, M, N, K, true, A, C, ws, stream);
        return v;
    }
    const Q8Kernel &e = kQ8Kernels[c.id];
    Q8TnParams p;
    p.A = static_cast<const uint16_t *>(A);
    p.codes = static_cast<const uint8_t *>(codes);
    p.scales = static_cast<const uint16_t *>(scales);
    p.C = static_cast<uint16_t *>(C);
    p.partial = c.splits > 1 ? static_cast<float *>(workspace) : nullptr;
    p.stride = c.blocks * c.m_tiles * e.mt * e.cb * 256;
    p.T = static_cast<int32_t>(K);
    p.M = static_cast<int32_t>(M);
    p.N = static_cast<int32_t>(N);
    p.ng = static_cast<int32_t>(s.groups);
    p.blocks = static_cast<int32_t>(c.blocks);
    p.m_tiles = static_cast<int32_t>(c.m_tiles);
    p.t_split = static_cast<int32_t>(c.t_split);
    const int v = launch(e.fn, c.blocks * c.m_tiles * c.splits, 64 * e.waves, &p, stream);
    if (v != GEMM_F16_OK || c.splits == 1) return v;
    Q8JoinParams q;
    q.partial = p.partial;
    q.C = static_cast<uint16_t *>(C);
    q.stride = p.stride;
    q.M = p.M;
    q.N = static_cast<int32_t>(N);
    q.m_tiles = p.m_tiles;
    q.splits = static_cast<int32_t>(c.splits);
    q.mt = e.mt;
    q.cb = e.cb;
    return launch(reinterpret_cast<const void *>(&q8_join_kernel), cdiv(p.stride, 1024), 256, &q,
                  stream);
}

}  // namespace gemm_f16_lowbit

// ---------------------------------------------------------------------------
// C ABI
// ---------------------------------------------------------------------------
using namespace gemm_f16_lowbit;

extern "C" int gemm_f16_w4_sizes(int64_t N, int64_t K, int32_t group, int64_t *words_bytes,
                                 int64_t *scales_bytes)
{
    if (!words_bytes || !scales_bytes) return GEMM_F16_INVALID_ARG;
    W4Shape s;
    const int v = w4_shape(N, K, group, &s);
    if (v != GEMM_F16_OK) return v;
    *words_bytes = s.words;
    *scales_bytes = s.scales;
    return GEMM_F16_OK;
}

extern "C" int gemm_f16_w4_quantize(int64_t N, int64_t K, int32_t group, const void *W,
                                    void *words, void *scales, hipStream_t stream)
{
    return w4_encode(N, K, group, W, nullptr, nullptr, words, scales, stream);
}

extern "C" int gemm_f16_w4_pack(int64_t N, int64_t K, int32_t group, const void *codes,
                                const void *in_scales, void *words, void *scales,
                                hipStream_t stream)
{
    if (N > 0 && K > 0 && !codes) return GEMM_F16_INVALID_ARG;
    return w4_encode(N, K, group, nullptr, codes, in_scales, words, scales, stream);
}

extern "C" int gemm_f16_w4_dequantize(int64_t N, int64_t K, int32_t group, const void *words,
                                      const void *scales, void *W, hipStream_t stream)
{
    W4Shape s;
    const int v = w4_shape(N, K, group, &s);
    if (v != GEMM_F16_OK) return v;
    const Array arrays[3] = {
        {words, s.words, 16, false}, {scales, s.scales, 8, false}, {W, N * K * 2, 2, true}};
    const int a = check_arrays(arrays, 3);
    if (a != GEMM_F16_OK || s.tiles == 0) return a;
    return w4_decode(N, K, s, words, scales, W, K, stream);
}

extern "C" int gemm_f16_nt_w4_plan(int64_t M, int64_t N, int64_t K, int32_t group,
                                   int32_t num_cus, gemm_f16_lowbit_plan_t *plan)
{
    return plan ? w4_plan(M, N, K, group, num_cus, plan) : GEMM_F16_INVALID_ARG;
}

extern "C" int gemm_f16_nt_w4(int64_t M, int64_t N, int64_t K, int32_t group, const void *A,
                              const void *words, const void *scales, void *C, void *workspace,
                              int64_t workspace_bytes, hipStream_t stream)
{
    W4Shape s;
    int v = w4_shape(N, K, group, &s);
    if (v != GEMM_F16_OK) return v;
    if (M < 0 || workspace_bytes < 0) return GEMM_F16_INVALID_ARG;
    if (M > INT32_MAX) return GEMM_F16_UNSUPPORTED;
    const Array arrays[5] = {{A, M * K * 2, 2, false},
                             {words, s.words, 16, false},
                             {scales, s.scales, 8, false},
                             {C, M * N * 2, 2, true},
                             {workspace, workspace ? workspace_bytes : 0, 256, true}};
    v = check_arrays(arrays, 5);
    if (v != GEMM_F16_OK || M == 0 || N == 0) return v;
    if (K == 0) return gemm_f16_nt(M, N, 0, A, nullptr, C, stream);
    int32_t cus = 0;
    v = gemm_f16_device_cus(&cus);
    if (v != GEMM_F16_OK) return v;
    const W4Choice choice = w4_choose(M, K, s, cus);
    gemm_f16_lowbit_plan_t plan{};
    plan.splits = 1;
    v = w4_plan_choice(choice, M, N, K, s, cus, &plan);
    if (v != GEMM_F16_OK) return v;
    if (plan.workspace_bytes > (workspace ? workspace_bytes : 0)) return GEMM_F16_INVALID_ARG;
    return w4_run(choice, plan, M, N, K, s, A, words, scales, C, workspace, cus, stream);
}

extern "C" int gemm_f16_q8_quantize(int64_t R, int64_t N, const void *X, void *codes,
                                    void *scales, hipStream_t stream)
{
    Q8Shape s;
    const int v = q8_shape(R, N, &s);
    if (v != GEMM_F16_OK) return v;
    const Array arrays[3] = {
        {X, R * N * 2, 2, false}, {codes, s.codes, 16, true}, {scales, s.scales, 2, true}};
    const int a = check_arrays(arrays, 3);
    if (a != GEMM_F16_OK || s.codes == 0) return a;
    return q8_launch(reinterpret_cast<const void *>(&q8_encode_kernel), R, N, s, X, nullptr, 0, codes,
                     scales, stream);
}

extern "C" int gemm_f16_q8_dequantize(int64_t R, int64_t N, const void *codes, const void *scales,
                                      void *X, hipStream_t stream)
{
    Q8Shape s;
    const int v = q8_shape(R, N, &s);
    if (v != GEMM_F16_OK) return v;
    const Array arrays[3] = {
        {codes, s.codes, 16, false}, {scales, s.scales, 2, false}, {X, R * N * 2, 2, true}};
    const int a = check_arrays(arrays, 3);
    if (a != GEMM_F16_OK || s.codes == 0) return a;
    return q8_launch(reinterpret_cast<const void *>(&q8_decode_kernel), R, N, s, nullptr, X, N, codes,
                     scales, stream);
}

extern "C" int gemm_f16_tn_q8_plan(int64_t M, int64_t N, int64_t K, int32_t num_cus,
                                   gemm_f16_lowbit_plan_t *plan)
{
    return plan ? q8_plan(M, N, K, num_cus, plan) : GEMM_F16_INVALID_ARG;
}

extern "C" int gemm_f16_tn_q8(int64_t M, int64_t N, int64_t K, const void *A, const void *codes,
                              const void *scales, void *C, void *workspace,
                              int64_t workspace_bytes, hipStream_t stream)
{
    Q8Shape s;
    int v = q8_shape(K, N, &s);
    if (v != GEMM_F16_OK) return v;
    if (M < 0 || workspace_bytes < 0) return GEMM_F16_INVALID_ARG;
    if (M > INT32_MAX) return GEMM_F16_UNSUPPORTED;
    const Array arrays[5] = {{A, K * M * 2, 2, false},
                             {codes, s.codes, 16, false},
                             {scales, s.scales, 2, false},
                             {C, M * N * 2, 2, true},
                             {workspace, workspace ? workspace_bytes : 0, 256, true}};
    v = check_arrays(arrays, 5);
    if (v != GEMM_F16_OK || M == 0 || N == 0) return v;
    if (K == 0) return gemm_f16_tn(M, N, 0, A, nullptr, C, stream);
    int32_t cus = 0;
    v = gemm_f16_device_cus(&cus);
    if (v != GEMM_F16_OK) return v;
    const Q8Choice choice = q8_choose(M, N, K, s, cus);
    gemm_f16_lowbit_plan_t plan{};
    v = q8_plan_choice(choice, M, N, K, cus, &plan);
    if (v != GEMM_F16_OK) return v;
    if (plan.workspace_bytes > (workspace ? workspace_bytes : 0)) return GEMM_F16_INVALID_ARG;
    return q8_run(choice, M, N, K, s, A, codes, scales, C, workspace, cus, stream);
}
