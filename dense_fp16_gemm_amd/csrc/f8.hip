// Operands in 8-bit floating point with a scale for each 128 values: quantising,
// reading back, and the products, of one matrix or of many experts' (see
// gemm_f16_f8.h for the storage).

#include <hip/hip_runtime.h>

#include <algorithm>
#include <stddef.h>
#include <stdint.h>

#include "gemm_f16_f8.h"

namespace gemm_f16_f8 {

typedef _Float16 half4_t __attribute__((ext_vector_type(4)));
typedef _Float16 half8_t __attribute__((ext_vector_type(8)));
// 16 (8) bytes at any 2-byte alignment (the target's unaligned-access mode)
typedef _Float16 half8_u_t __attribute__((ext_vector_type(8), aligned(2)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef int32_t i32x4_t __attribute__((ext_vector_type(4)));
typedef int32_t i32x8_t __attribute__((ext_vector_type(8)));
typedef uint16_t u16x2_t __attribute__((ext_vector_type(2)));
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));

constexpr int GROUP = GEMM_F16_F8_GROUP;

template <class T, class S>
__device__ __forceinline__ T bits_as(S s)
{
    static_assert(sizeof(T) == sizeof(S), "same size");
    return __builtin_bit_cast(T, s);
}

// The wave's index in its workgroup, in a scalar register.
__device__ __forceinline__ int wave_index() { return __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); }

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

__device__ __forceinline__ float half_of(u32x4_t v, int i)
{
    return static_cast<float>(bits_as<_Float16>(static_cast<uint16_t>(v[i / 2] >> (16 * (i % 2)))));
}

__device__ __forceinline__ u16x2_t max2(u16x2_t a, uint32_t b)
{
    return __builtin_elementwise_max(a, bits_as<u16x2_t>(b & 0x7fff7fffu));
}

// Two halves with infinities and NaN replaced by zero.
__device__ __forceinline__ uint32_t finite2(uint32_t v)
{
    v &= 0x7fff7fffu;
    if ((v & 0xffffu) >= 0x7c00u) v &= 0xffff0000u;
    if (v >= 0x7c000000u) v &= 0xffffu;
    return v;
}

// Largest finite magnitude of eight halves, as fp16 bits (which order as
// integers; infinities and NaN come last, and are looked for only if there).
__device__ __forceinline__ uint32_t largest8(u32x4_t v)
{
    u16x2_t m = {0, 0};
#pragma unroll
    for (int i = 0; i < 4; ++i) m = max2(m, v[i]);
    if (m[0] >= 0x7c00 || m[1] >= 0x7c00) {
        m = u16x2_t{0, 0};
#pragma unroll
        for (int i = 0; i < 4; ++i) m = max2(m, finite2(v[i]));
    }
    return m[0] > m[1] ? m[0] : m[1];
}

// The scale's byte for a largest magnitude of fp16 bits `big`: with big = 1.f
// 2^e, the exponent is e - 8 where 1.f is at most 1.75 (448 = 1.75 2^8), else
// e - 7; at least -32.
__device__ __forceinline__ uint32_t scale_byte(uint32_t big)
{
    const uint32_t b =
        bits_as<uint32_t>(static_cast<float>(bits_as<_Float16>(static_cast<uint16_t>(big))));
    const uint32_t s = (b >> 23) - ((b & 0x7fffffu) > 0x600000u ? 7u : 8u);
    return big == 0 ? 95u : max(static_cast<int32_t>(s), 95);
}

// 1 / scale; byte from 95 to 135.
__device__ __forceinline__ float inverse(uint32_t byte) { return bits_as<float>((254u - byte) << 23); }

// Four codes of products that are exact (a half times a power of two), rounded
// by the conversion to nearest, ties to even.
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d)
{
    int32_t v = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
    return static_cast<uint32_t>(__builtin_amdgcn_cvt_pk_fp8_f32(c, d, v, true));
}

// ---------------------------------------------------------------------------
// Quantising rows: a scale for each 128 values of a row
// ---------------------------------------------------------------------------
// A wave takes 512 columns (eight a lane, the 16 lanes of a DPP row one group) of
// ROWS rows, so that several loads are in flight.
constexpr int ROWS = 4;

struct RowsParams {
    const uint16_t *X;
    uint8_t *codes;
    uint8_t *scales;
    int64_t rows;              // of all matrices
    int32_t R, K, kp, kq;      // rows of a matrix, columns, as stored, dwords of scales a row
};

__device__ __forceinline__ uint32_t row16_max(uint32_t v)
{
    // rotations by 8, 4, 2 and 1 of the 16 lanes
    v = max(v, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, v, 0x128, 0xf, 0xf, true)));
    v = max(v, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, v, 0x124, 0xf, 0xf, true)));
    v = max(v, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, v, 0x122, 0xf, 0xf, true)));
    return max(v, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, v, 0x121, 0xf, 0xf, true)));
}

__global__ __launch_bounds__(256) void f8_rows_kernel(RowsParams p)
{
    const int lane = threadIdx.x & 63;
    const int64_t unit = static_cast<int64_t>(xcd_unit()) * 4 + wave_index();
    const int32_t q = static_cast<int32_t>(unit % p.kq);
    const int64_t r0 = unit / p.kq * ROWS;
    const int32_t c = q * 512 + lane * 8;
    u32x4_t v[ROWS];
#pragma unroll
    for (int i = 0; i < ROWS; ++i)
        v[i] = r0 + i < p.rows ? load8(p.X + (r0 + i) * p.K, c, p.K) : u32x4_t{0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
        const int64_t r = r0 + i;
        if (r >= p.rows) break;
        const uint32_t byte = scale_byte(row16_max(largest8(v[i])));
        const float inv = inverse(byte);
        u32x2_t codes;
#pragma unroll
        for (int h = 0; h < 2; ++h)
            codes[h] = codes4(half_of(v[i], 4 * h) * inv, half_of(v[i], 4 * h + 1) * inv,
                              half_of(v[i], 4 * h + 2) * inv, half_of(v[i], 4 * h + 3) * inv);
        if (c < p.kp) *reinterpret_cast<u32x2_t *>(p.codes + r * p.kp + c) = codes;
        const int64_t matrix = r / p.R;
        const int64_t at = (matrix * p.kq + q) * p.R + (r - matrix * p.R);
        if ((lane & 15) == 0) p.scales[at * 4 + lane / 16] = static_cast<uint8_t>(byte);
    }
}

// ---------------------------------------------------------------------------
// Quantising 128 x 128 values: blocks of them, or either form of the transpose
// ---------------------------------------------------------------------------
// A workgroup takes 128 x 128 values of X, eight rows by eight columns a thread:
// thread (ty, tx) = (tid / 16, tid % 16) rows 8 ty .., columns 8 tx .. .
struct SquareParams {
    const uint16_t *X;
    uint8_t *codes;
    uint8_t *scales;
    const int32_t *rows, *offsets;   // experts: where X's rows come from
    int32_t XR, XC;                  // rows and columns of X (a matrix of it)
    int32_t kp, kq, blocks;          // as stored: columns, dwords of scales, blocks of rows
    int32_t tiles_r, tiles_c;        // of X, in 128s
    int32_t E, top;
};

// The largest finite magnitude of each of a thread's eight columns.
__device__ __forceinline__ void columns8(const u32x4_t (&v)[8], u16x2_t (&m)[4])
{
    bool odd = false;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        m[j] = u16x2_t{0, 0};
#pragma unroll
        for (int i = 0; i < 8; ++i) m[j] = max2(m[j], v[i][j]);
        odd |= m[j][0] >= 0x7c00 || m[j][1] >= 0x7c00;
    }
    if (odd) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            m[j] = u16x2_t{0, 0};
#pragma unroll
            for (int i = 0; i < 8; ++i) m[j] = max2(m[j], finite2(v[i][j]));
        }
    }
}

// Where position p's range of an experts' order lies, found by a whole wave:
// the expert with the id-th unit, units being ceil(rows / size) an expert.
// Returns the expert, or -1 and the units left over in `id`.
struct Found {
    int32_t e;        // expert, -1: past the last
    int32_t index;    // which of its units (or of those past the last)
    int32_t lo, hi;   // its positions (or those of no expert)
};

__device__ __forceinline__ int32_t inclusive_scan(int32_t v, int lane)
{
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const int32_t o = __shfl_up(v, d);
        if (lane >= d) v += o;
    }
    return v;
}

__device__ __forceinline__ Found find_unit(const int32_t *offsets, int32_t E, int32_t S, int32_t size,
                                           int32_t id, int lane)
{
    for (int32_t c = 0; c < E; c += 64) {
        int32_t lo = 0, hi = 0;
        if (c + lane < E) {
            lo = min(max(offsets[c + lane], 0), S);
            hi = max(min(max(offsets[c + lane + 1], 0), S), lo);
        }
        const int32_t units = (hi - lo + size - 1) / size;
        const int32_t upto = inclusive_scan(units, lane);
        const int32_t all = __builtin_amdgcn_readlane(upto, 63);
        if (id < all) {
            const int l = __builtin_ctzll(__ballot(upto > id));
            Found f;
            f.e = c + l;
            f.index = id - (__builtin_amdgcn_readlane(upto, l) - __builtin_amdgcn_readlane(units, l));
            f.lo = __builtin_amdgcn_readlane(lo, l);
            f.hi = __builtin_amdgcn_readlane(hi, l);
            return f;
        }
        id -= all;
    }
    return Found{-1, id, __builtin_amdgcn_readfirstlane(min(max(offsets[E], 0), S)), S};
}

// BLOCK: one scale for all values.  TRANSPOSED: stored the other way round.
// EXPERTS: X's rows are those of the experts' positions, and each expert's are
// padded to a multiple of 128.
template <bool BLOCK, bool TRANSPOSED, bool EXPERTS>
__global__ __launch_bounds__(256) void f8_square_kernel(SquareParams p)
{
    __shared__ __attribute__((aligned(16))) uint8_t smem[128 * 128];
    __shared__ __attribute__((aligned(16))) uint16_t most[4 * 128];
    const int tid = threadIdx.x, lane = tid & 63, wave = wave_index();
    const int tx = tid & 15, ty = tid >> 4;
    int64_t unit = xcd_unit();
    const int32_t tc = static_cast<int32_t>(unit % p.tiles_c);
    unit /= p.tiles_c;
    const int32_t tr = static_cast<int32_t>(unit % p.tiles_r);
    const int64_t matrix = unit / p.tiles_r;
    const uint16_t *X = p.X + matrix * p.XR * p.XC;
    const int32_t c0 = tc * 128 + tx * 8;
    u32x4_t v[8];
    if constexpr (EXPERTS) {
        const Found f = find_unit(p.offsets, p.E, p.XR, 128, tr, lane);
        if (f.e < 0) return;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int32_t pos = f.lo + f.index * 128 + ty * 8 + i;
            v[i] = u32x4_t{0, 0, 0, 0};
            if (pos < f.hi) {
                int64_t row = pos;
                if (p.top > 0) row = min(max(p.rows[pos], 0), p.XR - 1) / p.top;
                v[i] = load8(X + row * p.XC, c0, p.XC);
            }
        }
    } else {
        const int32_t r0 = tr * 128 + ty * 8;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v[i] = r0 + i < p.XR ? load8(X + static_cast<int64_t>(r0 + i) * p.XC, c0, p.XC)
                                 : u32x4_t{0, 0, 0, 0};
    }
    u16x2_t m[4];
    columns8(v, m);
    // over the four threads of a wave that share columns, then over the waves
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        m[j] = __builtin_elementwise_max(m[j], bits_as<u16x2_t>(__shfl_xor(bits_as<uint32_t>(m[j]), 16)));
        m[j] = __builtin_elementwise_max(m[j], bits_as<u16x2_t>(__shfl_xor(bits_as<uint32_t>(m[j]), 32)));
    }
    if (lane < 16) {
        u32x4_t w;
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = bits_as<uint32_t>(m[j]);
        *reinterpret_cast<u32x4_t *>(&most[wave * 128 + tx * 8]) = w;
    }
    __syncthreads();
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        const u32x4_t o = *reinterpret_cast<const u32x4_t *>(&most[w * 128 + tx * 8]);
#pragma unroll
        for (int j = 0; j < 4; ++j) m[j] = __builtin_elementwise_max(m[j], bits_as<u16x2_t>(o[j]));
    }
    uint32_t byte[8];
    float inv[8];
    if constexpr (BLOCK) {
        uint32_t big = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) big = max(big, static_cast<uint32_t>(m[j / 2][j % 2]));
        byte[0] = scale_byte(row16_max(big));
#pragma unroll
        for (int j = 0; j < 8; ++j) inv[j] = inverse(byte[0]);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            byte[j] = scale_byte(m[j / 2][j % 2]);
            inv[j] = inverse(byte[j]);
        }
    }
    // scales: bytes past the last group (of a dword's four) are written too
    const int32_t group = TRANSPOSED ? tr : tc, block0 = TRANSPOSED ? tc : tr;
    const int32_t groups = p.kp / 128;
    const int last = !EXPERTS && group == groups - 1 ? 3 : group & 3;
    uint8_t *scales = p.scales + (matrix * p.kq + group / 4) * p.blocks * 4;
    if constexpr (BLOCK) {
        if (tid == 0)
            for (int i = group & 3; i <= last; ++i)
                scales[static_cast<int64_t>(block0) * 4 + i] = static_cast<uint8_t>(byte[0]);
    } else {
        static_assert(BLOCK || TRANSPOSED, "f8_rows_kernel");
        if (ty == 0)
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (c0 + j < p.XC)
                    for (int i = group & 3; i <= last; ++i)
                        scales[static_cast<int64_t>(c0 + j) * 4 + i] = static_cast<uint8_t>(byte[j]);
    }
    if constexpr (!TRANSPOSED) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int32_t r = tr * 128 + ty * 8 + i;
            u32x2_t codes;
#pragma unroll
            for (int h = 0; h < 2; ++h)
                codes[h] = codes4(half_of(v[i], 4 * h) * inv[0], half_of(v[i], 4 * h + 1) * inv[0],
                                  half_of(v[i], 4 * h + 2) * inv[0], half_of(v[i], 4 * h + 3) * inv[0]);
            if (r < p.XR)
                *reinterpret_cast<u32x2_t *>(p.codes + (matrix * p.XR + r) * p.kp + c0) = codes;
        }
        return;
    }
    // eight codes of a column at a time to LDS, at [column][8 rows], the eight-byte
    // places of a row XORed with tx so that 16 threads write to 16 of them
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        u32x2_t codes;
#pragma unroll
        for (int h = 0; h < 2; ++h)
            codes[h] = codes4(half_of(v[4 * h], j) * inv[j], half_of(v[4 * h + 1], j) * inv[j],
                              half_of(v[4 * h + 2], j) * inv[j], half_of(v[4 * h + 3], j) * inv[j]);
        *reinterpret_cast<u32x2_t *>(&smem[(tx * 8 + j) * 128 + ((ty ^ tx) * 8)]) = codes;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int row = i * 32 + tid / 8, at = tid % 8 * 2;
        const int32_t r = tc * 128 + row;
        if (r >= p.XC) break;
        const u32x2_t lo = *reinterpret_cast<const u32x2_t *>(&smem[row * 128 + ((at ^ (row / 8)) * 8)]);
        const u32x2_t hi =
            *reinterpret_cast<const u32x2_t *>(&smem[row * 128 + (((at + 1) ^ (row / 8)) * 8)]);
        *reinterpret_cast<u32x4_t *>(p.codes + (matrix * p.XC + r) * p.kp +
                                     static_cast<int64_t>(tr) * 128 + at * 8) =
            u32x4_t{lo[0], lo[1], hi[0], hi[1]};
    }
}

// ---------------------------------------------------------------------------
// Reading back
// ---------------------------------------------------------------------------
struct DecodeParams {
    const uint8_t *codes;
    const uint8_t *scales;
    uint16_t *X;
    int64_t rows;
    int32_t R, K, kp, kq, shift, blocks;
};

__global__ __launch_bounds__(256) void f8_decode_kernel(DecodeParams p)
{
    const int lane = threadIdx.x & 63;
    const int64_t unit = static_cast<int64_t>(xcd_unit()) * 4 + wave_index();
    const int32_t q = static_cast<int32_t>(unit % p.kq);
    const int64_t r0 = unit / p.kq * ROWS;
    const int32_t c = q * 512 + lane * 8;
    if (c >= p.K) return;
    u32x2_t v[ROWS];
    int32_t e[ROWS];
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
        const int64_t r = min(r0 + i, p.rows - 1);
        const int64_t matrix = r / p.R;
        const int64_t block = (r - matrix * p.R) >> p.shift;
        v[i] = *reinterpret_cast<const u32x2_t *>(p.codes + r * p.kp + c);
        e[i] = p.scales[((matrix * p.kq + q) * p.blocks + block) * 4 + lane / 16];
    }
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
        if (r0 + i >= p.rows) break;
        half8_t h;
#pragma unroll
        for (int w = 0; w < 2; ++w) {
            const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8(v[i][w], false);
            const auto hi = __builtin_amdgcn_cvt_pk_f32_fp8(v[i][w], true);
            const float f[4] = {lo[0], lo[1], hi[0], hi[1]};
#pragma unroll
            for (int j = 0; j < 4; ++j)
                h[4 * w + j] = static_cast<_Float16>(
                    e[i] == 255 ? __builtin_nanf("") : __builtin_ldexpf(f[j], e[i] - 127));
        }
        store8(p.X + (r0 + i) * p.K, c, p.K, h);
    }
}

// ---------------------------------------------------------------------------
// Products
// ---------------------------------------------------------------------------
enum { DENSE = 0, EXPERTS = 1, GRAD = 2 };

struct Params {
    const uint8_t *a, *b;
    const uint32_t *as, *bs;    // four scales of a row (block) a dword
    uint16_t *c;
    const int32_t *rows, *offsets;
    int64_t a_ld, b_ld;         // bytes a row
    int32_t M, N;               // rows and columns of C (one matrix of it)
    int32_t kb;                 // groups of 128 columns
    int32_t a_rows;             // rows of A
    int32_t b_blocks, b_shift;  // blocks of rows of B, log2 of their size
    int32_t E, top;
    int32_t tiles_m, tiles_n;
};

// A scale of each operand for its row comes from the lane that holds the row,
// so any order of the 128 columns in the lanes' registers is right that is the
// same for both.
__device__ __forceinline__ i32x8_t load_codes(const uint8_t *row, int kq)
{
    const i32x4_t lo = *reinterpret_cast<const i32x4_t *>(row + kq * 16);
    const i32x4_t hi = *reinterpret_cast<const i32x4_t *>(row + 64 + kq * 16);
    return i32x8_t{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
}

// A workgroup's part of C and of K.
struct Unit {
    int64_t matrix;             // of B (experts' products) and of C (gradients)
    int32_t m0, m1, n0;         // rows of C, its first column
    int32_t kb0, kb1;           // groups of 128 columns
    bool none;
};

template <int MODE, int BM, int BN>
__device__ __forceinline__ Unit make_unit(const Params &p, int32_t unit, int lane)
{
    Unit u;
    u.none = false;
    u.matrix = 0;
    u.kb0 = 0;
    u.kb1 = p.kb;
    if constexpr (MODE == EXPERTS) {
        u.n0 = unit % p.tiles_n * BN;
        const Found f = find_unit(p.offsets, p.E, p.M, BM, unit / p.tiles_n, lane);
        u.m0 = f.lo + f.index * BM;
        u.m1 = min(f.hi, u.m0 + BM);
        u.none = u.m0 >= f.hi;
        if (f.e < 0) u.kb1 = 0;
        u.matrix = max(f.e, 0);
    } else {
        u.n0 = unit % p.tiles_n * BN;
        unit /= p.tiles_n;
        u.m0 = unit % p.tiles_m * BM;
        u.m1 = min(p.M, u.m0 + BM);
        if constexpr (MODE == GRAD) {
            u.matrix = unit / p.tiles_m;
            const int32_t S = p.top;   // slots
            int32_t before = 0, mine = 0;
            for (int32_t e = lane; e <= u.matrix; e += 64) {
                const int32_t lo = min(max(p.offsets[e], 0), S);
                const int32_t hi = max(min(max(p.offsets[e + 1], 0), S), lo);
                const int32_t groups = (hi - lo + 127) / 128;
                if (e < u.matrix) before += groups; else mine = groups;
            }
#pragma unroll
            for (int d = 1; d < 64; d *= 2) {
                before += __shfl_xor(before, d);
                mine += __shfl_xor(mine, d);
            }
            u.kb0 = min(__builtin_amdgcn_readfirstlane(before), p.kb);
            u.kb1 = min(u.kb0 + __builtin_amdgcn_readfirstlane(mine), p.kb);
        }
    }
    return u;
}

// 64 x 64 of C a workgroup, 16 x 64 a wave, operands straight from memory.
template <int MODE>
__global__ __launch_bounds__(256) void f8_product_kernel(Params p)
{
    const int lane = threadIdx.x & 63, wave = wave_index();
    const int r = lane & 15, kq = lane >> 4;
    const Unit u = make_unit<MODE, 64, 64>(p, xcd_unit(), lane);
    if (u.none) return;
    const int32_t m = min(u.m0 + wave * 16 + r, u.m1 - 1);
    int64_t ar = m;
    if (MODE == EXPERTS && p.top > 0)
        ar = min(max(p.rows[m], 0) / p.top, p.a_rows - 1);
    const uint8_t *a = p.a + ar * p.a_ld;
    const int64_t bm = MODE == EXPERTS ? u.matrix : 0;
    const uint32_t *bs = p.bs + bm * ((p.kb + 3) / 4) * p.b_blocks;
    f32x4_t acc[4] = {};
    for (int32_t kb = u.kb0; kb < u.kb1; ++kb) {
        const i32x8_t af = load_codes(a + static_cast<int64_t>(kb) * 128, kq);
        const int sa = p.as[static_cast<int64_t>(kb >> 2) * p.a_rows + ar] >> (8 * (kb & 3));
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int32_t n = min(u.n0 + j * 16 + r, p.N - 1);
            const i32x8_t bf =
                load_codes(p.b + (bm * p.N + n) * p.b_ld + static_cast<int64_t>(kb) * 128, kq);
            const int sb = bs[static_cast<int64_t>(kb >> 2) * p.b_blocks + (n >> p.b_shift)] >> (8 * (kb & 3));
            acc[j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(bf, af, acc[j], 0, 0, 0, sb, 0, sa);
        }
    }
    const int32_t mo = u.m0 + wave * 16 + r;
    if (mo >= u.m1) return;
    uint16_t *c = p.c + (MODE == GRAD ? u.matrix * p.M * p.N : 0) + static_cast<int64_t>(mo) * p.N;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const half4_t h = __builtin_convertvector(acc[j], half4_t);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int32_t n = u.n0 + j * 16 + kq * 4 + e;
            if (n < p.N) c[n] = bits_as<uint16_t>(_Float16(h[e]));
        }
    }
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
template <class K>
static const void *address(K *kernel) { return reinterpret_cast<const void *>(kernel); }

// Threads of a launch stay within 32 bits.
constexpr int64_t MOST_THREADS = int64_t(1) << 32;

struct Shape {
    int64_t kp, kq, blocks, codes, scales;   // columns stored, dwords of scales, blocks of rows, bytes
    int32_t shift;
};

static int shape_of(int64_t count, int64_t R, int64_t K, int32_t block, Shape *s)
{
    if (count < 0 || R < 0 || K < 0 || (block != 1 && block != 128)) return GEMM_F16_INVALID_ARG;
    constexpr int64_t most = (int64_t(1) << 31) - 128;
    if (K > (1 << 23) || R > most || count > most || (count > 0 && R > most / count))
        return GEMM_F16_UNSUPPORTED;
    s->shift = block == 128 ? 7 : 0;
    s->kp = round_up(K, GROUP);
    s->kq = cdiv(K, 4 * GROUP);
    s->blocks = cdiv(R, block);
    s->codes = count * R * s->kp;
    s->scales = count * s->kq * s->blocks * 4;
    return s->codes > (int64_t(1) << 40) ? GEMM_F16_UNSUPPORTED : GEMM_F16_OK;
}

static int quantize(int64_t count, int64_t R, int64_t K, int32_t block, bool transposed,
                    const Shape &s, const void *X, void *codes, void *scales, hipStream_t stream)
{
    if (block == 1 && !transposed) {
        RowsParams p;
        p.X = static_cast<const uint16_t *>(X);
        p.codes = static_cast<uint8_t *>(codes);
        p.scales = static_cast<uint8_t *>(scales);
        p.rows = count * R;
        p.R = static_cast<int32_t>(R);
        p.K = static_cast<int32_t>(K);
        p.kp = static_cast<int32_t>(s.kp);
        p.kq = static_cast<int32_t>(s.kq);
        // 2048 codes and more a wave, up to a row's padding to 512
        const int64_t grid = cdiv(cdiv(count * R, ROWS) * s.kq, 4);
        if (grid * 256 >= MOST_THREADS) return GEMM_F16_UNSUPPORTED;
        return launch(address(f8_rows_kernel), grid, 256, &p, stream);
    }
    SquareParams p{};
    p.X = static_cast<const uint16_t *>(X);
    p.codes = static_cast<uint8_t *>(codes);
    p.scales = static_cast<uint8_t *>(scales);
    p.XR = static_cast<int32_t>(transposed ? K : R);
    p.XC = static_cast<int32_t>(transposed ? R : K);
    p.kp = static_cast<int32_t>(s.kp);
    p.kq = static_cast<int32_t>(s.kq);
    p.blocks = static_cast<int32_t>(s.blocks);
    p.tiles_r = static_cast<int32_t>(cdiv(p.XR, 128));
    p.tiles_c = static_cast<int32_t>(cdiv(p.XC, 128));
    const int64_t grid = count * p.tiles_r * p.tiles_c;
    if (grid * 256 >= MOST_THREADS) return GEMM_F16_UNSUPPORTED;
    const void *fn = !transposed  ? address(f8_square_kernel<true, false, false>)
                     : block == 1 ? address(f8_square_kernel<false, true, false>)
                                  : address(f8_square_kernel<true, true, false>);
    return launch(fn, grid, 256, &p, stream);
}

// ---- products ---------------------------------------------------------------
struct Call {
    int mode;
    int64_t M, N, K;             // C's rows and columns (of a matrix), columns of A and B
    int64_t a_rows, matrices;    // rows of A, matrices of B (experts) or C (gradients)
    int32_t top;
    Shape a, b;
    bool a_f16;
};

constexpr int64_t MOST_EXPERTS = 1024;

static int plan_call(const Call &c, int32_t num_cus, gemm_f16_lowbit_plan_t *plan)
{
    *plan = gemm_f16_lowbit_plan_t{};
    plan->splits = 1;
    if (num_cus <= 0) return GEMM_F16_INVALID_ARG;
    if (cdiv(c.M, 16) * cdiv(c.N, 16) > INT32_MAX / (c.mode == GRAD ? c.matrices : 1))
        return GEMM_F16_UNSUPPORTED;
    if (c.M == 0 || c.N == 0) return GEMM_F16_OK;
    int64_t tiles = cdiv(c.M, 64);
    if (c.mode == EXPERTS) tiles = c.M / 64 + std::min(c.matrices, c.M) + 1;
    const int64_t grid = (c.mode == GRAD ? c.matrices : 1) * tiles * cdiv(c.N, 64);
    if (grid * 256 >= MOST_THREADS) return GEMM_F16_UNSUPPORTED;
    plan->kernel = GEMM_F16_LOWBIT_STREAM;
    plan->block_m = plan->block_n = 64;
    plan->waves = 4;
    plan->grid = static_cast<int32_t>(grid);
    if (c.a_f16) plan->workspace_bytes = round_up(c.a.codes, 256) + round_up(c.a.scales, 256);
    return GEMM_F16_OK;
}

static int run_call(const Call &c, const void *X, const void *a_codes, const void *a_scales,
                    const void *b_codes, const void *b_scales, const void *rows,
                    const void *offsets, void *C, void *workspace, int64_t workspace_bytes,
                    hipStream_t stream)
{
    int32_t cus = 0;
    int v = gemm_f16_device_cus(&cus);
    if (v != GEMM_F16_OK) return v;
    gemm_f16_lowbit_plan_t plan;
    v = plan_call(c, cus, &plan);
    if (v != GEMM_F16_OK) return v;
    if (plan.workspace_bytes > (workspace ? workspace_bytes : 0)) return GEMM_F16_INVALID_ARG;
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    if (c.a_f16 && c.a.codes > 0) {
        v = quantize(1, c.a_rows, c.K, 1, false, c.a, X, ws, ws + round_up(c.a.codes, 256), stream);
        if (v != GEMM_F16_OK) return v;
        a_codes = ws;
        a_scales = ws + round_up(c.a.codes, 256);
    }
    Params p;
    p.a = static_cast<const uint8_t *>(a_codes);
    p.b = static_cast<const uint8_t *>(b_codes);
    p.as = static_cast<const uint32_t *>(a_scales);
    p.bs = static_cast<const uint32_t *>(b_scales);
    p.c = static_cast<uint16_t *>(C);
    p.rows = static_cast<const int32_t *>(rows);
    p.offsets = static_cast<const int32_t *>(offsets);
    p.a_ld = c.a.kp;
    p.b_ld = c.b.kp;
    p.M = static_cast<int32_t>(c.M);
    p.N = static_cast<int32_t>(c.N);
    p.kb = static_cast<int32_t>(c.a.kp / GROUP);
    p.a_rows = static_cast<int32_t>(c.a_rows);
    p.b_blocks = static_cast<int32_t>(c.b.blocks);
    p.b_shift = c.b.shift;
    p.E = static_cast<int32_t>(c.matrices);
    p.top = c.top;
    p.tiles_m = static_cast<int32_t>(cdiv(c.M, 64));
    p.tiles_n = static_cast<int32_t>(cdiv(c.N, 64));
    const void *fn = c.mode == DENSE     ? address(f8_product_kernel<DENSE>)
                     : c.mode == EXPERTS ? address(f8_product_kernel<EXPERTS>)
                                         : address(f8_product_kernel<GRAD>);
    return launch(fn, plan.grid, 256, &p, stream);
}

static int dense_call(int64_t M, int64_t N, int64_t K, int32_t b_block, bool a_f16, Call *c)
{
    *c = Call{};
    c->mode = DENSE;
    c->M = M;
    c->N = N;
    c->K = K;
    c->a_rows = M;
    c->matrices = 1;
    c->a_f16 = a_f16;
    const int v = shape_of(1, M, K, 1, &c->a);
    return v != GEMM_F16_OK ? v : shape_of(1, N, K, b_block, &c->b);
}

static int nt_f8(int64_t M, int64_t N, int64_t K, const void *X, const void *a_codes,
                 const void *a_scales, int32_t b_block, const void *b_codes, const void *b_scales,
                 void *C, void *workspace, int64_t workspace_bytes, hipStream_t stream, bool a_f16)
{
    Call c;
    int v = dense_call(M, N, K, b_block, a_f16, &c);
    if (v != GEMM_F16_OK) return v;
    if (workspace_bytes < 0) return GEMM_F16_INVALID_ARG;
    const Array arrays[7] = {{X, a_f16 ? M * K * 2 : 0, 2, false},
                             {a_codes, a_f16 ? 0 : c.a.codes, 16, false},
                             {a_scales, a_f16 ? 0 : c.a.scales, 4, false},
                             {b_codes, c.b.codes, 16, false},
                             {b_scales, c.b.scales, 4, false},
                             {C, M * N * 2, 2, true},
                             {workspace, workspace ? workspace_bytes : 0, 256, true}};
    v = check_arrays(arrays, 7);
    if (v != GEMM_F16_OK || M == 0 || N == 0) return v;
    if (K == 0) return gemm_f16_nt(M, N, 0, nullptr, nullptr, C, stream);
    return run_call(c, X, a_codes, a_scales, b_codes, b_scales, nullptr, nullptr, C, workspace,
                    workspace_bytes, stream);
}

static int experts_call(int64_t S, int64_t E, int64_t N, int64_t K, int32_t top, bool a_f16, Call *c)
{
    *c = Call{};
    if (S < 0 || E < 1 || N < 0 || top < 0 || (top > 0 && S % top != 0)) return GEMM_F16_INVALID_ARG;
    if (E > MOST_EXPERTS || S > INT32_MAX - 1023) return GEMM_F16_UNSUPPORTED;
    c->mode = EXPERTS;
    c->M = S;
    c->N = N;
    c->K = K;
    c->a_rows = top > 0 ? S / top : S;
    c->matrices = E;
    c->top = top;
    c->a_f16 = a_f16;
    int v = shape_of(1, c->a_rows, K, 1, &c->a);
    if (v == GEMM_F16_OK) v = shape_of(E, N, K, 128, &c->b);
    if (v == GEMM_F16_OK && top > 0 && c->a.codes >= int64_t(1) << 32) v = GEMM_F16_UNSUPPORTED;
    return v;
}

static int nt_f8_experts(int64_t S, int64_t E, int64_t N, int64_t K, int32_t top, const void *X,
                         const void *a_codes, const void *a_scales, const void *w_codes,
                         const void *w_scales, const void *rows, const void *offsets, void *C,
                         void *workspace, int64_t workspace_bytes, hipStream_t stream, bool a_f16)
{
    Call c;
    int v = experts_call(S, E, N, K, top, a_f16, &c);
    if (v != GEMM_F16_OK) return v;
    if (workspace_bytes < 0) return GEMM_F16_INVALID_ARG;
    const Array arrays[9] = {{X, a_f16 ? c.a_rows * K * 2 : 0, 2, false},
                             {a_codes, a_f16 ? 0 : c.a.codes, 16, false},
                             {a_scales, a_f16 ? 0 : c.a.scales, 4, false},
                             {w_codes, c.b.codes, 16, false},
                             {w_scales, c.b.scales, 4, false},
                             {rows, top > 0 ? S * 4 : 0, 4, false},
                             {offsets, (E + 1) * 4, 4, false},
                             {C, S * N * 2, 2, true},
                             {workspace, workspace ? workspace_bytes : 0, 256, true}};
    v = check_arrays(arrays, 9);
    if (v != GEMM_F16_OK || S == 0 || N == 0) return v;
    if (K == 0) return gemm_f16_nt(S, N, 0, nullptr, nullptr, C, stream);
    return run_call(c, X, a_codes, a_scales, w_codes, w_scales, rows, offsets, C, workspace,
                    workspace_bytes, stream);
}

static int experts_columns(int64_t S, int64_t E, int64_t *columns)
{
    if (S < 0 || E < 1) return GEMM_F16_INVALID_ARG;
    if (E > MOST_EXPERTS || S > INT32_MAX - 1023) return GEMM_F16_UNSUPPORTED;
    *columns = 128 * (S / 128 + std::min(E, S));
    return GEMM_F16_OK;
}

}  // namespace gemm_f16_f8

using namespace gemm_f16_f8;

extern "C" int gemm_f16_f8_sizes(int64_t count, int64_t R, int64_t K, int32_t block,
                                 int64_t *codes_bytes, int64_t *scales_bytes)
{
    if (!codes_bytes || !scales_bytes) return GEMM_F16_INVALID_ARG;
    Shape s;
    const int v = shape_of(count, R, K, block, &s);
    if (v != GEMM_F16_OK) return v;
    *codes_bytes = s.codes;
    *scales_bytes = s.scales;
    return GEMM_F16_OK;
}

extern "C" int gemm_f16_f8_quantize(int64_t count, int64_t R, int64_t K, int32_t block,
                                    int32_t transposed, const void *X, void *codes, void *scales,
                                    hipStream_t stream)
{
    Shape s;
    int v = shape_of(count, R, K, block, &s);
    if (v != GEMM_F16_OK) return v;
    if (transposed != 0 && transposed != 1) return GEMM_F16_INVALID_ARG;
    const Array arrays[3] = {{X, count * R * K * 2, 2, false},
                             {codes, s.codes, 16, true},
                             {scales, s.scales, 4, true}};
    v = check_arrays(arrays, 3);
    if (v != GEMM_F16_OK || s.codes == 0) return v;
    return quantize(count, R, K, block, transposed != 0, s, X, codes, scales, stream);
}

extern "C" int gemm_f16_f8_dequantize(int64_t count, int64_t R, int64_t K, int32_t block,
                                      const void *codes, const void *scales, void *X,
                                      hipStream_t stream)
{
    Shape s;
    int v = shape_of(count, R, K, block, &s);
    if (v != GEMM_F16_OK) return v;
    const Array arrays[3] = {{codes, s.codes, 16, false},
                             {scales, s.scales, 4, false},
                             {X, count * R * K * 2, 2, true}};
    v = check_arrays(arrays, 3);
    if (v != GEMM_F16_OK || s.codes == 0) return v;
    DecodeParams p;
    p.codes = static_cast<const uint8_t *>(codes);
    p.scales = static_cast<const uint8_t *>(scales);
    p.X = static_cast<uint16_t *>(X);
    p.rows = count * R;
    p.R = static_cast<int32_t>(R);
    p.K = static_cast<int32_t>(K);
    p.kp = static_cast<int32_t>(s.kp);
    p.kq = static_cast<int32_t>(s.kq);
    p.shift = s.shift;
    p.blocks = static_cast<int32_t>(s.blocks);
    const int64_t grid = cdiv(cdiv(count * R, ROWS) * s.kq, 4);
    if (grid * 256 >= MOST_THREADS) return GEMM_F16_UNSUPPORTED;
    return launch(address(f8_decode_kernel), grid, 256, &p, stream);
}

extern "C" int gemm_f16_nt_f8_plan(int64_t M, int64_t N, int64_t K, int32_t b_block, int32_t a_f16,
                                   int32_t num_cus, gemm_f16_lowbit_plan_t *plan)
{
    if (!plan) return GEMM_F16_INVALID_ARG;
    Call c;
    const int v = dense_call(M, N, K, b_block, a_f16 != 0, &c);
    return v != GEMM_F16_OK ? v : plan_call(c, num_cus, plan);
}

extern "C" int gemm_f16_nt_f8(int64_t M, int64_t N, int64_t K, const void *a_codes,
                              const void *a_scales, int32_t b_block, const void *b_codes,
                              const void *b_scales, void *C, void *workspace,
                              int64_t workspace_bytes, hipStream_t stream)
{
    return nt_f8(M, N, K, nullptr, a_codes, a_scales, b_block, b_codes, b_scales, C, workspace,
                 workspace_bytes, stream, false);
}

extern "C" int gemm_f16_nt_f8_x(int64_t M, int64_t N, int64_t K, const void *X, int32_t b_block,
                                const void *b_codes, const void *b_scales, void *C,
                                void *workspace, int64_t workspace_bytes, hipStream_t stream)
{
    return nt_f8(M, N, K, X, nullptr, nullptr, b_block, b_codes, b_scales, C, workspace,
                 workspace_bytes, stream, true);
}

extern "C" int gemm_f16_nt_f8_experts_plan(int64_t S, int64_t E, int64_t N, int64_t K, int32_t top,
                                           int32_t a_f16, int32_t num_cus,
                                           gemm_f16_lowbit_plan_t *plan)
{
    if (!plan) return GEMM_F16_INVALID_ARG;
    Call c;
    const int v = experts_call(S, E, N, K, top, a_f16 != 0, &c);
    return v != GEMM_F16_OK ? v : plan_call(c, num_cus, plan);
}

extern "C" int gemm_f16_nt_f8_experts(int64_t S, int64_t E, int64_t N, int64_t K, int32_t top,
                                      const void *a_codes, const void *a_scales,
                                      const void *w_codes, const void *w_scales, const void *rows,
                                      const void *offsets, void *C, void *workspace,
                                      int64_t workspace_bytes, hipStream_t stream)
{
    return nt_f8_experts(S, E, N, K, top, nullptr, a_codes, a_scales, w_codes, w_scales, rows,
                         offsets, C, workspace, workspace_bytes, stream, false);
}

extern "C" int gemm_f16_nt_f8_experts_x(int64_t S, int64_t E, int64_t N, int64_t K, int32_t top,
                                        const void *X, const void *w_codes, const void *w_scales,
                                        const void *rows, const void *offsets, void *C,
                                        void *workspace, int64_t workspace_bytes,
                                        hipStream_t stream)
{
    return nt_f8_experts(S, E, N, K, top, X, nullptr, nullptr, w_codes, w_scales, rows, offsets, C,
                         workspace, workspace_bytes, stream, true);
}

extern "C" int gemm_f16_f8_experts_columns(int64_t S, int64_t E, int64_t *columns)
{
    return columns ? experts_columns(S, E, columns) : GEMM_F16_INVALID_ARG;
}

extern "C" int gemm_f16_f8_quantize_experts(int64_t S, int64_t E, int64_t R, int32_t top,
                                            const void *X, const void *rows, const void *offsets,
                                            void *codes, void *scales, hipStream_t stream)
{
    int64_t columns = 0;
    int v = experts_columns(S, E, &columns);
    if (v != GEMM_F16_OK) return v;
    if (R < 0 || top < 0 || (top > 0 && S % top != 0)) return GEMM_F16_INVALID_ARG;
    Shape s;
    v = shape_of(1, R, columns, 1, &s);
    if (v != GEMM_F16_OK) return v;
    const int64_t x_rows = top > 0 ? S / top : S;
    const Array arrays[5] = {{X, x_rows * R * 2, 2, false},
                             {rows, top > 0 ? S * 4 : 0, 4, false},
                             {offsets, (E + 1) * 4, 4, false},
                             {codes, s.codes, 16, true},
                             {scales, s.scales, 4, true}};
    v = check_arrays(arrays, 5);
    if (v != GEMM_F16_OK || s.codes == 0) return v;
    SquareParams p{};
    p.X = static_cast<const uint16_t *>(X);
    p.codes = static_cast<uint8_t *>(codes);
    p.scales = static_cast<uint8_t *>(scales);
    p.rows = static_cast<const int32_t *>(rows);
    p.offsets = static_cast<const int32_t *>(offsets);
    p.XR = static_cast<int32_t>(S);
    p.XC = static_cast<int32_t>(R);
    p.kp = static_cast<int32_t>(s.kp);
    p.kq = static_cast<int32_t>(s.kq);
    p.blocks = static_cast<int32_t>(s.blocks);
    p.tiles_r = static_cast<int32_t>(columns / 128);
    p.tiles_c = static_cast<int32_t>(cdiv(R, 128));
    p.E = static_cast<int32_t>(E);
    p.top = top;
    const int64_t grid = int64_t(p.tiles_r) * p.tiles_c;
    if (grid * 256 >= MOST_THREADS) return GEMM_F16_UNSUPPORTED;
    return launch(address(f8_square_kernel<false, true, true>), grid, 256, &p, stream);
}

extern "C" int gemm_f16_nt_f8_experts_grad(int64_t S, int64_t E, int64_t M, int64_t N,
                                           const void *a_codes, const void *a_scales,
                                           const void *b_codes, const void *b_scales,
                                           const void *offsets, void *C, hipStream_t stream)
{
    int64_t columns = 0;
    int v = experts_columns(S, E, &columns);
    if (v != GEMM_F16_OK) return v;
    Call c{};
    c.mode = GRAD;
    c.M = M;
    c.N = N;
    c.K = columns;
    c.a_rows = M;
    c.matrices = E;
    c.top = static_cast<int32_t>(S);
    v = shape_of(1, M, columns, 1, &c.a);
    if (v == GEMM_F16_OK) v = shape_of(1, N, columns, 1, &c.b);
    if (v != GEMM_F16_OK) return v;
    if (cdiv(M, 16) * cdiv(N, 16) > INT32_MAX / E) return GEMM_F16_UNSUPPORTED;
    const Array arrays[6] = {{a_codes, c.a.codes, 16, false}, {a_scales, c.a.scales, 4, false},
                             {b_codes, c.b.codes, 16, false}, {b_scales, c.b.scales, 4, false},
                             {offsets, (E + 1) * 4, 4, false}, {C, E * M * N * 2, 2, true}};
    v = check_arrays(arrays, 6);
    if (v != GEMM_F16_OK || M == 0 || N == 0) return v;
    if (S == 0) return gemm_f16_nt(E * M, N, 0, nullptr, nullptr, C, stream);
    return run_call(c, nullptr, a_codes, a_scales, b_codes, b_scales, nullptr, offsets, C, nullptr,
                    0, stream);
}
