// Operands in 8-bit floating point with a scale for each 128 values: quantising,
// reading back, and the products, of one matrix or of many experts' (see
// gemm_f16_f8.h for the storage).

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <type_traits>
#include <stddef.h>
#include <stdint.h>

#include "gemm_f16_f8.h"

namespace gemm_f16_f8 {

typedef _Float16 half2_t __attribute__((ext_vector_type(2)));
typedef _Float16 half4_t __attribute__((ext_vector_type(4)));
typedef _Float16 half8_t __attribute__((ext_vector_type(8)));
// 16 (8) bytes at any 2-byte alignment (the target's unaligned-access mode)
typedef _Float16 half8_u_t __attribute__((ext_vector_type(8), aligned(2)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef int32_t i32x4_t __attribute__((ext_vector_type(4)));
typedef int32_t i32x8_t __attribute__((ext_vector_type(8)));
typedef int16_t i16x2_t __attribute__((ext_vector_type(2)));
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
__device__ __forceinline__ int32_t xcd_unit(int32_t id, int32_t count)
{
    const int32_t q = count >> 3, rem = count & 7, x = id & 7;
    return x * q + (x < rem ? x : rem) + (id >> 3);
}
__device__ __forceinline__ int32_t xcd_unit() { return xcd_unit(blockIdx.x, gridDim.x); }

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

// Four codes of two pairs of halves over the scale of `byte` (95 to 135): quotients by
// a power of two are exact, and the conversion rounds them to nearest, ties to
// even.  (Through fp32 and a product a value takes 3.5 instructions instead of one
// half.)
__device__ __forceinline__ uint32_t codes4(uint32_t a, uint32_t b, uint32_t byte)
{
    const float s = bits_as<float>(byte << 23);
    i16x2_t w = {0, 0};
    w = __builtin_amdgcn_cvt_scalef32_pk_fp8_f16(w, bits_as<half2_t>(a), s, false);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp8_f16(w, bits_as<half2_t>(b), s, true);
    return bits_as<uint32_t>(w);
}

__device__ __forceinline__ u32x2_t codes8(u32x4_t v, uint32_t byte)
{
    return u32x2_t{codes4(v[0], v[1], byte), codes4(v[2], v[3], byte)};
}

// Between a wave's LDS writes and its other lanes' reads of them: see that the
// compiler keeps their order (a wave's LDS operations are done in order).
__device__ __forceinline__ void wave_lds_fence()
{
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront", "local");
    __builtin_amdgcn_wave_barrier();
}

// ---------------------------------------------------------------------------
// Quantising rows: a scale for each 128 values of a row
// ---------------------------------------------------------------------------
// A wave takes 512 columns (eight a lane, the 16 lanes of a DPP row one group) of
// ROWS rows, so that several loads are in flight.  Bound by HBM: 4096 x 8192 in 21 us,
// 4.8 TB/s.
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
        if (c < p.kp) *reinterpret_cast<u32x2_t *>(p.codes + r * p.kp + c) = codes8(v[i], byte);
        const int64_t matrix = r / p.R;
        const int64_t at = (matrix * p.kq + q) * p.R + (r - matrix * p.R);
        if ((lane & 15) == 0) p.scales[at * 4 + lane / 16] = static_cast<uint8_t>(byte);
    }
}

// ---------------------------------------------------------------------------
// Quantising 128 x 128 values: blocks of them, or either form of the transpose
// ---------------------------------------------------------------------------
// A workgroup takes 128 x 128 values of X, eight rows by eight columns a thread:
// thread (ty, tx) = (tid / 16, tid % 16) rows 8 ty .., columns 8 tx .. .  The transpose
// goes through LDS as codes, so that both sides move 128 bytes and more at once: 4999
// x 8192 in 24 us, 5 TB/s.  By expert, where each workgroup first finds its rows,
// 16396 x 1408 in 16 us and x 2048, gathered from 4099 rows, in 20.5: their way through
// memory three times in a row.
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

// What an expert has of some units of work: ceil(rows / size) times `per`.
struct Found {
    int32_t e;        // expert, -1: past the last
    int32_t index;    // which of its units (or of those past the last)
    int32_t lo, hi;   // its positions (or those of no expert)
};

// Sums of units stop here: only offsets that overlap reach it, and what is computed
// of those does not matter, but stays inside the arrays.
constexpr int32_t MOST_UNITS = 1 << 29;

__device__ __forceinline__ int32_t add_units(int32_t a, int32_t b) { return min(a + b, MOST_UNITS); }

__device__ __forceinline__ int32_t inclusive_scan(int32_t v, int lane)
{
    v = min(v, MOST_UNITS);
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const int32_t o = __shfl_up(v, d);
        if (lane >= d) v = add_units(v, o);
    }
    return v;
}

// The positions of expert e, held to 0 .. S whatever `offsets` says.
__device__ __forceinline__ void positions(const int32_t *offsets, int32_t E, int32_t S, int32_t e,
                                          int32_t &lo, int32_t &hi)
{
    lo = hi = 0;
    if (e < E) {
        lo = min(max(offsets[e], 0), S);
        hi = max(min(max(offsets[e + 1], 0), S), lo);
    }
}

// The expert that unit `id` of all experts' belongs to, found by a whole wave, 64
// experts at a time.  PER_XCD: `id` counts workgroups, and each XCD (workgroups
// mod 8) takes a contiguous range of the units that there are, the rows of no
// expert (ceil(rows / size) times per, too) last.
template <bool PER_XCD>
__device__ __forceinline__ Found find_unit(const int32_t *offsets, int32_t E, int32_t S, int32_t size,
                                           int32_t per, int32_t id, int lane)
{
    int32_t lo, hi;
    positions(offsets, E, S, lane, lo, hi);
    int32_t units = (hi - lo + size - 1) / size * per;
    int32_t upto = inclusive_scan(units, lane);
    const int32_t end = __builtin_amdgcn_readfirstlane(min(max(offsets[E], 0), S));
    if constexpr (PER_XCD) {
        int32_t total = __builtin_amdgcn_readlane(upto, 63) + (S - end + size - 1) / size * per;
        for (int32_t c = 64; c < E; c += 64) {
            int32_t l, h;
            positions(offsets, E, S, c + lane, l, h);
            total = add_units(total, __builtin_amdgcn_readlane(inclusive_scan((h - l + size - 1) / size * per, lane), 63));
        }
        const int32_t x = id & 7, i = id >> 3, q = total >> 3, rem = total & 7;
        if (i >= q + (x < rem ? 1 : 0)) return Found{-1, 0, S, S};
        id = x * q + min(x, rem) + i;
    }
    for (int32_t c = 0;;) {
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
        c += 64;
        if (c >= E) break;
        positions(offsets, E, S, c + lane, lo, hi);
        units = (hi - lo + size - 1) / size * per;
        upto = inclusive_scan(units, lane);
    }
    return Found{-1, id, end, S};
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
    // an XCD's workgroups go along what is stored together; where it is transposed and
    // its rows gathered several times, a slab of 128 columns then stays in the L2 (the
    // other way 25, 17.4 and 23 us at the sizes above)
    const int32_t inner = TRANSPOSED ? p.tiles_r : p.tiles_c, outer = TRANSPOSED ? p.tiles_c : p.tiles_r;
    const int32_t near = static_cast<int32_t>(unit % inner);
    unit /= inner;
    const int32_t far = static_cast<int32_t>(unit % outer);
    const int64_t matrix = unit / outer;
    const int32_t tc = TRANSPOSED ? far : near, tr = TRANSPOSED ? near : far;
    const uint16_t *X = p.X + matrix * p.XR * p.XC;
    const int32_t c0 = tc * 128 + tx * 8;
    u32x4_t v[8];
    if constexpr (EXPERTS) {
        const Found f = find_unit<false>(p.offsets, p.E, p.XR, 128, 1, tr, lane);
        if (f.e < 0) return;
        const int32_t pos = f.lo + f.index * 128 + ty * 8;
        int32_t row[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            row[i] = min(pos + i, f.hi - 1);
            if (p.top > 0) row[i] = min(max(p.rows[row[i]], 0), p.XR - 1) / p.top;
        }
        // rows past the expert's last are read as that one, then dropped
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            v[i] = load8(X + static_cast<int64_t>(row[i]) * p.XC, c0, p.XC);
            if (pos + i >= f.hi) v[i] = u32x4_t{0, 0, 0, 0};
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
    if constexpr (BLOCK) {
        uint32_t big = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) big = max(big, static_cast<uint32_t>(m[j / 2][j % 2]));
        byte[0] = scale_byte(row16_max(big));
#pragma unroll
        for (int j = 1; j < 8; ++j) byte[j] = byte[0];
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) byte[j] = scale_byte(m[j / 2][j % 2]);
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
            if (r < p.XR)
                *reinterpret_cast<u32x2_t *>(p.codes + (matrix * p.XR + r) * p.kp + c0) = codes8(v[i], byte[0]);
        }
        return;
    }
    // eight codes of a column at a time to LDS, at [column][8 rows], the eight-byte
    // places of a row XORed with tx so that 16 threads write to 16 of them
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        u32x4_t w;   // column j's halves of two rows a dword
#pragma unroll
        for (int i = 0; i < 4; ++i)
            w[i] = __builtin_amdgcn_perm(v[2 * i + 1][j / 2], v[2 * i][j / 2], j % 2 ? 0x07060302u : 0x05040100u);
        *reinterpret_cast<u32x2_t *>(&smem[(tx * 8 + j) * 128 + ((ty ^ tx) * 8)]) = codes8(w, byte[j]);
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

// Sums are fp32, but for what the matrix units drop of each eight neighbouring
// products: all below 2^-13 of the largest one's leading bit (4.5e-5 of the result for
// activations with a few large channels; gemm_f16_f8.h).  Their instructions for 8 bits
// know no other way; products in fp16 would keep those bits at half the rate.

// A scale of each operand for its row comes from the lane that holds the row, so
// any order of a group's columns in the lanes' registers is right that is the
// same for both operands.
struct Params {
    const uint8_t *a, *b;
    const uint16_t *x;          // A in fp16, quantised by the kernel
    const uint32_t *as, *bs;    // four scales of a row (block) a dword
    uint16_t *c;
    const int32_t *rows, *offsets;
    int64_t a_ld, b_ld;         // bytes a row
    int32_t M, N, K;            // rows and columns of C (one matrix of it), columns of A
    int32_t kb;                 // groups of 128 columns
    int32_t a_rows;             // rows of A
    int32_t b_blocks, b_shift;  // blocks of rows of B, log2 of their size
    int32_t E, top;
    int32_t tiles_m, tiles_n;
    int32_t units;              // at most, where a workgroup takes more than one
    int32_t splits, kb_split;   // ranges of K (dense), groups of each
    float *partial;             // their sums
};

// Four neighbouring columns of a row of C.
__device__ __forceinline__ void store4(uint16_t *row, int32_t n, int32_t N, f32x4_t v)
{
    const half4_t h = __builtin_convertvector(v, half4_t);
    if (n + 4 <= N) {
        __builtin_memcpy(row + n, &h, 8);   // any 2-byte alignment
        return;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e)
        if (n + e < N) row[n + e] = bits_as<uint16_t>(_Float16(h[e]));
}

// A workgroup's part of C and of K.
struct Unit {
    int64_t matrix;             // of B (experts' products) and of C (gradients)
    int32_t m0, m1, n0;         // rows of C, its first column
    int32_t kb0, kb1;           // groups of 128 columns
    int32_t split, tile;        // which range of K, which tile of C
    bool none;
};

// Tile `tile` of tiles_m x tiles_n: neighbours (which share an XCD's L2) are tiles
// of a few rows of tiles at a time, one column after the other.
constexpr int32_t RASTER = 8;

__device__ __forceinline__ void find_tile(int32_t tile, int32_t tiles_m, int32_t tiles_n, int32_t &tm, int32_t &tn)
{
    if (tiles_m == 1) {
        tm = 0;
        tn = tile;
        return;
    }
    const int32_t group = tile / (RASTER * tiles_n), first = group * RASTER;
    const int32_t height = min(RASTER, tiles_m - first), rest = tile - group * RASTER * tiles_n;
    tm = first + rest % height;
    tn = rest / height;
}

// Rows lo .. hi - 1 of expert e (-1: of none), `index` of their tiles.
template <int BM, int BN>
__device__ __forceinline__ Unit expert_unit(const Params &p, const Found &f)
{
    Unit u{};
    const int32_t tiles = max((f.hi - f.lo + BM - 1) / BM, 1);
    const int32_t tm = f.index % tiles, tn = f.index / tiles;
    u.m0 = f.lo + tm * BM;
    u.m1 = min(f.hi, u.m0 + BM);
    u.n0 = tn * BN;
    u.none = f.lo >= f.hi;
    u.kb1 = f.e < 0 ? 0 : p.kb;
    u.matrix = max(f.e, 0);
    return u;
}

// Unit `id` of `count` of a product of two matrices, K in p.splits ranges, or of the
// gradients (whose range of K is not found here).
template <int MODE, int BM, int BN>
__device__ __forceinline__ Unit matrix_unit(const Params &p, int32_t id, int32_t count)
{
    Unit u{};
    int32_t unit = 0, tm, tn;
    u.kb1 = p.kb;
    if constexpr (MODE == GRAD) {
        // Each XCD (workgroups mod 8) takes a share of every expert's tiles, since some
        // have many more rows than others: of the e-th expert the share x + e mod 8,
        // which makes eight experts' shares even.
        const int32_t tiles = p.tiles_m * p.tiles_n, q = tiles >> 3, rem = tiles & 7;
        const int32_t x = id & 7, i = id >> 3, eight = i / tiles;
        int32_t at = i - eight * tiles, e = 0, share = x;
        for (; e < 7; ++e, share = (share + 1) & 7) {
            const int32_t mine = q + (share < rem ? 1 : 0);
            if (at < mine) break;
            at -= mine;
        }
        u.matrix = eight * 8 + e;
        u.none = u.matrix >= p.E;
        unit = share * q + min(share, rem) + at;
    } else {
        unit = xcd_unit(id, count);
    }
    if (MODE == DENSE && p.splits > 1) {
        u.split = unit % p.splits;
        unit /= p.splits;
        u.kb0 = u.split * p.kb_split;
        u.kb1 = min(u.kb0 + p.kb_split, p.kb);
    }
    find_tile(unit, p.tiles_m, p.tiles_n, tm, tn);
    u.m0 = tm * BM;
    u.m1 = min(p.M, u.m0 + BM);
    u.n0 = tn * BN;
    u.tile = unit;
    return u;
}

// A workgroup's only unit.
template <int MODE, int BM, int BN>
__device__ __forceinline__ Unit make_unit(const Params &p, int lane)
{
    if constexpr (MODE == EXPERTS)
        return expert_unit<BM, BN>(p, find_unit<true>(p.offsets, p.E, p.M, BM, p.tiles_n, blockIdx.x, lane));
    Unit u = matrix_unit<MODE, BM, BN>(p, blockIdx.x, gridDim.x);
    if (MODE == GRAD && !u.none) {
        int32_t before = 0, mine = 0;
        for (int32_t e = lane; e <= u.matrix; e += 64) {
            int32_t lo, hi;
            positions(p.offsets, p.E, p.top, e, lo, hi);   // top: slots
            const int32_t groups = (hi - lo + 127) / 128;
            if (e < u.matrix) before = add_units(before, groups); else mine = groups;
        }
#pragma unroll
        for (int d = 1; d < 64; d *= 2) {
            before = add_units(before, __shfl_xor(before, d));
            mine += __shfl_xor(mine, d);
        }
        u.kb0 = min(__builtin_amdgcn_readfirstlane(before), p.kb);
        u.kb1 = min(u.kb0 + __builtin_amdgcn_readfirstlane(mine), p.kb);
    }
    return u;
}

// Up to and with each expert, its units of ceil(rows / size) times `per`, in LDS, for
// workgroups that take one unit after the other.
struct Experts {
    int32_t upto[1024], sums[16];

    // By all W waves of the workgroup, a barrier at the end.
    template <int W>
    __device__ __forceinline__ void fill(const int32_t *offsets, int32_t E, int32_t S, int32_t size, int32_t per)
    {
        const int tid = threadIdx.x, lane = tid & 63, wave = wave_index();
        int32_t before = 0;
        for (int32_t e0 = 0; e0 < E; e0 += 64 * W) {
            int32_t l, h;
            positions(offsets, E, S, e0 + tid, l, h);
            int32_t up = inclusive_scan((h - l + size - 1) / size * per, lane);
            if (lane == 63) sums[wave] = up;
            __syncthreads();
            int32_t all = before;
            for (int w = 0; w < W; ++w) {
                if (w == wave) up = add_units(up, all);
                all = add_units(all, sums[w]);
            }
            before = all;
            if (e0 + tid < E) upto[e0 + tid] = up;
            __syncthreads();
        }
    }

    // As find_unit<true>.
    __device__ __forceinline__ Found find(const int32_t *offsets, int32_t E, int32_t S, int32_t size, int32_t per,
                                          int32_t id, int lane) const
    {
        const int32_t last = min(max(offsets[E], 0), S);
        const int32_t all = __builtin_amdgcn_readfirstlane(upto[E - 1]);
        const int32_t total = all + (S - last + size - 1) / size * per;
        const int32_t x = id & 7, i = id >> 3, q = total >> 3, rem = total & 7;
        if (i >= q + (x < rem ? 1 : 0)) return Found{-1, 0, S, S};
        id = x * q + min(x, rem) + i;
        if (id >= all) return Found{-1, id - all, last, S};
        int32_t e = 0;
        for (;; e += 64) {
            const uint64_t over = __ballot(upto[min(e + lane, E - 1)] > id);
            if (over) {
                e += __builtin_ctzll(over);
                break;
            }
        }
        Found f;
        f.e = e;
        f.index = id - (e > 0 ? __builtin_amdgcn_readfirstlane(upto[e - 1]) : 0);
        positions(offsets, E, S, e, f.lo, f.hi);
        return f;
    }
};

__device__ __forceinline__ i32x8_t whole(const i32x4_t (&v)[2])
{
    return i32x8_t{v[0][0], v[0][1], v[0][2], v[0][3], v[1][0], v[1][1], v[1][2], v[1][3]};
}

// ---- codes straight from memory ---------------------------------------------------
// The largest of eight neighbouring lanes' values.
__device__ __forceinline__ uint32_t eight_max(uint32_t v)
{
    v = max(v, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, v, 0xb1, 0xf, 0xf, true)));   // lane ^ 1
    v = max(v, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, v, 0x4e, 0xf, 0xf, true)));   // lane ^ 2
    return max(v, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, v, 0x141, 0xf, 0xf, true)));   // 7 - lane
}

// A few rows of halves against 16 rows of B a workgroup, straight from memory.  The
// workgroup quantises A's rows to LDS itself, which costs less than a launch for
// it (a few microseconds) while they are short; its W waves then take every W-th Q
// groups of 128 columns each and add up at the end.  B is read once, by 16 bytes a
// lane in the order in which the MFMA takes it, so it goes through no LDS.  Bound by
// HBM, behind 3 us of launch and of quantising: 1 x 4096 x 14336 13 to 14 us (59 MB),
// 5 x 7001 x 4160 11 to 13.
template <int MODE, int W, int Q>
__global__ __launch_bounds__(64 * W) void f8_stream_kernel(Params p)
{
    static_assert(W * Q % 4 == 0, "a wave's groups all start at the same byte of a dword of scales");
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    const int lane = threadIdx.x & 63, wave = wave_index();
    const int r = lane & 15, kq = lane >> 4;
    const Unit u = make_unit<MODE, 16, 16>(p, lane);
    if (u.none) return;
    const int rows = u.m1 - u.m0;
    const int64_t bm = MODE == EXPERTS ? u.matrix : 0;
    const int32_t bn = min(u.n0 + r, p.N - 1);
    const uint8_t *b = p.b + (bm * p.N + bn) * p.b_ld + kq * 16;
    const uint32_t *bs = p.bs + bm * ((p.kb + 3) / 4) * p.b_blocks + (bn >> p.b_shift);
    const int32_t kb = MODE == EXPERTS ? u.kb1 : p.kb;   // none for rows of no expert
    i32x4_t bv[2][Q][2];
    uint32_t sb[2];
    // Groups Q i .. + Q - 1 for i = wave, wave + W, ..., in two buffers: one's loads
    // fly while the other's are multiplied.  Past the end the last group is loaded
    // again, so that the waits on one buffer leave the other's in flight.
    auto load = [&](int buf, int32_t i) {
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            const i32x4_t *at = reinterpret_cast<const i32x4_t *>(b + static_cast<int64_t>(min(i * Q + q, kb - 1)) * 128);
            bv[buf][q][0] = __builtin_nontemporal_load(at);
            bv[buf][q][1] = __builtin_nontemporal_load(at + 4);
        }
        sb[buf] = bs[static_cast<int64_t>(min(i * Q, kb - 1) >> 2) * p.b_blocks];
    };
    const int32_t steps = (kb + Q - 1) / Q;
    const int32_t count = steps > wave ? (steps - wave + W - 1) / W : 0;
    auto at = [&](int32_t i) { return wave + min(i, count - 1) * W; };
    // A's codes and, after them, scales in LDS: rows apart by 16 bytes in the banks
    const int pitch = kb * 128 + 16;
    uint8_t *const lds_s = lds + rows * pitch;
    {
        // each thread 16 values of a row, eight threads a group; the codes' own loads
        // go out before the last of them is waited for
        const int per = kb * 8, all = rows * per;
        int o = threadIdx.x;
        u32x4_t lo, hi;
        auto fetch = [&](int o) {
            const int row = o / per, c = (o - row * per) * 16;
            int64_t m = u.m0 + row;
            if (MODE == EXPERTS && p.top > 0) m = min(max(p.rows[m], 0) / p.top, p.a_rows - 1);
            const uint16_t *x = p.x + m * p.K;
            lo = load8(x, c, p.K);
            hi = load8(x, c + 8, p.K);
        };
        auto put = [&](int o) {
            const int row = o / per, c = o - row * per;
            const uint32_t byte = scale_byte(eight_max(max(largest8(lo), largest8(hi))));
            const u32x2_t first = codes8(lo, byte), second = codes8(hi, byte);
            *reinterpret_cast<u32x4_t *>(lds + row * pitch + c * 16) = u32x4_t{first[0], first[1], second[0], second[1]};
            if (c % 8 == 0) lds_s[row * kb + c / 8] = static_cast<uint8_t>(byte);
        };
        for (; o + 64 * W < all; o += 64 * W) {
            fetch(o);
            put(o);
        }
        if (o < all) fetch(o);
        if (count > 0) load(0, at(0));
        if (o < all) put(o);
        __syncthreads();
    }
    // rows past the last are that row: not stored
    const int ar = min(r, rows - 1);
    const uint8_t *const la = lds + ar * pitch + kq * 16;
    const uint8_t *const ls = lds_s + ar * kb;
    const int first = wave * Q & 3;   // the byte of a step's first group
    f32x4_t acc = {};
    auto mma = [&](int buf, int32_t i) {
        const int32_t g0 = (wave + i * W) * Q;
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            if (g0 + q >= kb) break;
            const i32x4_t x[2] = {*reinterpret_cast<const i32x4_t *>(la + (g0 + q) * 128),
                                  *reinterpret_cast<const i32x4_t *>(la + (g0 + q) * 128 + 64)};
            acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(whole(bv[buf][q]), whole(x), acc, 0, 0, 0,
                                                                   sb[buf] >> (8 * (first + q)), 0, ls[g0 + q]);
        }
    };
    if (count > 0) {
        int32_t i = 0;
        for (; i + 2 <= count; i += 2) {
            load(1, at(i + 1));
            __builtin_amdgcn_sched_barrier(0);
            mma(0, i);
            __builtin_amdgcn_sched_barrier(0);
            load(0, at(i + 2));
            __builtin_amdgcn_sched_barrier(0);
            mma(1, i + 1);
            __builtin_amdgcn_sched_barrier(0);
        }
        if (i < count) mma(0, i);
    }
    // the waves' sums: lane l holds columns 4 (l / 16) .. + 3, row l % 16
    __syncthreads();
    f32x4_t *const red = reinterpret_cast<f32x4_t *>(lds);
    red[wave * 64 + lane] = acc;
    __syncthreads();
    if (wave > 0) return;
    f32x4_t v = red[lane];
#pragma unroll
    for (int w = 1; w < W; ++w) v += red[w * 64 + lane];
    const int32_t m = u.m0 + r;
    if (m < u.m1) store4(p.c + static_cast<int64_t>(m) * p.N, u.n0 + kq * 4, p.N, v);
}

// ---- tiles through LDS --------------------------------------------------------
typedef float f32x16_t __attribute__((ext_vector_type(16)));

// The lane, for a part of a loop over units: what is made of it there is not kept in
// registers over the rest of the loop, which has none to spare.
__device__ __forceinline__ int anew(int lane)
{
    asm volatile("" : "+v"(lane));
    return lane;
}

// Buffer resource for raw byte addressing from `base` on, 2^32 - 1 bytes: what
// is loaded lies inside the arrays by its rows and columns, which are held to
// those that exist.
__device__ __forceinline__ i32x4_t make_rsrc(const void *base)
{
    const uint64_t a = reinterpret_cast<uint64_t>(base);
    i32x4_t r;
    r.x = __builtin_amdgcn_readfirstlane(static_cast<int32_t>(a & 0xffffffffu));
    r.y = __builtin_amdgcn_readfirstlane(static_cast<int32_t>((a >> 32) & 0xffffu));
    r.z = -1;
    r.w = 0x00020000;
    return r;
}

// Direct-to-LDS loads: lane l copies 16 (4) bytes from rsrc + voff + soff to LDS
// byte address lds + 16 l (4 l).  M0 carries the wave-uniform LDS base; the s_nop
// covers the M0-write hazard, which the compiler cannot see inside an asm.
__device__ __forceinline__ void dma16(i32x4_t rsrc, uint32_t voff, uint32_t soff, uint32_t lds)
{
    asm volatile("s_nop 0\n\tbuffer_load_dwordx4 %0, %1, %2 offen lds"
                 :
                 : "v"(voff), "s"(rsrc), "s"(soff), "{m0}"(lds));
}

__device__ __forceinline__ void dma4(i32x4_t rsrc, uint32_t voff, uint32_t lds)
{
    asm volatile("s_nop 0\n\tbuffer_load_dword %0, %1, 0 offen lds"
                 :
                 : "v"(voff), "s"(rsrc), "{m0}"(lds));
}

// A workgroup's tile of WM x WN waves, each FM x FN blocks of 32 x 32, in LDS:
// stages of 128 columns of A's rows, then B's, then a dword of scales for each.
// Rows of 128 bytes start on two banks' worth of places, so the 16-byte chunks of
// row r are XORed with a number of r that spreads a fragment's reads over them,
// applied where the chunks are fetched.
template <int WM_, int WN_, int FM_, int FN_, int S_>
struct Tile {
    static constexpr int WM = WM_, WN = WN_, FM = FM_, FN = FN_, S = S_;
    static constexpr int W = WM * WN, BM = WM * FM * 32, BN = WN * FN * 32;
    static constexpr int AL = (BM / 8 + W - 1) / W, BL = (BN / 8 + W - 1) / W;   // loads of codes a wave and step
    static constexpr int SA = (BM + 64 * W - 1) / (64 * W), SB = (BN + 64 * W - 1) / (64 * W);
    static constexpr int LOADS = AL + BL + SA + SB;
    static constexpr int A_BYTES = BM * 128, B_BYTES = BN * 128;
    static constexpr int SCALES = (BM > 64 ? BM : 64) * 4;   // bytes of A's: whole loads
    static constexpr int STAGE = (A_BYTES + B_BYTES + SCALES + BN * 4 + 1023) / 1024 * 1024;
    static constexpr int PITCH = BN * 2 + 16;   // of C's rows
    // of the tile kernel: blocks and bytes of a wave's part for C, its stores of a tile
    static constexpr int PJ = FM * FN <= 4 ? 1 : FN % 2 == 0 ? 2 : FN, PART = PJ * 32 * 64, STORES = FM * FN * 2;
    static constexpr int LDS = S * STAGE > BM * PITCH ? S * STAGE : BM * PITCH;
    static_assert(BM % 64 == 0 || BM == 32, "whole loads of scales, or half a one");
    static_assert(BN % 64 == 0, "whole loads of scales");
    static_assert(LDS <= 160 * 1024, "LDS");
};

__device__ __forceinline__ int swizzle(int row) { return (row & 7) ^ ((row >> 3) & 3); }

// Where a wave's loads come from, and the loads.  Rows past the tile's last are
// that row again, columns past the last group that group: every load is inside
// its array, and every step has the same number.
template <int MODE, class T>
struct Loads {
    i32x4_t ra, rb;
    uint32_t va[T::AL], vb[T::BL], vsa[T::SA], vsb[T::SB], lds0;
    const uint32_t *as, *bs;
    int32_t last, a_rows, b_blocks;
    int wave;

    __device__ __forceinline__ Loads(const uint8_t *smem, int wave_) : wave(wave_)
    {
        lds0 = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(smem));
    }

    __device__ __forceinline__ void set(const Params &p, const Unit &u, int lane)
    {
        constexpr int W = T::W, FM = T::FM, FN = T::FN;
        lane = anew(lane);
        const int32_t m0 = u.m0, rows = u.m1 - u.m0, cols = min(T::BN, p.N - u.n0);
        const int64_t bm = MODE == EXPERTS ? u.matrix : 0;
        const bool gather = MODE == EXPERTS && p.top > 0;
        ra = make_rsrc(p.a + (gather ? 0 : m0) * p.a_ld);
        rb = make_rsrc(p.b + (bm * p.N + u.n0) * p.b_ld);
        auto a_row = [&](int row) -> uint32_t {   // from ra's
            const int32_t m = min(row, rows - 1);
            if (!gather) return m;
            return min(max(p.rows[m0 + m], 0) / p.top, p.a_rows - 1);
        };
        // load d of a wave fills rows 8 (d W + wave) .. + 7: waves without rows
        // of their own load the last ones again
#pragma unroll
        for (int i = 0; i < T::AL; ++i) {
            const int row = min(i * W + wave, T::BM / 8 - 1) * 8 + lane / 8;
            va[i] = a_row(row) * static_cast<uint32_t>(p.a_ld) + ((lane & 7) ^ swizzle(row)) * 16;
        }
#pragma unroll
        for (int i = 0; i < T::BL; ++i) {
            const int row = min(i * W + wave, T::BN / 8 - 1) * 8 + lane / 8;
            vb[i] = static_cast<uint32_t>(min(row, cols - 1)) * static_cast<uint32_t>(p.b_ld) +
                    ((lane & 7) ^ swizzle(row)) * 16;
        }
        // scales in LDS: [wave][row of 32][block], so that a lane's are neighbours
#pragma unroll
        for (int i = 0; i < T::SA; ++i) {
            const int d = min((i * W + wave) * 64, T::BM > 64 ? T::BM - 64 : 0) + lane;
            vsa[i] = a_row(d / (32 * FM) * (32 * FM) + d % FM * 32 + d / FM % 32) * 4;
        }
#pragma unroll
        for (int i = 0; i < T::SB; ++i) {
            const int d = min((i * W + wave) * 64, T::BN - 64) + lane;
            const int row = min(d / (32 * FN) * (32 * FN) + d % FN * 32 + d / FN % 32, cols - 1);
            vsb[i] = static_cast<uint32_t>(((u.n0 + row) >> p.b_shift) - (u.n0 >> p.b_shift)) * 4;
        }
        as = p.as + (gather ? 0 : m0);
        bs = p.bs + bm * ((p.kb + 3) / 4) * p.b_blocks + (u.n0 >> p.b_shift);
        a_rows = p.a_rows;
        b_blocks = p.b_blocks;
        last = u.kb1 - 1;
    }

    // Load d (a constant) of group kb to a stage.
    __device__ __forceinline__ void fetch(int stage, int32_t kb, int d) const
    {
        constexpr int W = T::W;
        kb = min(kb, last);
        const uint32_t base = lds0 + stage * T::STAGE;
        const uint32_t soff = static_cast<uint32_t>(kb) * 128u;
        if (d < T::AL) {
            dma16(ra, va[d], soff, base + min(d * W + wave, T::BM / 8 - 1) * 1024);
        } else if (d < T::AL + T::BL) {
            const int i = d - T::AL;
            dma16(rb, vb[i], soff, base + T::A_BYTES + min(i * W + wave, T::BN / 8 - 1) * 1024);
        } else if (d < T::AL + T::BL + T::SA) {
            const int i = d - T::AL - T::BL;
            dma4(make_rsrc(as + static_cast<int64_t>(kb >> 2) * a_rows), vsa[i],
                 base + T::A_BYTES + T::B_BYTES + min((i * W + wave) * 64, T::BM > 64 ? T::BM - 64 : 0) * 4);
        } else {
            const int i = d - T::AL - T::BL - T::SA;
            dma4(make_rsrc(bs + static_cast<int64_t>(kb >> 2) * b_blocks), vsb[i],
                 base + T::A_BYTES + T::B_BYTES + T::SCALES + min((i * W + wave) * 64, T::BN - 64) * 4);
        }
    }
};

// C from the waves' sums, through LDS, so that a row's columns leave in one run.
template <int MODE, class T>
__device__ __forceinline__ void store_tile(const Params &p, const Unit &u, uint16_t *c, uint8_t *smem,
                                           const f32x16_t (&acc)[T::FM][T::FN], int wm, int wn, int lane)
{
    const int r = lane & 31, h = lane >> 5, rows = u.m1 - u.m0;
#pragma unroll
    for (int i = 0; i < T::FM; ++i)
#pragma unroll
        for (int j = 0; j < T::FN; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const f32x4_t v = {acc[i][j][4 * e], acc[i][j][4 * e + 1], acc[i][j][4 * e + 2],
                                   acc[i][j][4 * e + 3]};
                *reinterpret_cast<half4_t *>(smem + ((wm * T::FM + i) * 32 + r) * T::PITCH +
                                             ((wn * T::FN + j) * 32 + 8 * e + 4 * h) * 2) =
                    __builtin_convertvector(v, half4_t);
            }
    __syncthreads();
#pragma unroll 4
    for (int o = threadIdx.x; o < T::BM * T::BN / 8; o += 64 * T::W) {
        const int row = o / (T::BN / 8), col = o % (T::BN / 8) * 8;
        if (row >= rows || u.n0 + col >= p.N) continue;
        store8(c + static_cast<int64_t>(row) * p.N, u.n0 + col, p.N,
               *reinterpret_cast<const half8_t *>(smem + row * T::PITCH + col * 2));
    }
}

// A block's sums are held to the accumulation registers: a wave's 128 x 128 values
// need all 256, and the compiler left to itself splits them between both files and
// spills.  It then cannot see these MFMAs, so the kernel supplies the wait states
// around them.  LAST: before the code's next branch, where the compiler may copy
// sums from register to register, as it did: the wait states of a read of the
// result, more than any MFMA asks for, are part of the statement.  (The host's
// pass of the compiler knows no such registers.)
template <bool LAST>
__device__ __forceinline__ void mfma(f32x16_t &acc, i32x8_t b, i32x8_t a, uint32_t sb, uint32_t sa)
{
#ifdef __HIP_DEVICE_COMPILE__
    if constexpr (LAST)
        asm volatile("v_mfma_scale_f32_32x32x64_f8f6f4 %0, %1, %2, %0, %3, %4 op_sel_hi:[0,0,0]\n\t"
                     "s_nop 7\n\ts_nop 7\n\ts_nop 7"
                     : "+a"(acc)
                     : "v"(b), "v"(a), "v"(sb), "v"(sa));
    else
        asm volatile("v_mfma_scale_f32_32x32x64_f8f6f4 %0, %1, %2, %0, %3, %4 op_sel_hi:[0,0,0]"
                     : "+a"(acc)
                     : "v"(b), "v"(a), "v"(sb), "v"(sa));
#endif
}

__device__ __forceinline__ void keep(f32x16_t &acc)
{
#ifdef __HIP_DEVICE_COMPILE__
    asm volatile("" : "+a"(acc));
#endif
}

// A range's sums, in the order in which lanes hold them.
template <class T>
__device__ __forceinline__ void store_partial(const Params &p, const Unit &u, f32x16_t (&acc)[T::FM][T::FN],
                                              int wave, int lane)
{
    lane = anew(lane);
    const int64_t tiles = p.tiles_m * p.tiles_n;
    float *to = p.partial + ((u.split * tiles + u.tile) * T::W + wave) * (T::FM * T::FN * 1024) + lane * 4;
#pragma unroll
    for (int i = 0; i < T::FM; ++i)
#pragma unroll
        for (int j = 0; j < T::FN; ++j) {
            keep(acc[i][j]);   // read here, not before
#pragma unroll
            for (int e = 0; e < 4; ++e)
                *reinterpret_cast<f32x4_t *>(to + ((i * T::FN + j) * 4 + e) * 256) =
                    f32x4_t{acc[i][j][4 * e], acc[i][j][4 * e + 1], acc[i][j][4 * e + 2], acc[i][j][4 * e + 3]};
            __builtin_amdgcn_sched_barrier(0);
        }
}

// Zeros: rows of no expert, an expert without rows.
template <class T>
__device__ __forceinline__ void store_zeros(const Params &p, const Unit &u, uint16_t *c)
{
    for (int o = anew(threadIdx.x); o < T::BM * T::BN / 8; o += 64 * T::W) {
        const int row = o / (T::BN / 8), col = o % (T::BN / 8) * 8;
        if (row < u.m1 - u.m0 && u.n0 + col < p.N)
            store8(c + static_cast<int64_t>(row) * p.N, u.n0 + col, p.N, half8_t{});
    }
}

// C from the waves' sums, by T::STORES stores of the wave where no part of the tile is
// missing, else after its loads have landed: 32 rows of T::PJ blocks at a time
// through the wave's own part of LDS, so that lanes write neighbouring columns.
template <class T, bool ALL>
__device__ __forceinline__ void store_blocks(const Params &p, const Unit &u, uint16_t *c,
                                             f32x16_t (&acc)[T::FM][T::FN], uint8_t *part, int wm, int wn, int lane)
{
    lane = anew(lane);
    const int r = lane & 31, h = lane >> 5, rows = u.m1 - u.m0;
    auto put = [&](int row, int32_t n, half8_t v) {
        uint16_t *to = c + static_cast<int64_t>(row) * p.N;
        if constexpr (ALL)
            // past the L2, which they would fill (16396 rows of 32 experts, 2048 x 1408: 87 us, 82 so)
            __builtin_nontemporal_store(v, reinterpret_cast<half8_u_t *>(to + n));
        else if (row < rows && n < p.N)
            store8(to, n, p.N, v);
    };
    auto four = [&](int i, int j, int e) {
        return __builtin_convertvector(
            f32x4_t{acc[i][j][4 * e], acc[i][j][4 * e + 1], acc[i][j][4 * e + 2], acc[i][j][4 * e + 3]}, half4_t);
    };
#pragma unroll
    for (int i = 0; i < T::FM; ++i) {
        const int row0 = (wm * T::FM + i) * 32;
        constexpr int CH = T::PJ * 4;   // 16-byte chunks of a row
#pragma unroll
        for (int j0 = 0; j0 < T::FN; j0 += T::PJ) {
            // chunks XORed within fours with the row: lanes' writes spread over the banks
#pragma unroll
            for (int j = 0; j < T::PJ; ++j) {
                keep(acc[i][j0 + j]);   // read here, not before
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    *reinterpret_cast<half4_t *>(part + r * (CH * 16) + (j * 4 + (e ^ (r & 3))) * 16 + h * 8) =
                        four(i, j0 + j, e);
            }
            wave_lds_fence();
#pragma unroll
            for (int o0 = 0; o0 < 32 * CH; o0 += 64) {
                const int o = o0 + lane, row = o / CH, ch = o % CH;
                put(row0 + row, u.n0 + (wn * T::FN + j0) * 32 + ch * 8,
                    *reinterpret_cast<const half8_t *>(part + row * (CH * 16) + (ch ^ (row & 3)) * 16));
            }
            wave_lds_fence();
            __builtin_amdgcn_sched_barrier(0);
        }
    }
}

template <class T>
__device__ __forceinline__ void store_sums(const Params &p, const Unit &u, uint16_t *c,
                                           f32x16_t (&acc)[T::FM][T::FN], uint8_t *part, int wm, int wn, int lane)
{
    if (u.m1 - u.m0 == T::BM && u.n0 + T::BN <= p.N) {
        store_blocks<T, true>(p, u, c, acc, part, wm, wn, lane);
    } else {
        asm volatile("s_waitcnt vmcnt(0)" : : : "memory");
        store_blocks<T, false>(p, u, c, acc, part, wm, wn, lane);
    }
}

// Two stages; a step's MFMAs are its two halves' (64 columns), each half's
// fragments read from LDS while the other's are multiplied.  A workgroup takes one
// unit after the other without a pause: the last two steps of one load the first
// groups of the next before C leaves.  Memory operations return in order, so C's
// stores are waited for with the first loads behind them, in a unit's second step;
// and a register spilled in between would wait for them at once (20 us a tile).
//
// 256 x 256 is the largest tile whose sums the registers hold: 64 KB of loads a step
// for 17 MFLOP.  4096 x 8192 x 8192: 205 to 237 us by box, 2.3 to 2.7 PFLOP/s, MFMA busy
// 67%, at the power limit (1.8 to 1.9 GHz).  256 x 192 and 128 x 128 (two workgroups a
// CU) for shapes that their rounds fit better: 3818 x 5760 x 1152 36.8, 31.6 and 34.2 us,
// 1024 x 8192 x 8192 88.5, 80.1 and 76.2.
template <int MODE, class T, int OCC>
__global__ __launch_bounds__(64 * T::W)
__attribute__((amdgpu_waves_per_eu(OCC, OCC)))
void f8_tile_kernel(Params p)
{
    constexpr int FM = T::FM, FN = T::FN, LOADS = T::LOADS;
    static_assert(T::S == 2, "two stages");
    static_assert(T::STORES <= 63 && T::STORES <= FM * FN * 4, "vmcnt counts at most 63");
    __shared__ __attribute__((aligned(1024))) uint8_t smem[T::S * T::STAGE];
    __shared__ __attribute__((aligned(16))) uint8_t parts[T::W][T::PART];
    __shared__ Experts experts;
    const int lane = threadIdx.x & 63, wave = wave_index();
    const int wm = wave / T::WN, wn = wave % T::WN;
    const int r = lane & 31, h = lane >> 5;
    if constexpr (MODE == EXPERTS) experts.template fill<T::W>(p.offsets, p.E, p.M, T::BM, p.tiles_n);
    if constexpr (MODE == GRAD) experts.template fill<T::W>(p.offsets, p.E, p.top, 128, 1);
    auto c_of = [&](const Unit &u) {
        return p.c + (MODE == GRAD ? u.matrix * p.M * p.N : 0) + static_cast<int64_t>(u.m0) * p.N;
    };
    int32_t id = blockIdx.x;
    // the next unit that has something to multiply; zeros for those before it
    auto next = [&](Unit &u) {
        for (; id < p.units; id += gridDim.x) {
            if constexpr (MODE == EXPERTS)
                u = expert_unit<T::BM, T::BN>(p, experts.find(p.offsets, p.E, p.M, T::BM, p.tiles_n, id, lane));
            else
                u = matrix_unit<MODE, T::BM, T::BN>(p, id, p.units);
            if (MODE == GRAD && !u.none) {
                const int32_t e = static_cast<int32_t>(u.matrix);
                u.kb0 = e > 0 ? min(__builtin_amdgcn_readfirstlane(experts.upto[e - 1]), p.kb) : 0;
                u.kb1 = min(__builtin_amdgcn_readfirstlane(experts.upto[e]), p.kb);
            }
            if (u.none) continue;
            if (MODE != DENSE && u.kb0 >= u.kb1) {
                store_zeros<T>(p, u, c_of(u));
                continue;
            }
            id += gridDim.x;
            return true;
        }
        return false;
    };
    Unit u, nu;
    if (!next(u)) return;
    Loads<MODE, T> loads(smem, wave);
    loads.set(p, u, lane);
    f32x16_t acc[FM][FN];
    int off[4];   // a lane's 16-byte chunks in a tile's rows
#pragma unroll
    for (int kk = 0; kk < 2; ++kk)
#pragma unroll
        for (int w = 0; w < 2; ++w) off[kk * 2 + w] = r * 128 + (((kk * 4 + h * 2 + w) ^ swizzle(r)) * 16);
    i32x4_t af[2][FM][2], bf[2][FN][2];
    uint32_t sa[FM], sb[FN], na[FM], nb[FN];
    auto read = [&](int stage, int kk, int d) {   // one of 2 (FM + FN)
        const uint8_t *st = smem + stage * T::STAGE;
        if (d < 2 * FM)
            af[kk][d / 2][d % 2] = *reinterpret_cast<const i32x4_t *>(
                st + wm * FM * 4096 + d / 2 * 4096 + off[kk * 2 + d % 2]);
        else
            bf[kk][d / 2 - FM][d % 2] = *reinterpret_cast<const i32x4_t *>(
                st + T::A_BYTES + wn * FN * 4096 + (d / 2 - FM) * 4096 + off[kk * 2 + d % 2]);
    };
    auto read_scales = [&](int stage) {
        const uint8_t *st = smem + stage * T::STAGE + T::A_BYTES + T::B_BYTES;
#pragma unroll
        for (int i = 0; i < FM; ++i)
            na[i] = *reinterpret_cast<const uint32_t *>(st + ((wm * 32 + r) * FM + i) * 4);
#pragma unroll
        for (int i = 0; i < FN; ++i)
            nb[i] = *reinterpret_cast<const uint32_t *>(st + T::SCALES + ((wn * 32 + r) * FN + i) * 4);
    };
    auto take_scales = [&](int32_t kb) {
        const int s = 8 * (kb & 3);
#pragma unroll
        for (int i = 0; i < FM; ++i) sa[i] = na[i] >> s;
#pragma unroll
        for (int i = 0; i < FN; ++i) sb[i] = nb[i] >> s;
        // two wait states between a VALU's result and an MFMA that reads it
#pragma unroll
        for (int i = 0; i < FM; ++i) asm volatile("" : "+v"(sa[i]));
#pragma unroll
        for (int i = 0; i < FN; ++i) asm volatile("" : "+v"(sb[i]));
        asm volatile("s_nop 1");
    };
    constexpr int READS = 2 * (FM + FN), MFMAS = FM * FN;
    // the MFMAs of half a step, the next half's reads and the loads between them
    auto compute = [&](int kk, auto each) {
#pragma unroll
        for (int t = 0; t < MFMAS; ++t) {
            const int i = t / FN, j = t % FN;
            if (kk == 1 && t == MFMAS - 1)
                mfma<true>(acc[i][j], whole(bf[kk][j]), whole(af[kk][i]), sb[j], sa[i]);
            else
                mfma<false>(acc[i][j], whole(bf[kk][j]), whole(af[kk][i]), sb[j], sa[i]);
            each(t);
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    // One group from `stage`; group `fetch` of `loads` then takes its place, and the
    // next step's is group `after`.  FIRST of a unit: T::STORES stores of the unit
    // before or more are behind the loads that are waited for, or those are there.
    auto step = [&](auto first, int stage, int32_t fetch, int32_t after) {
        compute(0, [&](int t) {
#pragma unroll
            for (int d = 0; d < READS; ++d)
                if (d * MFMAS / READS == t) read(stage, 1, d);
        });
        // this stage is read to the end, the next one has landed
        asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" : : "n"(first ? T::STORES : 0) : "memory");
        read_scales(stage ^ 1);
        compute(1, [&](int t) {
#pragma unroll
            for (int d = 0; d < READS; ++d)
                if (d * MFMAS / READS == t) read(stage ^ 1, 0, d);
#pragma unroll
            for (int d = 0; d < LOADS; ++d)
                if (d * MFMAS / LOADS == t) loads.fetch(stage, fetch, d);
        });
        take_scales(after);
    };
    auto clear = [&] {
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
            for (int j = 0; j < FN; ++j) {
                acc[i][j] = f32x16_t{};
                keep(acc[i][j]);
            }
        asm volatile("s_nop 4");   // between those writes and the first MFMA
    };
    auto fetch_all = [&](int stage, int32_t kb) {
#pragma unroll
        for (int d = 0; d < LOADS; ++d) loads.fetch(stage, kb, d);
    };
    fetch_all(0, u.kb0);
    fetch_all(1, u.kb0 + 1);
    bool more = next(nu);
    asm volatile("s_waitcnt vmcnt(0)\n\ts_barrier" : : : "memory");
#pragma unroll
    for (int d = 0; d < READS; ++d) read(0, 0, d);
    read_scales(0);
    take_scales(u.kb0);
    clear();
    for (int stage = 0;;) {
        if (u.kb1 - u.kb0 == 1 && more) {
            // the step before could not know the unit after this one
            loads.set(p, nu, lane);
            fetch_all(stage ^ 1, nu.kb0);
            asm volatile("s_waitcnt vmcnt(0)" : : : "memory");
        }
        const int32_t over = more ? nu.kb0 - u.kb1 : 0;   // of a group past this unit's last
        auto group = [&](int32_t kb) { return kb < u.kb1 ? kb : kb + over; };
        if (u.kb0 + 2 == u.kb1 && more) loads.set(p, nu, lane);
        step(std::true_type{}, stage, group(u.kb0 + 2), group(u.kb0 + 1));
        stage ^= 1;
        for (int32_t kb = u.kb0 + 1; kb < u.kb1; ++kb) {
            if (kb + 2 == u.kb1 && more) loads.set(p, nu, lane);
            step(std::false_type{}, stage, group(kb + 2), group(kb + 1));
            stage ^= 1;
        }
        __builtin_amdgcn_sched_barrier(0);
        if (MODE == DENSE && p.splits > 1)
            store_partial<T>(p, u, acc, wave, lane);
        else
            store_sums<T>(p, u, c_of(u), acc, parts[wave], wm, wn, lane);
        __builtin_amdgcn_sched_barrier(0);
        if (!more) break;
        clear();
        u = nu;
        more = next(nu);
    }
    // no load may still be on its way to this LDS
    asm volatile("s_waitcnt vmcnt(0)" : : : "memory");
}

// A ring of S stages for few rows, where reading B bounds the call: S - 1 groups
// are on their way while one is multiplied.  With p.splits > 1 (dense) K is
// split into ranges of p.kb_split groups, and the ranges' sums go to p.partial in
// the order in which lanes hold them.  Two workgroups fit on a CU.  16 x 16384 x 16384
// 51 to 56 us (268 MB at 4.8 to 5.2 TB/s), 64 x 4096 x 4096 10.4 (in four ranges, unsplit
// 11.2), 8 experts of one token, 2048 x 4096, 13.1 (67 MB).
template <int MODE, class T>
__global__ __launch_bounds__(64 * T::W) void f8_ring_kernel(Params p)
{
    constexpr int FM = T::FM, FN = T::FN, LOADS = T::LOADS, S = T::S;
    static_assert((S - 2) * LOADS <= 63, "vmcnt counts at most 63 loads");
    __shared__ __attribute__((aligned(1024))) uint8_t smem[T::LDS];
    const int lane = threadIdx.x & 63, wave = wave_index();
    const int wm = wave / T::WN, wn = wave % T::WN;
    const int r = lane & 31, h = lane >> 5;
    Unit u = make_unit<MODE, T::BM, T::BN>(p, lane);
    if (u.none) return;
    uint16_t *c = p.c + (MODE == GRAD ? u.matrix * p.M * p.N : 0) + static_cast<int64_t>(u.m0) * p.N;
    if (MODE != DENSE && u.kb0 >= u.kb1) return store_zeros<T>(p, u, c);
    Loads<MODE, T> loads(smem, wave);
    loads.set(p, u, lane);
    f32x16_t acc[FM][FN] = {};
    int off[4];
#pragma unroll
    for (int kk = 0; kk < 2; ++kk)
#pragma unroll
        for (int w = 0; w < 2; ++w) off[kk * 2 + w] = r * 128 + (((kk * 4 + h * 2 + w) ^ swizzle(r)) * 16);
#pragma unroll
    for (int s = 0; s < S - 1; ++s)
#pragma unroll
        for (int d = 0; d < LOADS; ++d) loads.fetch(s, u.kb0 + s, d);
    int stage = 0;
    for (int32_t kb = u.kb0; kb < u.kb1; ++kb) {
        // this stage's loads (the oldest) have landed, and every wave is done with
        // the stage before it, which is filled again
        asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" : : "n"((S - 2) * LOADS) : "memory");
#pragma unroll
        for (int d = 0; d < LOADS; ++d) loads.fetch(stage == 0 ? S - 1 : stage - 1, kb + S - 1, d);
        const uint8_t *st = smem + stage * T::STAGE;
        const uint8_t *ss = st + T::A_BYTES + T::B_BYTES;
        const int s = 8 * (kb & 3);
        uint32_t sa[FM], sb[FN];
#pragma unroll
        for (int i = 0; i < FM; ++i)
            sa[i] = *reinterpret_cast<const uint32_t *>(ss + ((wm * 32 + r) * FM + i) * 4) >> s;
#pragma unroll
        for (int i = 0; i < FN; ++i)
            sb[i] = *reinterpret_cast<const uint32_t *>(ss + T::SCALES + ((wn * 32 + r) * FN + i) * 4) >> s;
#pragma unroll
        for (int kk = 0; kk < 2; ++kk) {
            i32x4_t af[FM][2], bf[FN][2];
#pragma unroll
            for (int w = 0; w < 2; ++w) {
#pragma unroll
                for (int i = 0; i < FM; ++i)
                    af[i][w] = *reinterpret_cast<const i32x4_t *>(st + (wm * FM + i) * 4096 + off[kk * 2 + w]);
#pragma unroll
                for (int j = 0; j < FN; ++j)
                    bf[j][w] = *reinterpret_cast<const i32x4_t *>(st + T::A_BYTES + (wn * FN + j) * 4096 +
                                                                  off[kk * 2 + w]);
            }
#pragma unroll
            for (int i = 0; i < FM; ++i)
#pragma unroll
                for (int j = 0; j < FN; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
                        whole(bf[j]), whole(af[i]), acc[i][j], 0, 0, 0, sb[j], 0, sa[i]);
        }
        stage = stage == S - 1 ? 0 : stage + 1;
    }
    // no load may still be on its way to this LDS
    asm volatile("s_waitcnt vmcnt(0)" : : : "memory");
    if (MODE == DENSE && p.splits > 1) return store_partial<T>(p, u, acc, wave, lane);
    __syncthreads();
    store_tile<MODE, T>(p, u, c, smem, acc, wm, wn, lane);
}

// C from the ranges' sums, in order; four columns a thread.
struct JoinParams {
    const float *partial;
    uint16_t *c;
    int64_t stride;                    // values between two ranges' sums
    int32_t M, N, tiles_m, tiles_n, splits;
    int32_t wn, fm, fn, waves;
};

__global__ __launch_bounds__(256) void f8_join_kernel(JoinParams p)
{
    const int64_t idx = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    if (idx * 4 >= p.stride) return;
    const int lane = threadIdx.x & 63, r = lane & 31, h = lane >> 5;
    int32_t rest = static_cast<int32_t>(idx >> 6);
    const int e = rest % 4;
    rest /= 4;
    const int j = rest % p.fn;
    rest /= p.fn;
    const int i = rest % p.fm;
    rest /= p.fm;
    const int wave = rest % p.waves;
    int32_t tm, tn;
    find_tile(rest / p.waves, p.tiles_m, p.tiles_n, tm, tn);
    const int wm = wave / p.wn, wn = wave % p.wn;
    const int32_t m = ((tm * (p.waves / p.wn) + wm) * p.fm + i) * 32 + r;
    const int32_t n = ((tn * p.wn + wn) * p.fn + j) * 32 + 8 * e + 4 * h;
    if (m >= p.M || n >= p.N) return;
    const float *from = p.partial + idx * 4;
    f32x4_t sum = *reinterpret_cast<const f32x4_t *>(from);
#pragma unroll 4
    for (int32_t s = 1; s < p.splits; ++s) sum += *reinterpret_cast<const f32x4_t *>(from + s * p.stride);
    store4(p.c + static_cast<int64_t>(m) * p.N, n, p.N, sum);
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

static int launch(const void *fn, int64_t grid, int threads, void *params, hipStream_t stream,
                  int lds = 0)
{
    // the launch's own status only: the thread's sticky error state is neither
    // read nor cleared
    void *args[] = {params};
    const hipError_t err = hipLaunchKernel(fn, dim3(static_cast<uint32_t>(grid)),
                                           dim3(static_cast<uint32_t>(threads)), args, lds, stream);
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

struct Kernel {
    int32_t kind, bm, bn, waves;
    int32_t lds;               // for the waves' sums
    int32_t wn, fm, fn;        // of a kernel whose K may be split
    int32_t slots;             // workgroups on a compute unit
    bool persistent;           // which take one unit after the other
    double start, step, full;  // us: a workgroup's start and end, 128 columns with one and with all slots taken
    const void *run[3];        // by mode
};
#define STREAM(W, Q)                                                                              \
    {GEMM_F16_LOWBIT_STREAM, 16, 16, W, W * 1024, 0, 0, 0, 0, false, 0, 0, 0,                     \
     {address(f8_stream_kernel<DENSE, W, Q>), address(f8_stream_kernel<EXPERTS, W, Q>), nullptr}}
#define TILE(WM, WN, FM, FN, OCC, START, STEP, FULL)                                              \
    {GEMM_F16_LOWBIT_TILE, WM * FM * 32, WN * FN * 32, WM * WN, 0, WN, FM, FN, OCC, true, START, STEP, FULL, \
     {address(f8_tile_kernel<DENSE, Tile<WM, WN, FM, FN, 2>, OCC>),                               \
      address(f8_tile_kernel<EXPERTS, Tile<WM, WN, FM, FN, 2>, OCC>),                             \
      address(f8_tile_kernel<GRAD, Tile<WM, WN, FM, FN, 2>, OCC>)}}
#define RING(WM, WN, FM, FN, S, START, STEP, FULL)                                                \
    {GEMM_F16_LOWBIT_TILE, WM * FM * 32, WN * FN * 32, WM * WN, 0, WN, FM, FN, 2, false, START, STEP, FULL, \
     {address(f8_ring_kernel<DENSE, Tile<WM, WN, FM, FN, S>>),                                    \
      address(f8_ring_kernel<EXPERTS, Tile<WM, WN, FM, FN, S>>),                                  \
      address(f8_ring_kernel<GRAD, Tile<WM, WN, FM, FN, S>>)}}
static const Kernel kKernels[] = {
    TILE(2, 2, 4, 4, 1, 6.26, 1.022, 1.022), TILE(2, 2, 4, 3, 1, 5.43, 0.849, 0.849),
    TILE(2, 2, 2, 2, 2, 1.91, 0.586, 0.794), RING(1, 2, 1, 1, 6, 1.26, 0.208, 0.249),
    RING(2, 2, 1, 1, 4, 1.27, 0.231, 0.341), RING(1, 4, 2, 1, 3, 1.54, 0.347, 0.563),
    STREAM(8, 2), STREAM(16, 2),
};
#undef TILE
#undef RING
#undef STREAM
constexpr int32_t TILES = 6, STREAM8 = 6, STREAM16 = 7;

// The kernel of a call, an index of kKernels, and the ranges of K (dense).
struct Choice {
    int32_t id, splits, units;
};

// Time in us of `wgs` workgroups with `steps` groups of columns each, their K in
// `splits` ranges; bytes of the operands and C.  Rounds of workgroups over the CUs,
// bytes and multiplications at a rate each, and for ranges their sums' way through
// memory and the join.  All constants are fitted (planner_fit/fit_f8_model.py, with its
// timings): that of the multiplications is 1.99 PFLOP/s, a mean over tiles of every size,
// below what the largest tiles reach.
static double model(const Kernel &e, double wgs, double steps, int64_t splits, double bytes, int32_t cus)
{
    const double slots = static_cast<double>(cus) * e.slots;
    const double all = std::floor(wgs / slots), rest = wgs - all * slots;
    const double taken = e.full * steps + e.start * e.slots, tile = static_cast<double>(e.bm) * e.bn;
    double us = all * taken;
    if (rest > 0) us += rest <= cus ? e.step * steps + e.start : taken;
    const double memory = bytes / 5.475e6, matrix = wgs * tile * steps * GROUP / 9.928e8;
    auto fourth = [](double x) { return x * x * x * x; };
    us = std::sqrt(std::sqrt(fourth(us) + fourth(memory) + fourth(matrix)));
    return us + 3.16 + (splits > 1 ? 1.76 + 4.0 * wgs * tile / 5.045e6 : 0.0);
}

// The tile and ring kernels and ranges of K by that model, fitted to 2,184 timings
// of 142 shapes (1 to 8192 rows, N and K of 64 to 16384, 8 to 256 experts, operands from
// HBM).  Its error, as rms of the logarithm over the shapes, is 6 to 19% by kernel and
// call; the longest products take less than it says (4096 x 8192 x 8192: 285 us, measured
// 205 to 237).  What it chose took 2.6% (products), 1.7% (experts) and 2.3% (gradients)
// longer than the best of each shape in the mean, 13, 40 and 12% in the worst (2095 tokens,
// 2 of 256 experts, 3264 x 192: 91.6 us, with 128 x 128 tiles 65.3).
static Choice search(const Call &c, int32_t num_cus)
{
    const double M = static_cast<double>(c.M), N = static_cast<double>(c.N), K = static_cast<double>(c.a.kp);
    const int64_t kb = std::max<int64_t>(c.a.kp / GROUP, 1);
    // experts that have rows, if each row's is drawn alike
    const double E = static_cast<double>(c.matrices);
    const double used = c.mode == DENSE ? 1.0 : E * (1.0 - std::pow(1.0 - 1.0 / E, c.mode == EXPERTS ? M : c.top));
    const double bytes = c.mode == GRAD ? c.top * (M + N) + 2.0 * E * M * N : used * N * K + M * K + 2.0 * M * N;
    Choice best{};
    // Halves that the product's kernel quantises itself: up to 16 rows, and 2^15
    // values of them a workgroup; of experts' tiles not many more than run at once.
    // (5 x 7001 x 4160 12.7 us, quantised first 13.3; 14 x 4544 x 8064 26.3 and 14.8; one token's 8
    // experts of 1216 x 512 5.5 and 7.9, 48 experts of 256, 3328 x 192, 69 and 24.)  Sixteen waves
    // for 13 to 36 groups, whose steps of 32 are then one or two and eight's of 16 up to three
    // (16 x 448 x 1728 5.9 us, eight 6.8; 1 x 4096 x 14336 16.2 and 14.6; 8 x 15936 x 832 10.4 and
    // 8.3).  Their time over that of eight, the mean over 1 to 16 rows and N of 448 to 15936, by
    // groups: 12 1.06, 13 to 16 1.05 (of 16 rows alone 0.98), 20 0.94, 24 0.88, 32 0.81, 33 0.87,
    // 36 0.89, 40 0.96, 44 1.04, 48 1.10.
    const double rows = c.mode == EXPERTS ? M / used : M;
    if (c.a_f16 && c.mode != GRAD && rows <= 16 && std::min(M, 16.0) * K <= 32768 &&
        (c.mode == DENSE || used * static_cast<double>(cdiv(c.N, 16)) <= 3.0 * num_cus)) {
        best.id = kb > 12 && kb <= 36 ? STREAM16 : STREAM8;
        best.splits = 1;
        return best;
    }
    double best_us = 0;
    for (int32_t id = 0; id < TILES; ++id) {
        const Kernel &e = kKernels[id];
        const int64_t tiles = cdiv(c.M, e.bm) * cdiv(c.N, e.bn);
        auto consider = [&](double wgs, double steps, int64_t splits) {
            const double us = model(e, wgs, steps, splits, bytes, num_cus);
            if (best_us > 0 && us >= best_us) return;
            best_us = us;
            best = Choice{id, static_cast<int32_t>(splits), 0};
        };
        if (c.mode == GRAD) {
            consider(E * static_cast<double>(tiles), c.top > 64.0 * E ? c.top / E / GROUP + 0.5 : 1.0, 1);
        } else if (c.mode == EXPERTS) {
            // tiles of an expert whose rows are anything up to twice the mean
            const double most = 2.0 * M / (used * e.bm), whole = std::floor(most);
            const double down = used * (most <= 1.0 ? 1.0 : (0.5 * whole + most - whole) * (whole + 1.0) / most);
            consider(std::ceil(static_cast<double>(cdiv(c.N, e.bn)) * down), static_cast<double>(kb), 1);
        } else {
            int64_t last = 0;
            for (int64_t sp = 1; sp <= std::min<int64_t>(kb, 32); ++sp) {
                const int64_t per = cdiv(kb, sp), splits = cdiv(kb, per);
                if (per == last) continue;   // the same ranges
                last = per;
                if (sp > 1 && tiles * splits > 4 * e.slots * num_cus) break;
                consider(static_cast<double>(tiles * splits), static_cast<double>(per), splits);
            }
        }
    }
    return best;
}

// The search takes microseconds: each thread keeps its last few choices.
static Choice choose(const Call &c, int32_t num_cus)
{
    struct Entry {
        int64_t M, N, K, matrices;
        int32_t mode, top, cus;
        bool a_f16;
        Choice choice;
    };
    static thread_local Entry cache[8] = {};
    static thread_local int next = 0;
    for (const Entry &o : cache)
        if (o.cus == num_cus && o.M == c.M && o.N == c.N && o.K == c.K && o.matrices == c.matrices &&
            o.mode == c.mode && o.top == c.top && o.a_f16 == c.a_f16)
            return o.choice;
    const Choice choice = search(c, num_cus);
    cache[next] = Entry{c.M, c.N, c.K, c.matrices, c.mode, c.top, num_cus, c.a_f16, choice};
    next = (next + 1) % 8;
    return choice;
}

// The bytes of LDS in which a workgroup of a stream kernel quantises A's rows.
static int64_t stream_lds(const Call &c, const Kernel &e)
{
    const int64_t rows = std::min<int64_t>(16, c.M);
    return std::max<int64_t>(rows * (c.a.kp + 16) + round_up(rows * (c.a.kp / GROUP), 16), e.lds);
}

// The bytes of one range's sums.
static int64_t partial_bytes(const Call &c, const Kernel &e)
{
    return cdiv(c.M, e.bm) * cdiv(c.N, e.bn) * e.bm * e.bn * 4;
}

static int plan_call(const Call &c, int32_t num_cus, gemm_f16_lowbit_plan_t *plan, Choice *r)
{
    *plan = gemm_f16_lowbit_plan_t{};
    plan->splits = 1;
    if (num_cus <= 0) return GEMM_F16_INVALID_ARG;
    const int64_t matrices = c.mode == GRAD ? round_up(c.matrices, 8) : 1;
    if (cdiv(c.M, 16) * cdiv(c.N, 16) > INT32_MAX / matrices) return GEMM_F16_UNSUPPORTED;
    if (c.M == 0 || c.N == 0) return GEMM_F16_OK;
    *r = choose(c, num_cus);
    const Kernel &e = kKernels[r->id];
    // the kernels compute the ends of their tiles in 32 bits
    if (round_up(c.M, e.bm) > INT32_MAX || round_up(c.N, e.bn) > INT32_MAX) return GEMM_F16_UNSUPPORTED;
    // every expert, and the rows of none, may end inside a tile
    const int64_t tiles = c.mode == EXPERTS ? c.M / e.bm + std::min(c.matrices, c.M) + 1 : cdiv(c.M, e.bm);
    const int64_t grid = matrices * tiles * cdiv(c.N, e.bn) * r->splits;
    if (grid * 64 * e.waves >= MOST_THREADS) return GEMM_F16_UNSUPPORTED;
    plan->kernel = e.kind;
    plan->block_m = e.bm;
    plan->block_n = e.bn;
    plan->waves = e.waves;
    plan->splits = r->splits;
    // the tile kernels' workgroups take several units each
    plan->grid = static_cast<int32_t>(e.persistent ? std::min<int64_t>(grid, int64_t(num_cus) * e.slots) : grid);
    r->units = static_cast<int32_t>(grid);
    if (r->splits > 1) plan->workspace_bytes = r->splits * partial_bytes(c, e);
    if (c.a_f16 && r->id < TILES)
        plan->workspace_bytes += round_up(c.a.codes, 256) + round_up(c.a.scales, 256);
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
    Choice r{};
    v = plan_call(c, cus, &plan, &r);
    if (v != GEMM_F16_OK) return v;
    if (plan.workspace_bytes > (workspace ? workspace_bytes : 0)) return GEMM_F16_INVALID_ARG;
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    const Kernel &e = kKernels[r.id];
    const bool fused = r.id >= TILES;
    const int64_t a_bytes = c.a_f16 && !fused ? round_up(c.a.codes, 256) + round_up(c.a.scales, 256) : 0;
    if (a_bytes > 0) {
        v = quantize(1, c.a_rows, c.K, 1, false, c.a, X, ws, ws + round_up(c.a.codes, 256), stream);
        if (v != GEMM_F16_OK) return v;
        a_codes = ws;
        a_scales = ws + round_up(c.a.codes, 256);
    }
    Params p;
    const int64_t partial = plan.splits > 1 ? partial_bytes(c, e) : 0;
    p.partial = reinterpret_cast<float *>(ws + a_bytes);
    p.units = r.units;
    p.splits = plan.splits;
    p.kb_split = static_cast<int32_t>(cdiv(c.a.kp / GROUP, plan.splits));
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
    p.K = static_cast<int32_t>(c.K);
    p.x = static_cast<const uint16_t *>(X);
    p.kb = static_cast<int32_t>(c.a.kp / GROUP);
    p.a_rows = static_cast<int32_t>(c.a_rows);
    p.b_blocks = static_cast<int32_t>(c.b.blocks);
    p.b_shift = c.b.shift;
    p.E = static_cast<int32_t>(c.matrices);
    p.top = c.top;
    p.tiles_m = static_cast<int32_t>(cdiv(c.M, e.bm));
    p.tiles_n = static_cast<int32_t>(cdiv(c.N, e.bn));
    v = launch(e.run[c.mode], plan.grid, 64 * e.waves, &p, stream,
               static_cast<int>(fused ? stream_lds(c, e) : 0));
    if (v != GEMM_F16_OK || plan.splits == 1) return v;
    JoinParams q;
    q.partial = p.partial;
    q.c = p.c;
    q.stride = partial / 4;
    q.M = p.M;
    q.N = p.N;
    q.tiles_m = p.tiles_m;
    q.tiles_n = p.tiles_n;
    q.splits = p.splits;
    q.wn = e.wn;
    q.fm = e.fm;
    q.fn = e.fn;
    q.waves = e.waves;
    return launch(address(f8_join_kernel), cdiv(partial, 4096), 256, &q, stream);
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

static int grad_call(int64_t S, int64_t E, int64_t M, int64_t N, Call *c)
{
    int64_t columns = 0;
    int v = experts_columns(S, E, &columns);
    if (v != GEMM_F16_OK) return v;
    *c = Call{};
    c->mode = GRAD;
    c->M = M;
    c->N = N;
    c->K = columns;
    c->a_rows = M;
    c->matrices = E;
    c->top = static_cast<int32_t>(S);
    v = shape_of(1, M, columns, 1, &c->a);
    return v != GEMM_F16_OK ? v : shape_of(1, N, columns, 1, &c->b);
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
    Choice r{};
    const int v = dense_call(M, N, K, b_block, a_f16 != 0, &c);
    return v != GEMM_F16_OK ? v : plan_call(c, num_cus, plan, &r);
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
    Choice r{};
    const int v = experts_call(S, E, N, K, top, a_f16 != 0, &c);
    return v != GEMM_F16_OK ? v : plan_call(c, num_cus, plan, &r);
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

extern "C" int gemm_f16_nt_f8_experts_grad_plan(int64_t S, int64_t E, int64_t M, int64_t N,
                                                int32_t num_cus, gemm_f16_lowbit_plan_t *plan)
{
    if (!plan) return GEMM_F16_INVALID_ARG;
    Call c;
    Choice r{};
    const int v = grad_call(S, E, M, N, &c);
    return v != GEMM_F16_OK ? v : plan_call(c, num_cus, plan, &r);
}

extern "C" int gemm_f16_nt_f8_experts_grad(int64_t S, int64_t E, int64_t M, int64_t N,
                                           const void *a_codes, const void *a_scales,
                                           const void *b_codes, const void *b_scales,
                                           const void *offsets, void *C, hipStream_t stream)
{
    Call c;
    int v = grad_call(S, E, M, N, &c);
    if (v != GEMM_F16_OK) return v;
    if (cdiv(M, 16) * cdiv(N, 16) > INT32_MAX / round_up(E, 8)) return GEMM_F16_UNSUPPORTED;
    const Array arrays[6] = {{a_codes, c.a.codes, 16, false}, {a_scales, c.a.scales, 4, false},
                             {b_codes, c.b.codes, 16, false}, {b_scales, c.b.scales, 4, false},
                             {offsets, (E + 1) * 4, 4, false}, {C, E * M * N * 2, 2, true}};
    v = check_arrays(arrays, 6);
    if (v != GEMM_F16_OK || M == 0 || N == 0) return v;
    if (S == 0) return gemm_f16_nt(E * M, N, 0, nullptr, nullptr, C, stream);
    return run_call(c, nullptr, a_codes, a_scales, b_codes, b_scales, nullptr, offsets, C, nullptr,
                    0, stream);
}
