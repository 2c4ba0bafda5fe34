// Conversions of the low-bit formats: 2-byte weights to packed 4-bit codes with
// group scales and zero points and back, and 2-byte activations to 8-bit codes
// with a scale per column of 128 rows and back. All are bound by memory: each
// block reads its tile once in 16-byte loads, keeps it on chip (shared memory
// where the tile changes orientation, registers elsewhere) and writes once.
//
// At 8192 x 8192: w4 quantise 47 to 50 us (0.50 to 0.53 of the measured copy rate: some 15
// instructions a weight, two bytes at a time from shared memory) and dequantise
// 35 to 37 us (0.67 to 0.72), pack 44 us (one byte at a time; 0.33), q8 quantise 45 to
// 47 us (0.64 to 0.67: three blocks of 80 registers to an SM, each waiting for its
// tile before it converts) and dequantise 32 to 34 us (0.88 to 0.94).
//
// 4-bit weights, W (K x N) in groups of `group` k of one column n:
//     hi = max(0, max w), lo = min(0, min w)
//     with zero points:    s = round_type((hi - lo) * (1/15)), z = rint(-lo / s)
//                          (hi * (1/15) - lo * (1/15) where hi - lo is beyond fp32)
//     without:             s = round_type(max |w| * (1/7)),    z = 8
//     q = clamp(rint(w / s) + z, 0, 15), and W is read back as (q - z) * s.
// The scale is rounded to the weights' type before it divides, so the codes fit
// the scale that is kept. w / s is one fp32 multiplication by 1 / s (a full
// division a weight would cost more than its bytes). A group whose scale is
// zero (or below 2^-126, and taken as zero) has q = z (8, or 0 with zero points); a group with a weight that is not
// finite gets a NaN scale and reads back as NaN.
//
// 8-bit activations, X (M x K) in columns of 128 rows: s = max |x| * (1/127),
// q = rint(x / s), the same way; a column of magnitudes below 2^-100 (whose 1/s
// would leave the fp32 range) is saved as zeros with scale 0, a column with a
// value that is not finite as zeros with scale NaN.
#include <cstdint>
#include <cuda_runtime.h>

#include "lowbit.h"
#include "lowbit_types.cuh"

namespace rtm {
namespace lbq {

constexpr int kThreads = 256;
constexpr int TN = 64;       // columns of a 4-bit tile
constexpr int PITCH = 66;    // 2-byte values per tile row in shared memory: the four
                             // quarters of a block (8 rows apart) fall 8 banks apart

// Rounding and conversion by addition, on the full-rate pipe (the conversion
// instructions issue at a quarter of it or less: both directions at 8192 x 8192
// took 90 us with them). 1.5 * 2^23 has ulp 1: adding it rounds a small value to
// the nearest integer, halves to even, and leaves that integer in the low bits.
// 2^23 with an integer in its low bits is the way back.
constexpr float kRound = 12582912.f;
constexpr uint32_t kTwo23 = 0x4b000000u;
constexpr float kTwo23f = 8388608.f;

// Rows k0 .. k0+127, columns n0 .. n0+63 of W into shared memory, zeros outside.
template <typename E, bool VEC>
__device__ __forceinline__ void load_tile(uint16_t (*tile)[PITCH], const E *W, int64_t K, int64_t N,
                                          int64_t k0, int64_t n0)
{
    if constexpr (VEC) {  // 2-byte values, rows on 16-byte boundaries (N % 8 == 0)
        const int seg = threadIdx.x & 7, row = threadIdx.x >> 3;
        uint4 v[4];
#pragma unroll
        for (int p = 0; p < 4; ++p) {
            const int64_t k = k0 + row + 32 * p, n = n0 + seg * 8;
            v[p] = k < K && n < N ? __ldg(reinterpret_cast<const uint4 *>(W + k * N + n))
                                  : make_uint4(0u, 0u, 0u, 0u);
        }
#pragma unroll
        for (int p = 0; p < 4; ++p) {
            uint32_t *d = reinterpret_cast<uint32_t *>(&tile[row + 32 * p][seg * 8]);
            d[0] = v[p].x;
            d[1] = v[p].y;
            d[2] = v[p].z;
            d[3] = v[p].w;
        }
    } else {
        const int col = threadIdx.x & 63;
#pragma unroll 8
        for (int row = threadIdx.x >> 6; row < kW4Block; row += kThreads / TN) {
            const int64_t k = k0 + row, n = n0 + col;
            tile[row][col] = k < K && n < N ? (uint16_t)__ldg(W + k * N + n) : (uint16_t)0;
        }
    }
}

// One block: 64 columns x 128 k. Thread 4 n + c owns the 16-byte quarter c of
// column n's packed block: k = 32 w + 8 c + i in word w, i = 0..7. A group of
// 32, 64 or 128 k is one, two or four whole words of the four quarters, so its
// range is a reduction over a thread's words and two lane exchanges.
template <bool F16, int GROUP, bool ZEROS, bool VEC>
__global__ void __launch_bounds__(kThreads)
    w4_quantize_kernel(int64_t K, int64_t N, const uint16_t *__restrict__ W,
                       uint8_t *__restrict__ codes, uint16_t *__restrict__ scales,
                       uint8_t *__restrict__ zeros)
{
    __shared__ uint16_t tile[kW4Block][PITCH];
    const int64_t tiles_n = (N + TN - 1) / TN;
    const int64_t kb = blockIdx.x / tiles_n, n0 = (blockIdx.x - kb * tiles_n) * TN;
    const int64_t k0 = kb * kW4Block;
    load_tile<uint16_t, VEC>(tile, W, K, N, k0, n0);
    __syncthreads();
    const int c = threadIdx.x & 3, col = threadIdx.x >> 2;
    const int64_t n = n0 + col;
    constexpr int WORDS = GROUP / 32;  // words of a thread in one group
    uint32_t out[4];
#pragma unroll
    for (int g = 0; g < 4 / WORDS; ++g) {
        float v[WORDS][8];
        float hi = 0.f, lo = 0.f, bad = 0.f;  // bad: 0, or NaN once a value is not finite
#pragma unroll
        for (int w = 0; w < WORDS; ++w)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float x = to_f32<F16>(tile[(g * WORDS + w) * 32 + 8 * c + i][col]);
                v[w][i] = x;
                hi = fmaxf(hi, x);
                lo = fminf(lo, x);
                bad = fmaf(x, 0.f, bad);
            }
#pragma unroll
        for (int d = 1; d <= 2; d *= 2) {
            hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, d));
            lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, d));
            bad += __shfl_xor_sync(0xffffffffu, bad, d);
        }
        constexpr float PART = ZEROS ? 1.0f / 15.0f : 1.0f / 7.0f;
        const float range = ZEROS ? hi - lo : fmaxf(hi, -lo);
        float part = __fmul_rn(range, PART);
        if constexpr (ZEROS && !F16)
            if (range > 3.402823466e38f)  // beyond fp32, though hi and lo are not
                part = __fsub_rn(__fmul_rn(hi, PART), __fmul_rn(lo, PART));
        uint16_t sbits = from_f32<F16>(__fadd_rn(part, bad));
        if (to_f32<F16>(sbits) < 0x1p-126f)
            sbits = 0;  // its reciprocal would leave the fp32 range
        const float s = to_f32<F16>(sbits);
        const float inv = s == 0.f ? 0.f : __frcp_rn(s);  // s == 0: every code is the zero point
        float z = 8.f;
        if constexpr (ZEROS)
            z = fminf(fmaxf(rintf(__fmul_rn(-lo, inv)), 0.f), 15.f);
        const float least = kRound - z, most = least + 15.f;  // codes 0 and 15, before z is added
        const uint32_t zi = (uint32_t)z;
#pragma unroll
        for (int w = 0; w < WORDS; ++w) {
            uint32_t word = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float q = __fadd_rn(__fmul_rn(v[w][i], inv), kRound);
                word |= (__float_as_uint(fminf(fmaxf(q, least), most)) + zi & 15u) << w4_shift(i);
            }
            out[g * WORDS + w] = word;
        }
        const int64_t k = k0 + g * GROUP;
        if (c == 0 && n < N && k < K) {
            scales[k / GROUP * N + n] = sbits;
            if constexpr (ZEROS)
                zeros[k / GROUP * N + n] = (uint8_t)zi;
        }
    }
    if (n < N)
        *reinterpret_cast<uint4 *>(codes + n * w4_row_bytes(K) + kb * kW4BlockBytes + c * 16) =
            make_uint4(out[0], out[1], out[2], out[3]);
}

// Codes one to a byte (K x N, the low four bits) into packed blocks.
__global__ void __launch_bounds__(kThreads)
    w4_pack_kernel(int64_t K, int64_t N, const uint8_t *__restrict__ q, uint8_t *__restrict__ codes)
{
    __shared__ uint16_t tile[kW4Block][PITCH];
    const int64_t tiles_n = (N + TN - 1) / TN;
    const int64_t kb = blockIdx.x / tiles_n, n0 = (blockIdx.x - kb * tiles_n) * TN;
    load_tile<uint8_t, false>(tile, q, K, N, kb * kW4Block, n0);
    __syncthreads();
    const int c = threadIdx.x & 3, col = threadIdx.x >> 2;
    uint32_t out[4];
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        out[w] = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            out[w] |= (uint32_t)(tile[w * 32 + 8 * c + i][col] & 15) << w4_shift(i);
    }
    if (n0 + col < N)
        *reinterpret_cast<uint4 *>(codes + (n0 + col) * w4_row_bytes(K) + kb * kW4BlockBytes +
                                   c * 16) = make_uint4(out[0], out[1], out[2], out[3]);
}

// The way back: packed blocks to 2-byte values (q - z) * s, rounded once.
template <bool F16, int GROUP, bool VEC>
__global__ void __launch_bounds__(kThreads)
    w4_dequantize_kernel(int64_t K, int64_t N, const uint8_t *__restrict__ codes,
                         const uint16_t *__restrict__ scales, const uint8_t *__restrict__ zeros,
                         uint16_t *__restrict__ W)
{
    __shared__ uint16_t tile[kW4Block][PITCH];
    const int64_t tiles_n = (N + TN - 1) / TN;
    const int64_t kb = blockIdx.x / tiles_n, n0 = (blockIdx.x - kb * tiles_n) * TN;
    const int64_t k0 = kb * kW4Block;
    const int c = threadIdx.x & 3, col = threadIdx.x >> 2;
    const int64_t n = n0 + col;
    if (n < N) {
        const uint4 v = __ldg(reinterpret_cast<const uint4 *>(codes + n * w4_row_bytes(K) +
                                                              kb * kW4BlockBytes + c * 16));
        const uint32_t words[4] = {v.x, v.y, v.z, v.w};
        float s = 0.f, z = kTwo23f + 8.f;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            if (w % (GROUP / 32) == 0) {
                const int64_t k = k0 + w * 32;
                if (k < K) {
                    s = to_f32<F16>(__ldg(scales + k / GROUP * N + n));
                    if (zeros)
                        z = __uint_as_float(kTwo23 | (__ldg(zeros + k / GROUP * N + n) & 15u));
                }
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float q = __uint_as_float(and_or(words[w] >> w4_shift(i), 15u, kTwo23));
                tile[w * 32 + 8 * c + i][col] = from_f32<F16>((q - z) * s);
            }
        }
    }
    __syncthreads();
    if constexpr (VEC) {
        const int seg = threadIdx.x & 7, row = threadIdx.x >> 3;
#pragma unroll
        for (int p = 0; p < 4; ++p) {
            const int64_t k = k0 + row + 32 * p, nn = n0 + seg * 8;
            const uint32_t *d = reinterpret_cast<const uint32_t *>(&tile[row + 32 * p][seg * 8]);
            if (k < K && nn < N)
                *reinterpret_cast<uint4 *>(W + k * N + nn) = make_uint4(d[0], d[1], d[2], d[3]);
        }
    } else {
        const int cc = threadIdx.x & 63;
#pragma unroll 4
        for (int row = threadIdx.x >> 6; row < kW4Block; row += kThreads / TN)
            if (k0 + row < K && n0 + cc < N)
                W[(k0 + row) * N + n0 + cc] = tile[row][cc];
    }
}

// ---------------------------------------------------------------- 8 bits
// One block: 128 rows x 128 columns; 16 threads span a row (8 columns each),
// 16 rows a pass, 8 passes held in registers between the range and the codes.
constexpr int QN = 128;

template <bool VEC>
__device__ __forceinline__ uint4 load8(const uint16_t *row, int64_t col, int64_t K)
{
    if constexpr (VEC)
        return col < K ? __ldg(reinterpret_cast<const uint4 *>(row + col))
                       : make_uint4(0u, 0u, 0u, 0u);
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const uint32_t a = col + 2 * j < K ? __ldg(row + col + 2 * j) : 0;
        const uint32_t b = col + 2 * j + 1 < K ? __ldg(row + col + 2 * j + 1) : 0;
        w[j] = a | b << 16;
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

template <bool F16, bool VEC>
__global__ void __launch_bounds__(kThreads)
    q8_quantize_kernel(int64_t M, int64_t K, const uint16_t *__restrict__ X,
                       int8_t *__restrict__ codes, float *__restrict__ scales)
{
    __shared__ uint4 tops[8][16];  // per warp: the largest |x| bits of its rows, 8 columns a thread
    const int64_t tiles_k = (K + QN - 1) / QN;
    const int64_t mb = blockIdx.x / tiles_k, c0 = (blockIdx.x - mb * tiles_k) * QN;
    const int seg = threadIdx.x & 15, r0 = threadIdx.x >> 4;
    const int64_t col = c0 + seg * 8, m0 = mb * kQ8Rows;
    uint4 v[8];
#pragma unroll
    for (int p = 0; p < 8; ++p) {
        const int64_t m = m0 + r0 + 16 * p;
        v[p] = m < M ? load8<VEC>(X + m * K, col, K) : make_uint4(0u, 0u, 0u, 0u);
    }
    // Magnitudes compared as 16-bit integers: the order of the values, with
    // infinities above every finite value and NaNs above those.
    uint4 top = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
    for (int p = 0; p < 8; ++p) {
        top.x = __vmaxu2(top.x, v[p].x & 0x7fff7fffu);
        top.y = __vmaxu2(top.y, v[p].y & 0x7fff7fffu);
        top.z = __vmaxu2(top.z, v[p].z & 0x7fff7fffu);
        top.w = __vmaxu2(top.w, v[p].w & 0x7fff7fffu);
    }
    top.x = __vmaxu2(top.x, __shfl_xor_sync(0xffffffffu, top.x, 16));
    top.y = __vmaxu2(top.y, __shfl_xor_sync(0xffffffffu, top.y, 16));
    top.z = __vmaxu2(top.z, __shfl_xor_sync(0xffffffffu, top.z, 16));
    top.w = __vmaxu2(top.w, __shfl_xor_sync(0xffffffffu, top.w, 16));
    if ((threadIdx.x & 31) < 16)
        tops[threadIdx.x >> 5][seg] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < 8; ++w) {
        const uint4 t = tops[w][seg];
        top.x = __vmaxu2(top.x, t.x);
        top.y = __vmaxu2(top.y, t.y);
        top.z = __vmaxu2(top.z, t.z);
        top.w = __vmaxu2(top.w, t.w);
    }
    const uint32_t tw[4] = {top.x, top.y, top.z, top.w};
    float inv[8];
    uint32_t keep[4] = {~0u, ~0u, ~0u, ~0u};  // of two columns each: 0 where the scale is NaN
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const float amax = to_f32<F16>((uint16_t)(tw[j >> 1] >> (16 * (j & 1))));
        float s = __fmul_rn(amax, 1.0f / 127.0f);
        s = amax < 0x1p-100f ? 0.f : amax <= 3.402823466e38f ? s : __int_as_float(0x7fffffff);
        inv[j] = s > 0.f ? __frcp_rn(s) : 0.f;  // codes 0 for scales of 0 and NaN
        if (!(s >= 0.f))
            keep[j >> 1] &= j & 1 ? 0x0000ffffu : 0xffff0000u;
        if (r0 == 0 && col + j < K)
            scales[mb * K + col + j] = s;
    }
    const int64_t pitch = q8_pitch(K);
    if (col >= pitch)
        return;
#pragma unroll
    for (int p = 0; p < 8; ++p) {
        const int64_t m = m0 + r0 + 16 * p;
        if (m >= M)
            break;
        const uint32_t w[4] = {v[p].x & keep[0], v[p].y & keep[1], v[p].z & keep[2],
                               v[p].w & keep[3]};
        uint32_t q[8];  // the code in the low byte
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float x = to_f32<F16>((uint16_t)(w[j >> 1] >> (16 * (j & 1))));
            const float r = __fadd_rn(__fmul_rn(x, inv[j]), kRound);
            q[j] = __float_as_uint(fminf(fmaxf(r, kRound - 127.f), kRound + 127.f));
        }
        auto four = [](uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
            return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
        };
        *reinterpret_cast<uint2 *>(codes + m * pitch + col) =
            make_uint2(four(q[0], q[1], q[2], q[3]), four(q[4], q[5], q[6], q[7]));
    }
}

template <bool F16, bool VEC>
__global__ void __launch_bounds__(kThreads)
    q8_dequantize_kernel(int64_t M, int64_t K, const int8_t *__restrict__ codes,
                         const float *__restrict__ scales, uint16_t *__restrict__ X)
{
    const int64_t tiles_k = (K + QN - 1) / QN;
    const int64_t mb = blockIdx.x / tiles_k, c0 = (blockIdx.x - mb * tiles_k) * QN;
    const int seg = threadIdx.x & 15, r0 = threadIdx.x >> 4;
    const int64_t col = c0 + seg * 8, m0 = mb * kQ8Rows, pitch = q8_pitch(K);
    if (col >= K)
        return;
    uint2 v[8];
#pragma unroll
    for (int p = 0; p < 8; ++p) {
        const int64_t m = m0 + r0 + 16 * p;
        v[p] = m < M ? __ldg(reinterpret_cast<const uint2 *>(codes + m * pitch + col))
                     : make_uint2(0u, 0u);
    }
    float s[8];
#pragma unroll
    for (int j = 0; j < 8; ++j)
        s[j] = col + j < K ? __ldg(scales + mb * K + col + j) : 0.f;
#pragma unroll
    for (int p = 0; p < 8; ++p) {
        const int64_t m = m0 + r0 + 16 * p;
        if (m >= M)
            break;
        float x[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {  // code + 128 in the low byte of 2^23
            const uint32_t u = __byte_perm((j < 4 ? v[p].x : v[p].y) ^ 0x80808080u, kTwo23,
                                           0x7440 | (j & 3));
            x[j] = (__uint_as_float(u) - (kTwo23f + 128.f)) * s[j];
        }
        uint16_t *dst = X + m * K + col;
        if constexpr (VEC) {
            *reinterpret_cast<uint4 *>(dst) =
                make_uint4(pack2_f32<F16>(x[0], x[1]), pack2_f32<F16>(x[2], x[3]),
                           pack2_f32<F16>(x[4], x[5]), pack2_f32<F16>(x[6], x[7]));
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (col + j < K)
                    dst[j] = from_f32<F16>(x[j]);
        }
    }
}

// Tiles of rows x cols, 128 x `width` each, as a one-dimensional grid; 0 if
// there are more than a grid holds.
static unsigned grid_tiles(int64_t rows, int64_t cols, int width)
{
    const int64_t tiles = (rows + 127) / 128 * ((cols + width - 1) / width);
    return tiles <= 0x7fffffff ? (unsigned)tiles : 0u;
}

static bool rows16(const void *p, int64_t cols)
{
    return cols % 8 == 0 && (reinterpret_cast<uintptr_t>(p) & 15) == 0;
}

template <bool F16, int GROUP>
static void quantize_group(unsigned grid, int64_t K, int64_t N, const uint16_t *W, uint8_t *codes,
                           uint16_t *scales, uint8_t *zeros, cudaStream_t s)
{
    const bool vec = rows16(W, N);
    if (zeros && vec)
        w4_quantize_kernel<F16, GROUP, true, true><<<grid, kThreads, 0, s>>>(K, N, W, codes, scales, zeros);
    else if (zeros)
        w4_quantize_kernel<F16, GROUP, true, false><<<grid, kThreads, 0, s>>>(K, N, W, codes, scales, zeros);
    else if (vec)
        w4_quantize_kernel<F16, GROUP, false, true><<<grid, kThreads, 0, s>>>(K, N, W, codes, scales, zeros);
    else
        w4_quantize_kernel<F16, GROUP, false, false><<<grid, kThreads, 0, s>>>(K, N, W, codes, scales, zeros);
}

template <bool F16, int GROUP>
static void dequantize_group(unsigned grid, int64_t K, int64_t N, const uint8_t *codes,
                             const uint16_t *scales, const uint8_t *zeros, uint16_t *W,
                             cudaStream_t s)
{
    if (rows16(W, N))
        w4_dequantize_kernel<F16, GROUP, true><<<grid, kThreads, 0, s>>>(K, N, codes, scales, zeros, W);
    else
        w4_dequantize_kernel<F16, GROUP, false><<<grid, kThreads, 0, s>>>(K, N, codes, scales, zeros, W);
}

} // namespace lbq

cudaError_t launch_w4_quantize(int64_t K, int64_t N, int group, int f16, const uint16_t *W,
                               uint8_t *codes, uint16_t *scales, uint8_t *zeros,
                               cudaStream_t stream)
{
    using namespace lbq;
    const unsigned grid = grid_tiles(K, N, TN);
    if (!grid)
        return cudaErrorInvalidValue;
    auto fn = f16 ? (group == 32   ? quantize_group<true, 32>
                     : group == 64 ? quantize_group<true, 64>
                                   : quantize_group<true, 128>)
                  : (group == 32   ? quantize_group<false, 32>
                     : group == 64 ? quantize_group<false, 64>
                                   : quantize_group<false, 128>);
    fn(grid, K, N, W, codes, scales, zeros, stream);
    return cudaGetLastError();
}

cudaError_t launch_w4_pack(int64_t K, int64_t N, const uint8_t *q, uint8_t *codes,
                           cudaStream_t stream)
{
    using namespace lbq;
    const unsigned grid = grid_tiles(K, N, TN);
    if (!grid)
        return cudaErrorInvalidValue;
    w4_pack_kernel<<<grid, kThreads, 0, stream>>>(K, N, q, codes);
    return cudaGetLastError();
}

cudaError_t launch_w4_dequantize(int64_t K, int64_t N, int group, int f16, const uint8_t *codes,
                                 const uint16_t *scales, const uint8_t *zeros, uint16_t *W,
                                 cudaStream_t stream)
{
    using namespace lbq;
    const unsigned grid = grid_tiles(K, N, TN);
    if (!grid)
        return cudaErrorInvalidValue;
    auto fn = f16 ? (group == 32   ? dequantize_group<true, 32>
                     : group == 64 ? dequantize_group<true, 64>
                                   : dequantize_group<true, 128>)
                  : (group == 32   ? dequantize_group<false, 32>
                     : group == 64 ? dequantize_group<false, 64>
                                   : dequantize_group<false, 128>);
    fn(grid, K, N, codes, scales, zeros, W, stream);
    return cudaGetLastError();
}

cudaError_t launch_q8_quantize(int64_t M, int64_t K, int f16, const uint16_t *X, int8_t *codes,
                               float *scales, cudaStream_t stream)
{
    using namespace lbq;
    const unsigned grid = grid_tiles(M, K, QN);
    if (!grid)
        return cudaErrorInvalidValue;
    const bool vec = rows16(X, K);
    auto fn = f16 ? (vec ? q8_quantize_kernel<true, true> : q8_quantize_kernel<true, false>)
                  : (vec ? q8_quantize_kernel<false, true> : q8_quantize_kernel<false, false>);
    fn<<<grid, kThreads, 0, stream>>>(M, K, X, codes, scales);
    return cudaGetLastError();
}

cudaError_t launch_q8_dequantize(int64_t M, int64_t K, int f16, const int8_t *codes,
                                 const float *scales, uint16_t *X, cudaStream_t stream)
{
    using namespace lbq;
    const unsigned grid = grid_tiles(M, K, QN);
    if (!grid)
        return cudaErrorInvalidValue;
    const bool vec = rows16(X, K);
    auto fn = f16 ? (vec ? q8_dequantize_kernel<true, true> : q8_dequantize_kernel<true, false>)
                  : (vec ? q8_dequantize_kernel<false, true> : q8_dequantize_kernel<false, false>);
    fn<<<grid, kThreads, 0, stream>>>(M, K, codes, scales, X);
    return cudaGetLastError();
}

} // namespace rtm
