// Values to e4m3 codes with a scale for each block of 128, and back.
//
//     s = 2^i, the least with max|x| <= 448 * 2^i over the block;  code = e4m3(x / s)
//
// A power of two makes x / s exact, so the code's rounding (half a step of 2^-3, halves to
// even) is the only one, and the same value gets the same code along either axis while the
// scales agree. It costs up to one binade of e4m3's 18, no precision. Blocks are 128 values of
// a row (activations in a product), 128 of a column (the operands of a weight gradient, which
// sums over rows), or 128 x 128 (weights).
//
// A block owns 128 columns of some rows (128 where a scale spans them): thread (tid & 15, tid >> 4)
// holds eight neighbouring columns of P rows in registers, as they came, so X is read once whatever
// is made of it and several blocks fit an SM to cover each other's loads. A row's maximum meets
// in 16 lanes, a column's in registers, two lanes and shared memory. Maxima are of the
// magnitudes' bits, two 16-bit values at a time: their order is the values', and a NaN exceeds all.
#include <atomic>
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "f8.h"
#include "kernels.h"
#include "ptx.cuh"

namespace rtm {
namespace f8q {

constexpr int kThreads = 256;
constexpr uint32_t kTinyBits = 27u << 23;  // 2^-100
constexpr uint32_t kInfBits = 0x7f800000u;

// The scale of a block whose largest magnitude has these bits, and its inverse; both exact.
// Below 2^-100 the scale is 0, with a value that is not finite NaN; the codes are then 0.
struct Scale {
    float s, inv;
    bool nil;
};
__device__ __forceinline__ Scale scale_of(uint32_t top)
{
    if (top >= kInfBits)
        return {__uint_as_float(0x7fc00000u), 0.f, true};
    if (top < kTinyBits)
        return {0.f, 0.f, true};
    const uint32_t e = (top >> 23) - 8 + ((top & 0x7fffffu) > 0x600000u);  // 448 = 1.75 * 2^8
    return {__uint_as_float(e << 23), __uint_as_float((254u - e) << 23), false};
}

__device__ __forceinline__ uint32_t codes2(float a, float b)
{
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %2, %1;" : "=h"(r) : "f"(a), "f"(b));
    return r;
}

// Two products at a time; + 0 makes a -0 a 0, so that the bytes past a row's end are 0.
__device__ __forceinline__ void mul2(float &v0, float &v1, float s0, float s1)
{
    asm("{\n\t.reg .b64 v, s, z;\n\t"
        "mov.b64 v, {%0, %1};\n\t"
        "mov.b64 s, {%2, %3};\n\t"
        "mov.b64 z, {%4, %4};\n\t"
        "fma.rn.f32x2 v, v, s, z;\n\t"
        "mov.b64 {%0, %1}, v;\n\t}\n"
        : "+f"(v0), "+f"(v1)
        : "f"(s0), "f"(s1), "f"(0.f));
}

__device__ __forceinline__ uint2 codes8(const float (&v)[8])
{
    return make_uint2(codes2(v[0], v[1]) | codes2(v[2], v[3]) << 16,
                      codes2(v[4], v[5]) | codes2(v[6], v[7]) << 16);
}

__device__ __forceinline__ uint2 codes8(float (&v)[8], float inv, bool nil)
{
#pragma unroll
    for (int j = 0; j < 8; j += 2)
        mul2(v[j], v[j + 1], inv, inv);
    return nil ? make_uint2(0u, 0u) : codes8(v);
}

// The larger of a and |b|; NaN where one is.
__device__ __forceinline__ float max_magnitude(float a, float b)
{
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(fabsf(b)));
    return d;
}

// Eight values as they lie in memory.
template <int TYPE>
struct Raw {
    static constexpr int WORDS = TYPE == kF32 ? 8 : 4;
    uint32_t w[WORDS];

    __device__ __forceinline__ void clear()
    {
#pragma unroll
        for (int j = 0; j < WORDS; ++j)
            w[j] = 0;
    }
    // From i on; i's address on 16 bytes.
    __device__ __forceinline__ void load(const void *X, int64_t i)
    {
        const uint4 *p = reinterpret_cast<const uint4 *>(static_cast<const uint8_t *>(X) +
                                                         i * (TYPE == kF32 ? 4 : 2));
#pragma unroll
        for (int j = 0; j < WORDS; j += 4) {
            const uint4 a = __ldg(p + j / 4);
            w[j] = a.x, w[j + 1] = a.y, w[j + 2] = a.z, w[j + 3] = a.w;
        }
    }
    // The first n of them.
    __device__ __forceinline__ void load_some(const void *X, int64_t i, int n)
    {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (j < n) {
                if constexpr (TYPE == kF32)
                    w[j] = __ldg(static_cast<const uint32_t *>(X) + i + j);
                else
                    w[j / 2] |= (uint32_t)__ldg(static_cast<const uint16_t *>(X) + i + j) << (16 * (j & 1));
            }
    }
    __device__ __forceinline__ void values(float (&v)[8]) const
    {
#pragma unroll
        for (int j = 0; j < WORDS; ++j) {
            if constexpr (TYPE == kF32) {
                v[j] = __uint_as_float(w[j]);
            } else if constexpr (TYPE == kBf16) {
                v[2 * j] = __uint_as_float(w[j] << 16);
                v[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
            } else {
                const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w[j]));
                v[2 * j] = f.x;
                v[2 * j + 1] = f.y;
            }
        }
    }
};

__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b)  // of two 16-bit halves
{
    uint32_t d;
    asm("max.u16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// The fp32 bits of a 16-bit magnitude.
template <int TYPE>
__device__ __forceinline__ uint32_t widen(uint32_t half)
{
    if constexpr (TYPE == kBf16)
        return half << 16;
    else
        return __float_as_uint(__half2float(__ushort_as_half((unsigned short)half)));
}

struct Params {
    int64_t M, K, source;  // M: rows of one matrix
    uint32_t fan;
    const void *X;
    const int32_t *rows;
    const float *factors;
    uint8_t *row_codes, *col_codes;  // kTiles: row_codes, row_scales
    float *row_scales, *col_scales;
    int64_t col_blocks, row_blocks;  // of one matrix
    int64_t blocks;  // of rows, of all matrices
    int vec;  // X's rows on 16-byte boundaries
};

enum Kind { kRows = 1, kColumns = 2, kBoth = 3, kTiles = 4 };

// Threads of a block: twice as many where a scale spans 128 rows, so that a thread holds four of
// them (eight, and their products by factors, left two blocks of 256 on an SM).
__host__ __device__ constexpr int threads_of(int kind) { return kind == kRows ? 256 : 512; }

template <int TYPE, int KIND, int P, bool FACTORS>
__global__ void __launch_bounds__(threads_of(KIND), KIND == kRows ? 4 : KIND == kTiles ? 1 : TYPE != kF32 && !FACTORS ? 3 : 2)
    f8_quantize_kernel(const Params p)
{
    constexpr bool DOWN = KIND != kRows;  // a scale spans rows
    constexpr bool HALVES = TYPE != kF32 && !FACTORS;  // maxima of 16-bit magnitudes
    constexpr int TOPS = HALVES ? 4 : 8;
    constexpr int SPAN = threads_of(KIND) / 16;  // rows that a block takes at once
    static_assert(!DOWN || P * SPAN == kF8Block, "128 rows");
    constexpr int WARPS = threads_of(KIND) / 32;
    __shared__ uint32_t top_of[DOWN ? WARPS : 1][DOWN ? 128 : 1];
    __shared__ __align__(16) float inverse[DOWN ? 128 : 4];
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4, warp = threadIdx.x >> 5;
    const int cb = blockIdx.x;
    const int64_t all = blockIdx.y + (int64_t)gridDim.y * blockIdx.z;
    if (all >= p.blocks)
        return;
    const int64_t e = KIND == kTiles ? all / p.row_blocks : 0;
    const int64_t rb = KIND == kTiles ? all - e * p.row_blocks : all;
    // Rows and columns are below 2^31; what they address is not.
    const int M = (int)p.M, K = (int)p.K, pitch = (K + 15) & ~15;
    const int c0 = cb * kF8Block + tx * 8, r0 = (int)rb * (SPAN * P) + ty;
    const int64_t base = e * p.M;  // first row of this matrix

    Raw<TYPE> raw[P];
    float factor[FACTORS ? P : 1];
#pragma unroll
    for (int i = 0; i < P; ++i) {
        const int r = r0 + SPAN * i;
        raw[i].clear();
        if constexpr (FACTORS)
            factor[i] = 0.f;
        if (r >= M)
            continue;
        int64_t from = base + r;
        if (KIND != kTiles && p.rows) {
            const int slot = __ldg(p.rows + r);
            from = (uint32_t)slot / p.fan;
            if (slot < 0 || from >= p.source)
                continue;
            if constexpr (FACTORS)
                factor[i] = __ldg(p.factors + slot);
        }
        if (p.vec && c0 + 8 <= K)
            raw[i].load(p.X, from * p.K + c0);
        else
            raw[i].load_some(p.X, from * p.K + c0, K - c0);
    }
    auto values = [&](int i, float (&v)[8]) {
        raw[i].values(v);
        if constexpr (FACTORS) {
#pragma unroll
            for (int j = 0; j < 8; j += 2)
                mul2(v[j], v[j + 1], factor[i], factor[i]);
        }
    };
    auto larger = [](uint32_t a, uint32_t b) { return HALVES ? max2(a, b) : max(a, b); };

    // A row's largest magnitude is that of X's row times the factor's: rounding keeps order.
    // A column's is found among the products.
    uint32_t tops[DOWN ? TOPS : 1];  // of the columns: fp32 bits, or two 16-bit ones a word
    float column[DOWN && !HALVES ? 8 : 1];
#pragma unroll
    for (int j = 0; j < (DOWN ? TOPS : 0); ++j)
        tops[j] = 0;
#pragma unroll
    for (int j = 0; j < (DOWN && !HALVES ? 8 : 0); ++j)
        column[j] = 0.f;
#pragma unroll
    for (int i = 0; i < P; ++i) {
        if constexpr (DOWN && HALVES) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                tops[j] = max2(tops[j], raw[i].w[j] & 0x7fff7fffu);
        } else if constexpr (DOWN) {
            float v[8];
            values(i, v);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                column[j] = max_magnitude(column[j], v[j]);
        }
        if constexpr (KIND & kRows) {
            uint32_t top;
            if constexpr (TYPE != kF32) {
                top = raw[i].w[0] & 0x7fff7fffu;
#pragma unroll
                for (int j = 1; j < 4; ++j)
                    top = max2(top, raw[i].w[j] & 0x7fff7fffu);
#pragma unroll
                for (int o = 1; o < 16; o *= 2)
                    top = max2(top, __shfl_xor_sync(0xffffffffu, top, o));
                top = widen<TYPE>(max(top & 0xffffu, top >> 16));
            } else {
                top = raw[i].w[0] & 0x7fffffffu;
#pragma unroll
                for (int j = 1; j < 8; ++j)
                    top = max(top, raw[i].w[j] & 0x7fffffffu);
#pragma unroll
                for (int o = 1; o < 16; o *= 2)
                    top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
            }
            if constexpr (FACTORS)
                top = __float_as_uint(__uint_as_float(top) * factor[i]) & 0x7fffffffu;
            const Scale s = scale_of(top);
            const int r = r0 + SPAN * i;
            if (r < M) {
                float v[8];
                values(i, v);
                if (c0 < pitch)
                    *reinterpret_cast<uint2 *>(p.row_codes + (int64_t)r * pitch + c0) = codes8(v, s.inv, s.nil);
                if (tx == 0)
                    p.row_scales[(int64_t)r * p.col_blocks + cb] = s.s;
            }
        }
    }
    if constexpr (DOWN && !HALVES) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            tops[j] = __float_as_uint(column[j]);
    }

    if constexpr (DOWN) {
#pragma unroll
        for (int j = 0; j < TOPS; ++j)
            tops[j] = larger(tops[j], __shfl_xor_sync(0xffffffffu, tops[j], 16));
        if ((threadIdx.x & 16) == 0) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                top_of[warp][tx * 8 + j] =
                    HALVES ? widen<TYPE == kF32 ? kBf16 : TYPE>(j & 1 ? tops[j / 2] >> 16
                                                                     : tops[j / 2] & 0xffffu)
                           : tops[j % TOPS];
        }
        __syncthreads();
        bool bad = false;  // a value that is not finite
        if (threadIdx.x < 128) {
            uint32_t t = top_of[0][threadIdx.x];
#pragma unroll
            for (int w = 1; w < WARPS; ++w)
                t = max(t, top_of[w][threadIdx.x]);
            if constexpr (KIND == kTiles) {
                top_of[0][threadIdx.x] = __reduce_max_sync(0xffffffffu, t);
            } else {
                const Scale s = scale_of(t);
                inverse[threadIdx.x] = s.inv;
                bad = t >= kInfBits;
                const int c = cb * kF8Block + threadIdx.x;
                if (c < K)
                    p.col_scales[rb * p.K + c] = s.s;
            }
        }
        bad = __syncthreads_or(bad);
        if constexpr (KIND == kTiles) {
            const Scale s = scale_of(max(max(top_of[0][0], top_of[0][32]),
                                         max(top_of[0][64], top_of[0][96])));
            if (threadIdx.x == 0)
                p.row_scales[(e * p.row_blocks + rb) * p.col_blocks + cb] = s.s;
#pragma unroll
            for (int i = 0; i < P; ++i) {
                const int r = r0 + SPAN * i;
                float v[8];
                values(i, v);
                if (r < M && c0 < pitch)
                    *reinterpret_cast<uint2 *>(p.row_codes + (base + r) * pitch + c0) =
                        codes8(v, s.inv, s.nil);
            }
        } else {
            float inv[8];
#pragma unroll
            for (int j = 0; j < 8; j += 4) {
                const float4 f = *reinterpret_cast<const float4 *>(inverse + tx * 8 + j);
                inv[j] = f.x, inv[j + 1] = f.y, inv[j + 2] = f.z, inv[j + 3] = f.w;
            }
#pragma unroll
            for (int i = 0; i < P; ++i) {
                const int r = r0 + SPAN * i;
                float v[8];
                values(i, v);
                if (bad) {
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        v[j] = inv[j] == 0.f ? 0.f : v[j];
                }
#pragma unroll
                for (int j = 0; j < 8; j += 2)
                    mul2(v[j], v[j + 1], inv[j], inv[j + 1]);
                if (r < M && c0 < pitch)
                    *reinterpret_cast<uint2 *>(p.col_codes + (int64_t)r * pitch + c0) = codes8(v);
            }
        }
    }
}

// Rows alone, of whole sixteens on 32-byte boundaries: a thread takes 16 values in one or two
// 32-byte loads and stores their codes in one of 16 bytes, eight lanes a block, four rows a
// thread. Half the reductions, scales and stores of the kernel above: 8192 x 8192 bf16 39 us
// against 42.
template <int TYPE, bool FACTORS>
__global__ void __launch_bounds__(256) f8_quantize_rows_kernel(const Params p)
{
    constexpr int P = 4, HALVES = TYPE == kF32 ? 2 : 1;  // loads of 32 bytes a row
    const int tx = threadIdx.x & 7, ty = threadIdx.x >> 3;
    const int64_t block = blockIdx.y + (int64_t)gridDim.y * blockIdx.z;
    if (block >= p.blocks)
        return;
    const int M = (int)p.M, K = (int)p.K, cb = blockIdx.x;
    const int c0 = cb * kF8Block + tx * 16, r0 = (int)block * (32 * P) + ty;

    uint32_t raw[P][8 * HALVES];
    float factor[FACTORS ? P : 1];
#pragma unroll
    for (int i = 0; i < P; ++i) {
        const int r = r0 + 32 * i;
#pragma unroll
        for (int j = 0; j < 8 * HALVES; ++j)
            raw[i][j] = 0;
        if constexpr (FACTORS)
            factor[i] = 0.f;
        if (r >= M || c0 >= K)
            continue;
        int64_t from = r;
        if (p.rows) {
            const int slot = __ldg(p.rows + r);
            from = (uint32_t)slot / p.fan;
            if (slot < 0 || from >= p.source)
                continue;
            if constexpr (FACTORS)
                factor[i] = __ldg(p.factors + slot);
        }
        const uint8_t *x = static_cast<const uint8_t *>(p.X) + (from * p.K + c0) * (TYPE == kF32 ? 4 : 2);
#pragma unroll
        for (int h = 0; h < HALVES; ++h) {
            uint32_t(&w)[8] = *reinterpret_cast<uint32_t(*)[8]>(raw[i] + 8 * h);
            asm("ld.global.nc.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]),
                  "=r"(w[6]), "=r"(w[7])
                : "l"(x + 32 * h));
        }
    }
#pragma unroll
    for (int i = 0; i < P; ++i) {
        uint32_t top = 0;
        if constexpr (TYPE == kF32) {
#pragma unroll
            for (int j = 0; j < 16; ++j)
                top = max(top, raw[i][j] & 0x7fffffffu);
#pragma unroll
            for (int o = 1; o < 8; o *= 2)
                top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                top = max2(top, raw[i][j] & 0x7fff7fffu);
#pragma unroll
            for (int o = 1; o < 8; o *= 2)
                top = max2(top, __shfl_xor_sync(0xffffffffu, top, o));
            top = widen<TYPE>(max(top & 0xffffu, top >> 16));
        }
        if constexpr (FACTORS)
            top = __float_as_uint(__uint_as_float(top) * factor[i]) & 0x7fffffffu;
        const Scale s = scale_of(top);
        uint2 q[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float v[8];
            Raw<TYPE> eight;
#pragma unroll
            for (int j = 0; j < Raw<TYPE>::WORDS; ++j)
                eight.w[j] = raw[i][h * Raw<TYPE>::WORDS + j];
            eight.values(v);
            if constexpr (FACTORS) {
#pragma unroll
                for (int j = 0; j < 8; j += 2)
                    mul2(v[j], v[j + 1], factor[i], factor[i]);
            }
            q[h] = codes8(v, s.inv, s.nil);
        }
        const int r = r0 + 32 * i;
        if (r < M) {
            if (c0 < K)
                *reinterpret_cast<uint4 *>(p.row_codes + (int64_t)r * K + c0) =
                    make_uint4(q[0].x, q[0].y, q[1].x, q[1].y);
            if (tx == 0)
                p.row_scales[(int64_t)r * p.col_blocks + cb] = s.s;
        }
    }
}

// Scales that span rows, for rows of whole sixteens on 16-byte boundaries: the 128 x 128 values
// of a block are copied to shared memory, 16 bytes at a time and zeros where there are none, and
// read there once for the maxima and the row codes and once for the other codes. Held in
// registers they leave two or three blocks on an SM; so it has five (fp32 three), which cover each
// other's copies. A thread has 16 columns of four rows. us, and with the kernel above: 8192 x 8192
// bf16 columns 41 (49), both 51 (64), tiles 36 (50); 32768 gathered rows of 2048, both ways, 59
// (80), with factors 66 (84); fp32 tiles 57 (82). fp32 columns 66 (61) and both 80 (73) stay
// above: their values take half an SM's shared memory twice over, and no more are in flight.
template <int TYPE>
struct Staged {
    static constexpr int SIZE = TYPE == kF32 ? 4 : 2, CHUNKS = 8 * SIZE;  // of 16 bytes in 128 values
    static constexpr uint32_t ROW = 128 * SIZE, BYTES = 128 * ROW;
    // Chunk c of a row: the chunks that eight lanes read at once lie in different banks.
    __device__ static uint32_t at(int row, int c)
    {
        return row * ROW + ((TYPE == kF32 ? c ^ (c >> 3 & 3) : c ^ (c >> 3 & 1)) << 4);
    }
};

template <int TYPE, int KIND, bool FACTORS>
__global__ void __launch_bounds__(256, TYPE == kF32 ? 3 : 5)
    f8_quantize_staged_kernel(const Params p)
{
    using St = Staged<TYPE>;
    constexpr int P = 4, SPAN = 32, WARPS = 8;  // rows of a thread, SPAN apart
    constexpr bool PAIRS = TYPE != kF32 && !FACTORS;  // columns' maxima of 16-bit magnitudes, two a word
    constexpr int TOPS = PAIRS ? 8 : 16, WORDS = TYPE == kF32 ? 16 : 8;
    extern __shared__ __align__(16) uint8_t staged[];
    __shared__ __align__(16) uint32_t top_of[WARPS][8 * TOPS];
    __shared__ __align__(16) float inverse[128];
    __shared__ float factors[FACTORS ? 128 : 1];
    const int64_t all = blockIdx.y + (int64_t)gridDim.y * blockIdx.z;
    if (all >= p.blocks)
        return;
    const int64_t e = KIND == kTiles ? all / p.row_blocks : 0;
    const int64_t rb = KIND == kTiles ? all - e * p.row_blocks : all;
    const int64_t base = e * p.M;  // first row of this matrix
    const int M = (int)p.M, K = (int)p.K, cb = blockIdx.x, row0 = (int)rb * kF8Block;
    const uint32_t to = (uint32_t)__cvta_generic_to_shared(staged);
    {
        constexpr int STEP = 256 / St::CHUNKS;  // rows copied at once
        const int chunk = threadIdx.x % St::CHUNKS, c = cb * kF8Block + chunk * (16 / St::SIZE);
#pragma unroll
        for (int i = 0; i < 128 / STEP; ++i) {
            const int l = threadIdx.x / St::CHUNKS + i * STEP, r = row0 + l;
            int64_t from = base + r;
            bool held = r < M && c < K;
            if (KIND != kTiles && held && p.rows) {
                const int slot = __ldg(p.rows + r);
                from = (uint32_t)slot / p.fan;
                held = slot >= 0 && from < p.source;
            }
            const void *x = static_cast<const uint8_t *>(p.X) + (held ? (from * p.K + c) * St::SIZE : 0);
            cp_async_16(to + St::at(l, chunk), x, held ? 16u : 0u);
        }
        cp_async_commit();
    }
    const int tx = threadIdx.x & 7, ty = threadIdx.x >> 3;
    const int c0 = cb * kF8Block + tx * 16, r0 = row0 + ty;
    if constexpr (FACTORS) {
        if (threadIdx.x < 128) {
            const int r = row0 + threadIdx.x, slot = r < M ? __ldg(p.rows + r) : -1;
            factors[threadIdx.x] =
                slot >= 0 && (uint32_t)slot / p.fan < p.source ? __ldg(p.factors + slot) : 0.f;
        }
    }
    cp_async_wait<0>();
    __syncthreads();
    // Words of row i, as they came.
    auto read = [&](int i, uint32_t (&w)[WORDS]) {
#pragma unroll
        for (int q = 0; q < WORDS / 4; ++q) {
            const uint4 a = *reinterpret_cast<const uint4 *>(staged + St::at(ty + SPAN * i, tx * (WORDS / 4) + q));
            w[4 * q] = a.x, w[4 * q + 1] = a.y, w[4 * q + 2] = a.z, w[4 * q + 3] = a.w;
        }
    };
    // Eight of them, times the row's factor.
    auto values = [&](const uint32_t (&w)[WORDS], int i, int h, float (&v)[8]) {
        Raw<TYPE> eight;
#pragma unroll
        for (int j = 0; j < WORDS / 2; ++j)
            eight.w[j] = w[h * (WORDS / 2) + j];
        eight.values(v);
        if constexpr (FACTORS) {
#pragma unroll
            for (int j = 0; j < 8; j += 2)
                mul2(v[j], v[j + 1], factors[ty + SPAN * i], factors[ty + SPAN * i]);
        }
    };

    uint32_t tops[TOPS] = {};  // magnitudes' bits: their order is the values', NaN above all
#pragma unroll(FACTORS ? 2 : P)  // two: registers for five blocks
    for (int i = 0; i < P; ++i) {
        uint32_t w[WORDS];
        read(i, w);
        uint32_t top = 0;
        if constexpr (PAIRS) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                tops[j] = max2(tops[j], w[j] & 0x7fff7fffu);
        }
        if constexpr (KIND & kRows) {
            if constexpr (TYPE == kF32) {
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    top = max(top, w[j] & 0x7fffffffu);
#pragma unroll
                for (int o = 1; o < 8; o *= 2)
                    top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    top = max2(top, w[j] & 0x7fff7fffu);
#pragma unroll
                for (int o = 1; o < 8; o *= 2)
                    top = max2(top, __shfl_xor_sync(0xffffffffu, top, o));
                top = widen<TYPE>(max(top & 0xffffu, top >> 16));
            }
            // That of X's row times the factor's is the products': rounding keeps order.
            if constexpr (FACTORS)
                top = __float_as_uint(__uint_as_float(top) * factors[ty + SPAN * i]) & 0x7fffffffu;
        }
        const Scale s = scale_of(top);
        uint2 q[2];
        if constexpr (!PAIRS || (KIND & kRows)) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float v[8];
                values(w, i, h, v);
                if constexpr (!PAIRS) {
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        tops[8 * h + j] = max(tops[8 * h + j], __float_as_uint(v[j]) & 0x7fffffffu);
                }
                if constexpr (KIND & kRows)
                    q[h] = codes8(v, s.inv, s.nil);
            }
        }
        if constexpr (KIND & kRows) {
            const int r = r0 + SPAN * i;
            if (r < M) {
                if (c0 < K)
                    *reinterpret_cast<uint4 *>(p.row_codes + (int64_t)r * K + c0) =
                        make_uint4(q[0].x, q[0].y, q[1].x, q[1].y);
                if (tx == 0)
                    p.row_scales[(int64_t)r * p.col_blocks + cb] = s.s;
            }
        }
    }
#pragma unroll
    for (int j = 0; j < TOPS; ++j)
#pragma unroll
        for (int o = 8; o < 32; o *= 2) {
            const uint32_t t = __shfl_xor_sync(0xffffffffu, tops[j], o);
            tops[j] = PAIRS ? max2(tops[j], t) : max(tops[j], t);
        }
    if ((threadIdx.x & 31) < 8) {
#pragma unroll
        for (int j = 0; j < TOPS; j += 4)
            *reinterpret_cast<uint4 *>(&top_of[threadIdx.x >> 5][tx * TOPS + j]) =
                make_uint4(tops[j], tops[j + 1], tops[j + 2], tops[j + 3]);
    }
    __syncthreads();
    bool bad = false;  // a value that is not finite
    if (threadIdx.x < 8 * TOPS) {
        uint32_t t = top_of[0][threadIdx.x];
#pragma unroll
        for (int w = 1; w < WARPS; ++w)
            t = PAIRS ? max2(t, top_of[w][threadIdx.x]) : max(t, top_of[w][threadIdx.x]);
        if constexpr (KIND == kTiles) {
            top_of[0][threadIdx.x] =
                __reduce_max_sync(0xffffffffu, PAIRS ? widen<TYPE == kF32 ? kBf16 : TYPE>(max(t & 0xffffu, t >> 16)) : t);
        } else {
#pragma unroll
            for (int j = 0; j < (PAIRS ? 2 : 1); ++j) {
                const uint32_t bits = PAIRS ? widen<TYPE == kF32 ? kBf16 : TYPE>(j ? t >> 16 : t & 0xffffu) : t;
                const int at = PAIRS ? 2 * threadIdx.x + j : threadIdx.x;
                const Scale s = scale_of(bits);
                inverse[at] = s.inv;
                bad |= bits >= kInfBits;
                if (cb * kF8Block + at < K)
                    p.col_scales[rb * p.K + cb * kF8Block + at] = s.s;
            }
        }
    }
    bad = __syncthreads_or(bad);
    uint8_t *codes = p.col_codes;
    Scale tile;
    if constexpr (KIND == kTiles) {
        uint32_t t = 0;
#pragma unroll
        for (int j = 0; j < 8 * TOPS; j += 32)
            t = max(t, top_of[0][j]);
        tile = scale_of(t);
        if (threadIdx.x == 0)
            p.row_scales[(e * p.row_blocks + rb) * p.col_blocks + cb] = tile.s;
        bad = tile.nil;
        codes = p.row_codes;
    }
    float inv[16];
#pragma unroll
    for (int j = 0; j < 16; j += 4) {
        float4 f;
        if constexpr (KIND == kTiles)
            f = make_float4(tile.inv, tile.inv, tile.inv, tile.inv);
        else
            f = *reinterpret_cast<const float4 *>(inverse + tx * 16 + j);
        inv[j] = f.x, inv[j + 1] = f.y, inv[j + 2] = f.z, inv[j + 3] = f.w;
    }
#pragma unroll
    for (int i = 0; i < P; ++i) {
        uint32_t w[WORDS];
        read(i, w);
        uint2 q[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float v[8];
            values(w, i, h, v);
            if (bad) {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    v[j] = inv[8 * h + j] == 0.f ? 0.f : v[j];
            }
#pragma unroll
            for (int j = 0; j < 8; j += 2)
                mul2(v[j], v[j + 1], inv[8 * h + j], inv[8 * h + j + 1]);
            q[h] = codes8(v);
        }
        const int r = r0 + SPAN * i;
        if (r < M && c0 < K)
            *reinterpret_cast<uint4 *>(codes + (base + r) * K + c0) =
                make_uint4(q[0].x, q[0].y, q[1].x, q[1].y);
    }
}

template <int TYPE, int KIND, bool FACTORS>
static cudaError_t launch_staged(const Params &p, cudaStream_t stream)
{
    auto kernel = f8_quantize_staged_kernel<TYPE, KIND, FACTORS>;
    static std::atomic<uint64_t> done{0};
    const cudaError_t e = set_smem_limit_once(kernel, (int)Staged<TYPE>::BYTES, done);
    if (e != cudaSuccess)
        return e;
    const int64_t y = p.blocks < 65535 ? p.blocks : 65535, z = (p.blocks + y - 1) / y;
    if (z > 65535 || p.col_blocks > 0x7fffffff)
        return cudaErrorInvalidValue;
    kernel<<<dim3((unsigned)p.col_blocks, (unsigned)y, (unsigned)z), 256, Staged<TYPE>::BYTES, stream>>>(p);
    return cudaGetLastError();
}

template <bool FACTORS>
static cudaError_t launch_rows(int type, Params p, cudaStream_t stream)
{
    p.blocks = (p.M + 127) / 128;
    const int64_t y = p.blocks < 65535 ? p.blocks : 65535, z = (p.blocks + y - 1) / y;
    if (z > 65535 || p.col_blocks > 0x7fffffff)
        return cudaErrorInvalidValue;
    const dim3 grid((unsigned)p.col_blocks, (unsigned)y, (unsigned)z);
    if (type == kF32)
        f8_quantize_rows_kernel<kF32, FACTORS><<<grid, 256, 0, stream>>>(p);
    else if (type == kBf16)
        f8_quantize_rows_kernel<kBf16, FACTORS><<<grid, 256, 0, stream>>>(p);
    else
        f8_quantize_rows_kernel<kF16, FACTORS><<<grid, 256, 0, stream>>>(p);
    return cudaGetLastError();
}

template <int KIND, int P, bool FACTORS>
static cudaError_t launch_kind(int type, Params p, int64_t blocks, cudaStream_t stream)
{
    if constexpr (KIND != kRows) {
        if (p.K % 16 == 0 && p.vec) {
            p.blocks = blocks;
            if (type == kBf16)
                return launch_staged<kBf16, KIND, FACTORS>(p, stream);
            if (type == kF16)
                return launch_staged<kF16, KIND, FACTORS>(p, stream);
            if constexpr (KIND == kTiles)
                return launch_staged<kF32, KIND, FACTORS>(p, stream);
        }
    }
    const int64_t y = blocks < 65535 ? blocks : 65535, z = (blocks + y - 1) / y;
    if (z > 65535 || p.col_blocks > 0x7fffffff)
        return cudaErrorInvalidValue;
    p.blocks = blocks;
    const dim3 grid((unsigned)p.col_blocks, (unsigned)y, (unsigned)z);
    if (type == kF32)
        f8_quantize_kernel<kF32, KIND, P, FACTORS><<<grid, threads_of(KIND), 0, stream>>>(p);
    else if (type == kBf16)
        f8_quantize_kernel<kBf16, KIND, P, FACTORS><<<grid, threads_of(KIND), 0, stream>>>(p);
    else
        f8_quantize_kernel<kF16, KIND, P, FACTORS><<<grid, threads_of(KIND), 0, stream>>>(p);
    return cudaGetLastError();
}

template <bool FACTORS>
static cudaError_t launch_rows_and_columns(int type, const Params &p, cudaStream_t stream)
{
    const int64_t down = f8_blocks(p.M);
    if (p.row_codes && p.col_codes)
        return launch_kind<kBoth, 4, FACTORS>(type, p, down, stream);
    if (p.col_codes)
        return launch_kind<kColumns, 4, FACTORS>(type, p, down, stream);
    // Four rows a thread, whose loads cover each other, where that still makes many blocks: 8192 x
    // 8200 bf16 44 us against 52, at the least size 2048 x 8200 17.5 against 19.6, below it the
    // same (1024 x 8192 13.4). Rows off 16 bytes are loaded value by value, one row a thread:
    // 8192 x 8191 58 us against 62.
    if (p.M * p.col_blocks >= 64 * 2048 && p.vec) {
        if (p.K % 16 == 0 && (reinterpret_cast<uintptr_t>(p.X) & 31) == 0)
            return launch_rows<FACTORS>(type, p, stream);
        return launch_kind<kRows, 4, FACTORS>(type, p, (p.M + 63) / 64, stream);
    }
    return launch_kind<kRows, 1, FACTORS>(type, p, (p.M + 15) / 16, stream);
}

static bool rows_on_16(int type, const void *X, int64_t K)
{
    return K * (type == kF32 ? 4 : 2) % 16 == 0 && (reinterpret_cast<uintptr_t>(X) & 15) == 0;
}

// A warp takes 512 codes of a row, a thread V at a time 32 * V apart, so that loads and stores
// of a warp are whole lines: eight where rows of X are whole eights on 32-byte boundaries
// (8192 x 8192 by columns to fp32 70 us in fours, 57 in eights; by rows to bf16 43, 40), else four.
struct BackParams {
    int64_t rows, M, K, ld, chunks;  // rows: of all matrices; chunks of 512 codes a row
    const uint8_t *codes;
    const float *scales;
    void *X;
    int bm_shift, bk_shift;
    int64_t row_blocks, col_blocks;
    int vec;  // X's rows on 16-byte boundaries
};

template <int TYPE, int V>
__global__ void __launch_bounds__(kThreads) f8_dequantize_kernel(const BackParams p)
{
    constexpr int STEPS = 16 / V, WORDS = V / 4;
    const int lane = threadIdx.x & 31;
    const int64_t at = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    if (at >= p.rows * p.chunks)
        return;
    const int64_t r = at / p.chunks, e = r / p.M, m = r - e * p.M;
    const int64_t c0 = (at - r * p.chunks) * 512 + lane * V;
    const float *s = p.scales + (e * p.row_blocks + (m >> p.bm_shift)) * p.col_blocks;
    const uint8_t *q = p.codes + r * p.ld;
    uint32_t word[STEPS][WORDS];
#pragma unroll
    for (int i = 0; i < STEPS; ++i) {
        const int64_t c = c0 + 32 * V * i;
#pragma unroll
        for (int j = 0; j < WORDS; ++j)
            word[i][j] = 0;
        if (c + V <= p.K) {  // rows lie on 16 bytes
            if constexpr (V == 8) {
                const uint2 w = __ldg(reinterpret_cast<const uint2 *>(q + c));
                word[i][0] = w.x, word[i][1] = w.y;
            } else {
                word[i][0] = __ldg(reinterpret_cast<const uint32_t *>(q + c));
            }
        } else if constexpr (V == 4) {  // (rows of whole eights end with one)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (c + j < p.K)
                    word[i][0] |= (uint32_t)__ldg(q + c + j) << (8 * j);
        }
    }
#pragma unroll
    for (int i = 0; i < STEPS; ++i) {
        const int64_t c = c0 + 32 * V * i, left = p.K - c;
        if (left <= 0)
            return;
        float v[V];
#pragma unroll
        for (int j = 0; j < V / 2; ++j) {
            uint32_t h;
            const uint16_t two = (uint16_t)(word[i][j / 2] >> (16 * (j & 1)));
            asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(two));
            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h));
            v[2 * j] = f.x;
            v[2 * j + 1] = f.y;
        }
        if (p.bk_shift) {
            const float one = __ldg(s + (c >> p.bk_shift));
#pragma unroll
            for (int j = 0; j < V; ++j)
                v[j] *= one;
        } else if constexpr (V == 8) {
#pragma unroll
            for (int j = 0; j < 8; j += 4) {
                const float4 f = __ldg(reinterpret_cast<const float4 *>(s + c + j));
                v[j] *= f.x, v[j + 1] *= f.y, v[j + 2] *= f.z, v[j + 3] *= f.w;
            }
        } else {
#pragma unroll
            for (int j = 0; j < V; ++j)
                if (j < left)
                    v[j] *= __ldg(s + c + j);
        }
        const int64_t to = r * p.K + c;
        if (V == 8 || (p.vec && left >= 4)) {
            if constexpr (TYPE == kF32) {
                float *x = static_cast<float *>(p.X) + to;
                if constexpr (V == 8)
                    asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};"
                                 :: "l"(x), "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]),
                                    "f"(v[5]), "f"(v[6]), "f"(v[7]) : "memory");
                else
                    *reinterpret_cast<float4 *>(x) = make_float4(v[0], v[1], v[2], v[3]);
            } else {
                uint32_t o[V / 2];
#pragma unroll
                for (int j = 0; j < V / 2; ++j) {
                    if constexpr (TYPE == kBf16) {
                        const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
                        o[j] = *reinterpret_cast<const uint32_t *>(&b);
                    } else {
                        const __half2 b = __floats2half2_rn(v[2 * j], v[2 * j + 1]);
                        o[j] = *reinterpret_cast<const uint32_t *>(&b);
                    }
                }
                uint16_t *x = static_cast<uint16_t *>(p.X) + to;
                if constexpr (V == 8)
                    *reinterpret_cast<uint4 *>(x) = make_uint4(o[0], o[1], o[2], o[3]);
                else
                    *reinterpret_cast<uint2 *>(x) = make_uint2(o[0], o[1]);
            }
        } else {
#pragma unroll
            for (int j = 0; j < V; ++j)
                if (j < left) {
                    if constexpr (TYPE == kF32)
                        static_cast<float *>(p.X)[to + j] = v[j];
                    else if constexpr (TYPE == kBf16)
                        static_cast<__nv_bfloat16 *>(p.X)[to + j] = __float2bfloat16_rn(v[j]);
                    else
                        static_cast<__half *>(p.X)[to + j] = __float2half_rn(v[j]);
                }
        }
    }
}

} // namespace f8q

cudaError_t launch_f8_quantize(const F8QuantLaunch &L, cudaStream_t stream)
{
    using namespace f8q;
    Params p = {};
    p.M = L.M;
    p.K = L.K;
    p.source = L.source;
    p.fan = (uint32_t)L.fan;
    p.X = L.X;
    p.rows = L.rows;
    p.factors = L.factors;
    p.row_codes = L.row_codes;
    p.row_scales = L.row_scales;
    p.col_codes = L.col_codes;
    p.col_scales = L.col_scales;
    p.col_blocks = f8_blocks(L.K);
    p.vec = rows_on_16(L.type, L.X, L.K);
    return L.factors ? launch_rows_and_columns<true>(L.type, p, stream)
                     : launch_rows_and_columns<false>(L.type, p, stream);
}

cudaError_t launch_f8_quantize_tiles(int64_t E, int64_t K, int64_t N, int type, const void *W,
                                     uint8_t *codes, float *scales, cudaStream_t stream)
{
    using namespace f8q;
    Params p = {};
    p.M = K;
    p.K = N;
    p.X = W;
    p.row_codes = codes;
    p.row_scales = scales;
    p.row_blocks = f8_blocks(K);
    p.col_blocks = f8_blocks(N);
    p.vec = rows_on_16(type, W, N);
    return launch_kind<kTiles, 4, false>(type, p, E * p.row_blocks, stream);
}

cudaError_t launch_f8_dequantize(int64_t E, int64_t M, int64_t K, int bm, int bk, int type,
                                 const uint8_t *codes, int64_t ld, const float *scales, void *X,
                                 cudaStream_t stream)
{
    using namespace f8q;
    BackParams p = {};
    p.rows = E * M;
    p.M = M;
    p.K = K;
    p.ld = ld;
    p.chunks = (K + 511) / 512;
    p.codes = codes;
    p.scales = scales;
    p.X = X;
    p.bm_shift = bm == 1 ? 0 : 7;
    p.bk_shift = bk == 1 ? 0 : 7;
    p.row_blocks = bm == 1 ? M : f8_blocks(M);
    p.col_blocks = bk == 1 ? K : f8_blocks(K);
    p.vec = rows_on_16(type, X, K);
    const int64_t blocks = (p.rows * p.chunks + kThreads / 32 - 1) / (kThreads / 32);
    if (blocks > 0x7fffffff)
        return cudaErrorInvalidValue;
    const bool eights = K % 8 == 0 && (reinterpret_cast<uintptr_t>(X) & 31) == 0 &&
                        (bk != 1 || (reinterpret_cast<uintptr_t>(scales) & 15) == 0);
    auto launch = [&](auto kernel) { kernel<<<(unsigned)blocks, kThreads, 0, stream>>>(p); };
    if (type == kF32)
        launch(eights ? f8_dequantize_kernel<kF32, 8> : f8_dequantize_kernel<kF32, 4>);
    else if (type == kBf16)
        launch(eights ? f8_dequantize_kernel<kBf16, 8> : f8_dequantize_kernel<kBf16, 4>);
    else
        launch(eights ? f8_dequantize_kernel<kF16, 8> : f8_dequantize_kernel<kF16, 4>);
    return cudaGetLastError();
}

} // namespace rtm
