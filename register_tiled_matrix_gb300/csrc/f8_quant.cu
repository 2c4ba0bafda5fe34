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
// A block of 256 threads owns 128 columns of 16 P rows: thread (tid & 15, tid >> 4) holds eight
// neighbouring columns of P rows 16 apart in registers, so X is read once whatever is made of
// it. A row's maximum meets in 16 lanes, a column's in registers, two lanes and shared memory.
// Maxima are of the magnitudes' bits: their order is the values', and a NaN exceeds all.
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "f8.h"

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

__device__ __forceinline__ uint2 codes8(const float (&v)[8], float inv, bool nil)
{
    if (nil)
        return make_uint2(0u, 0u);
    return make_uint2(codes2(v[0] * inv, v[1] * inv) | codes2(v[2] * inv, v[3] * inv) << 16,
                      codes2(v[4] * inv, v[5] * inv) | codes2(v[6] * inv, v[7] * inv) << 16);
}

__device__ __forceinline__ uint32_t magnitude(float v) { return __float_as_uint(v) & 0x7fffffffu; }

template <int TYPE>
__device__ __forceinline__ float load1(const void *X, int64_t i)
{
    if constexpr (TYPE == kF32)
        return static_cast<const float *>(X)[i];
    else if constexpr (TYPE == kBf16)
        return __bfloat162float(static_cast<const __nv_bfloat16 *>(X)[i]);
    else
        return __half2float(static_cast<const __half *>(X)[i]);
}

// Eight values from i on; i's address on 16 bytes.
template <int TYPE>
__device__ __forceinline__ void load8(const void *X, int64_t i, float (&v)[8])
{
    if constexpr (TYPE == kF32) {
        const float4 *p = reinterpret_cast<const float4 *>(static_cast<const float *>(X) + i);
        const float4 a = __ldg(p), b = __ldg(p + 1);
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
        v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    } else {
        const uint4 a =
            __ldg(reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(X) + i));
        const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if constexpr (TYPE == kBf16) {
                v[2 * j] = __uint_as_float(w[j] << 16);
                v[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
            } else {
                const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w[j]));
                v[2 * j] = f.x;
                v[2 * j + 1] = f.y;
            }
        }
    }
}

struct Params {
    int64_t M, K, source, fan;  // M: rows of one matrix
    const void *X;
    const int32_t *rows;
    const float *factors;
    uint8_t *row_codes, *col_codes;  // kTiles: row_codes, row_scales
    float *row_scales, *col_scales;
    int64_t col_blocks, row_blocks;  // of one matrix
    int vec;  // X's rows on 16-byte boundaries
};

enum Kind { kRows = 1, kColumns = 2, kBoth = 3, kTiles = 4 };

template <int TYPE, int KIND, int P>
__global__ void __launch_bounds__(kThreads) f8_quantize_kernel(const Params p)
{
    constexpr bool DOWN = KIND != kRows;  // a scale spans rows
    static_assert(!DOWN || P == 8, "128 rows");
    __shared__ uint32_t top_of[DOWN ? 8 : 1][DOWN ? 128 : 1];
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4, warp = threadIdx.x >> 5;
    const int64_t cb = blockIdx.x % p.col_blocks, all = blockIdx.x / p.col_blocks;
    const int64_t rb = KIND == kTiles ? all % p.row_blocks : all;
    const int64_t e = KIND == kTiles ? all / p.row_blocks : 0;
    const int64_t c0 = cb * kF8Block + tx * 8;
    const int64_t r0 = rb * (16 * P) + ty;
    const int64_t base = e * p.M;  // first row of this matrix
    const int64_t pitch = f8_pitch(p.K);

    float v[P][8];
#pragma unroll
    for (int i = 0; i < P; ++i) {
        const int64_t r = r0 + 16 * i;
#pragma unroll
        for (int j = 0; j < 8; ++j)
            v[i][j] = 0.f;
        if (r >= p.M)
            continue;
        int64_t from = base + r;
        float factor = 1.f;
        if (KIND != kTiles && p.rows) {
            const int64_t slot = __ldg(p.rows + r);
            from = slot / p.fan;
            if (slot < 0 || from >= p.source)
                continue;
            if (p.factors)
                factor = __ldg(p.factors + slot);
        }
        if (p.vec && c0 + 8 <= p.K) {
            load8<TYPE>(p.X, from * p.K + c0, v[i]);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (c0 + j < p.K)
                    v[i][j] = load1<TYPE>(p.X, from * p.K + c0 + j);
        }
        if (KIND != kTiles && p.factors) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                v[i][j] = fmaf(v[i][j], factor, 0.f);  // one rounding; no -0 past the row's end
        }
    }

    if constexpr (KIND & kRows) {
#pragma unroll
        for (int i = 0; i < P; ++i) {
            uint32_t top = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j)
                top = max(top, magnitude(v[i][j]));
#pragma unroll
            for (int m = 1; m < 16; m *= 2)
                top = max(top, __shfl_xor_sync(0xffffffffu, top, m));
            const Scale s = scale_of(top);
            const int64_t r = r0 + 16 * i;
            if (r < p.M) {
                if (c0 < pitch)
                    *reinterpret_cast<uint2 *>(p.row_codes + r * pitch + c0) =
                        codes8(v[i], s.inv, s.nil);
                if (tx == 0)
                    p.row_scales[r * p.col_blocks + cb] = s.s;
            }
        }
    }

    if constexpr (DOWN) {
        uint32_t top[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            top[j] = 0;
#pragma unroll
            for (int i = 0; i < P; ++i)
                top[j] = max(top[j], magnitude(v[i][j]));
            top[j] = max(top[j], __shfl_xor_sync(0xffffffffu, top[j], 16));
        }
        if ((threadIdx.x & 16) == 0) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                top_of[warp][tx * 8 + j] = top[j];
        }
        __syncthreads();
        if (threadIdx.x < 128) {
            uint32_t t = top_of[0][threadIdx.x];
#pragma unroll
            for (int w = 1; w < 8; ++w)
                t = max(t, top_of[w][threadIdx.x]);
            if constexpr (KIND == kTiles)
                t = __reduce_max_sync(0xffffffffu, t);
            top_of[0][threadIdx.x] = t;
            const int64_t c = cb * kF8Block + threadIdx.x;
            if (KIND != kTiles && c < p.K)
                p.col_scales[rb * p.K + c] = scale_of(t).s;
        }
        __syncthreads();
        if constexpr (KIND == kTiles) {
            const Scale s = scale_of(max(max(top_of[0][0], top_of[0][32]),
                                         max(top_of[0][64], top_of[0][96])));
            if (threadIdx.x == 0)
                p.row_scales[(e * p.row_blocks + rb) * p.col_blocks + cb] = s.s;
#pragma unroll
            for (int i = 0; i < P; ++i) {
                const int64_t r = r0 + 16 * i;
                if (r < p.M && c0 < pitch)
                    *reinterpret_cast<uint2 *>(p.row_codes + (base + r) * pitch + c0) =
                        codes8(v[i], s.inv, s.nil);
            }
        } else {
            float inv[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const Scale s = scale_of(top_of[0][tx * 8 + j]);
                inv[j] = s.inv;
                if (s.nil) {
#pragma unroll
                    for (int i = 0; i < P; ++i)
                        v[i][j] = 0.f;
                }
            }
#pragma unroll
            for (int i = 0; i < P; ++i) {
                const int64_t r = r0 + 16 * i;
                if (r >= p.M || c0 >= pitch)
                    continue;
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    v[i][j] *= inv[j];
                *reinterpret_cast<uint2 *>(p.col_codes + r * pitch + c0) =
                    codes8(v[i], 1.f, false);
            }
        }
    }
}

template <int KIND, int P>
static cudaError_t launch_kind(int type, const Params &p, int64_t blocks, cudaStream_t stream)
{
    if (blocks > 0x7fffffff)
        return cudaErrorInvalidValue;
    const unsigned grid = (unsigned)blocks;
    if (type == kF32)
        f8_quantize_kernel<kF32, KIND, P><<<grid, kThreads, 0, stream>>>(p);
    else if (type == kBf16)
        f8_quantize_kernel<kBf16, KIND, P><<<grid, kThreads, 0, stream>>>(p);
    else
        f8_quantize_kernel<kF16, KIND, P><<<grid, kThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

static bool rows_on_16(int type, const void *X, int64_t K)
{
    return K * (type == kF32 ? 4 : 2) % 16 == 0 && (reinterpret_cast<uintptr_t>(X) & 15) == 0;
}

// Sixteen codes a thread.
struct BackParams {
    int64_t rows, M, K, ld, chunks;  // rows: of all matrices; chunks of 16 codes a row
    const uint8_t *codes;
    const float *scales;
    void *X;
    int bm_shift, bk_shift;
    int64_t row_blocks, col_blocks;
    int vec;  // X's rows on 16-byte boundaries
};

template <int TYPE>
__global__ void __launch_bounds__(kThreads) f8_dequantize_kernel(const BackParams p)
{
    const int64_t at = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (at >= p.rows * p.chunks)
        return;
    const int64_t r = at / p.chunks, c0 = (at - r * p.chunks) * 16;
    const int64_t e = r / p.M, m = r - e * p.M;
    const float *s = p.scales + (e * p.row_blocks + (m >> p.bm_shift)) * p.col_blocks;
    const uint8_t *q = p.codes + r * p.ld + c0;
    uint32_t word[4] = {0, 0, 0, 0};
    if (c0 + 16 <= p.K) {
        const uint4 w = __ldg(reinterpret_cast<const uint4 *>(q));  // rows lie on 16 bytes
        word[0] = w.x, word[1] = w.y, word[2] = w.z, word[3] = w.w;
    } else {
#pragma unroll
        for (int j = 0; j < 16; ++j)
            if (c0 + j < p.K)
                word[j / 4] |= (uint32_t)__ldg(q + j) << (8 * (j & 3));
    }
    float v[16];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        uint32_t h;
        const uint16_t two = (uint16_t)(word[j / 2] >> (16 * (j & 1)));
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(two));
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h));
        v[2 * j] = f.x;
        v[2 * j + 1] = f.y;
    }
    const int64_t left = p.K - c0;
#pragma unroll
    for (int j = 0; j < 16; ++j)
        if (j < left)
            v[j] *= __ldg(s + ((c0 + j) >> p.bk_shift));
    const int64_t to = r * p.K + c0;
    if (p.vec && left >= 16) {
        if constexpr (TYPE == kF32) {
            float4 *x = reinterpret_cast<float4 *>(static_cast<float *>(p.X) + to);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                x[j] = make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
        } else {
            uint32_t o[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                if constexpr (TYPE == kBf16) {
                    const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
                    o[j] = *reinterpret_cast<const uint32_t *>(&b);
                } else {
                    const __half2 b = __floats2half2_rn(v[2 * j], v[2 * j + 1]);
                    o[j] = *reinterpret_cast<const uint32_t *>(&b);
                }
            }
            uint4 *x = reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p.X) + to);
            x[0] = make_uint4(o[0], o[1], o[2], o[3]);
            x[1] = make_uint4(o[4], o[5], o[6], o[7]);
        }
        return;
    }
#pragma unroll
    for (int j = 0; j < 16; ++j)
        if (j < left) {
            if constexpr (TYPE == kF32)
                static_cast<float *>(p.X)[to + j] = v[j];
            else if constexpr (TYPE == kBf16)
                static_cast<__nv_bfloat16 *>(p.X)[to + j] = __float2bfloat16_rn(v[j]);
            else
                static_cast<__half *>(p.X)[to + j] = __float2half_rn(v[j]);
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
    p.fan = L.fan;
    p.X = L.X;
    p.rows = L.rows;
    p.factors = L.factors;
    p.row_codes = L.row_codes;
    p.row_scales = L.row_scales;
    p.col_codes = L.col_codes;
    p.col_scales = L.col_scales;
    p.col_blocks = f8_blocks(L.K);
    p.vec = rows_on_16(L.type, L.X, L.K);
    const int64_t down = f8_blocks(L.M) * p.col_blocks;
    if (L.row_codes && L.col_codes)
        return launch_kind<kBoth, 8>(L.type, p, down, stream);
    if (L.col_codes)
        return launch_kind<kColumns, 8>(L.type, p, down, stream);
    return launch_kind<kRows, 1>(L.type, p, (L.M + 15) / 16 * p.col_blocks, stream);
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
    return launch_kind<kTiles, 8>(type, p, E * p.row_blocks * p.col_blocks, stream);
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
    p.chunks = (K + 15) / 16;
    p.codes = codes;
    p.scales = scales;
    p.X = X;
    p.bm_shift = bm == 1 ? 0 : 7;
    p.bk_shift = bk == 1 ? 0 : 7;
    p.row_blocks = bm == 1 ? M : f8_blocks(M);
    p.col_blocks = bk == 1 ? K : f8_blocks(K);
    p.vec = rows_on_16(type, X, K);
    const int64_t blocks = (p.rows * p.chunks + kThreads - 1) / kThreads;
    if (blocks > 0x7fffffff)
        return cudaErrorInvalidValue;
    const unsigned grid = (unsigned)blocks;
    if (type == kF32)
        f8_dequantize_kernel<kF32><<<grid, kThreads, 0, stream>>>(p);
    else if (type == kBf16)
        f8_dequantize_kernel<kBf16><<<grid, kThreads, 0, stream>>>(p);
    else
        f8_dequantize_kernel<kF16><<<grid, kThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

} // namespace rtm
