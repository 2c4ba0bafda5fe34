// C = A.W for few rows of A (a decoded token, a small batch) and W in 4 bits:
//
//     C[m][n] = sum_g s[g][n] * sum_{k in g} A[m][k] * (q[k][n] - z[g][n])
//
// Every weight is used M times, so the product is bound by the weights' bytes
// (8192 x 8192: 35 MB, 5.2 us at the measured HBM rate) as long as decoding them
// costs few instructions. mma.sync m16n8k16 takes 16 columns of W on its row side
// and 8 rows of A on its column side: with one row of A seven eighths of the
// product is zeros, but the tensor core has the time, and a weight costs about
// one and a half integer instructions where a multiplication of its own in
// fp32 would add a conversion and an addition.
//
// A block of 8 warps owns 16 T columns of W (rows of its packed form); warp w
// takes the 128-deep blocks w, w + 8, .. of k, so the warps together read 512
// consecutive bytes of each row. A lane loads 16 bytes of a row: the packing
// puts word w of quarter c at k = 32 w + 8 c, so a word's eight codes are the
// operand rows of two instructions, whose other operand is the 16 bytes of A at
// the same k. Codes, scales and zero points are copied to shared memory several
// blocks ahead (asynchronous copies that each lane makes and waits for itself),
// A is loaded one block ahead.
// Integers (codes minus zero point) are exact in both types; the group's sum
// is fp32 and is scaled when it is added to the fp32 total. The eight warps'
// totals are added in order through shared memory.
#include <cstdint>
#include <cuda_runtime.h>

#include "kernels.h"
#include "lowbit.h"
#include "lowbit_types.cuh"
#include "ptx.cuh"

namespace rtm {
namespace w4r {

constexpr int kWarps = 8, kThreads = 32 * kWarps;

template <bool F16>
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1)
{
    if constexpr (F16)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, "
                     "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, "
                     "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Eight consecutive values of a row of A from k, zeros from `left` values on.
// V: values per load (8, 2 or 1), the most that rows of K values allow.
template <int V>
__device__ __forceinline__ uint4 load_values(const uint16_t *p, int left)
{
    if (left <= 0)
        return make_uint4(0u, 0u, 0u, 0u);
    if constexpr (V == 8)  // K % 8 == 0: all or none
        return __ldg(reinterpret_cast<const uint4 *>(p));
    uint32_t w[4] = {};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (V == 2) {
            w[i] = 2 * i < left ? __ldg(reinterpret_cast<const uint32_t *>(p) + i) : 0u;
        } else {
            const uint32_t lo = 2 * i < left ? __ldg(p + 2 * i) : 0;
            const uint32_t hi = 2 * i + 1 < left ? __ldg(p + 2 * i + 1) : 0;
            w[i] = lo | hi << 16;
        }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// A warp's ring in shared memory: per block of k and 16 columns the lanes' codes
// (16 bytes of rows r and r + 8) and the words that hold their scales and zero
// points. Each lane copies and reads its own bytes.
template <int T>
struct Ring {
    static constexpr int DEPTH = T == 1 ? 6 : 4;
    static constexpr uint32_t META = T * 2 * 512;             // codes come first
    static constexpr uint32_t SLOT = META + T * 2 * 2 * 128;  // 1.5 KB for each 16 columns
    static constexpr uint32_t BYTES = kWarps * DEPTH * SLOT;
};

template <bool F16, int T, int NB, int V>
__global__ void __launch_bounds__(kThreads, T * NB == 1 ? 3 : T * NB == 4 && V < 8 ? 1 : 2)
    w4_rows_kernel(const W4Launch p, int gs)
{
    using R = Ring<T>;
    extern __shared__ __align__(16) uint8_t ring[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int r = lane >> 2, c = lane & 3;
    const int n0 = blockIdx.x * (16 * T), m0 = blockIdx.y * (8 * NB);
    const int blocks = (p.K + kW4Block - 1) / kW4Block;
    const int G = (p.K + p.group - 1) >> gs;
    const int per_block = 7 - gs;  // log2 of the groups of a block
    const uint32_t mine = smem_u32(ring) + warp * R::DEPTH * R::SLOT;
    const int64_t pitch = w4_row_bytes(p.K);
    // Columns past the end read the last one's bytes; they are not stored.
    const uint8_t *row[T][2];
    uint32_t col[T][2];
#pragma unroll
    for (int t = 0; t < T; ++t)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            col[t][h] = (uint32_t)min(n0 + 16 * t + 8 * h + r, p.N - 1);
            row[t][h] = p.codes + col[t][h] * pitch + c * 16;
        }
    // Each of a row's four lanes holds one group's scale and zero point of a
    // block (of 1, 2 or 4 groups); the others get it by a lane exchange. A scale
    // (2 bytes) and a zero point (1 byte) are copied with the aligned word around them.
    const int own = c & ((1 << per_block) - 1);
    auto fetch = [&](int b, int slot) {
        if (b < blocks) {
            const uint32_t dst = mine + slot * R::SLOT;
            const int64_t at = (int64_t)min((b << per_block) + own, G - 1) * p.N;
#pragma unroll
            for (int t = 0; t < T; ++t)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int i = 2 * t + h;
                    cp_async_16_full(dst + i * 512 + lane * 16, row[t][h] + (int64_t)b * kW4BlockBytes);
                    const uintptr_t sp = reinterpret_cast<uintptr_t>(p.scales + at + col[t][h]);
                    cp_async_4_full(dst + R::META + i * 256 + lane * 4,
                                    reinterpret_cast<const void *>(sp & ~uintptr_t(3)));
                    if (p.zeros) {
                        const uintptr_t zp = reinterpret_cast<uintptr_t>(p.zeros + at + col[t][h]);
                        cp_async_4_full(dst + R::META + i * 256 + 128 + lane * 4,
                                        reinterpret_cast<const void *>(zp & ~uintptr_t(3)));
                    }
                }
        }
        cp_async_commit();
    };
    uint4 x[NB][4];  // A at the block's four words; each is loaded a block ahead of its use
    auto load_x = [&](int b, int w) {
#pragma unroll
        for (int j = 0; j < NB; ++j) {
            const int m = m0 + 8 * j + r, k = b * kW4Block + 32 * w + 8 * c;
            x[j][w] = load_values<V>(p.A + (int64_t)m * p.K + k, m < p.M ? p.K - k : 0);
        }
    };
    float total[T][NB][4] = {}, sum[T][NB][4] = {};
    int b = warp, slot = 0;
#pragma unroll 1
    for (int a = 0; a < R::DEPTH - 1; ++a)
        fetch(b + a * kWarps, a);
#pragma unroll
    for (int w = 0; w < 4; ++w)
        load_x(b, w);
#pragma unroll 1
    for (; b < blocks; b += kWarps) {
        cp_async_wait<R::DEPTH - 2>();
        const uint32_t src = mine + slot * R::SLOT;
        uint4 q[T][2];
        uint32_t scale[T][2], zero[T][2], zz[T][2];
        const int gl = (b << per_block) + own;
        const int64_t at = (int64_t)min(gl, G - 1) * p.N;
#pragma unroll
        for (int t = 0; t < T; ++t)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int i = 2 * t + h;
                q[t][h] = lds128(src + i * 512 + lane * 16);
                const uint32_t sp =
                    (uint32_t)reinterpret_cast<uintptr_t>(p.scales) + 2 * (uint32_t)(at + col[t][h]);
                scale[t][h] = lds32(src + R::META + i * 256 + lane * 4) >> (8 * (sp & 2));
                if (gl >= G)
                    scale[t][h] = 0;  // codes of k >= K: sums of zeros
                zero[t][h] = 8;
                if (p.zeros) {
                    const uint32_t zp =
                        (uint32_t)reinterpret_cast<uintptr_t>(p.zeros) + (uint32_t)(at + col[t][h]);
                    zero[t][h] =
                        (lds32(src + R::META + i * 256 + 128 + lane * 4) >> (8 * (zp & 3))) & 15u;
                }
            }
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            if ((w * 32 & (p.group - 1)) == 0)
#pragma unroll
                for (int t = 0; t < T; ++t)
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        zz[t][h] = magic2<F16>() |
                                   __shfl_sync(0xffffffffu, zero[t][h],
                                               (lane & 28) | ((w * 32) >> gs)) * 0x00010001u;
#pragma unroll
            for (int t = 0; t < T; ++t) {
                const uint4 &qa = q[t][0], &qb = q[t][1];
                const uint4 va = w4_values<F16>(w == 0 ? qa.x : w == 1 ? qa.y : w == 2 ? qa.z : qa.w,
                                                zz[t][0]);
                const uint4 vb = w4_values<F16>(w == 0 ? qb.x : w == 1 ? qb.y : w == 2 ? qb.z : qb.w,
                                                zz[t][1]);
#pragma unroll
                for (int j = 0; j < NB; ++j) {
                    mma16816<F16>(sum[t][j], va.x, vb.x, va.y, vb.y, x[j][w].x, x[j][w].y);
                    mma16816<F16>(sum[t][j], va.z, vb.z, va.w, vb.w, x[j][w].z, x[j][w].w);
                }
            }
            load_x(b + kWarps, w);
            if (((w + 1) * 32 & (p.group - 1)) == 0)
#pragma unroll
                for (int t = 0; t < T; ++t) {
                    float s[2];
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        s[h] = to_f32<F16>((uint16_t)__shfl_sync(0xffffffffu, scale[t][h],
                                                                 (lane & 28) | ((w * 32) >> gs)));
#pragma unroll
                    for (int j = 0; j < NB; ++j)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            total[t][j][e] = fmaf(s[e >> 1], sum[t][j][e], total[t][j][e]);
                            sum[t][j][e] = 0.f;
                        }
                }
        }
        // The slot read in the block before this one (its words are long used).
        fetch(b + (R::DEPTH - 1) * kWarps, slot == 0 ? R::DEPTH - 1 : slot - 1);
        slot = slot + 1 == R::DEPTH ? 0 : slot + 1;
    }
    cp_async_wait<0>();
    __syncthreads();
    float(*red)[16 * T][8 * NB + 1] = reinterpret_cast<float(*)[16 * T][8 * NB + 1]>(ring);
#pragma unroll
    for (int t = 0; t < T; ++t)
#pragma unroll
        for (int j = 0; j < NB; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                red[warp][16 * t + 8 * (e >> 1) + r][8 * j + 2 * c + (e & 1)] = total[t][j][e];
    __syncthreads();
    for (int i = threadIdx.x; i < 16 * T * 8 * NB; i += kThreads) {
        const int nn = i % (16 * T), mm = i / (16 * T);
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w)
            v += red[w][nn][mm];
        if (n0 + nn < p.N && m0 + mm < p.M)
            p.C[(int64_t)(m0 + mm) * p.N + n0 + nn] = v;
    }
}

template <bool F16, int T, int NB, int V>
static cudaError_t launch_kernel(const W4Launch &L, dim3 grid, int gs, cudaStream_t stream)
{
    using R = Ring<T>;
    static_assert(kWarps * 16 * T * (8 * NB + 1) * 4 <= R::BYTES, "the totals fit the ring");
    auto kernel = w4_rows_kernel<F16, T, NB, V>;
    static std::atomic<uint64_t> done{0};
    const cudaError_t e = set_smem_limit_once(kernel, (int)R::BYTES, done, 100);
    if (e != cudaSuccess)
        return e;
    kernel<<<grid, kThreads, R::BYTES, stream>>>(L, gs);
    return cudaGetLastError();
}

template <bool F16, int T, int NB>
static cudaError_t launch_v(const W4Launch &L, dim3 grid, int gs, cudaStream_t stream)
{
    const uintptr_t a = reinterpret_cast<uintptr_t>(L.A);
    if (L.K % 8 == 0 && a % 16 == 0)
        return launch_kernel<F16, T, NB, 8>(L, grid, gs, stream);
    if (L.K % 2 == 0 && a % 4 == 0)
        return launch_kernel<F16, T, NB, 2>(L, grid, gs, stream);
    return launch_kernel<F16, T, NB, 1>(L, grid, gs, stream);
}

template <bool F16>
static cudaError_t launch_f(const W4Launch &L, int sms, cudaStream_t stream)
{
    const int gs = L.group == 32 ? 5 : L.group == 64 ? 6 : 7;
    const bool two = L.M > 8;
    const int nb = two ? 2 : 1;
    // 32 columns a block while that still gives every SM two blocks.
    const int t = (L.N + 31) / 32 >= 2 * sms ? 2 : 1;
    const dim3 grid((unsigned)((L.N + 16 * t - 1) / (16 * t)), (unsigned)((L.M + 8 * nb - 1) / (8 * nb)));
    if (t == 2)
        return two ? launch_v<F16, 2, 2>(L, grid, gs, stream)
                   : launch_v<F16, 2, 1>(L, grid, gs, stream);
    return two ? launch_v<F16, 1, 2>(L, grid, gs, stream)
               : launch_v<F16, 1, 1>(L, grid, gs, stream);
}

} // namespace w4r

cudaError_t launch_w4_rows(const W4Launch &L, int sms, cudaStream_t stream)
{
    return L.f16 ? w4r::launch_f<true>(L, sms, stream) : w4r::launch_f<false>(L, sms, stream);
}

} // namespace rtm
