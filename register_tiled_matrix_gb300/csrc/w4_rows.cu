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
// blocks of k ahead, A with them, by asynchronous copies that each lane makes and
// waits for itself.
// Integers (codes minus zero point) are exact in both types; the group's sum
// is fp32 and is scaled when it is added to the fp32 total. The eight warps'
// totals are added in order through shared memory.
//
// What bounds it: 1 x 32768 x 8192 takes 33.0 us in a graph (35 us call by call), 0.59
// to 0.63 of the measured copy rate (1 x 8192 x 8192 12.1 to 12.6 us, 16 x 8192 x 8192
// 17.5 to 18.1 us, 1 x 1024 x 1024 2.1 us in a graph). 16 columns x 128 k cost 167 warp
// instructions (88 decode), half of the issue slots; without decoding and multiplying
// the copies of this launch alone took 31 to 35 us, whether a lane group took 64 bytes
// of a row or a whole line, with rings of four or eight blocks: at K = 8192 a warp has
// eight blocks of k, so a block of threads spends much of its time filling and draining
// its rings, and 1 x 8192 x 8192 ends in a second wave of a few blocks. Tried and no faster: a range of k to a warp in place of every eighth
// block (35 to 41 us), clusters over k, shifts on the multiplier pipe (43.6 us).
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

// Eight 4-bit codes minus their zero point, in order. nz: -(magic + z), twice.
// fp16 has mantissa bits to spare: a code four bits up adds 16 times itself to
// 1024, and one fused multiply-add takes it down and subtracts 64 + z (nz16),
// exactly, which saves two of the three shifts.
template <bool F16>
__device__ __forceinline__ uint4 values_of(uint32_t word, uint32_t nz, uint32_t nz16)
{
    auto low = [&](uint32_t w) {
        const uint32_t v = and_or(w, 0x000f000fu, magic2<F16>());
        uint32_t d;
        if constexpr (F16)
            asm("add.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(v), "r"(nz));
        else
            asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(v), "r"(0x3f803f80u), "r"(nz));
        return d;
    };
    auto up = [&](uint32_t w) {
        uint32_t d;
        asm("fma.rn.f16x2 %0, %1, %2, %3;"
            : "=r"(d)
            : "r"(and_or(w, 0x00f000f0u, 0x64006400u)), "r"(0x2c002c00u), "r"(nz16));
        return d;
    };
    if constexpr (F16)
        return make_uint4(low(word), up(word), low(word >> 8), up(word >> 8));
    else
        return make_uint4(low(word), low(word >> 4), low(word >> 8), low(word >> 12));
}

// Eight consecutive values of a row of A to shared memory, zeros from `left`
// values on. V: values a copy moves, the most that rows of K values allow (8, 2);
// single values (1) have no asynchronous copy and go through registers.
template <int V>
__device__ __forceinline__ void copy_values(uint32_t dst, const uint16_t *p, int left)
{
    if constexpr (V == 8) {  // K % 8 == 0: all or none
        cp_async_16(dst, left > 0 ? p : nullptr, left > 0 ? 16u : 0u);
    } else if constexpr (V == 2) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            cp_async_4(dst + 4 * i, 2 * i < left ? p + 2 * i : nullptr, 2 * i < left ? 4u : 0u);
    } else {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t lo = 2 * i < left ? __ldg(p + 2 * i) : 0;
            const uint32_t hi = 2 * i + 1 < left ? __ldg(p + 2 * i + 1) : 0;
            w[i] = lo | hi << 16;
        }
        asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(dst), "r"(w[0]), "r"(w[1]),
                     "r"(w[2]), "r"(w[3])
                     : "memory");
    }
}

constexpr int DEPTH = 4;  // blocks in a warp's ring, and the unrolling of its loop

// Shared memory of a warp: the scale and zero point of four groups of each
// column, ready for use, and a ring of blocks. A block holds 16 bytes a lane for
// rows r and r + 8 of each 16 columns, then its 128 values of the rows of A (256
// bytes each; odd rows with their 64-byte halves exchanged, so that two rows'
// quarters fall on different banks). Each lane copies and reads its own bytes.
template <int T>
struct Warp {
    static constexpr uint32_t META = 4 * T * 16 * 8;
    static constexpr uint32_t CODES = T * 1024;
};
inline __host__ __device__ constexpr uint32_t slot_bytes(int t, int rows) { return t * 1024 + rows * 256; }
inline __host__ __device__ constexpr uint32_t warp_bytes(int t, int rows)
{
    return 4 * t * 16 * 8 + DEPTH * slot_bytes(t, rows);
}

// GS: log2 of the group. V: see copy_values.
template <bool F16, int T, int NB, int V, int GS>
__global__ void __launch_bounds__(kThreads, NB == 2 ? 1 : T == 1 && V == 8 && GS == 7 ? 3 : 2)
    w4_rows_kernel(const W4Launch p)
{
    constexpr int GROUP = 1 << GS;
    constexpr int GPB = kW4Block / GROUP;  // groups of a block
    constexpr int SPAN = 4 / GPB;          // blocks of this warp that four groups cover
    using S = Warp<T>;
    extern __shared__ __align__(256) uint8_t shared[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int r = lane >> 2, c = lane & 3;
    const int n0 = blockIdx.x * (16 * T);
    const int blocks = (p.K + kW4Block - 1) / kW4Block;
    const int G = (p.K + GROUP - 1) / GROUP;
    const uint32_t slot = slot_bytes(T, p.M);  // M <= 8 NB
    const uint32_t mine = smem_u32(shared) + warp * warp_bytes(T, p.M);
    const uint32_t meta = mine + r * 8;
    const uint32_t ring = mine + S::META, codes = ring + lane * 16;
    // A's values for words 0 and 2 are at xring, + 128; for words 1 and 3 at xother, + 128.
    const uint32_t xring = ring + S::CODES + r * 256 + c * 16 + (r & 1) * 64;
    const uint32_t xother = xring ^ 64u;
    const int64_t pitch = w4_row_bytes(p.K);
    // Columns past the end read the last one's bytes; they are not stored.
    const uint8_t *row[T][2];  // at this warp's first block of the loop's round
    int col[T][2];
#pragma unroll
    for (int t = 0; t < T; ++t)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            col[t][h] = min(n0 + 16 * t + 8 * h + r, p.N - 1);
            row[t][h] = p.codes + col[t][h] * pitch + (int64_t)warp * kW4BlockBytes + c * 16;
        }
    // Rows of A: lanes of rows past M copy and read nothing.
    const uint16_t *a[NB];
    bool in[NB];
#pragma unroll
    for (int j = 0; j < NB; ++j) {
        const int m = 8 * j + r;
        in[j] = m < p.M;
        a[j] = p.A + (int64_t)m * p.K + 8 * c + (int64_t)warp * kW4Block;
    }
    // Copies this warp's block `ahead` of the round (block b) to slot `at`.
    auto fetch = [&](int b, int ahead, int at) {
        if (b < blocks) {
#pragma unroll
            for (int t = 0; t < T; ++t)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    cp_async_16_full(codes + at * slot + (2 * t + h) * 512,
                                     row[t][h] + ahead * (kWarps * kW4BlockBytes));
            const int left = p.K - b * kW4Block - 8 * c;
            const bool whole = (b + 1) * (int64_t)kW4Block <= p.K;
#pragma unroll
            for (int j = 0; j < NB; ++j)
                if (in[j])
#pragma unroll
                    for (int w = 0; w < 4; ++w) {
                        const uint32_t dst =
                            (w & 1 ? xother : xring) + at * slot + j * 2048 + (w & 2) * 64;
                        const uint16_t *src = a[j] + ahead * (kWarps * kW4Block) + 32 * w;
                        if (V == 8 && whole)
                            cp_async_16_full(dst, src);
                        else
                            copy_values<V>(dst, src, left - 32 * w);
                    }
        }
        cp_async_commit();
    };
    // Lane c of a row's four loads the scale and zero point of the c-th of the four
    // groups that begin with block b, one span ahead of their use.
    uint16_t scale[T][2];
    uint8_t zero[T][2];
    auto load_meta = [&](int b) {
        const int g = (b + c / GPB * kWarps) * GPB + c % GPB;
        const int64_t at = (int64_t)g * p.N;
#pragma unroll
        for (int t = 0; t < T; ++t)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                // codes of k >= K: sums of zeros
                scale[t][h] = g < G ? __ldg(p.scales + at + col[t][h]) : (uint16_t)0;
                zero[t][h] = p.zeros && g < G ? __ldg(p.zeros + at + col[t][h]) : (uint8_t)8;
            }
    };
    auto store_meta = [&]() {
        __syncwarp();  // the last span's values have been read
#pragma unroll
        for (int t = 0; t < T; ++t)
#pragma unroll
            for (int h = 0; h < 2; ++h)
                asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(
                                 meta + (c * T * 16 + 16 * t + 8 * h) * 8),
                             "r"(__float_as_uint(to_f32<F16>(scale[t][h]))),
                             "r"(magic2<F16>() | 0x80008000u | (zero[t][h] & 15u) * 0x00010001u)
                             : "memory");
        __syncwarp();
    };
    uint4 x[NB][4];  // lanes of rows past M keep zeros
#pragma unroll
    for (int j = 0; j < NB; ++j)
#pragma unroll
        for (int w = 0; w < 4; ++w)
            x[j][w] = make_uint4(0u, 0u, 0u, 0u);
    float total[T][NB][4] = {};
#pragma unroll
    for (int i = 0; i < DEPTH - 1; ++i)
        fetch(warp + i * kWarps, i, i);
    load_meta(warp);
#pragma unroll 1
    for (int b0 = warp; b0 < blocks; b0 += DEPTH * kWarps) {
#pragma unroll
        for (int i = 0; i < DEPTH; ++i) {
            const int b = b0 + i * kWarps;
            if (b >= blocks)
                break;
            if (i % SPAN == 0) {
                store_meta();
                load_meta(b + SPAN * kWarps);
            }
            cp_async_wait<DEPTH - 2>();
            uint4 q[T][2];
#pragma unroll
            for (int t = 0; t < T; ++t)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    q[t][h] = lds128(codes + i * slot + (2 * t + h) * 512);
            float sum[T][NB][4], s[T][2];
            uint32_t nz[T][2], nz16[T][2];  // -(magic + z); fp16: -(64 + z)
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                const bool begin = w * 32 % GROUP == 0, end = (w + 1) * 32 % GROUP == 0;
                const int group = i % SPAN * GPB + w * 32 / GROUP;  // of the span's four
#pragma unroll
                for (int j = 0; j < NB; ++j)
                    if (in[j])
                        x[j][w] = lds128((w & 1 ? xother : xring) + i * slot + j * 2048 + (w & 2) * 64);
#pragma unroll
                for (int t = 0; t < T; ++t) {
                    if (begin)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];"
                                         : "=f"(s[t][h]), "=r"(nz[t][h])
                                         : "r"(meta + (group * T * 16 + 16 * t + 8 * h) * 8)
                                         : "memory");
                            nz16[t][h] = F16 ? (nz[t][h] << 4 & 0x00f000f0u) | 0xd400d400u : 0u;
                        }
                    const uint4 &qa = q[t][0], &qb = q[t][1];
                    const uint4 va = values_of<F16>(
                        w == 0 ? qa.x : w == 1 ? qa.y : w == 2 ? qa.z : qa.w, nz[t][0], nz16[t][0]);
                    const uint4 vb = values_of<F16>(
                        w == 0 ? qb.x : w == 1 ? qb.y : w == 2 ? qb.z : qb.w, nz[t][1], nz16[t][1]);
#pragma unroll
                    for (int j = 0; j < NB; ++j) {
                        if (begin)
                            sum[t][j][0] = sum[t][j][1] = sum[t][j][2] = sum[t][j][3] = 0.f;
                        mma16816<F16>(sum[t][j], va.x, vb.x, va.y, vb.y, x[j][w].x, x[j][w].y);
                        mma16816<F16>(sum[t][j], va.z, vb.z, va.w, vb.w, x[j][w].z, x[j][w].w);
                        if (end)
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                total[t][j][e] = fmaf(s[t][e >> 1], sum[t][j][e], total[t][j][e]);
                    }
                }
            }
            // Into the slot of the block before this one.
            fetch(b + (DEPTH - 1) * kWarps, i + DEPTH - 1, (i + DEPTH - 1) % DEPTH);
        }
#pragma unroll
        for (int t = 0; t < T; ++t)
#pragma unroll
            for (int h = 0; h < 2; ++h)
                row[t][h] += DEPTH * kWarps * kW4BlockBytes;
#pragma unroll
        for (int j = 0; j < NB; ++j)
            a[j] += DEPTH * kWarps * kW4Block;
    }
    cp_async_wait<0>();
    __syncthreads();
    float(*red)[16 * T][8 * NB + 1] = reinterpret_cast<float(*)[16 * T][8 * NB + 1]>(shared);
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
        if (n0 + nn < p.N && mm < p.M)
            p.C[(int64_t)mm * p.N + n0 + nn] = v;
    }
}

template <bool F16, int T, int NB, int V, int GS>
static cudaError_t launch_kernel(const W4Launch &L, cudaStream_t stream)
{
    static_assert(kWarps * 16 * T * (8 * NB + 1) * 4 <= kWarps * warp_bytes(T, 1), "the totals fit");
    auto kernel = w4_rows_kernel<F16, T, NB, V, GS>;
    static std::atomic<uint64_t> done{0};
    const cudaError_t e =
        set_smem_limit_once(kernel, kWarps * (int)warp_bytes(T, 8 * NB), done, 100);
    if (e != cudaSuccess)
        return e;
    const unsigned grid = (unsigned)((L.N + 16 * T - 1) / (16 * T));
    kernel<<<grid, kThreads, kWarps * warp_bytes(T, L.M), stream>>>(L);
    return cudaGetLastError();
}

template <bool F16, int T, int NB, int GS>
static cudaError_t launch_v(const W4Launch &L, cudaStream_t stream)
{
    const uintptr_t a = reinterpret_cast<uintptr_t>(L.A);
    return L.K % 8 == 0 && a % 16 == 0  ? launch_kernel<F16, T, NB, 8, GS>(L, stream)
           : L.K % 2 == 0 && a % 4 == 0 ? launch_kernel<F16, T, NB, 2, GS>(L, stream)
                                        : launch_kernel<F16, T, NB, 1, GS>(L, stream);
}

template <bool F16, int GS>
static cudaError_t launch_f(const W4Launch &L, int sms, cudaStream_t stream)
{
    if (L.M > 8)
        return launch_v<F16, 2, 2, GS>(L, stream);
    // 32 columns a block (A's values are read once for both halves) where that
    // still gives every SM two blocks and few rows of A leave the shared memory:
    // 1 x 32768 x 8192 34.8 us against 38.7 us with 16. Finer groups need the
    // registers for their scales.
    if constexpr (GS == 7)
        if ((L.N + 31) / 32 >= 2 * sms && L.M <= 4)
            return launch_v<F16, 2, 1, GS>(L, stream);
    return launch_v<F16, 1, 1, GS>(L, stream);
}

} // namespace w4r

cudaError_t launch_w4_rows(const W4Launch &L, int sms, cudaStream_t stream)
{
    using namespace w4r;
    if (L.f16)
        return L.group == 32   ? launch_f<true, 5>(L, sms, stream)
               : L.group == 64 ? launch_f<true, 6>(L, sms, stream)
                               : launch_f<true, 7>(L, sms, stream);
    return L.group == 32   ? launch_f<false, 5>(L, sms, stream)
           : L.group == 64 ? launch_f<false, 6>(L, sms, stream)
                           : launch_f<false, 7>(L, sms, stream);
}

} // namespace rtm
