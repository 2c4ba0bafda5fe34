// The low-bit products on the FP32 pipes: 64 x 64 tiles of C, 4 x 4 outputs a
// thread, both operands turned into fp32 values as their 16-deep slices are
// stored to shared memory. Every size and alignment; no workspace: for operands
// whose rows are off 16-byte boundaries where the caller gives none. w4 4096 x
// 8192 x 8192 takes 33 ms, q8t 8192^3 53 ms (tensor cores 0.41 and 0.86): each
// operand is decoded anew in every 64 x 64 tile.
//
//     w4:  C[m][n] = sum_k A[m][k] * (q[k][n] - z[g][n]) * s[g][n],  g = k / group
//     q8t: C[k][n] = sum_m q[m][k] * s[m / 128][k] * dY[m][n]
#include <cstdint>
#include <cuda_runtime.h>

#include "lowbit.h"
#include "lowbit_types.cuh"

namespace rtm {
namespace lbs {

constexpr int T = 64, DEPTH = 16, kThreads = 256;

template <bool F16>
struct W4Operands {
    W4Launch p;
    __device__ int rows() const { return p.M; }
    __device__ int cols() const { return p.N; }
    __device__ int depth() const { return p.K; }
    __device__ float left(int64_t m, int64_t k) const { return to_f32<F16>(p.A[m * p.K + k]); }
    __device__ float right(int64_t k, int64_t n) const
    {
        const unsigned r = (unsigned)k % kW4Block, w = r / 32, c = r % 32 / 8, i = r % 8;
        const uint32_t word = *reinterpret_cast<const uint32_t *>(
            p.codes + n * w4_row_bytes(p.K) + (unsigned)k / kW4Block * kW4BlockBytes + c * 16 + w * 4);
        const int64_t g = (int64_t)((unsigned)k / (unsigned)p.group) * p.N + n;
        const float z = p.zeros ? (float)(p.zeros[g] & 15) : 8.f;
        return ((float)((word >> w4_shift((int)i)) & 15u) - z) * to_f32<F16>(p.scales[g]);
    }
};

template <bool F16>
struct Q8tOperands {
    Q8tLaunch p;
    __device__ int rows() const { return p.K; }
    __device__ int cols() const { return p.N; }
    __device__ int depth() const { return p.M; }
    __device__ float left(int64_t k, int64_t m) const
    {
        return (float)p.codes[m * q8_pitch(p.K) + k] * p.scales[m / kQ8Rows * p.K + k];
    }
    __device__ float right(int64_t m, int64_t n) const { return to_f32<F16>(p.dY[m * p.N + n]); }
};

template <typename Ops>
__global__ void __launch_bounds__(kThreads) lowbit_simt_kernel(const Ops ops, float *C)
{
    __shared__ float a[DEPTH][T + 1], b[DEPTH][T];
    const int rows = ops.rows(), cols = ops.cols(), depth = ops.depth();
    const unsigned tiles_n = ((unsigned)cols + T - 1) / T;
    const int64_t i0 = (int64_t)(blockIdx.x / tiles_n) * T, j0 = (int64_t)(blockIdx.x % tiles_n) * T;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    float acc[4][4] = {};
    for (int64_t d0 = 0; d0 < depth; d0 += DEPTH) {
#pragma unroll 1
        for (int e = threadIdx.x; e < T * DEPTH; e += kThreads) {
            const int64_t i = i0 + e / DEPTH, da = d0 + e % DEPTH;
            a[e % DEPTH][e / DEPTH] = i < rows && da < depth ? ops.left(i, da) : 0.f;
            const int64_t j = j0 + e % T, db = d0 + e / T;
            b[e / T][e % T] = j < cols && db < depth ? ops.right(db, j) : 0.f;
        }
        __syncthreads();
#pragma unroll
        for (int d = 0; d < DEPTH; ++d)
#pragma unroll
            for (int y = 0; y < 4; ++y)
#pragma unroll
                for (int x = 0; x < 4; ++x)
                    acc[y][x] = fmaf(a[d][ty + 16 * y], b[d][tx + 16 * x], acc[y][x]);
        __syncthreads();
    }
#pragma unroll
    for (int y = 0; y < 4; ++y)
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            const int64_t i = i0 + ty + 16 * y, j = j0 + tx + 16 * x;
            if (i < rows && j < cols)
                C[i * cols + j] = acc[y][x];
        }
}

template <typename Ops>
static cudaError_t launch(const Ops &ops, int64_t rows, int64_t cols, float *C, cudaStream_t stream)
{
    const int64_t tiles = (rows + T - 1) / T * ((cols + T - 1) / T);
    if (tiles > 0x7fffffff)
        return cudaErrorInvalidValue;
    lowbit_simt_kernel<<<(unsigned)tiles, kThreads, 0, stream>>>(ops, C);
    return cudaGetLastError();
}

} // namespace lbs

cudaError_t launch_w4_simt(const W4Launch &L, cudaStream_t stream)
{
    return L.f16 ? lbs::launch(lbs::W4Operands<true>{L}, L.M, L.N, L.C, stream)
                 : lbs::launch(lbs::W4Operands<false>{L}, L.M, L.N, L.C, stream);
}

cudaError_t launch_q8t_simt(const Q8tLaunch &L, cudaStream_t stream)
{
    return L.f16 ? lbs::launch(lbs::Q8tOperands<true>{L}, L.K, L.N, L.C, stream)
                 : lbs::launch(lbs::Q8tOperands<false>{L}, L.K, L.N, L.C, stream);
}

} // namespace rtm
