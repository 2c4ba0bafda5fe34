// Internal declarations of the 8-bit floating-point products (e4m3 codes, an fp32 scale for
// each block of 128) and of the experts' layer. Arguments are validated by the caller (f8_api.cu).
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "lowbit.h"

namespace rtm {

constexpr int kF8Block = 128;        // values that share a scale, along each blocked axis
constexpr int kRouteMaxExperts = 1024;
constexpr int kRouteMaxChosen = 32;  // a lane of the token's warp holds one
constexpr int kRouteMaxGroups = 32;

enum F8Type { kF32 = 0, kBf16 = 1, kF16 = 2 };

inline __host__ __device__ int64_t f8_blocks(int64_t n) { return (n + kF8Block - 1) / kF8Block; }
inline __host__ __device__ int64_t f8_pitch(int64_t n) { return (n + 15) / 16 * 16; }

// f8_quant.cu. X (source x K) -> M rows of codes: row i is X's row i, or with `rows` the row
// rows[i] / fan times factors[rows[i]] (factors may be null), zeros where rows[i] is outside
// 0 .. source * fan - 1. Row codes (a scale for 128 values of a row) and column codes (for 128
// values of a column): either pair may be null.
struct F8QuantLaunch {
    int64_t M, K, source;
    int type;
    const void *X;
    const int32_t *rows;
    int64_t fan;
    const float *factors;
    uint8_t *row_codes;
    float *row_scales;
    uint8_t *col_codes;
    float *col_scales;
};
cudaError_t launch_f8_quantize(const F8QuantLaunch &L, cudaStream_t stream);
// E matrices of K x N, a scale for each 128 x 128 tile.
cudaError_t launch_f8_quantize_tiles(int64_t E, int64_t K, int64_t N, int type, const void *W,
                                     uint8_t *codes, float *scales, cudaStream_t stream);
// E matrices of M x K (rows `ld` bytes apart) back to values; bm, bk: 128 along a blocked axis, else 1.
cudaError_t launch_f8_dequantize(int64_t E, int64_t M, int64_t K, int bm, int bk, int type,
                                 const uint8_t *codes, int64_t ld, const float *scales, void *X,
                                 cudaStream_t stream);

// A product on the tensor cores (f8_tc.cu). The product sums over `depth`:
//   kF8Forward  C (rows x cols) = A (rows x depth) . W (depth x cols)
//   kF8Input    C (rows x cols) = dY (rows x depth) . W^T, W (cols x depth)
//   kF8Weight   C (rows x cols) = X^T . dY, X (depth x rows), dY (depth x cols)
// With `offsets` (experts + 1 ascending values, on the device) rows offsets[e] .. offsets[e+1]-1
// of A (dY) and C belong to expert e and its matrix of W; kF8Weight sums over them and gives
// `experts` matrices C. Without, experts is 1.
enum F8Mode { kF8Forward = 0, kF8Input = 1, kF8Weight = 2 };
struct F8Launch {
    int mode;
    int experts;
    int64_t rows, cols, depth;
    const uint8_t *a;  // A, dY or X
    int64_t lda;       // bytes
    const float *a_scales;
    const uint8_t *b;  // W or dY
    int64_t ldb;
    const float *b_scales;
    const int32_t *offsets;
    float *C;
};
cudaError_t launch_f8_tc(const F8Launch &L, const DeviceContext &d, bool mute, cudaStream_t stream);

// route.cu
struct RouteLaunch {
    int64_t T;
    int E, k, type;
    const void *logits;
    const float *bias;  // may be null
    int groups, top_groups, sigmoid, renormalise;
    float scale;
    int align;
    int64_t R;  // entries of rows
    int32_t *experts;
    float *weights;
    int32_t *slots, *rows, *offsets;
    int32_t *counts;  // workspace
};
int64_t route_rows(int64_t T, int E, int k, int align);
int64_t route_workspace_ints(int64_t T, int E);
cudaError_t launch_route(const RouteLaunch &L, cudaStream_t stream);
cudaError_t launch_route_backward(const RouteLaunch &L, const int32_t *experts,
                                  const float *dweights, float *dlogits, cudaStream_t stream);
// y (T x N) = sum_j weights[t][j] * C[slots[t][j]]; weights may be null (ones).
cudaError_t launch_experts_join(int64_t T, int64_t N, int k, int64_t R, const float *C,
                                const int32_t *slots, const float *weights, float *Y,
                                cudaStream_t stream);
// dweights[t][j] = dY[t] . C[slots[t][j]]
cudaError_t launch_experts_join_backward(int64_t T, int64_t N, int k, int64_t R, int type,
                                         const void *dY, const float *C, const int32_t *slots,
                                         float *dweights, cudaStream_t stream);

} // namespace rtm
