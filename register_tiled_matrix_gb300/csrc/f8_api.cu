// C entry points of the 8-bit floating-point products and of the experts' layer (declared in
// include/gemm.h): argument checks, then one launch function each.
#include <cstdint>
#include <cuda_runtime.h>

#include "api_checks.h"
#include "f8.h"
#include "gemm.h"
#include "kernels.h"

namespace {

using namespace rtm::api;
using rtm::f8_blocks;
using rtm::f8_pitch;

int64_t type_bytes(int type) { return type == rtm::kF32 ? 4 : 2; }

// batch matrices of rows x cols: each size and all elements within the limits.
bool batch_ok(int64_t batch, int64_t rows, int64_t cols)
{
    return size_ok(rows, cols) && batch >= 0 && batch <= kMaxDim &&
           (rows == 0 || cols == 0 || batch <= kMaxElements / rows / cols);
}

// A row pitch in bytes: at least the row, a multiple of 16, the matrix within the limits.
bool pitch_ok(int64_t batch, int64_t rows, int64_t cols, int64_t ld)
{
    return ld >= cols && ld % 16 == 0 && batch_ok(batch, rows, ld);
}

int context(rtm::DeviceContext *d, int64_t wait_limit_ns = 0)
{
    const int st = rtm::device_context(d);
    if (st == GEMM_OK && !d->encode_tiled)
        return GEMM_ERR_LAUNCH;
    if (wait_limit_ns > 0)
        d->wait_limit_ns = (uint64_t)wait_limit_ns;
    return st;
}

// No output overlaps an input or another output.
template <int OUT, int IN>
bool disjoint(const Range (&out)[OUT], const Range (&in)[IN])
{
    for (int i = 0; i < OUT; ++i)
        if (overlaps(out[i], in, IN) || overlaps(out[i], out, i))
            return false;
    return true;
}

int quantize(int64_t M, int64_t K, int type, const void *X, int64_t source, const int32_t *rows,
             int64_t fan, const float *factors, uint8_t *row_codes, float *row_scales,
             uint8_t *col_codes, float *col_scales, void *stream)
{
    if (!size_ok(M, f8_pitch(K)) || !size_ok(source, K) || fan < 1 || fan > kMaxDim ||
        source > kMaxDim / fan || !row_codes != !row_scales || !col_codes != !col_scales)
        return GEMM_ERR_INVALID_ARG;
    if (M == 0 || K == 0)
        return GEMM_OK;
    if ((!rows && (source != M || fan != 1 || factors)) || (source > 0 && !X) || (!row_codes && !col_codes))
        return GEMM_ERR_INVALID_ARG;
    const Range out[4] = {{row_codes, M * f8_pitch(K)},
                          {row_scales, M * f8_blocks(K) * 4},
                          {col_codes, M * f8_pitch(K)},
                          {col_scales, f8_blocks(M) * K * 4}};
    const Range in[3] = {{X, source * K * type_bytes(type)},
                         {rows, M * 4},
                         {factors, source * fan * 4}};
    if (!disjoint(out, in))
        return GEMM_ERR_INVALID_ARG;
    if (misaligned(X, type_bytes(type)) || misaligned(rows, 4) || misaligned(factors, 4) ||
        misaligned(row_codes, 16) || misaligned(col_codes, 16) || misaligned(row_scales, 4) ||
        misaligned(col_scales, 4))
        return GEMM_ERR_ALIGNMENT;
    rtm::DeviceContext d;
    const int st = rtm::device_context(&d);
    if (st != GEMM_OK)
        return st;
    rtm::F8QuantLaunch L;
    L.M = M;
    L.K = K;
    L.source = source;
    L.type = type;
    L.X = X;
    L.rows = rows;
    L.fan = fan;
    L.factors = factors;
    L.row_codes = row_codes;
    L.row_scales = row_scales;
    L.col_codes = col_codes;
    L.col_scales = col_scales;
    return finish(rtm::launch_f8_quantize(L, static_cast<cudaStream_t>(stream)));
}

int quantize_tiles(int64_t E, int64_t K, int64_t N, int type, const void *W, uint8_t *codes,
                   float *scales, void *stream)
{
    if (!batch_ok(E, K, f8_pitch(N)))
        return GEMM_ERR_INVALID_ARG;
    if (E == 0 || K == 0 || N == 0)
        return GEMM_OK;
    if (!W || !codes || !scales)
        return GEMM_ERR_INVALID_ARG;
    const Range out[2] = {{codes, E * K * f8_pitch(N)},
                          {scales, E * f8_blocks(K) * f8_blocks(N) * 4}};
    const Range in[1] = {{W, E * K * N * type_bytes(type)}};
    if (!disjoint(out, in))
        return GEMM_ERR_INVALID_ARG;
    if (misaligned(W, type_bytes(type)) || misaligned(codes, 16) || misaligned(scales, 4))
        return GEMM_ERR_ALIGNMENT;
    rtm::DeviceContext d;
    const int st = rtm::device_context(&d);
    if (st != GEMM_OK)
        return st;
    return finish(rtm::launch_f8_quantize_tiles(E, K, N, type, W, codes, scales,
                                                static_cast<cudaStream_t>(stream)));
}

int dequantize(int64_t E, int64_t M, int64_t K, int kind, int type, const uint8_t *codes,
               int64_t ld, const float *scales, void *X, void *stream)
{
    if (kind < GEMM_F8_ROWS || kind > GEMM_F8_TILES || !batch_ok(E, M, K) || !pitch_ok(E, M, K, ld))
        return GEMM_ERR_INVALID_ARG;
    if (E == 0 || M == 0 || K == 0)
        return GEMM_OK;
    if (!codes || !scales || !X)
        return GEMM_ERR_INVALID_ARG;
    const int bm = kind == GEMM_F8_ROWS ? 1 : rtm::kF8Block;
    const int bk = kind == GEMM_F8_COLUMNS ? 1 : rtm::kF8Block;
    const int64_t held = E * (bm == 1 ? M : f8_blocks(M)) * (bk == 1 ? K : f8_blocks(K));
    const Range out[1] = {{X, E * M * K * type_bytes(type)}};
    const Range in[2] = {{codes, (E * M - 1) * ld + K}, {scales, held * 4}};
    if (!disjoint(out, in))
        return GEMM_ERR_INVALID_ARG;
    if (misaligned(X, type_bytes(type)) || misaligned(codes, 16) || misaligned(scales, 4))
        return GEMM_ERR_ALIGNMENT;
    rtm::DeviceContext d;
    const int st = rtm::device_context(&d);
    if (st != GEMM_OK)
        return st;
    return finish(rtm::launch_f8_dequantize(E, M, K, bm, bk, type, codes, ld, scales, X,
                                            static_cast<cudaStream_t>(stream)));
}

// Every product. rows, cols: of one matrix C; `a` has `rows` rows (weight: depth rows), W
// `experts` matrices. wait_limit_ns > 0: the failure-detection self-test.
int product(int mode, int64_t experts, int64_t rows, int64_t cols, int64_t depth, const uint8_t *a,
            int64_t lda, const float *a_scales, const uint8_t *b, int64_t ldb, const float *b_scales,
            const int32_t *offsets, bool grouped, float *C, int64_t wait_limit_ns, void *stream)
{
    const bool weight = mode == rtm::kF8Weight;
    const int64_t ar = weight ? depth : rows, ac = weight ? rows : depth;
    const int64_t br = mode == rtm::kF8Input ? cols : depth, bc = mode == rtm::kF8Input ? depth : cols;
    const int64_t cs = weight ? experts : 1, bs = weight ? 1 : experts;
    if (!size_ok(rows, cols) || !size_ok(ar, ac) || !size_ok(br, bc) || experts < 0 ||
        experts > rtm::kRouteMaxExperts || !batch_ok(cs, rows, cols) || !pitch_ok(1, ar, ac, lda) ||
        !pitch_ok(bs, br, bc, ldb))
        return GEMM_ERR_INVALID_ARG;
    if (rows == 0 || cols == 0 || experts == 0)
        return GEMM_OK;
    if (!C || (depth > 0 && (!a || !a_scales || !b || !b_scales || (grouped && !offsets))))
        return GEMM_ERR_INVALID_ARG;
    const int64_t sa = weight ? f8_blocks(depth) * rows : rows * f8_blocks(depth);
    const int64_t sb = weight ? f8_blocks(depth) * cols : experts * f8_blocks(br) * f8_blocks(bc);
    const Range out[1] = {{C, cs * rows * cols * 4}};
    const Range in[5] = {{a, ar > 0 ? (ar - 1) * lda + ac : 0},
                         {a_scales, sa * 4},
                         {b, br > 0 ? (bs * br - 1) * ldb + bc : 0},
                         {b_scales, sb * 4},
                         {offsets, grouped ? (experts + 1) * 4 : 0}};
    if (depth > 0 && !disjoint(out, in))
        return GEMM_ERR_INVALID_ARG;
    if (misaligned(C, 4) || (depth > 0 && (misaligned(a, 16) || misaligned(b, 16) ||
                                           misaligned(a_scales, 4) || misaligned(b_scales, 4) ||
                                           misaligned(offsets, 4))))
        return GEMM_ERR_ALIGNMENT;
    rtm::DeviceContext d;
    const int st = context(&d, wait_limit_ns);
    if (st != GEMM_OK)
        return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (depth == 0)
        return finish(rtm::launch_zero_fill(C, cs * rows * cols, s));
    rtm::F8Launch L;
    L.mode = mode;
    L.experts = (int)experts;
    L.rows = rows;
    L.cols = cols;
    L.depth = depth;
    L.a = a;
    L.lda = lda;
    L.a_scales = a_scales;
    L.b = b;
    L.ldb = ldb;
    L.b_scales = b_scales;
    L.offsets = grouped ? offsets : nullptr;
    L.C = C;
    return finish(rtm::launch_f8_tc(L, d, wait_limit_ns > 0, s));
}

bool route_ok(int64_t T, int64_t E, int64_t k, int64_t groups, int64_t top_groups, int64_t align)
{
    return T >= 0 && E >= 1 && E <= rtm::kRouteMaxExperts && k >= 1 && k <= rtm::kRouteMaxChosen &&
           k <= E && groups >= 1 && groups <= rtm::kRouteMaxGroups && E % groups == 0 &&
           top_groups >= 1 && top_groups <= groups && k <= top_groups * (E / groups) && align >= 1 &&
           align <= 1024 && T <= kMaxDim / k && T <= kMaxElements / E &&
           T * k + E * align <= kMaxDim;
}

int route(int64_t T, int64_t E, int64_t k, int type, const void *logits, const float *bias,
          int64_t groups, int64_t top_groups, int sigmoid, int renormalise, float scale,
          int64_t align, int32_t *experts, float *weights, int32_t *slots, int32_t *rows,
          int32_t *offsets, void *workspace, int64_t workspace_bytes, void *stream)
{
    if (!route_ok(T, E, k, groups, top_groups, align) || workspace_bytes < 0 ||
        (workspace_bytes > 0 && !workspace))
        return GEMM_ERR_INVALID_ARG;
    const int64_t R = rtm::route_rows(T, (int)E, (int)k, (int)align);
    const int64_t need = rtm::route_workspace_ints(T, (int)E) * 4;
    if (!offsets || (T > 0 && (!logits || !experts || !weights || !slots || !rows)) ||
        workspace_bytes < need)
        return GEMM_ERR_INVALID_ARG;
    const Range out[6] = {{experts, T * k * 4}, {weights, T * k * 4}, {slots, T * k * 4},
                          {rows, R * 4},        {offsets, (E + 1) * 4}, {workspace, need}};
    const Range in[2] = {{logits, T * E * type_bytes(type)}, {bias, E * 4}};
    if (!disjoint(out, in))
        return GEMM_ERR_INVALID_ARG;
    if (misaligned(logits, type_bytes(type)) || misaligned(bias, 4) || misaligned(experts, 4) ||
        misaligned(weights, 4) || misaligned(slots, 4) || misaligned(rows, 4) ||
        misaligned(offsets, 4) || (need > 0 && misaligned(workspace, 4)))
        return GEMM_ERR_ALIGNMENT;
    rtm::DeviceContext d;
    const int st = rtm::device_context(&d);
    if (st != GEMM_OK)
        return st;
    rtm::RouteLaunch L = {};
    L.T = T;
    L.E = (int)E;
    L.k = (int)k;
    L.type = type;
    L.logits = logits;
    L.bias = bias;
    L.groups = (int)groups;
    L.top_groups = (int)top_groups;
    L.sigmoid = sigmoid != 0;
    L.renormalise = renormalise != 0;
    L.scale = scale;
    L.align = (int)align;
    L.R = R;
    L.experts = experts;
    L.weights = weights;
    L.slots = slots;
    L.rows = rows;
    L.offsets = offsets;
    L.counts = static_cast<int32_t *>(workspace);
    return finish(rtm::launch_route(L, static_cast<cudaStream_t>(stream)));
}

int route_backward(int64_t T, int64_t E, int64_t k, int type, const void *logits, int sigmoid,
                   int renormalise, float scale, const int32_t *experts, const float *dweights,
                   float *dlogits, void *stream)
{
    if (!route_ok(T, E, k, 1, 1, 1))
        return GEMM_ERR_INVALID_ARG;
    if (T == 0)
        return GEMM_OK;
    if (!logits || !experts || !dweights || !dlogits)
        return GEMM_ERR_INVALID_ARG;
    const Range out[1] = {{dlogits, T * E * 4}};
    const Range in[3] = {{logits, T * E * type_bytes(type)}, {experts, T * k * 4}, {dweights, T * k * 4}};
    if (!disjoint(out, in))
        return GEMM_ERR_INVALID_ARG;
    if (misaligned(logits, type_bytes(type)) || misaligned(experts, 4) || misaligned(dweights, 4) ||
        misaligned(dlogits, 4))
        return GEMM_ERR_ALIGNMENT;
    rtm::DeviceContext d;
    const int st = rtm::device_context(&d);
    if (st != GEMM_OK)
        return st;
    rtm::RouteLaunch L = {};
    L.T = T;
    L.E = (int)E;
    L.k = (int)k;
    L.type = type;
    L.logits = logits;
    L.sigmoid = sigmoid != 0;
    L.renormalise = renormalise != 0;
    L.scale = scale;
    return finish(rtm::launch_route_backward(L, experts, dweights, dlogits,
                                             static_cast<cudaStream_t>(stream)));
}

bool join_ok(int64_t T, int64_t N, int64_t k, int64_t R)
{
    return size_ok(T, N) && size_ok(R, N) && k >= 1 && k <= rtm::kRouteMaxChosen && T <= kMaxDim / k;
}

int join_backward(int64_t T, int64_t N, int64_t k, int64_t R, int type, const void *dY,
                  const float *C, const int32_t *slots, float *dweights, void *stream)
{
    if (!join_ok(T, N, k, R))
        return GEMM_ERR_INVALID_ARG;
    if (T == 0)
        return GEMM_OK;
    if (!dweights || !slots || (N > 0 && (!dY || (R > 0 && !C))))
        return GEMM_ERR_INVALID_ARG;
    const Range out[1] = {{dweights, T * k * 4}};
    const Range in[3] = {{dY, T * N * type_bytes(type)}, {C, R * N * 4}, {slots, T * k * 4}};
    if (!disjoint(out, in))
        return GEMM_ERR_INVALID_ARG;
    if (misaligned(dY, type_bytes(type)) || misaligned(C, 4) || misaligned(slots, 4) ||
        misaligned(dweights, 4))
        return GEMM_ERR_ALIGNMENT;
    rtm::DeviceContext d;
    const int st = rtm::device_context(&d);
    if (st != GEMM_OK)
        return st;
    return finish(rtm::launch_experts_join_backward(T, N, (int)k, R, type, dY, C, slots, dweights,
                                                    static_cast<cudaStream_t>(stream)));
}

} // namespace

extern "C" {

int64_t gemm_f8_pitch(int64_t K)
{
    return K >= 0 && K <= kMaxDim ? f8_pitch(K) : GEMM_ERR_INVALID_ARG;
}

#define RTM_F8_TYPED(NAME, T, TYPE)                                                                \
    int gemm_##NAME##_f8_quantize(int64_t M, int64_t K, const T *X, int64_t source_rows,           \
                                  const int32_t *rows, int64_t fan, const float *factors,          \
                                  uint8_t *row_codes, float *row_scales, uint8_t *col_codes,       \
                                  float *col_scales, void *stream)                                 \
    {                                                                                              \
        return quantize(M, K, TYPE, X, source_rows, rows, fan, factors, row_codes, row_scales,     \
                        col_codes, col_scales, stream);                                            \
    }                                                                                              \
    int gemm_##NAME##_f8_quantize_tiles(int64_t E, int64_t K, int64_t N, const T *W,               \
                                        uint8_t *codes, float *scales, void *stream)               \
    {                                                                                              \
        return quantize_tiles(E, K, N, TYPE, W, codes, scales, stream);                            \
    }                                                                                              \
    int gemm_##NAME##_f8_dequantize(int64_t E, int64_t M, int64_t K, int kind,                     \
                                    const uint8_t *codes, int64_t ld, const float *scales, T *X,   \
                                    void *stream)                                                  \
    {                                                                                              \
        return dequantize(E, M, K, kind, TYPE, codes, ld, scales, X, stream);                      \
    }                                                                                              \
    int gemm_##NAME##_route(int64_t T_, int64_t E, int64_t k, const T *logits, const float *bias,  \
                            int64_t groups, int64_t top_groups, int sigmoid, int renormalise,      \
                            float scale, int64_t align, int32_t *experts, float *weights,          \
                            int32_t *slots, int32_t *rows, int32_t *offsets, void *workspace,      \
                            int64_t workspace_bytes, void *stream)                                 \
    {                                                                                              \
        return route(T_, E, k, TYPE, logits, bias, groups, top_groups, sigmoid, renormalise,       \
                     scale, align, experts, weights, slots, rows, offsets, workspace,              \
                     workspace_bytes, stream);                                                     \
    }                                                                                              \
    int gemm_##NAME##_route_backward(int64_t T_, int64_t E, int64_t k, const T *logits,            \
                                     int sigmoid, int renormalise, float scale,                    \
                                     const int32_t *experts, const float *dweights,                \
                                     float *dlogits, void *stream)                                 \
    {                                                                                              \
        return route_backward(T_, E, k, TYPE, logits, sigmoid, renormalise, scale, experts,        \
                              dweights, dlogits, stream);                                          \
    }                                                                                              \
    int gemm_##NAME##_experts_join_backward(int64_t T_, int64_t N, int64_t k, int64_t R,           \
                                            const T *dY, const float *C, const int32_t *slots,     \
                                            float *dweights, void *stream)                         \
    {                                                                                              \
        return join_backward(T_, N, k, R, TYPE, dY, C, slots, dweights, stream);                   \
    }
RTM_F8_TYPED(f32, float, rtm::kF32)
RTM_F8_TYPED(bf16, uint16_t, rtm::kBf16)
RTM_F8_TYPED(f16, uint16_t, rtm::kF16)
#undef RTM_F8_TYPED

int gemm_f8w8f32(int64_t M, int64_t N, int64_t K, const uint8_t *A, int64_t lda,
                 const float *a_scales, const uint8_t *W, int64_t ldw, const float *w_scales,
                 float *C, void *stream)
{
    return product(rtm::kF8Forward, 1, M, N, K, A, lda, a_scales, W, ldw, w_scales, nullptr, false,
                   C, 0, stream);
}

int gemm_f8w8tf32(int64_t M, int64_t N, int64_t K, const uint8_t *dY, int64_t ldy,
                  const float *y_scales, const uint8_t *W, int64_t ldw, const float *w_scales,
                  float *dX, void *stream)
{
    return product(rtm::kF8Input, 1, M, K, N, dY, ldy, y_scales, W, ldw, w_scales, nullptr, false,
                   dX, 0, stream);
}

int gemm_f8tf8f32(int64_t M, int64_t N, int64_t K, const uint8_t *X, int64_t ldx,
                  const float *x_scales, const uint8_t *dY, int64_t ldy, const float *y_scales,
                  float *dW, void *stream)
{
    return product(rtm::kF8Weight, 1, K, N, M, X, ldx, x_scales, dY, ldy, y_scales, nullptr, false,
                   dW, 0, stream);
}

int gemm_f8w8f32_experts(int64_t R, int64_t N, int64_t K, int64_t E, const int32_t *offsets,
                         const uint8_t *A, int64_t lda, const float *a_scales, const uint8_t *W,
                         int64_t ldw, const float *w_scales, float *C, void *stream)
{
    return product(rtm::kF8Forward, E, R, N, K, A, lda, a_scales, W, ldw, w_scales, offsets, true,
                   C, 0, stream);
}

int gemm_f8w8tf32_experts(int64_t R, int64_t N, int64_t K, int64_t E, const int32_t *offsets,
                          const uint8_t *dY, int64_t ldy, const float *y_scales, const uint8_t *W,
                          int64_t ldw, const float *w_scales, float *dX, void *stream)
{
    return product(rtm::kF8Input, E, R, K, N, dY, ldy, y_scales, W, ldw, w_scales, offsets, true,
                   dX, 0, stream);
}

int gemm_f8tf8f32_experts(int64_t R, int64_t N, int64_t K, int64_t E, const int32_t *offsets,
                          const uint8_t *X, int64_t ldx, const float *x_scales, const uint8_t *dY,
                          int64_t ldy, const float *y_scales, float *dW, void *stream)
{
    return product(rtm::kF8Weight, E, K, N, R, X, ldx, x_scales, dY, ldy, y_scales, offsets, true,
                   dW, 0, stream);
}

int gemm_f8w8f32_selftest_timeout(int64_t M, int64_t N, int64_t K, const uint8_t *A, int64_t lda,
                                  const float *a_scales, const uint8_t *W, int64_t ldw,
                                  const float *w_scales, float *C, int64_t wait_limit_ns,
                                  void *stream)
{
    if (wait_limit_ns < 1000000 || wait_limit_ns > 10000000000LL || M < 1 || N < 1 || K < 1)
        return GEMM_ERR_INVALID_ARG;
    return product(rtm::kF8Forward, 1, M, N, K, A, lda, a_scales, W, ldw, w_scales, nullptr, false,
                   C, wait_limit_ns, stream);
}

int64_t gemm_route_rows(int64_t T, int64_t E, int64_t k, int64_t align)
{
    return route_ok(T, E, k, 1, 1, align) ? rtm::route_rows(T, (int)E, (int)k, (int)align)
                                          : GEMM_ERR_INVALID_ARG;
}

int64_t gemm_route_workspace_bytes(int64_t T, int64_t E)
{
    return route_ok(T, E, 1, 1, 1, 1) ? rtm::route_workspace_ints(T, (int)E) * 4
                                      : GEMM_ERR_INVALID_ARG;
}

int gemm_experts_join(int64_t T, int64_t N, int64_t k, int64_t R, const float *C,
                      const int32_t *slots, const float *weights, float *Y, void *stream)
{
    if (!join_ok(T, N, k, R))
        return GEMM_ERR_INVALID_ARG;
    if (T == 0 || N == 0)
        return GEMM_OK;
    if (!Y || !slots || (R > 0 && !C))
        return GEMM_ERR_INVALID_ARG;
    const Range out[1] = {{Y, T * N * 4}};
    const Range in[3] = {{C, R * N * 4}, {slots, T * k * 4}, {weights, T * k * 4}};
    if (!disjoint(out, in))
        return GEMM_ERR_INVALID_ARG;
    if (misaligned(C, 4) || misaligned(Y, 4) || misaligned(slots, 4) || misaligned(weights, 4))
        return GEMM_ERR_ALIGNMENT;
    rtm::DeviceContext d;
    const int st = rtm::device_context(&d);
    if (st != GEMM_OK)
        return st;
    return finish(rtm::launch_experts_join(T, N, (int)k, R, C, slots, weights, Y,
                                           static_cast<cudaStream_t>(stream)));
}

} // extern "C"
