// C entry points of the low-bit products (declared in include/gemm.h): argument
// checks, then one launch function each.
#include <cstdint>
#include <cuda_runtime.h>

#include "api_checks.h"
#include "gemm.h"
#include "kernels.h"
#include "lowbit.h"

namespace {

using namespace rtm::api;

bool group_ok(int group) { return group == 32 || group == 64 || group == 128; }

bool rows16(const void *p, int64_t cols) { return cols % 8 == 0 && !misaligned(p, 16); }

// Bytes of a copy of a rows x cols 2-byte matrix with its rows padded to 16 bytes.
int64_t padded_bytes(int64_t rows, int64_t cols)
{
    return (rows * ((cols + 7) / 8 * 8) * 2 + 255) / 256 * 256;
}

int64_t groups(int64_t K, int group) { return (K + group - 1) / group; }

// The checks and the launch of both quantise entries' outputs.
int w4_quantize(int64_t K, int64_t N, int group, int f16, const uint16_t *W, uint8_t *codes,
                uint16_t *scales, uint8_t *zeros, void *stream)
{
    if (!size_ok(K, N) || !group_ok(group))
        return GEMM_ERR_INVALID_ARG;
    if (K == 0 || N == 0)
        return GEMM_OK;
    if (!W || !codes || !scales)
        return GEMM_ERR_INVALID_ARG;
    const int64_t meta = groups(K, group) * N;
    const Range all[4] = {{W, K * N * 2},
                          {codes, N * rtm::w4_row_bytes(K)},
                          {scales, meta * 2},
                          {zeros, zeros ? meta : 0}};
    for (int i = 1; i < 4; ++i)
        if (overlaps(all[i], all, i))
            return GEMM_ERR_INVALID_ARG;
    if (misaligned(W, 2) || misaligned(codes, 16) || misaligned(scales, 2))
        return GEMM_ERR_ALIGNMENT;
    rtm::DeviceContext d;
    const int st = rtm::device_context(&d);
    if (st != GEMM_OK)
        return st;
    return finish(rtm::launch_w4_quantize(K, N, group, f16, W, codes, scales, zeros,
                                          static_cast<cudaStream_t>(stream)));
}

int w4_dequantize(int64_t K, int64_t N, int group, int f16, const uint8_t *codes,
                  const uint16_t *scales, const uint8_t *zeros, uint16_t *W, void *stream)
{
    if (!size_ok(K, N) || !group_ok(group))
        return GEMM_ERR_INVALID_ARG;
    if (K == 0 || N == 0)
        return GEMM_OK;
    if (!W || !codes || !scales)
        return GEMM_ERR_INVALID_ARG;
    const int64_t meta = groups(K, group) * N;
    const Range in[3] = {{codes, N * rtm::w4_row_bytes(K)}, {scales, meta * 2}, {zeros, meta}};
    if (overlaps({W, K * N * 2}, in, 3))
        return GEMM_ERR_INVALID_ARG;
    if (misaligned(W, 2) || misaligned(codes, 16) || misaligned(scales, 2))
        return GEMM_ERR_ALIGNMENT;
    rtm::DeviceContext d;
    const int st = rtm::device_context(&d);
    if (st != GEMM_OK)
        return st;
    return finish(rtm::launch_w4_dequantize(K, N, group, f16, codes, scales, zeros, W,
                                            static_cast<cudaStream_t>(stream)));
}

int q8_quantize(int64_t M, int64_t K, int f16, const uint16_t *X, int8_t *codes, float *scales,
                void *stream)
{
    if (!size_ok(M, K))
        return GEMM_ERR_INVALID_ARG;
    if (M == 0 || K == 0)
        return GEMM_OK;
    if (!X || !codes || !scales)
        return GEMM_ERR_INVALID_ARG;
    const Range all[3] = {{X, M * K * 2},
                          {codes, M * rtm::q8_pitch(K)},
                          {scales, groups(M, rtm::kQ8Rows) * K * 4}};
    for (int i = 1; i < 3; ++i)
        if (overlaps(all[i], all, i))
            return GEMM_ERR_INVALID_ARG;
    if (misaligned(X, 2) || misaligned(codes, 16) || misaligned(scales, 4))
        return GEMM_ERR_ALIGNMENT;
    rtm::DeviceContext d;
    const int st = rtm::device_context(&d);
    if (st != GEMM_OK)
        return st;
    return finish(rtm::launch_q8_quantize(M, K, f16, X, codes, scales,
                                          static_cast<cudaStream_t>(stream)));
}

int q8_dequantize(int64_t M, int64_t K, int f16, const int8_t *codes, const float *scales,
                  uint16_t *X, void *stream)
{
    if (!size_ok(M, K))
        return GEMM_ERR_INVALID_ARG;
    if (M == 0 || K == 0)
        return GEMM_OK;
    if (!X || !codes || !scales)
        return GEMM_ERR_INVALID_ARG;
    const Range in[2] = {{codes, M * rtm::q8_pitch(K)},
                         {scales, groups(M, rtm::kQ8Rows) * K * 4}};
    if (overlaps({X, M * K * 2}, in, 2))
        return GEMM_ERR_INVALID_ARG;
    if (misaligned(X, 2) || misaligned(codes, 16) || misaligned(scales, 4))
        return GEMM_ERR_ALIGNMENT;
    rtm::DeviceContext d;
    const int st = rtm::device_context(&d);
    if (st != GEMM_OK)
        return st;
    return finish(rtm::launch_q8_dequantize(M, K, f16, codes, scales, X,
                                            static_cast<cudaStream_t>(stream)));
}

int w4_product(int64_t M, int64_t N, int64_t K, int f16, const uint16_t *A, const uint8_t *codes,
               const uint16_t *scales, const uint8_t *zeros, int group, float *C, void *workspace,
               int64_t workspace_bytes, void *stream)
{
    if (!size_ok(M, K) || !size_ok(K, N) || !size_ok(M, N) || !group_ok(group) ||
        workspace_bytes < 0 || (workspace_bytes > 0 && !workspace))
        return GEMM_ERR_INVALID_ARG;
    if (M == 0 || N == 0)
        return GEMM_OK;
    if (!C || (K > 0 && (!A || !codes || !scales)))
        return GEMM_ERR_INVALID_ARG;
    const int64_t meta = groups(K, group) * N;
    const Range in[4] = {{A, M * K * 2},
                         {codes, N * rtm::w4_row_bytes(K)},
                         {scales, meta * 2},
                         {zeros, meta}};
    const Range out = {C, M * N * 4};
    if (K > 0 && overlaps(out, in, 4))
        return GEMM_ERR_INVALID_ARG;
    if (misaligned(C, 4) ||
        (K > 0 && (misaligned(A, 2) || misaligned(codes, 16) || misaligned(scales, 2))))
        return GEMM_ERR_ALIGNMENT;
    rtm::DeviceContext d;
    const int st = rtm::device_context(&d);
    if (st != GEMM_OK)
        return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (K == 0)
        return finish(rtm::launch_zero_fill(C, M * N, s));
    rtm::W4Launch L;
    L.M = (int)M;
    L.N = (int)N;
    L.K = (int)K;
    L.group = group;
    L.f16 = f16;
    L.A = A;
    L.codes = codes;
    L.scales = scales;
    L.zeros = zeros;
    L.C = C;
    if (M <= rtm::kW4RowsMax)
        return finish(rtm::launch_w4_rows(L, d.sms, s));
    if (d.encode_tiled && rows16(A, K))
        return finish(rtm::launch_w4_tc(L, K, d, false, s));
    const int64_t need = padded_bytes(M, K);
    if (d.encode_tiled && workspace && !misaligned(workspace, 16) && workspace_bytes >= need) {
        if (overlaps({workspace, need}, in, 4) || overlaps({workspace, need}, &out, 1))
            return GEMM_ERR_INVALID_ARG;
        const int64_t lda = (K + 7) / 8 * 8;
        uint16_t *copy = static_cast<uint16_t *>(workspace);
        const cudaError_t e = rtm::launch_pack_rows_2b(A, M, K, copy, lda, d.sms, s);
        if (e != cudaSuccess)
            return finish(e);
        L.A = copy;
        return finish(rtm::launch_w4_tc(L, lda, d, false, s));
    }
    return finish(rtm::launch_w4_simt(L, s));
}

int q8t_product(int64_t M, int64_t N, int64_t K, int f16, const int8_t *codes, const float *scales,
                const uint16_t *dY, float *C, void *workspace, int64_t workspace_bytes,
                void *stream)
{
    if (!size_ok(M, K) || !size_ok(K, N) || !size_ok(M, N) || workspace_bytes < 0 ||
        (workspace_bytes > 0 && !workspace))
        return GEMM_ERR_INVALID_ARG;
    if (K == 0 || N == 0)
        return GEMM_OK;
    if (!C || (M > 0 && (!codes || !scales || !dY)))
        return GEMM_ERR_INVALID_ARG;
    const Range in[3] = {{codes, M * rtm::q8_pitch(K)},
                         {scales, groups(M, rtm::kQ8Rows) * K * 4},
                         {dY, M * N * 2}};
    const Range out = {C, K * N * 4};
    if (M > 0 && overlaps(out, in, 3))
        return GEMM_ERR_INVALID_ARG;
    if (misaligned(C, 4) ||
        (M > 0 && (misaligned(codes, 16) || misaligned(scales, 4) || misaligned(dY, 2))))
        return GEMM_ERR_ALIGNMENT;
    rtm::DeviceContext d;
    const int st = rtm::device_context(&d);
    if (st != GEMM_OK)
        return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (M == 0)
        return finish(rtm::launch_zero_fill(C, K * N, s));
    rtm::Q8tLaunch L;
    L.M = (int)M;
    L.N = (int)N;
    L.K = (int)K;
    L.f16 = f16;
    L.codes = codes;
    L.scales = scales;
    L.dY = dY;
    L.C = C;
    if (d.encode_tiled && rows16(dY, N))
        return finish(rtm::launch_q8t_tc(L, N, d, false, s));
    const int64_t need = padded_bytes(M, N);
    if (d.encode_tiled && workspace && !misaligned(workspace, 16) && workspace_bytes >= need) {
        if (overlaps({workspace, need}, in, 3) || overlaps({workspace, need}, &out, 1))
            return GEMM_ERR_INVALID_ARG;
        const int64_t ldy = (N + 7) / 8 * 8;
        uint16_t *copy = static_cast<uint16_t *>(workspace);
        const cudaError_t e = rtm::launch_pack_rows_2b(dY, M, N, copy, ldy, d.sms, s);
        if (e != cudaSuccess)
            return finish(e);
        L.dY = copy;
        return finish(rtm::launch_q8t_tc(L, ldy, d, false, s));
    }
    return finish(rtm::launch_q8t_simt(L, s));
}

// wait_limit_ns > 0: the failure-detection self-test of the tensor-core kernel.
int device_with_limit(rtm::DeviceContext *d, int64_t wait_limit_ns)
{
    const int st = rtm::device_context(d);
    if (wait_limit_ns > 0)
        d->wait_limit_ns = (uint64_t)wait_limit_ns;
    return st == GEMM_OK && !d->encode_tiled ? GEMM_ERR_LAUNCH : st;
}

bool limit_ok(int64_t ns) { return ns >= 1000000 && ns <= 10000000000LL; }

} // namespace

extern "C" {

int gemm_bf16w4f32_selftest_timeout(int64_t M, int64_t N, int64_t K, const uint16_t *A,
                                    const uint8_t *codes, const uint16_t *scales,
                                    const uint8_t *zeros, int group, float *C,
                                    int64_t wait_limit_ns, void *stream)
{
    if (!limit_ok(wait_limit_ns) || M <= rtm::kW4RowsMax || N < 1 || K < 1 || !size_ok(M, K) ||
        !size_ok(K, N) || !size_ok(M, N) || !group_ok(group) || !A || !codes || !scales || !C ||
        !rows16(A, K) || misaligned(codes, 16) || misaligned(scales, 2) || misaligned(C, 4))
        return GEMM_ERR_INVALID_ARG;
    rtm::DeviceContext d;
    const int st = device_with_limit(&d, wait_limit_ns);
    if (st != GEMM_OK)
        return st;
    rtm::W4Launch L{(int)M, (int)N, (int)K, group, 0, A, codes, scales, zeros, C};
    return finish(rtm::launch_w4_tc(L, K, d, true, static_cast<cudaStream_t>(stream)));
}

int gemm_q8tbf16f32_selftest_timeout(int64_t M, int64_t N, int64_t K, const int8_t *codes,
                                     const float *scales, const uint16_t *dY, float *dW,
                                     int64_t wait_limit_ns, void *stream)
{
    if (!limit_ok(wait_limit_ns) || M < 1 || N < 1 || K < 1 || !size_ok(M, K) || !size_ok(K, N) ||
        !size_ok(M, N) || !codes || !scales || !dY || !dW || !rows16(dY, N) ||
        misaligned(codes, 16) || misaligned(scales, 4) || misaligned(dW, 4))
        return GEMM_ERR_INVALID_ARG;
    rtm::DeviceContext d;
    const int st = device_with_limit(&d, wait_limit_ns);
    if (st != GEMM_OK)
        return st;
    rtm::Q8tLaunch L{(int)M, (int)N, (int)K, 0, codes, scales, dY, dW};
    return finish(rtm::launch_q8t_tc(L, N, d, true, static_cast<cudaStream_t>(stream)));
}

int64_t gemm_w4_codes_bytes(int64_t K, int64_t N)
{
    return size_ok(K, N) ? N * rtm::w4_row_bytes(K) : GEMM_ERR_INVALID_ARG;
}

int gemm_bf16_w4_quantize(int64_t K, int64_t N, int group, const uint16_t *W, uint8_t *codes,
                          uint16_t *scales, uint8_t *zeros, void *stream)
{
    return w4_quantize(K, N, group, 0, W, codes, scales, zeros, stream);
}

int gemm_f16_w4_quantize(int64_t K, int64_t N, int group, const uint16_t *W, uint8_t *codes,
                         uint16_t *scales, uint8_t *zeros, void *stream)
{
    return w4_quantize(K, N, group, 1, W, codes, scales, zeros, stream);
}

int gemm_w4_pack(int64_t K, int64_t N, const uint8_t *q, uint8_t *codes, void *stream)
{
    if (!size_ok(K, N))
        return GEMM_ERR_INVALID_ARG;
    if (K == 0 || N == 0)
        return GEMM_OK;
    if (!q || !codes)
        return GEMM_ERR_INVALID_ARG;
    const Range in[1] = {{q, K * N}};
    if (overlaps({codes, N * rtm::w4_row_bytes(K)}, in, 1))
        return GEMM_ERR_INVALID_ARG;
    if (misaligned(codes, 16))
        return GEMM_ERR_ALIGNMENT;
    rtm::DeviceContext d;
    const int st = rtm::device_context(&d);
    if (st != GEMM_OK)
        return st;
    return finish(rtm::launch_w4_pack(K, N, q, codes, static_cast<cudaStream_t>(stream)));
}

int gemm_bf16_w4_dequantize(int64_t K, int64_t N, int group, const uint8_t *codes,
                            const uint16_t *scales, const uint8_t *zeros, uint16_t *W, void *stream)
{
    return w4_dequantize(K, N, group, 0, codes, scales, zeros, W, stream);
}

int gemm_f16_w4_dequantize(int64_t K, int64_t N, int group, const uint8_t *codes,
                           const uint16_t *scales, const uint8_t *zeros, uint16_t *W, void *stream)
{
    return w4_dequantize(K, N, group, 1, codes, scales, zeros, W, stream);
}

int gemm_bf16w4f32(int64_t M, int64_t N, int64_t K, const uint16_t *A, const uint8_t *codes,
                   const uint16_t *scales, const uint8_t *zeros, int group, float *C,
                   void *workspace, int64_t workspace_bytes, void *stream)
{
    return w4_product(M, N, K, 0, A, codes, scales, zeros, group, C, workspace, workspace_bytes,
                      stream);
}

int gemm_f16w4f32(int64_t M, int64_t N, int64_t K, const uint16_t *A, const uint8_t *codes,
                  const uint16_t *scales, const uint8_t *zeros, int group, float *C,
                  void *workspace, int64_t workspace_bytes, void *stream)
{
    return w4_product(M, N, K, 1, A, codes, scales, zeros, group, C, workspace, workspace_bytes,
                      stream);
}

int64_t gemm_w4_workspace_bytes(int64_t M, int64_t N, int64_t K)
{
    if (!size_ok(M, K) || !size_ok(K, N) || !size_ok(M, N))
        return GEMM_ERR_INVALID_ARG;
    return N > 0 && M > rtm::kW4RowsMax ? padded_bytes(M, K) : 0;
}

int64_t gemm_q8t_workspace_bytes(int64_t M, int64_t N, int64_t K)
{
    if (!size_ok(M, K) || !size_ok(K, N) || !size_ok(M, N))
        return GEMM_ERR_INVALID_ARG;
    return K > 0 ? padded_bytes(M, N) : 0;
}

int64_t gemm_q8_codes_bytes(int64_t M, int64_t K)
{
    return size_ok(M, K) ? M * rtm::q8_pitch(K) : GEMM_ERR_INVALID_ARG;
}

int gemm_bf16_q8_quantize(int64_t M, int64_t K, const uint16_t *X, int8_t *codes, float *scales,
                          void *stream)
{
    return q8_quantize(M, K, 0, X, codes, scales, stream);
}

int gemm_f16_q8_quantize(int64_t M, int64_t K, const uint16_t *X, int8_t *codes, float *scales,
                         void *stream)
{
    return q8_quantize(M, K, 1, X, codes, scales, stream);
}

int gemm_bf16_q8_dequantize(int64_t M, int64_t K, const int8_t *codes, const float *scales,
                            uint16_t *X, void *stream)
{
    return q8_dequantize(M, K, 0, codes, scales, X, stream);
}

int gemm_f16_q8_dequantize(int64_t M, int64_t K, const int8_t *codes, const float *scales,
                           uint16_t *X, void *stream)
{
    return q8_dequantize(M, K, 1, codes, scales, X, stream);
}

int gemm_q8tbf16f32(int64_t M, int64_t N, int64_t K, const int8_t *codes, const float *scales,
                    const uint16_t *dY, float *dW, void *workspace, int64_t workspace_bytes,
                    void *stream)
{
    return q8t_product(M, N, K, 0, codes, scales, dY, dW, workspace, workspace_bytes, stream);
}

int gemm_q8tf16f32(int64_t M, int64_t N, int64_t K, const int8_t *codes, const float *scales,
                   const uint16_t *dY, float *dW, void *workspace, int64_t workspace_bytes,
                   void *stream)
{
    return q8t_product(M, N, K, 1, codes, scales, dY, dW, workspace, workspace_bytes, stream);
}

} // extern "C"
