// Internal declarations of the low-bit products: 4-bit weights with group
// scales (w4) and activations saved in 8 bits (q8). Arguments are validated by
// the caller (lowbit_api.cu).
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace rtm {

constexpr int kW4Block = 128;        // k per packed block of one column
constexpr int kW4BlockBytes = 64;
constexpr int kQ8Rows = 128;         // rows sharing a scale
constexpr int kQ8Pad = 16;           // columns a saved row is padded to a multiple of

inline __host__ __device__ int64_t w4_row_bytes(int64_t K)
{
    return (K + kW4Block - 1) / kW4Block * kW4BlockBytes;
}
inline __host__ __device__ int64_t q8_pitch(int64_t K) { return (K + kQ8Pad - 1) / kQ8Pad * kQ8Pad; }

// What the entry points need of the current device (api.cu).
struct DeviceContext {
    int sms = 0;
    int *err = nullptr;            // device error word
    void *encode_tiled = nullptr;  // cuTensorMapEncodeTiled; null if unavailable
    uint64_t wait_limit_ns = 0;
};
int device_context(DeviceContext *out);  // GEMM_OK or an error status

// lowbit_quant.cu. f16: the 2-byte type (0 bf16, 1 fp16) of W, scales and X.
cudaError_t launch_w4_quantize(int64_t K, int64_t N, int group, int f16, const uint16_t *W,
                               uint8_t *codes, uint16_t *scales, uint8_t *zeros,
                               cudaStream_t stream);
cudaError_t launch_w4_pack(int64_t K, int64_t N, const uint8_t *q, uint8_t *codes,
                           cudaStream_t stream);
cudaError_t launch_w4_dequantize(int64_t K, int64_t N, int group, int f16, const uint8_t *codes,
                                 const uint16_t *scales, const uint8_t *zeros, uint16_t *W,
                                 cudaStream_t stream);
cudaError_t launch_q8_quantize(int64_t M, int64_t K, int f16, const uint16_t *X, int8_t *codes,
                               float *scales, cudaStream_t stream);
cudaError_t launch_q8_dequantize(int64_t M, int64_t K, int f16, const int8_t *codes,
                                 const float *scales, uint16_t *X, cudaStream_t stream);

// A product with 4-bit weights: C (M x N) = A (M x K) . W.
struct W4Launch {
    int M, N, K, group, f16;
    const uint16_t *A;
    const uint8_t *codes;
    const uint16_t *scales;
    const uint8_t *zeros;  // null: every zero point is 8
    float *C;
};
// dW (K x N) = X^T . dY with X (M x K) saved in 8 bits.
struct Q8tLaunch {
    int M, N, K, f16;
    const int8_t *codes;
    const float *scales;
    const uint16_t *dY;
    float *C;
};
// lowbit_tc.cu: the tensor cores. lda, ldy: row stride of A, dY in elements, rows
// on 16-byte boundaries. mute: the failure-detection self-test (no loads are
// issued, every wait runs out, C is left unspecified).
cudaError_t launch_w4_tc(const W4Launch &L, int64_t lda, const DeviceContext &d, bool mute,
                         cudaStream_t stream);
cudaError_t launch_q8t_tc(const Q8tLaunch &L, int64_t ldy, const DeviceContext &d, bool mute,
                          cudaStream_t stream);
// w4_rows.cu: few rows of A (M <= kW4RowsMax), any alignment. 16 rows x 8192 x
// 8192 take 17.5 to 18.1 us, 17 rows on the tensor-core kernel 30 us; a second pass over W
// for more rows was slower than that (24 rows: 37 us).
constexpr int kW4RowsMax = 16;
cudaError_t launch_w4_rows(const W4Launch &L, int sms, cudaStream_t stream);
// lowbit_simt.cu: any alignment.
cudaError_t launch_w4_simt(const W4Launch &L, cudaStream_t stream);
cudaError_t launch_q8t_simt(const Q8tLaunch &L, cudaStream_t stream);

} // namespace rtm
