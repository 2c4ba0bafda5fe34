// Checks of arguments that the low-bit and the 8-bit floating-point entry points share.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "gemm.h"

namespace rtm {
namespace api {

constexpr int64_t kMaxDim = 0x7fffff00;  // sizes rounded up to a tile stay below 2^31
constexpr int64_t kMaxElements = (int64_t)1 << 40;  // of one matrix

inline bool size_ok(int64_t rows, int64_t cols)
{
    return rows >= 0 && cols >= 0 && rows <= kMaxDim && cols <= kMaxDim &&
           (rows == 0 || cols <= kMaxElements / rows);
}

inline bool misaligned(const void *p, uintptr_t bytes)
{
    return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) != 0;
}

struct Range {
    const void *p;
    int64_t bytes;
};

// Whether what is written overlaps something that is read (or written).
inline bool overlaps(const Range &out, const Range *in, int count)
{
    const uintptr_t a = reinterpret_cast<uintptr_t>(out.p);
    for (int i = 0; i < count; ++i) {
        const uintptr_t b = reinterpret_cast<uintptr_t>(in[i].p);
        if (out.p && in[i].p && out.bytes > 0 && in[i].bytes > 0 &&
            a < b + (uintptr_t)in[i].bytes && b < a + (uintptr_t)out.bytes)
            return true;
    }
    return false;
}

inline int finish(cudaError_t e)
{
    if (e != cudaSuccess) {
        cudaGetLastError();
        return e == cudaErrorInvalidValue ? GEMM_ERR_INVALID_ARG : GEMM_ERR_LAUNCH;
    }
    return GEMM_OK;
}

} // namespace api
} // namespace rtm
