// The two 2-byte types of the low-bit products, by their bit patterns.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

namespace rtm {

template <bool F16>
__device__ __forceinline__ float to_f32(uint16_t bits)
{
    if constexpr (F16)
        return __half2float(__ushort_as_half(bits));
    else
        return __uint_as_float((uint32_t)bits << 16);
}

// Rounded to nearest even, once.
template <bool F16>
__device__ __forceinline__ uint16_t from_f32(float v)
{
    if constexpr (F16)
        return __half_as_ushort(__float2half_rn(v));
    else
        return __bfloat16_as_ushort(__float2bfloat16_rn(v));
}

template <bool F16>
__device__ __forceinline__ uint32_t pack2_f32(float lo, float hi)
{
    return (uint32_t)from_f32<F16>(lo) | ((uint32_t)from_f32<F16>(hi) << 16);
}

// Shift of value i (0..7) of a packed 4-bit word: even values in the low half,
// odd ones in the high half, so that (word >> 4 j) & 0x000f000f holds the
// consecutive pair 2 j, 2 j + 1.
__host__ __device__ constexpr int w4_shift(int i) { return 4 * (i >> 1) + 16 * (i & 1); }

} // namespace rtm
