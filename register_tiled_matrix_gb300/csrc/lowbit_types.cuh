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

template <bool F16>
__device__ __forceinline__ uint32_t sub2(uint32_t a, uint32_t b)
{
    uint32_t d;
    if constexpr (F16)
        asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    else
        asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// 2^7 in bf16 and 2^10 in fp16 have ulp 1: a small integer in the low mantissa
// bits adds itself, exactly.
template <bool F16>
__device__ __forceinline__ constexpr uint32_t magic2()
{
    return F16 ? 0x64006400u : 0x43004300u;
}

// (a & mask) | bits in one instruction: written out because the compiler makes two
// of it when mask and bits are both constants.
__device__ __forceinline__ uint32_t and_or(uint32_t a, uint32_t mask, uint32_t bits)
{
    uint32_t d;
    asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(d) : "r"(a), "r"(mask), "r"(bits));
    return d;
}

// Eight 4-bit codes minus their zero point, in order; zz = magic + z, twice.
template <bool F16>
__device__ __forceinline__ uint4 w4_values(uint32_t word, uint32_t zz)
{
    uint32_t v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
        v[j] = sub2<F16>(and_or(word >> (4 * j), 0x000f000fu, magic2<F16>()), zz);
    return make_uint4(v[0], v[1], v[2], v[3]);
}

__device__ __forceinline__ uint4 lds128(uint32_t addr)
{
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}

__device__ __forceinline__ uint32_t lds32(uint32_t addr)
{
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}

} // namespace rtm
