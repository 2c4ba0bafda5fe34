// What the role-specialised tensor-core kernels share: bounded waits by shared-memory address,
// rings of barriers, register splits and the MMAs' completion.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "kernels.h"
#include "ptx.cuh"

namespace rtm {
namespace roles {

__device__ __forceinline__ uint64_t sdesc_sw128(uint32_t saddr, uint32_t lbo, uint32_t sbo)
{
    return (uint64_t)((saddr >> 4) & 0x3FFFu) | ((uint64_t)((lbo >> 4) & 0x3FFFu) << 16) |
           ((uint64_t)((sbo >> 4) & 0x3FFFu) << 32) | (1ull << 46) | (2ull << 61);
}

__device__ __forceinline__ void give_up(int *err, volatile int *abort)
{
    atomicCAS(err, 0, kDevErrTimeout);
    *abort = 1;
}

// Barriers by their shared-memory address: the roles keep one address each and
// step through their rings by adding to it.
__device__ __forceinline__ bool try_wait(uint32_t bar, uint32_t parity)
{
    uint32_t done;
    asm volatile("{\n\t.reg .pred p;\n\t"
                 "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
                 "selp.u32 %0, 1, 0, p;\n\t}\n"
                 : "=r"(done)
                 : "r"(bar), "r"(parity)
                 : "memory");
    return done != 0;
}

// Whether the phase has completed, without waiting. A look at a barrier takes 130
// to 190 cycles here (shared memory is busy), more than issuing a stage's MMAs
// leaves; so the roles look ahead, before the work they have in hand, and wait
// only where the answer was no.
__device__ __forceinline__ bool peek(uint32_t bar, uint32_t parity)
{
    uint32_t done;
    asm volatile("{\n\t.reg .pred p;\n\t"
                 "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
                 "selp.u32 %0, 1, 0, p;\n\t}\n"
                 : "=r"(done)
                 : "r"(bar), "r"(parity)
                 : "memory");
    return done != 0;
}

__device__ __forceinline__ void arrive(uint32_t bar)
{
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

// Bounded wait: false when the limit passed or another warp gave up. A wait begun
// after that looks once at the barrier and once at the abort flag, so the roles'
// run-out (wait_on) costs its instructions and no polls, each of which may suspend
// the thread. While it polls, the clock and the flag are read once in 64.
__device__ __forceinline__ bool wait_bounded(uint32_t bar, uint32_t parity, uint64_t limit_ns,
                                             volatile int *abort)
{
    if (peek(bar, parity))
        return true;
    if (*abort)
        return false;
    uint64_t t0 = 0;
#pragma unroll 1
    for (uint32_t n = 1;; ++n) {
        if (try_wait(bar, parity))
            return true;
        if (n % 64 == 0) {
            if (*abort)
                return false;
            const uint64_t t = globaltimer_ns();
            if (t0 == 0)
                t0 = t;
            else if (t - t0 > limit_ns)
                return false;
        }
    }
}

// The same for a warp that waits as one. It returns in every case: after a wait
// that gave up (recorded in the error word and the abort flag, which ends the
// other waits too) the roles run through their loops on whatever is there, in
// bounds, so no lane leaves a loop that its mates stay in, and the result is
// unspecified. A vote of the lanes after each wait cost 3 to 8 %, a flag of its own
// in each thread 3 to 5 %. (After a copy that never lands, a barrier that waits for
// its bytes may so see more arrivals than its phase counts: of a product that is void
// already. Holding those arrivals back by a flag or sending them to spare barriers cost
// 2 to 4 % of a product that waits for nothing.)
__device__ __forceinline__ void wait_on(uint32_t bar, uint32_t parity, uint64_t limit_ns, int *err,
                                        volatile int *abort)
{
    if (!wait_bounded(bar, parity, limit_ns, abort))
        give_up(err, abort);
}

// A place in a ring of N barriers 8 bytes apart: its index and how often (mod 2)
// the ring has gone round.
template <int N>
struct Place {
    uint32_t at = 0, phase = 0;
    __device__ __forceinline__ void advance(uint32_t by = 1)
    {
        at += by;
        if (at >= N) {
            at -= N;
            phase ^= 1;
        }
    }
};

template <int R>
__device__ __forceinline__ void regs_dec()
{
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R));
}
template <int R>
__device__ __forceinline__ void regs_inc()
{
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R));
}

// acc += s * v, two at a time.
__device__ __forceinline__ void fma2(float &a0, float &a1, float s, float v0, float v1)
{
    asm("{\n\t.reg .b64 a, v, s;\n\t"
        "mov.b64 a, {%0, %1};\n\t"
        "mov.b64 v, {%2, %3};\n\t"
        "mov.b64 s, {%4, %4};\n\t"
        "fma.rn.f32x2 a, v, s, a;\n\t"
        "mov.b64 {%0, %1}, a;\n\t}\n"
        : "+f"(a0), "+f"(a1)
        : "f"(v0), "f"(v1), "f"(s));
}

__device__ __forceinline__ void sts128(uint32_t addr, uint4 v)
{
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y),
                 "r"(v.z), "r"(v.w)
                 : "memory");
}

// Arrive on `bar` (in both CTAs of a pair, or in `mask`) when the MMAs issued so far are done.
template <bool PAIR>
__device__ __forceinline__ void commit(uint64_t *bar, uint32_t mask)
{
    if constexpr (PAIR)
        umma_commit_pair_multicast(bar, (uint16_t)mask);
    else
        umma_commit(bar);
}

// One lane of the converged warp.
__device__ __forceinline__ bool elect_one()
{
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}\n"
                 : "=r"(p));
    return p != 0;
}

} // namespace roles
} // namespace rtm
