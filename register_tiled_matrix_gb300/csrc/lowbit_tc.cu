// Products with a low-bit operand on the sm_103a tensor cores (tcgen05):
//
//     w4:  C^T[n][m]  = sum_g s[g][n] * sum_{k in g} (q[k][n] - z[g][n]) * A[m][k]
//     q8t: dW[k][j]   = sum_b s[b][k] * sum_{m in b} q[m][k] * dY[m][j]
//
// Both are sums over a "depth" (k or m) of a low-bit operand, which owns the
// 128 lanes of the accumulator (n or k), times a 2-byte operand, which owns its
// columns (m or j). The scale is constant over a run of the depth (a group) and
// belongs to one lane, so nothing is rounded that the definition does not
// round: the codes minus their zero point are integers of at most 8 bits, exact
// in bf16 and fp16, the tensor core sums their products with the 2-byte values
// of one group in fp32, and the scale multiplies that sum when it is added to
// the running fp32 total. Applied to the codes instead, the scale would cost a
// rounding to 8 or 11 bits of every weight.
//
// One CTA computes 128 lanes x NT columns (NT = 32 .. 256) and its roles are
//  * a raw producer thread: TMA of the packed codes into a ring (8 KB slots);
//  * DW dequantising warpgroups: codes -> integers in bf16/fp16, written to the
//    128-byte-swizzled stage the MMA reads (a w4 thread owns a lane and reads
//    its 64-byte block, a q8 thread 16 channels of a row; neither store nor
//    load meets a bank conflict);
//  * a producer thread: TMA of the 2-byte operand into the same stages, 64 deep;
//  * an MMA thread: one accumulation set in tensor memory per group, SETS sets
//    in turn, so the next group is multiplied while the last one is read;
//  * PW promoting warpgroups: read a set (a lane a thread), multiply it by the
//    lane's scale, add it to fp32 totals in registers, and at the end of the
//    tile store them.
// Scales and zero points are 4-byte asynchronous copies that each thread makes
// for itself many groups ahead (the aligned word around a value of 2 bytes or
// one: it holds a byte of the array, so it lies in the array's pages). Registers move between the warpgroups: few for
// the issuing threads, most for the promoting ones, which keep up to 128 totals.
//
// With few tiles the depth is split over S CTAs of a cluster; their totals meet
// in shared memory and are added in rank order through distributed shared
// memory, so results repeat exactly. Without a split the CTAs are persistent,
// and the stores of one tile overlap the multiplications of the next.
//
// What bounds it: 4096 x 8192 x 8192 (w4) takes 0.41 to 0.43 ms and an 8192^3 weight
// gradient 0.86 to 0.91 ms, 1280 to 1350 and 1210 to 1280 TFLOP/s, 0.63 to 0.71 of the
// measured bf16 rate; groups of 64 take 0.49, of 32 0.82 ms. At 4096^3 the tensor pipe is
// active half of the time and no unit more. A stage passes through four roles, each a
// chain of shared-memory round trips of 130 to 190 cycles, and costs some 850 cycles
// where its MMAs take 512. Which role sets that pace is not measured; on CTA pairs one
// warpgroup converts every stage. Tried and slower: one CTA of 128 x 256 (twice the L2
// reads of the 2-byte operand: 0.77 and 1.58 ms), a forwarding thread with
// cluster-scope releases in the odd CTA (1.64 ms), an MMA loop rolled over the steps
// (1.14 ms), two CTAs an SM at NT <= 64 (64 x 8192 x 8192 38 us against 31).
//
// Every wait is bounded: a thread that gives up records GEMM_ERR_TIMEOUT in the
// device error word, and all threads still reach the barriers at the end.
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>
#include <type_traits>

#include "kernels.h"
#include "lowbit.h"
#include "lowbit_types.cuh"
#include "ptx.cuh"
#include "tc_roles.cuh"

namespace rtm {
namespace lbt {

using namespace roles;

constexpr int LANES = 128;
constexpr int BK = 64;        // depth of a stage: 64 2-byte values = a 128-byte swizzle row
constexpr int BLOCK = 128;    // depth of a raw w4 slot, and the granularity of a split
constexpr int UMMA_K = 16;
constexpr int kThreads = 512;  // four warpgroups: issuing, and three that convert or promote
constexpr uint32_t A_BYTES = LANES * BK * 2;   // 16 KB
constexpr uint32_t ATOM_BYTES = 64 * BK * 2;   // 8 KB: 64 columns x 64 depth, MN-major
constexpr uint32_t RAW_BYTES = 8192;           // w4: 128 lanes x 64 B; q8: 64 rows x 128 B
constexpr int SCALE_SLOTS = 16;
constexpr int SCALE_AHEAD = 14;                // groups a promoting thread copies ahead: a slot
                                               // is written two groups after its last use
constexpr int ZERO_SLOTS = 4;                  // blocks a dequantising thread copies ahead

enum Mode { kW4, kQ8t };

template <int NT>
struct Cfg {
    static constexpr bool PAIR = NT == 256;       // two CTAs to a tile
    static constexpr int TILE_LANES = PAIR ? 2 * LANES : LANES;
    static constexpr int BN = PAIR ? NT / 2 : NT;  // columns staged by a CTA
    static constexpr int DW = NT == 256 ? 1 : 2;  // dequantising warpgroups
    static constexpr int PW = 3 - DW;             // promoting warpgroups
    // Registers a thread after the split: the four warpgroups share what the block
    // was launched with, 4 x 128.
    static constexpr int R_ISSUE = 56, R_DEQUANT = NT == 256 ? 104 : NT == 128 ? 112 : 128;
    static constexpr int R_PROMOTE = NT >= 128 ? 176 : 192;
    static_assert(R_ISSUE + DW * R_DEQUANT + PW * R_PROMOTE <= 512, "register split");
    static constexpr int CPT = NT / PW;           // columns of a promoting thread
    static constexpr int SETS = NT == 256 ? 2 : 4;
    static constexpr uint32_t TMEM_COLS = SETS * NT;
    static constexpr uint32_t B_BYTES = BN * BK * 2;
    static constexpr uint32_t STAGE_BYTES = A_BYTES + B_BYTES;
    static constexpr int STAGES = NT == 256 ? 5 : 4;
    static constexpr int RAW = NT == 256 ? 4 : NT == 128 ? 6 : NT == 64 ? 10 : 12;
    static constexpr uint32_t OFF_RAW = STAGES * STAGE_BYTES;
    static constexpr uint32_t OFF_SCALE = OFF_RAW + RAW * RAW_BYTES;
    static constexpr uint32_t OFF_ZERO = OFF_SCALE + PW * SCALE_SLOTS * LANES * 4;
    static constexpr uint32_t OFF_BARS = OFF_ZERO + DW * ZERO_SLOTS * 4 * LANES * 4;
    static constexpr size_t SMEM_BYTES = OFF_BARS + 512 + 1024 /*align*/;
    static constexpr int PITCH = NT + 4;  // floats per lane of a partial tile
    static_assert(LANES * PITCH * 4 <= OFF_RAW, "a partial tile fits the stages");
    static_assert(SMEM_BYTES <= 227 * 1024, "shared memory");
};

struct Params {
    int lanes, cols, depth;  // w4: N, M, K; q8t: K, N, M
    int group;               // depth of a group: 32, 64 or 128
    const void *scales;      // w4: 2-byte, q8t: fp32; [group][lane]
    const uint8_t *zeros;    // w4: [group][lane], or null
    float *C;
    int *err;
    unsigned long long limit_ns;
    int splits;  // CTAs (pairs) of a cluster, each summing a range of the depth
    int tiles;
    int mute;    // failure-detection self-test: issue no loads
    uint32_t nil;  // 0, which the compiler cannot know (free_slot)
    int c_vec;   // q8t: rows of dW on 16-byte boundaries
};

// kind::f16, D fp32, M = 128 (256 for a pair), N = NT; w4: both operands K-major, q8t: both MN-major.
template <Mode MODE, bool F16, int NT>
__host__ __device__ constexpr uint32_t idesc()
{
    constexpr uint32_t mn = MODE == kQ8t ? 1u : 0u, t = F16 ? 0u : 1u;
    return (1u << 4) | (t << 7) | (t << 10) | (mn << 15) | (mn << 16) |
           ((uint32_t)(NT >> 3) << 17) | ((uint32_t)(Cfg<NT>::TILE_LANES >> 4) << 24);
}

// Four signed bytes, in order. fp16: 1024 + (q + 128) - 1152. bf16 has seven
// mantissa bits, so the sign bit goes to the subtrahend: with u = q mod 128 and
// the sign bit on the exponent's lowest bit, (128 + u) - (sign ? 256 : 128).
template <bool F16>
__device__ __forceinline__ uint2 q8_values(uint32_t word)
{
    if constexpr (F16) {
        const uint32_t u = word ^ 0x80808080u;
        return make_uint2(sub2<true>(__byte_perm(u, 0x64646464u, 0x4140), 0x64806480u),
                          sub2<true>(__byte_perm(u, 0x64646464u, 0x4342), 0x64806480u));
    } else {
        const uint32_t u = word & 0x7f7f7f7fu, s = word & 0x80808080u;
        return make_uint2(sub2<false>(__byte_perm(u, 0x43434343u, 0x4140),
                                      __byte_perm(s, 0x43434343u, 0x4140)),
                          sub2<false>(__byte_perm(u, 0x43434343u, 0x4342),
                                      __byte_perm(s, 0x43434343u, 0x4342)));
    }
}

// Gives a raw slot back to the copies once this warp has its words q, one load
// instruction each. Neither the order of the source nor the arrival's release holds
// back a load whose registers no instruction has asked for yet, and the next copy
// overtook such loads (whole blocks of the slot's next codes appeared). So the
// arrival asks for them: its address is made of a word of each load, masked by
// `nil`, and the vote asks for every lane's.
__device__ __forceinline__ void free_slot(uint32_t bar, const uint4 (&q)[4], uint32_t nil, int lane)
{
    const uint32_t words = q[0].x ^ q[1].x ^ q[2].x ^ q[3].x;
    const uint32_t none = __any_sync(0xffffffffu, (words & nil) != 0) ? 8u : 0u;
    if (lane == 0)
        arrive(bar + none);
}

// First lane and column of a tile, in bands of 2048 lanes, so that the tiles in
// flight share both operands in L2.
template <int NT>
__device__ __forceinline__ void tile_origin(int t, int lanes, int cols, int &l0, int &c0)
{
    constexpr int LT = Cfg<NT>::TILE_LANES, BAND = 2048 / LT;
    const int tl = (lanes + LT - 1) / LT, tc = (cols + NT - 1) / NT;
    const int band = t / (BAND * tc), first = band * BAND;
    const int rows = min(tl - first, BAND), in = t - band * BAND * tc;
    l0 = (first + in % rows) * LT;
    c0 = in / rows * NT;
}

// "This warp's part of a stage is written" to the leading CTA, whose thread issues the
// MMAs. See mbar_arrive_cluster_stage_written for why it is no release at cluster scope: with
// one, 4096 x 8192 x 8192 (w4) takes 802 us and an 8192^3 weight gradient 2204 us (408
// and 860 without).
template <bool PAIR>
__device__ __forceinline__ void arrive_stage(uint32_t bar)
{
    if constexpr (PAIR)
        mbar_arrive_cluster_stage_written(bar);
    else
        arrive(bar);
}

// "This warp has read its part of an accumulation set" to the leading CTA.
template <bool PAIR>
__device__ __forceinline__ void arrive_set(uint32_t bar)
{
    if constexpr (PAIR)
        mbar_arrive_cluster_tmem_free(bar);
    else
        arrive(bar);
}

// The MMA warp's loop; PG: 16-deep steps of a group (8, 4 or 2). The warp shares
// its scheduler with three busy warps, so the loop is kept short: every lane
// runs it (descriptors and counters stay in uniform registers) and one issues.
template <Mode MODE, bool F16, int NT, int PG>
__device__ __forceinline__ void issue_all(const Params &p, uint32_t smem0, uint32_t tmem_base,
                                          int unit, int units, int nstages, int depth,
                                          uint32_t pair_mask, uint64_t *full, uint64_t *empty,
                                          uint64_t *tfull, uint64_t *tempty, uint64_t *drain,
                                          volatile int *abort)
{
    using Cf = Cfg<NT>;
    constexpr bool PAIR = Cf::PAIR;
    constexpr int STEPS = BK / UMMA_K;
    // K-major: rows of 128 B, 8-row groups 1024 B apart, 32 B a step. MN-major:
    // 64-wide atoms ATOM_BYTES apart, 16 rows of 128 B a step.
    constexpr uint32_t LBO = MODE == kW4 ? 16 : ATOM_BYTES;
    constexpr uint32_t ADVANCE = (MODE == kW4 ? UMMA_K * 2 : UMMA_K * 128) >> 4;
    const uint64_t desc0 = sdesc_sw128(smem0, LBO, 1024);
    const bool elected = elect_one();
    const int tail = min(STEPS, (depth - (nstages - 1) * BK + UMMA_K - 1) / UMMA_K);
    Place<Cf::STAGES> stage;
    Place<Cf::SETS> set;
    const uint32_t full_at = smem_u32(full), tempty_at = smem_u32(tempty);
    bool full_seen = false, empty_seen = false;  // what the look ahead said
#pragma unroll 1
    for (int t = unit; t < p.tiles; t += units) {
#pragma unroll 1
        for (int i = 0; i < nstages; ++i) {
            if (!full_seen)
                wait_on(full_at + stage.at * 8, stage.phase, p.limit_ns, p.err, abort);
            tc_fence_after();
            const bool last = i == nstages - 1;
            const int steps = last ? tail : STEPS;
            const uint64_t adesc = desc0 + stage.at * (Cf::STAGE_BYTES >> 4);
            const uint64_t bdesc = adesc + (A_BYTES >> 4);
            Place<Cf::STAGES> next = stage;
            next.advance();
            full_seen = peek(full_at + next.at * 8, next.phase);
#pragma unroll
            for (int kk = 0; kk < STEPS; ++kk)
                if (kk < steps) {
                    const bool begin = PG == 8 ? kk == 0 && (i & 1) == 0 : kk % PG == 0;
                    if (begin) {
                        if (!empty_seen)
                            wait_on(tempty_at + set.at * 8, set.phase ^ 1, p.limit_ns, p.err, abort);
                        tc_fence_after();
                        Place<Cf::SETS> after = set;
                        after.advance();
                        empty_seen = peek(tempty_at + after.at * 8, after.phase ^ 1);
                    }
                    if (elected) {
                        if constexpr (PAIR)
                            umma_f16_pair(tmem_base + set.at * NT, adesc + kk * ADVANCE,
                                          bdesc + kk * ADVANCE, idesc<MODE, F16, NT>(), !begin);
                        else
                            umma_f16(tmem_base + set.at * NT, adesc + kk * ADVANCE,
                                     bdesc + kk * ADVANCE, idesc<MODE, F16, NT>(), !begin);
                    }
                    const bool end = PG == 8 ? kk == STEPS - 1 && (i & 1) == 1 : kk % PG == PG - 1;
                    if (end || (last && kk == steps - 1)) {
                        if (elected)
                            commit<PAIR>(tfull + set.at, pair_mask);
                        set.advance();
                    }
                }
            if (elected)
                commit<PAIR>(empty + stage.at, pair_mask);
            stage = next;
        }
    }
    if (nstages > 0 && unit < p.tiles) {
        if (elected)
            commit<PAIR>(drain, pair_mask & (~pair_mask + 1));  // the even CTA
        volatile int no_abort = 0;
        wait_bounded(smem_u32(drain), 0, p.limit_ns, &no_abort);  // before TMEM is freed
    }
}

template <Mode MODE, bool F16, int NT>
__global__ void __launch_bounds__(kThreads, 1)
    lowbit_tc_kernel(const __grid_constant__ CUtensorMap tm_codes,
                     const __grid_constant__ CUtensorMap tm_b, const Params p)
{
    using Cf = Cfg<NT>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + (-smem_u32(smem_raw) & 1023u);
    uint64_t *raw_full = reinterpret_cast<uint64_t *>(smem + Cf::OFF_BARS);
    uint64_t *raw_empty = raw_full + Cf::RAW;
    uint64_t *full = raw_empty + Cf::RAW;  // a stage: both operands
    uint64_t *empty = full + Cf::STAGES;
    uint64_t *tfull = empty + Cf::STAGES;
    uint64_t *tempty = tfull + Cf::SETS;
    uint64_t *drain = tempty + Cf::SETS;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(drain + 1);
    volatile int *abort = reinterpret_cast<volatile int *>(tmem_slot + 1);
    static_assert((2 * Cf::RAW + 2 * Cf::STAGES + 2 * Cf::SETS + 1) * 8 + 8 <= 512, "barriers");

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int wg = warp >> 2;
    constexpr bool PAIR = Cf::PAIR;
    constexpr int CTAS = PAIR ? 2 : 1;
    const int S = p.splits;
    const uint32_t cta = PAIR || S > 1 ? cluster_ctarank() : 0u;
    const uint32_t rank = cta / CTAS;               // of the depth split
    const uint32_t leader = cta - cta % CTAS;       // the pair's even CTA, which issues the MMAs
    const bool even = cta == leader;
    const int lane_half = even ? 0 : LANES;         // this CTA's lanes of a pair's tile
    const uint32_t pair_mask = 3u << leader;
    const int unit = blockIdx.x / (S * CTAS), units = gridDim.x / (S * CTAS);

    // This CTA's depth: whole blocks, the last one possibly ragged.
    const int blocks = (p.depth + BLOCK - 1) / BLOCK;
    const int per = (blocks + S - 1) / S;
    const int block0 = min(blocks, (int)rank * per), block1 = min(blocks, block0 + per);
    const int d0 = block0 * BLOCK;
    const int depth = max(0, (block1 == blocks ? p.depth : block1 * BLOCK) - d0);
    const int nstages = (depth + BK - 1) / BK;
    const int ngroups = (depth + p.group - 1) / p.group;
    const int group0 = d0 / p.group;

    if (threadIdx.x == 0) {
        for (int i = 0; i < Cf::RAW; ++i) {
            mbar_init(&raw_full[i], 1);
            mbar_init(&raw_empty[i], 4);  // the warps that read the slot
        }
        for (int i = 0; i < Cf::STAGES; ++i) {
            mbar_init(&full[i], 4 * CTAS + 1);  // the warps that write a stage, its bytes
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < Cf::SETS; ++i) {
            mbar_init(&tfull[i], 1);
            mbar_init(&tempty[i], 4 * Cf::PW * CTAS);
        }
        mbar_init(drain, 1);
        *abort = 0;
        fence_mbarrier_init();
        tma_prefetch_desc(&tm_codes);
        tma_prefetch_desc(&tm_b);
    }
    if (warp == 1) {
        if constexpr (PAIR) {
            tmem_alloc_pair(tmem_slot, Cf::TMEM_COLS);
            tmem_relinquish_pair();
        } else {
            tmem_alloc(tmem_slot, Cf::TMEM_COLS);
            tmem_relinquish();
        }
    }
    tc_fence_before();
    __syncthreads();
    if constexpr (PAIR)
        cluster_sync();  // the peer's barriers are initialised before any remote signal
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;

    if (wg == 0) {
        regs_dec<Cf::R_ISSUE>();
        if (warp == 0 && lane == 0 && !p.mute) {
            // ------------------------------------------------ codes
            uint32_t slot = 0, phase = 0, issued = 0, parity = 0;
            const int steps = MODE == kW4 ? (depth + BLOCK - 1) / BLOCK : nstages;
#pragma unroll 1
            for (int t = unit; t < p.tiles && !*abort; t += units) {
                int l0, c0;
                tile_origin<NT>(t, p.lanes, p.cols, l0, c0);
#pragma unroll 1
                for (int i = 0; i < steps; ++i) {
                    if (!wait_bounded(smem_u32(&raw_empty[slot]), phase ^ 1, p.limit_ns, abort)) {
                        give_up(p.err, abort);
                        break;
                    }
                    const uint32_t dst = smem_u32(smem + Cf::OFF_RAW + slot * RAW_BYTES);
                    mbar_arrive_expect_tx(&raw_full[slot], RAW_BYTES);
                    if constexpr (MODE == kW4)
                        tma_load_2d(dst, &tm_codes, &raw_full[slot], (block0 + i) * kW4BlockBytes,
                                    l0 + lane_half);
                    else
                        tma_load_2d(dst, &tm_codes, &raw_full[slot], l0 + lane_half, d0 + i * BK);
                    issued |= 1u << slot;
                    parity = (parity & ~(1u << slot)) | (phase << slot);
                    if (++slot == Cf::RAW) {
                        slot = 0;
                        phase ^= 1;
                    }
                }
            }
            // No copy into this CTA's shared memory may outlive it.
            volatile int no_abort = 0;
#pragma unroll 1
            for (int i = 0; i < Cf::RAW; ++i)
                if (issued & (1u << i))
                    wait_bounded(smem_u32(&raw_full[i]), (parity >> i) & 1u, p.limit_ns, &no_abort);
        } else if (warp == 2 && lane == 0 && !p.mute) {
            // ------------------------------------------------ 2-byte operand
            uint32_t stage = 0, phase = 0;
#pragma unroll 1
            for (int t = unit; t < p.tiles && !*abort; t += units) {
                int l0, c0;
                tile_origin<NT>(t, p.lanes, p.cols, l0, c0);
#pragma unroll 1
                for (int i = 0; i < nstages; ++i) {
                    if (!wait_bounded(smem_u32(&empty[stage]), phase ^ 1, p.limit_ns, abort)) {
                        give_up(p.err, abort);
                        break;
                    }
                    const uint32_t dst = smem_u32(smem + stage * Cf::STAGE_BYTES + A_BYTES);
                    if constexpr (PAIR) {  // each CTA half the columns, both signal the even CTA
                        if (even)
                            mbar_arrive_expect_tx(&full[stage], 2 * Cf::B_BYTES);
                        const uint32_t bar = mapa_shared(smem_u32(&full[stage]), leader);
                        const int cc = c0 + (even ? 0 : Cf::BN);
                        if constexpr (MODE == kW4) {
                            tma_load_2d_pair(dst, &tm_b, bar, d0 + i * BK, cc);
                        } else {
#pragma unroll
                            for (int j = 0; j < Cf::BN / 64; ++j)
                                tma_load_2d_pair(dst + j * ATOM_BYTES, &tm_b, bar, cc + 64 * j,
                                                 d0 + i * BK);
                        }
                    } else {
                        mbar_arrive_expect_tx(&full[stage], Cf::B_BYTES);
                        if constexpr (MODE == kW4) {
                            tma_load_2d(dst, &tm_b, &full[stage], d0 + i * BK, c0);
                        } else {
#pragma unroll
                            for (int j = 0; j < Cf::BN / 64; ++j)
                                tma_load_2d(dst + j * ATOM_BYTES, &tm_b, &full[stage],
                                            c0 + 64 * j, d0 + i * BK);
                        }
                    }
                    if (++stage == Cf::STAGES) {
                        stage = 0;
                        phase ^= 1;
                    }
                }
            }
        } else if (warp == 1 && even) {
            // ------------------------------------------------ MMA issuer
            if (MODE == kQ8t || p.group == 128)
                issue_all<MODE, F16, NT, 8>(p, smem_u32(smem), tmem_base, unit, units, nstages, depth,
                                         pair_mask, full, empty, tfull, tempty, drain, abort);
            else if (p.group == 64)
                issue_all<MODE, F16, NT, 4>(p, smem_u32(smem), tmem_base, unit, units, nstages, depth,
                                         pair_mask, full, empty, tfull, tempty, drain, abort);
            else
                issue_all<MODE, F16, NT, 2>(p, smem_u32(smem), tmem_base, unit, units, nstages, depth,
                                         pair_mask, full, empty, tfull, tempty, drain, abort);
        }
    } else if (wg <= Cf::DW) {
        // ------------------------------------------------ dequantise
        // Warpgroup d takes every DW-th raw slot, in order.
        regs_dec<Cf::R_DEQUANT>();
        // A stage is published (fence, arrival) after the next one's values have been
        // worked out, so the stores are done by then.
        const int d = wg - 1, tid = threadIdx.x & 127;
        const uint32_t base = smem_u32(smem);
        const uint32_t raw_full_at = smem_u32(raw_full), raw_empty_at = smem_u32(raw_empty);
        const uint32_t empty_at = smem_u32(empty);
        const uint32_t full_at =
            PAIR ? mapa_shared(smem_u32(full), leader) : smem_u32(full);
        uint32_t written = 0;  // the stage stored and not yet published: its barrier
        auto publish = [&]() {
            if (written) {
                fence_proxy_async_shared();
                __syncwarp();
                if (lane == 0)
                    arrive_stage<PAIR>(written);
                written = 0;
            }
        };
        Place<Cf::RAW> raw;  // the slot being converted
        raw.at = d;
        uint4 q[4];
        if constexpr (MODE == kW4) {
            const uint32_t zring =
                base + Cf::OFF_ZERO + (uint32_t)(d * ZERO_SLOTS * 4 * LANES + tid) * 4u;
            const int gs = p.group == 32 ? 5 : p.group == 64 ? 6 : 7;
            const int gpb = BLOCK >> gs;  // groups of a block: 1, 2 or 4
            const int nblocks = block1 - block0;
            const int glast = (p.depth - 1) >> gs;
            // 64-byte rows, 64-byte swizzle: quarter c of row r at c ^ (r / 2 mod 4).
            const uint32_t src0 = base + Cf::OFF_RAW + (uint32_t)(tid * 64 + ((tid & 6) << 3));
            const uint32_t dst0 = base + (uint32_t)(tid * 128 + ((tid & 7) << 4));
            auto load = [&]() {
                wait_on(raw_full_at + raw.at * 8, raw.phase, p.limit_ns, p.err, abort);
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    q[c] = lds128((src0 + raw.at * RAW_BYTES) ^ (uint32_t)(c << 4));
            };
            Place<Cf::STAGES> stage;
            int first = d;           // this warpgroup's first block of the tile
            uint32_t tile_stage = 0;  // stages of the tiles before
#pragma unroll 1
            for (int t = unit; t < p.tiles; t += units) {
                int l0, c0;
                tile_origin<NT>(t, p.lanes, p.cols, l0, c0);
                const int n = min(l0 + lane_half + tid, p.lanes - 1);  // past the end: any zero point
                // The words that hold the zero points of this lane in a block's groups:
                // the next block to copy and the low address bits of the next to use.
                int copied = first;
                uintptr_t zp = reinterpret_cast<uintptr_t>(p.zeros) +
                               (uintptr_t)(group0 + first * gpb) * p.lanes + n;
                uint32_t zbits = (uint32_t)zp, zslot = 0;
                auto fetch = [&](uint32_t slot) {
                    if (copied < nblocks)
#pragma unroll 1
                        for (int g = 0; g < gpb; ++g)
                            if (group0 + copied * gpb + g <= glast)
                                cp_async_4_full(zring + (slot * 4 + g) * (LANES * 4u),
                                                reinterpret_cast<const void *>(
                                                    (zp + (uintptr_t)g * p.lanes) & ~uintptr_t(3)));
                    copied += Cf::DW;
                    zp += (uintptr_t)(Cf::DW * gpb) * p.lanes;
                    cp_async_commit();
                };
                if (p.zeros)
#pragma unroll 1
                    for (int a = 0; a < ZERO_SLOTS - 1; ++a)
                        fetch(a);
                if (first < nblocks)
                    load();
                int i = first;
#pragma unroll 1
                for (; i < nblocks; i += Cf::DW) {
                    uint32_t zz[4];
#pragma unroll
                    for (int w = 0; w < 4; ++w)
                        zz[w] = magic2<F16>() | 0x00080008u;
                    if (p.zeros) {
                        fetch((zslot + ZERO_SLOTS - 1) % ZERO_SLOTS);
                        cp_async_wait<ZERO_SLOTS - 1>();
                        auto zero = [&](uint32_t g) {
                            const uint32_t word = lds32(zring + (zslot * 4 + g) * (LANES * 4u));
                            return magic2<F16>() |
                                   ((word >> (8 * ((zbits + g * p.lanes) & 3))) & 15u) * 0x00010001u;
                        };
                        zz[0] = zero(0);
                        zz[1] = gs == 5 ? zero(1) : zz[0];
                        zz[2] = gs < 7 ? zero(64u >> gs) : zz[0];
                        zz[3] = gs == 5 ? zero(3) : zz[2];
                        zbits += (uint32_t)(Cf::DW * gpb) * p.lanes;
                        zslot = (zslot + 1) % ZERO_SLOTS;
                    }
                    if constexpr (Cf::DW == 2) {
                        const uint32_t sn = tile_stage + 2 * i;
                        stage.at = sn % Cf::STAGES;
                        stage.phase = sn / Cf::STAGES & 1;
                    }
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const bool free = peek(empty_at + stage.at * 8, stage.phase ^ 1);
                        uint4 v[8];  // word w of quarter c: k = 32 w + 8 c and up
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            v[c] = w4_values<F16>(h == 0 ? q[c].x : q[c].z, zz[2 * h]);
                            v[4 + c] = w4_values<F16>(h == 0 ? q[c].y : q[c].w, zz[2 * h + 1]);
                        }
                        publish();
                        if (h == 1) {
                            free_slot(raw_empty_at + raw.at * 8, q, p.nil, lane);
                            raw.advance(Cf::DW);
                            if (i + Cf::DW < nblocks)
                                load();
                        }
                        if (2 * i + h >= nstages)
                            break;
                        if (!free)
                            wait_on(empty_at + stage.at * 8, stage.phase ^ 1, p.limit_ns, p.err,
                                    abort);
                        const uint32_t dst = dst0 + stage.at * Cf::STAGE_BYTES;
#pragma unroll
                        for (int c = 0; c < 8; ++c)
                            sts128(dst ^ (uint32_t)(c << 4), v[c]);
                        written = full_at + stage.at * 8;
                        stage.advance();
                    }
                }
                first = i - nblocks;  // the blocks of all tiles alternate
                tile_stage += nstages;
                cp_async_wait<0>();
            }
        } else {
            // Thread: 16 channels (chunk) of rows row + 16 j of a 64-row slot. The
            // chunks of the second 64 channels take the neighbouring row, whose swizzle
            // is off by one: a store's eight threads then cover all banks.
            const int chunk = tid & 7, row = (tid >> 3) ^ (chunk >> 2);
            const uint32_t src0 = base + Cf::OFF_RAW + (uint32_t)(row * 128 + chunk * 16);
            const uint32_t dst0 = base + (uint32_t)(chunk >> 2) * ATOM_BYTES +
                                  (uint32_t)row * 128u + (((2u * (chunk & 3)) ^ (row & 7u)) << 4);
            const int tiles = unit < p.tiles ? (p.tiles - unit + units - 1) / units : 0;
            const int64_t total = (int64_t)tiles * nstages;  // stages of this CTA, tile after tile
            auto load = [&]() {
                wait_on(raw_full_at + raw.at * 8, raw.phase, p.limit_ns, p.err, abort);
                const uint32_t src = src0 + raw.at * RAW_BYTES;
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    q[j] = lds128(src + j * 16 * 128);
            };
            Place<Cf::STAGES> stage;
            stage.at = d;
            if (d < total)
                load();
#pragma unroll 1
            for (int64_t sn = d; sn < total; sn += Cf::DW) {
                const bool free = peek(empty_at + stage.at * 8, stage.phase ^ 1);
                uint4 v[8];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint2 a = q8_values<F16>(q[j].x), b = q8_values<F16>(q[j].y);
                    const uint2 c = q8_values<F16>(q[j].z), e = q8_values<F16>(q[j].w);
                    v[2 * j] = make_uint4(a.x, a.y, b.x, b.y);
                    v[2 * j + 1] = make_uint4(c.x, c.y, e.x, e.y);
                }
                publish();
                free_slot(raw_empty_at + raw.at * 8, q, p.nil, lane);
                raw.advance(Cf::DW);
                if (sn + Cf::DW < total)
                    load();
                if (!free)
                    wait_on(empty_at + stage.at * 8, stage.phase ^ 1, p.limit_ns, p.err, abort);
                const uint32_t dst = dst0 + stage.at * Cf::STAGE_BYTES;
#pragma unroll
                for (int j = 0; j < 4; ++j) {  // rows 16 apart share the swizzle phase
                    sts128(dst + j * 16 * 128, v[2 * j]);
                    sts128((dst ^ 16u) + j * 16 * 128, v[2 * j + 1]);
                }
                written = full_at + stage.at * 8;
                stage.advance(Cf::DW);
            }
        }
        publish();
    } else {
        // ------------------------------------------------ promote and store
        regs_inc<Cf::R_PROMOTE>();
        const int pw = wg - 1 - Cf::DW, quarter = warp & 3;
        const int row = quarter * 32 + lane;  // TMEM lane
        const uint32_t sring =
            smem_u32(smem + Cf::OFF_SCALE) + (uint32_t)(pw * SCALE_SLOTS * LANES + row) * 4u;
        constexpr uintptr_t SB = MODE == kW4 ? 2 : 4;  // bytes of a scale
        const uint32_t tfull_at = smem_u32(tfull);
        const uint32_t tempty_at =
            PAIR ? mapa_shared(smem_u32(tempty), leader) : smem_u32(tempty);
        bool seen = false;
        uint32_t set = 0, set_phase = 0;
        int l0 = 0, c0 = 0;
        uintptr_t sp = 0;    // this lane's next scale to copy
        uint32_t sbyte = 0;  // the low bits of the address of the next scale to use
        // The aligned word that holds the scale of group i, one copy group each.
        auto fetch = [&](int i, int slot) {
            if (i < ngroups)
                cp_async_4_full(sring + (uint32_t)(slot * LANES) * 4u,
                                reinterpret_cast<const void *>(sp & ~uintptr_t(3)));
            sp += (uintptr_t)p.lanes * SB;
            cp_async_commit();
        };
        auto start = [&](int t) {
            tile_origin<NT>(t, p.lanes, p.cols, l0, c0);
            l0 += lane_half;
            const int ln = min(l0 + row, p.lanes - 1);
            sp = reinterpret_cast<uintptr_t>(p.scales) + ((uintptr_t)group0 * p.lanes + ln) * SB;
            sbyte = (uint32_t)sp;
#pragma unroll 1
            for (int a = 0; a < SCALE_AHEAD; ++a)
                fetch(a, a);
        };
        if (unit < p.tiles)
            start(unit);
        float acc[Cf::CPT];
#pragma unroll 1
        for (int t = unit; t < p.tiles; t += units) {
#pragma unroll
            for (int j = 0; j < Cf::CPT; ++j)
                acc[j] = 0.f;
#pragma unroll 1
            for (int i = 0; i < ngroups; ++i) {
                const int slot = i % SCALE_SLOTS;
                fetch(i + SCALE_AHEAD, (i + SCALE_AHEAD) % SCALE_SLOTS);
                cp_async_wait<SCALE_AHEAD>();
                const uint32_t word = lds32(sring + (uint32_t)(slot * LANES) * 4u);
                float s;
                if constexpr (MODE == kW4) {
                    s = to_f32<F16>((uint16_t)(word >> (8 * (sbyte & 2))));
                    sbyte += 2u * (uint32_t)p.lanes;
                } else {
                    s = __uint_as_float(word);
                }
                if (!seen)
                    wait_on(tfull_at + set * 8, set_phase, p.limit_ns, p.err, abort);
                __syncwarp();  // the lanes left the wait each for itself; the load is the warp's
                tc_fence_after();
                if constexpr (PAIR)  // (the other tiles' groups come too slowly for it to help)
                    seen = set + 1 == Cf::SETS ? peek(tfull_at, set_phase ^ 1)
                                               : peek(tfull_at + (set + 1) * 8, set_phase);
                const uint32_t taddr = tmem_base + ((uint32_t)(quarter * 32) << 16) + set * NT +
                                       (uint32_t)(pw * Cf::CPT);
#pragma unroll
                for (int c = 0; c < Cf::CPT; c += 32) {
                    uint32_t v[32];
                    tmem_ld_32x32b_x32(taddr + c, v);
                    tmem_wait_ld();
                    if (c + 32 == Cf::CPT) {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0)
                            arrive_set<PAIR>(tempty_at + set * 8);
                    }
#pragma unroll
                    for (int j = 0; j < 32; j += 2)
                        fma2(acc[c + j], acc[c + j + 1], s, __uint_as_float(v[j]),
                             __uint_as_float(v[j + 1]));
                }
                if (++set == Cf::SETS) {
                    set = 0;
                    set_phase ^= 1;
                }
            }
            if (S > 1) {
                const uint32_t part =
                    smem_u32(smem) + (uint32_t)(row * Cf::PITCH + pw * Cf::CPT) * 4u;
#pragma unroll
                for (int j = 0; j < Cf::CPT; j += 4)
                    sts128(part + 4 * j,
                           make_uint4(__float_as_uint(acc[j]), __float_as_uint(acc[j + 1]),
                                      __float_as_uint(acc[j + 2]), __float_as_uint(acc[j + 3])));
                break;
            }
            const int gl = l0 + row, gc = c0 + pw * Cf::CPT;
            if (t + units < p.tiles)
                start(t + units);
            if (gl < p.lanes) {
                if constexpr (MODE == kW4) {  // a warp's lanes: 32 consecutive floats of a row of C
                    float *cp = p.C + (int64_t)gc * p.lanes + gl;
                    const int rows = p.cols - gc;
#pragma unroll
                    for (int j = 0; j < Cf::CPT; ++j, cp += p.lanes)
                        if (j < rows)
                            *cp = acc[j];
                } else {
                    float *cp = p.C + (int64_t)gl * p.cols + gc;
                    const int cols = p.cols - gc;
#pragma unroll
                    for (int j = 0; j < Cf::CPT; j += 4) {
                        if (p.c_vec && j + 3 < cols) {
                            *reinterpret_cast<float4 *>(cp + j) =
                                make_float4(acc[j], acc[j + 1], acc[j + 2], acc[j + 3]);
                        } else {
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                if (j + e < cols)
                                    cp[j + e] = acc[j + e];
                        }
                    }
                }
            }
        }
        cp_async_wait<0>();
    }
    __syncwarp();  // the barriers below are the whole warp's

    if (S > 1) {
        cluster_sync();  // every partial tile of the cluster is in shared memory
        if (wg > Cf::DW) {
            int l0, c0;
            tile_origin<NT>(unit, p.lanes, p.cols, l0, c0);
            l0 += lane_half;
            const int row = threadIdx.x & 127, pw = wg - 1 - Cf::DW;
            const int cols = NT / S, first = (int)rank * cols;
            const uint32_t mine = smem_u32(smem) + (uint32_t)(row * Cf::PITCH) * 4u;
            const int gl = l0 + row;
            for (int cc = pw * 4; cc < cols; cc += 4 * Cf::PW) {
                const uint32_t off = (uint32_t)(first + cc) * 4u;
                float4 acc = ld_shared_cluster_v4(mapa_shared(mine + off, cta % CTAS));
                for (int q = 1; q < S; ++q) {
                    const float4 v = ld_shared_cluster_v4(
                        mapa_shared(mine + off, (uint32_t)q * CTAS + cta % CTAS));
                    acc.x += v.x;
                    acc.y += v.y;
                    acc.z += v.z;
                    acc.w += v.w;
                }
                const float a[4] = {acc.x, acc.y, acc.z, acc.w};
                const int gc = c0 + first + cc;
                if (gl < p.lanes) {
                    if constexpr (MODE == kW4) {
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (gc + e < p.cols)
                                p.C[(int64_t)(gc + e) * p.lanes + gl] = a[e];
                    } else {
                        float *cp = p.C + (int64_t)gl * p.cols + gc;
                        if (p.c_vec && gc + 3 < p.cols) {
                            *reinterpret_cast<float4 *>(cp) = acc;
                        } else {
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                if (gc + e < p.cols)
                                    cp[e] = a[e];
                        }
                    }
                }
            }
        }
        cluster_sync();  // no CTA leaves while a peer may still read its partial
    }

    tc_fence_before();
    __syncthreads();
    // No copy into this CTA's shared memory may outlive it. The MMAs waited for every
    // stage's bytes, unless a role gave up: then copies that nobody waited for get
    // the time of a wait to land. (A pair's CTAs leave together, below.)
    if (threadIdx.x == 0 && *abort) {
        const uint64_t t0 = globaltimer_ns();
        while (globaltimer_ns() - t0 < p.limit_ns) {
        }
    }
    __syncwarp();
    if constexpr (PAIR)
        cluster_sync();  // no CTA leaves while its peer may still signal or read it
    if (warp == 1) {
        tc_fence_after();
        if constexpr (PAIR)
            tmem_dealloc_pair(tmem_base, Cf::TMEM_COLS);
        else
            tmem_dealloc(tmem_base, Cf::TMEM_COLS);
    }
}

typedef CUresult (*EncodeTiledFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                  const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                  const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// rows x cols values of `elem` bytes, rows ld values apart, boxes of box_rows x box_cols.
static bool encode_map(EncodeTiledFn fn, CUtensorMap *map, CUtensorMapDataType type, int elem,
                       const void *base, uint64_t rows, uint64_t cols, uint64_t ld,
                       uint32_t box_rows, uint32_t box_cols, CUtensorMapSwizzle swizzle)
{
    cuuint64_t dims[2] = {cols, rows};
    cuuint64_t strides[1] = {ld * elem};
    cuuint32_t box[2] = {box_cols, box_rows};
    cuuint32_t estr[2] = {1, 1};
    return fn(map, type, 2, const_cast<void *>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <Mode MODE, bool F16, int NT>
static cudaError_t launch_nt(Params p, const CUtensorMap &codes, const CUtensorMap &b, int sms,
                             cudaStream_t stream)
{
    using Cf = Cfg<NT>;
    auto kernel = lowbit_tc_kernel<MODE, F16, NT>;
    static std::atomic<uint64_t> done{0};
    cudaError_t e = set_smem_limit_once(kernel, (int)Cf::SMEM_BYTES, done);
    if (e != cudaSuccess)
        return e;
    constexpr int CTAS = Cf::PAIR ? 2 : 1;
    const int64_t tiles = (int64_t)((p.lanes + Cf::TILE_LANES - 1) / Cf::TILE_LANES) *
                          ((p.cols + NT - 1) / NT);
    if (tiles > 0x1fffffff)
        return cudaErrorInvalidValue;
    p.tiles = (int)tiles;
    // Few tiles: split the depth while every CTA keeps at least two blocks (a pair
    // four) and all clusters (of at most 8 CTAs) are resident at once. Single CTAs
    // of two blocks against four: w4 24 x 1024 x 1024 7.6 and 8.8 us, 64 x 4096 x
    // 1024 9.8 and 10.7 us; pairs: w4 300 x 1000 x 504 16.2 and 14.0 us, q8t with
    // 1024 tokens of 1024 x 512 18.0 and 17.1 us.
    constexpr int LEAST = Cf::PAIR ? 4 : 2;
    const int blocks = (p.depth + BLOCK - 1) / BLOCK;
    int splits = 1;
    while (splits * CTAS < 8 && tiles * splits * CTAS * 2 <= sms && blocks >= splits * 2 * LEAST)
        splits *= 2;
    static std::atomic<int> resident[4][64] = {};  // clusters of 1, 2, 4, 8
    int fit = sms;
    for (; splits * CTAS > 1; splits /= 2) {
        const int size = splits * CTAS;
        const int slot = size == 2 ? 1 : size == 4 ? 2 : 3;
        fit = resident_clusters(kernel, size, kThreads, Cf::SMEM_BYTES, resident[slot]);
        if (fit <= 0)
            fit = sms / size;
        if (tiles <= fit || splits == 1)
            break;
    }
    if (splits * CTAS == 1)
        fit = sms;
    p.splits = splits;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((tiles < fit ? tiles : fit) * splits * CTAS), 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = Cf::SMEM_BYTES;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)(splits * CTAS);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, codes, b, p);
}

static int columns_of(int cols, bool narrow)
{
    return cols <= 32 && narrow ? 32 : cols <= 64 ? 64 : cols <= 128 ? 128 : 256;
}

static Params params_of(const DeviceContext &d, bool mute)
{
    Params p = {};
    p.err = d.err;
    p.limit_ns = d.wait_limit_ns;
    p.mute = mute ? 1 : 0;
    return p;
}

template <bool F16>
static cudaError_t w4_typed(const W4Launch &L, int64_t lda, const DeviceContext &d, bool mute,
                            cudaStream_t stream)
{
    auto fn = reinterpret_cast<EncodeTiledFn>(d.encode_tiled);
    const int nt = columns_of(L.M, true);
    CUtensorMap codes, b;
    if (!fn ||
        !encode_map(fn, &codes, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, L.codes, (uint64_t)L.N,
                    (uint64_t)w4_row_bytes(L.K), (uint64_t)w4_row_bytes(L.K), LANES, kW4BlockBytes,
                    CU_TENSOR_MAP_SWIZZLE_64B) ||
        !encode_map(fn, &b, F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                    2, L.A, (uint64_t)L.M, (uint64_t)L.K, (uint64_t)lda, (uint32_t)(nt < 128 ? nt : 128), BK,
                    CU_TENSOR_MAP_SWIZZLE_128B))
        return cudaErrorInvalidValue;
    Params p = params_of(d, mute);
    p.lanes = L.N;
    p.cols = L.M;
    p.depth = L.K;
    p.group = L.group;
    p.scales = L.scales;
    p.zeros = L.zeros;
    p.C = L.C;
    return nt == 32    ? launch_nt<kW4, F16, 32>(p, codes, b, d.sms, stream)
           : nt == 64  ? launch_nt<kW4, F16, 64>(p, codes, b, d.sms, stream)
           : nt == 128 ? launch_nt<kW4, F16, 128>(p, codes, b, d.sms, stream)
                       : launch_nt<kW4, F16, 256>(p, codes, b, d.sms, stream);
}

template <bool F16>
static cudaError_t q8t_typed(const Q8tLaunch &L, int64_t ldy, const DeviceContext &d, bool mute,
                             cudaStream_t stream)
{
    auto fn = reinterpret_cast<EncodeTiledFn>(d.encode_tiled);
    const int nt = columns_of(L.N, false);
    CUtensorMap codes, b;
    if (!fn ||
        !encode_map(fn, &codes, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, L.codes, (uint64_t)L.M,
                    (uint64_t)q8_pitch(L.K), (uint64_t)q8_pitch(L.K), BK, LANES,
                    CU_TENSOR_MAP_SWIZZLE_NONE) ||
        !encode_map(fn, &b, F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                    2, L.dY, (uint64_t)L.M, (uint64_t)L.N, (uint64_t)ldy, BK, 64,
                    CU_TENSOR_MAP_SWIZZLE_128B))
        return cudaErrorInvalidValue;
    Params p = params_of(d, mute);
    p.lanes = L.K;
    p.cols = L.N;
    p.depth = L.M;
    p.group = kQ8Rows;
    p.scales = L.scales;
    p.C = L.C;
    p.c_vec = L.N % 4 == 0 && (reinterpret_cast<uintptr_t>(L.C) & 15) == 0;
    return nt == 64    ? launch_nt<kQ8t, F16, 64>(p, codes, b, d.sms, stream)
           : nt == 128 ? launch_nt<kQ8t, F16, 128>(p, codes, b, d.sms, stream)
                       : launch_nt<kQ8t, F16, 256>(p, codes, b, d.sms, stream);
}

} // namespace lbt

cudaError_t launch_w4_tc(const W4Launch &L, int64_t lda, const DeviceContext &d, bool mute,
                         cudaStream_t stream)
{
    return L.f16 ? lbt::w4_typed<true>(L, lda, d, mute, stream)
                 : lbt::w4_typed<false>(L, lda, d, mute, stream);
}

cudaError_t launch_q8t_tc(const Q8tLaunch &L, int64_t ldy, const DeviceContext &d, bool mute,
                          cudaStream_t stream)
{
    return L.f16 ? lbt::q8t_typed<true>(L, ldy, d, mute, stream)
                 : lbt::q8t_typed<false>(L, ldy, d, mute, stream);
}

} // namespace rtm
