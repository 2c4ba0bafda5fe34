// Products of e4m3 operands with an fp32 scale for each block of 128, on the sm_103a tensor
// cores (tcgen05, kind::f8f6f4):
//
//     forward  Y[m][n]  = sum_b a[m][b] w[b][n/128] * sum_{k in b} A[m][k] W[k][n]
//     input    dX[m][k] = sum_b y[m][b] w[k/128][b] * sum_{n in b} dY[m][n] W[k][n]
//     weight   dW[k][n] = sum_b x[b][k] y[b][n]     * sum_{m in b} X[m][k] dY[m][n]
//
// The scales are constant over a block b of 128 of the summed axis (the depth), so the tensor
// core sums one block's products of codes in fp32 (a product of two codes is exact) and the
// scales multiply that sum as it is added to the running fp32 total.
//
// One CTA computes 128 lanes x NT columns, a pair of CTAs 256 x 256. Its roles are
//  * a producer thread: TMA of both operands' next 128 of depth into a ring of stages. A code is
//    a byte, so a stage's row is one 128-byte swizzle row, along the depth or across it: the
//    tensor core reads both, and no operand is ever transposed;
//  * an MMA warp: a stage is four steps of 32 into one accumulation set in tensor memory, SETS
//    sets in turn, so the next block is multiplied while the last one is read;
//  * PW promoting warpgroups: read a set (a lane a thread), scale it into fp32 totals in
//    registers, and store them at the end of the tile.
// Rows of A are the lanes: a thread's scale is its row's times the tile's of W. With few rows
// W's columns take the lanes instead (SWAP) and 16 to 64 rows of A the accumulator's columns,
// so that no lane idles and W is read once; the rows' scales then come through shared memory,
// as the columns' of a weight gradient do.
//
// Experts: rows offsets[e] .. offsets[e+1]-1 belong to expert e. The offsets stay on the device;
// every CTA turns them into a running count of tiles in shared memory and finds a tile's expert
// by bisection. Offsets are taken as ascending within 0 .. rows, whatever they hold, so no
// access leaves the arrays.
//
// With few tiles the depth is split over S CTAs (pairs) of a cluster; their totals meet in
// shared memory and are added in rank order, so results repeat exactly. Without a split the
// CTAs are persistent.
//
// Every wait is bounded: a thread that gives up records GEMM_ERR_TIMEOUT in the device error
// word, and all threads still reach the barriers at the end.
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "f8.h"
#include "kernels.h"
#include "lowbit_types.cuh"
#include "ptx.cuh"
#include "tc_roles.cuh"

namespace rtm {
namespace f8t {

using namespace roles;

constexpr int LANES = 128;
constexpr int BK = kF8Block;   // depth of a stage: 128 codes = a 128-byte swizzle row
constexpr int UMMA_K = 32;
constexpr uint32_t A_BYTES = LANES * BK;  // 16 KB
constexpr int kMaxGroups = kRouteMaxExperts;
// The scales' ring. A slot is written SCALE_AHEAD blocks ahead of use, when the accumulation set
// of SETS blocks ago is full, so the promoting warps are through with all but the last
// 2 * SETS + 2 blocks.
constexpr int SCALE_SLOTS = 16, SCALE_AHEAD = 6;
constexpr int SCALERS = 2;  // warps

template <int NT, bool SWAP>
struct Cfg {
    static constexpr bool PAIR = NT == 256;
    static constexpr int CTAS = PAIR ? 2 : 1;
    static constexpr int TILE_LANES = PAIR ? 2 * LANES : LANES;
    static constexpr int ROWS = SWAP ? NT : TILE_LANES;  // of C in a tile
    static constexpr int COLS = SWAP ? TILE_LANES : NT;
    static constexpr int BN = PAIR ? NT / 2 : NT;  // columns staged by a CTA
    static constexpr int PW = SWAP ? 1 : 2;        // promoting warpgroups
    static constexpr int THREADS = 128 * (1 + PW);
    // Registers a thread of a pair's warpgroups after the split of 3 x 168.
    static constexpr int R_ISSUE = 48, R_PROMOTE = 224;
    static constexpr int CPT = NT / PW;  // columns of a promoting thread
    static constexpr int CH = CPT < 32 ? CPT : 32;  // read from tensor memory at once
    static constexpr int SETS = PAIR ? 2 : 4;
    static constexpr uint32_t TMEM_COLS = SETS * NT;
    static constexpr uint32_t B_BYTES = BN * BK;
    static constexpr uint32_t STAGE_BYTES = A_BYTES + B_BYTES;
    // Floats of a slot: the lanes' scales or none, the columns' or none, the tiles'.
    static constexpr int SCALE_COLUMNS = SWAP ? 0 : LANES, SCALE_TILE = SCALE_COLUMNS + NT;
    static constexpr int SCALE_PITCH = SCALE_TILE + 4;

    static_assert(SCALE_AHEAD + 2 * SETS + 2 <= SCALE_SLOTS, "scales are read before their slot is written");
    // (Of a pair's six stages the sixth is the boxes' room: 8192^3 takes as long with five.)
    static constexpr int STAGES = PAIR ? 5 : NT >= 128 ? 6 : NT == 64 ? 8 : 10;
    static constexpr int PITCH = NT + 4;  // floats per lane of a partial tile
    // Partial tiles have room of their own where the stages are too small.
    static constexpr uint32_t OFF_GROUPS = STAGES * STAGE_BYTES;
    static constexpr uint32_t OFF_SCALE = OFF_GROUPS + 2 * (kMaxGroups + 4) * 4;
    // A pair's warps stage 16 columns of their 32 rows of C at a time, twice.
    static constexpr uint32_t BOX_BYTES = 32 * 16 * 4;
    static constexpr uint32_t OFF_BOXES = (OFF_SCALE + SCALE_SLOTS * SCALE_PITCH * 4 + 1023) / 1024 * 1024;
    static constexpr uint32_t OFF_BARS = PAIR ? OFF_BOXES + 4 * PW * 2 * BOX_BYTES
                                              : OFF_SCALE + SCALE_SLOTS * SCALE_PITCH * 4;
    static constexpr size_t SMEM_BYTES = OFF_BARS + 256 + 1024 /*align*/;
    static_assert(LANES * PITCH * 4 <= OFF_GROUPS, "a partial tile fits the stages");
    static_assert(SMEM_BYTES <= 227 * 1024, "shared memory");
};

// "This warp has read its part of an accumulation set" to the leading CTA.
template <bool PAIR>
__device__ __forceinline__ void arrive_set(uint32_t bar)
{
    if constexpr (PAIR)
        mbar_arrive_cluster_tmem_free(bar);
    else
        arrive(bar);
}

struct Params {
    int rows, cols;     // of C; weight: of one matrix C
    int depth;          // weight: rows of X and dY
    int groups;         // experts
    const int32_t *offsets;
    const float *a_scales, *b_scales;
    float *C;
    int *err;
    unsigned long long limit_ns;
    int splits;
    int mute;
    int c_vec;  // rows of C on 8-byte boundaries
    int c_boxes;  // on 16-byte boundaries: tiles of pairs are stored in boxes
};

// kind::f8f6f4, D fp32, both operands e4m3, M = 128 (256 for a pair), N = NT.
template <int NT, bool SWAP>
__host__ __device__ constexpr uint32_t idesc(bool lanes_mn, bool cols_mn)
{
    return (1u << 4) | ((lanes_mn ? 1u : 0u) << 15) | ((cols_mn ? 1u : 0u) << 16) |
           ((uint32_t)(NT >> 3) << 17) | ((uint32_t)(Cfg<NT, SWAP>::TILE_LANES >> 4) << 24);
}

// acc += v * (s0, s1), two at a time.
__device__ __forceinline__ void fma2_each(float &a0, float &a1, float v0, float v1, float s0, float s1)
{
    asm("{\n\t.reg .b64 a, v, s;\n\t"
        "mov.b64 a, {%0, %1};\n\t"
        "mov.b64 v, {%2, %3};\n\t"
        "mov.b64 s, {%4, %5};\n\t"
        "fma.rn.f32x2 a, v, s, a;\n\t"
        "mov.b64 {%0, %1}, a;\n\t}\n"
        : "+f"(a0), "+f"(a1)
        : "f"(v0), "f"(v1), "f"(s0), "f"(s1));
}

// v * s, two at a time.
__device__ __forceinline__ void mul2(float &v0, float &v1, float s)
{
    asm("{\n\t.reg .b64 v, s;\n\t"
        "mov.b64 v, {%0, %1};\n\t"
        "mov.b64 s, {%2, %2};\n\t"
        "mul.rn.f32x2 v, v, s;\n\t"
        "mov.b64 {%0, %1}, v;\n\t}\n"
        : "+f"(v0), "+f"(v1)
        : "f"(s));
}

template <int N>
__device__ __forceinline__ void tmem_load(uint32_t taddr, uint32_t (&v)[N])
{
    if constexpr (N == 16)
        tmem_ld_32x32b_x16(taddr, v);
    else
#pragma unroll
        for (int i = 0; i < N; i += 32)
            tmem_ld_32x32b_x32(taddr + i, *reinterpret_cast<uint32_t(*)[32]>(v + i));
}

// Waits for the loads so far; what uses v comes after.
template <int N>
__device__ __forceinline__ void tmem_arrived(uint32_t (&v)[N])
{
    tmem_wait_ld();
#pragma unroll
    for (int i = 0; i < N; ++i)
        asm volatile("" : "+r"(v[i]));
}

__device__ __forceinline__ float2 lds_f32x2(uint32_t addr)
{
    float2 v;
    asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr) : "memory");
    return v;
}

__device__ __forceinline__ void sts_f32x2(uint32_t addr, float a, float b)
{
    asm volatile("st.shared.v2.f32 [%0], {%1, %2};" ::"r"(addr), "f"(a), "f"(b) : "memory");
}

__device__ __forceinline__ float lds_f32(uint32_t addr) { return __uint_as_float(lds32(addr)); }

// What a tile is: its expert, first row and column of C, the rows' end, and the depth it sums.
struct Tile {
    int group, r0, c0, row_end;
    int d0, depth;  // weight: first row of X and dY, and how many
};

template <int MODE, int NT, bool SWAP>
struct Schedule {
    using Cf = Cfg<NT, SWAP>;
    uint32_t start;  // shared memory: groups + 1 row offsets, and as many running tile counts
    const Params *p;

    static constexpr uint32_t TILES = (kMaxGroups + 4) * 4;
    __device__ __forceinline__ int total() const { return (int)lds32(start + TILES + p->groups * 4); }

    __device__ __forceinline__ Tile at(int t) const
    {
        int lo = 0, hi = p->groups - 1;  // the last group with tiles[g] <= t
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if ((int)lds32(start + TILES + mid * 4) <= t)
                lo = mid;
            else
                hi = mid - 1;
        }
        Tile x;
        x.group = lo;
        const int begin = (int)lds32(start + lo * 4), end = (int)lds32(start + lo * 4 + 4);
        const int local = t - (int)lds32(start + TILES + lo * 4);
        const int first = MODE == kF8Weight ? 0 : begin;
        x.row_end = MODE == kF8Weight ? p->rows : end;
        x.d0 = MODE == kF8Weight ? begin : 0;
        x.depth = MODE == kF8Weight ? end - begin : p->depth;
        // In bands of 2048 rows, so that the tiles in flight share both operands in L2.
        constexpr int BAND = 2048 / Cf::ROWS;
        const int tr = (x.row_end - first + Cf::ROWS - 1) / Cf::ROWS;
        const int tc = (p->cols + Cf::COLS - 1) / Cf::COLS;
        const int band = local / (BAND * tc), row0 = band * BAND;
        const int rows = min(tr - row0, BAND), in = local - band * BAND * tc;
        x.r0 = first + (row0 + in % rows) * Cf::ROWS;
        x.c0 = in / rows * Cf::COLS;
        return x;
    }
};

// This CTA's blocks of a tile's depth.
struct Blocks {
    int first, count;
};
__device__ __forceinline__ Blocks blocks_of(const Tile &x, int splits, int rank)
{
    const int all = (x.depth + BK - 1) / BK, per = (all + splits - 1) / splits;
    const int first = min(all, rank * per);
    return {first, min(all, first + per) - first};
}

// Row offsets and running tile counts of the groups, by one warp.
template <int MODE, int NT, bool SWAP>
__device__ __forceinline__ void count_tiles(const Params &p, int32_t *start, int32_t *tiles, int lane)
{
    using Cf = Cfg<NT, SWAP>;
    const int most = MODE == kF8Weight ? p.depth : p.rows;
    const int tc = (p.cols + Cf::COLS - 1) / Cf::COLS;
    const int each = (p.rows + Cf::ROWS - 1) / Cf::ROWS * tc;  // weight: the same for every group
    int low = 0, sum = 0;
    if (p.offsets)
        low = min(max(p.offsets[0], 0), most);
    if (lane == 0) {
        start[0] = low;
        tiles[0] = 0;
    }
    for (int b = 0; b < p.groups; b += 32) {
        const int g = b + lane;
        int hi = 0;
        if (g < p.groups)
            hi = p.offsets ? min(max(p.offsets[g + 1], 0), most) : most;
        hi = max(hi, low);
#pragma unroll
        for (int o = 1; o < 32; o *= 2) {
            const int y = __shfl_up_sync(0xffffffffu, hi, o);
            if (lane >= o)
                hi = max(hi, y);
        }
        int before = __shfl_up_sync(0xffffffffu, hi, 1);
        if (lane == 0)
            before = low;
        int n = 0;
        if (g < p.groups)
            n = MODE == kF8Weight ? each : (hi - before + Cf::ROWS - 1) / Cf::ROWS * tc;
#pragma unroll
        for (int o = 1; o < 32; o *= 2) {
            const int y = __shfl_up_sync(0xffffffffu, n, o);
            if (lane >= o)
                n += y;
        }
        if (g < p.groups) {
            start[g + 1] = hi;
            tiles[g + 1] = sum + n;
        }
        sum += __shfl_sync(0xffffffffu, n, 31);
        low = __shfl_sync(0xffffffffu, hi, 31);
    }
}

template <int MODE, int NT, bool SWAP>
__global__ void __launch_bounds__(Cfg<NT, SWAP>::THREADS, 1)
    f8_tc_kernel(const __grid_constant__ CUtensorMap tm_lanes,
                 const __grid_constant__ CUtensorMap tm_cols,
                 const __grid_constant__ CUtensorMap tm_c, const Params p)
{
    using Cf = Cfg<NT, SWAP>;
    constexpr bool PAIR = Cf::PAIR;
    constexpr int CTAS = Cf::CTAS;
    // Which operand is W (batched by expert), and which lie with the depth along their rows.
    constexpr bool LANES_MN = SWAP ? MODE == kF8Forward : MODE == kF8Weight;
    constexpr bool COLS_MN = SWAP ? false : MODE != kF8Input;
    constexpr bool COLUMN_SCALES = SWAP || MODE == kF8Weight;
    // Read from tensor memory as matrix fragments: a thread then has 4 lanes of a quarter of the
    // columns, so a warp stores 32 bytes of each of eight rows of C at a time whatever their
    // alignment, and a weight gradient's thread loads half as many of the columns' scales (8192^3
    // 492 us, a lane a thread 550). On pairs a lane a thread is the faster form of the others:
    // one scale a thread, and shared memory is what they wait for (420 us, fragments 480).
    constexpr bool FRAGMENTS = !SWAP && (MODE == kF8Weight || !PAIR);
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + (-smem_u32(smem_raw) & 1023u);
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + Cf::OFF_BARS);
    uint64_t *empty = full + Cf::STAGES;
    uint64_t *tfull = empty + Cf::STAGES;
    uint64_t *tempty = tfull + Cf::SETS;
    uint64_t *drain = tempty + Cf::SETS;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(drain + 1);
    volatile int *abort = reinterpret_cast<volatile int *>(tmem_slot + 1);
    static_assert((2 * Cf::STAGES + 2 * Cf::SETS + 1) * 8 + 8 <= 256, "barriers");

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int wg = warp >> 2;
    const int S = p.splits;
    const uint32_t cta = PAIR || S > 1 ? cluster_ctarank() : 0u;
    const int rank = cta / CTAS;                   // of the depth split
    const uint32_t leader = cta - cta % CTAS;      // the pair's even CTA, which issues the MMAs
    const bool even = cta == leader;
    const int half = even ? 0 : LANES;             // this CTA's lanes of a pair's tile
    const uint32_t pair_mask = 3u << leader;
    const int unit = blockIdx.x / (S * CTAS), units = gridDim.x / (S * CTAS);

    if (threadIdx.x == 0) {
        for (int i = 0; i < Cf::STAGES; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < Cf::SETS; ++i) {
            mbar_init(&tfull[i], 1 + SCALERS);  // the MMAs, the block's scales
            mbar_init(&tempty[i], 4 * Cf::PW * CTAS);
        }
        mbar_init(drain, 1);
        *abort = 0;
        fence_mbarrier_init();
        tma_prefetch_desc(&tm_lanes);
        tma_prefetch_desc(&tm_cols);
        if (PAIR && p.c_boxes)
            tma_prefetch_desc(&tm_c);
    }
    __syncwarp();
    if (warp == 1) {
        if constexpr (PAIR) {
            tmem_alloc_pair(tmem_slot, Cf::TMEM_COLS);
            tmem_relinquish_pair();
        } else {
            tmem_alloc(tmem_slot, Cf::TMEM_COLS);
            tmem_relinquish();
        }
    }
    if (warp == 2) {
        int32_t *start = reinterpret_cast<int32_t *>(smem + Cf::OFF_GROUPS);
        count_tiles<MODE, NT, SWAP>(p, start, start + kMaxGroups + 4, lane);
    }
    tc_fence_before();
    __syncthreads();
    if constexpr (PAIR)
        cluster_sync();  // the peer's barriers are initialised before any remote signal
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    const Schedule<MODE, NT, SWAP> plan{smem_u32(smem + Cf::OFF_GROUPS), &p};
    const int tiles = plan.total();

    if (wg == 0) {
        if constexpr (PAIR)
            regs_dec<Cf::R_ISSUE>();
        if (warp == 0 && lane == 0 && !p.mute) {
            // ------------------------------------------------ producer
            Place<Cf::STAGES> stage;
            const uint32_t empty_at = smem_u32(empty), base = smem_u32(smem);
            const uint32_t full_at = PAIR ? mapa_shared(smem_u32(full), leader) : smem_u32(full);
            bool gave_up = false, seen = false;  // what the look ahead said
#pragma unroll 1
            for (int t = unit; t < tiles && !gave_up; t += units) {
                const Tile x = plan.at(t);
                const Blocks b = blocks_of(x, S, rank);
                const int l0 = (SWAP ? x.c0 : x.r0) + half;
                const int c0 = (SWAP ? x.r0 : x.c0) + (even ? 0 : Cf::BN);
                const int lane_batch = SWAP ? x.group : 0;
                const int col_batch = !SWAP && MODE != kF8Weight ? x.group : 0;
                int d = x.d0 + b.first * BK;
#pragma unroll 1
                for (int i = 0; i < b.count; ++i, d += BK) {
                    if (!seen &&
                        !wait_bounded(empty_at + stage.at * 8, stage.phase ^ 1, p.limit_ns, abort)) {
                        give_up(p.err, abort);
                        gave_up = true;
                        break;
                    }
                    Place<Cf::STAGES> next = stage;
                    next.advance();
                    seen = peek(empty_at + next.at * 8, next.phase ^ 1);
                    const uint32_t dst = base + stage.at * Cf::STAGE_BYTES;
                    const uint32_t bar = full_at + stage.at * 8;
                    const int lx = LANES_MN ? l0 : d, ly = LANES_MN ? d : l0;
                    const int cx = COLS_MN ? c0 : d, cy = COLS_MN ? d : c0;
                    if constexpr (PAIR) {  // both CTAs' bytes on the even one's barrier
                        if (even)
                            mbar_arrive_expect_tx(&full[stage.at], 2 * Cf::STAGE_BYTES);
                        tma_load_3d_pair(dst, &tm_lanes, bar, lx, ly, lane_batch);
                        tma_load_3d_pair(dst + A_BYTES, &tm_cols, bar, cx, cy, col_batch);
                    } else {
                        mbar_arrive_expect_tx(&full[stage.at], Cf::STAGE_BYTES);
                        tma_load_3d(dst, &tm_lanes, &full[stage.at], lx, ly, lane_batch);
                        tma_load_3d(dst + A_BYTES, &tm_cols, &full[stage.at], cx, cy, col_batch);
                    }
                    stage = next;
                }
            }
        } else if (warp == 1 && even) {
            // ------------------------------------------------ MMA
            // Along the depth: rows of 128 B, 8-row groups 1024 B apart, 32 B a step. Across
            // it: a row of 128 B for each of the depth, 32 rows a step.
            constexpr uint32_t LSTEP = (LANES_MN ? UMMA_K * 128 : UMMA_K) >> 4;
            constexpr uint32_t CSTEP = (COLS_MN ? UMMA_K * 128 : UMMA_K) >> 4;
            constexpr uint32_t ID = idesc<NT, SWAP>(LANES_MN, COLS_MN);
            const uint64_t ldesc0 = sdesc_sw128(smem_u32(smem), LANES_MN ? A_BYTES : 16, 1024);
            const uint64_t cdesc0 = sdesc_sw128(smem_u32(smem) + A_BYTES, COLS_MN ? A_BYTES : 16, 1024);
            const bool elected = elect_one();
            Place<Cf::STAGES> stage;
            Place<Cf::SETS> set;
            const uint32_t full_at = smem_u32(full), tempty_at = smem_u32(tempty);
            bool any = false;
            bool full_seen = false, empty_seen = false;  // what the look ahead said
#pragma unroll 1
            for (int t = unit; t < tiles; t += units) {
                const Blocks b = blocks_of(plan.at(t), S, rank);
#pragma unroll 1
                for (int i = 0; i < b.count; ++i) {
                    if (!empty_seen)
                        wait_on(tempty_at + set.at * 8, set.phase ^ 1, p.limit_ns, p.err, abort);
                    if (!full_seen)
                        wait_on(full_at + stage.at * 8, stage.phase, p.limit_ns, p.err, abort);
                    tc_fence_after();
                    Place<Cf::STAGES> next_stage = stage;
                    next_stage.advance();
                    Place<Cf::SETS> next_set = set;
                    next_set.advance();
                    full_seen = peek(full_at + next_stage.at * 8, next_stage.phase);
                    empty_seen = peek(tempty_at + next_set.at * 8, next_set.phase ^ 1);
                    const uint32_t d = tmem_base + set.at * NT;
                    const uint64_t ldesc = ldesc0 + stage.at * (Cf::STAGE_BYTES >> 4);
                    const uint64_t cdesc = cdesc0 + stage.at * (Cf::STAGE_BYTES >> 4);
                    if (elected) {
#pragma unroll
                        for (int kk = 0; kk < BK / UMMA_K; ++kk) {
                            if constexpr (PAIR)
                                umma_f8_pair(d, ldesc + kk * LSTEP, cdesc + kk * CSTEP, ID, kk > 0);
                            else
                                umma_f8(d, ldesc + kk * LSTEP, cdesc + kk * CSTEP, ID, kk > 0);
                        }
                        commit<PAIR>(tfull + set.at, pair_mask);
                        commit<PAIR>(empty + stage.at, pair_mask);
                    }
                    any = true;
                    set = next_set;
                    stage = next_stage;
                }
            }
            if (any) {
                if (elected)
                    commit<PAIR>(drain, pair_mask & (~pair_mask + 1));  // the even CTA
                volatile int no_abort = 0;
                wait_bounded(smem_u32(drain), 0, p.limit_ns, &no_abort);  // before TMEM is freed
            }
        } else if (warp >= 2) {
            // ------------------------------------------------ scales
            // A thread copies the scales of lanes (columns) id, id + 64, ...
            const int id = threadIdx.x & 63;
            const uint32_t ring = smem_u32(smem + Cf::OFF_SCALE), tfull_at = smem_u32(tfull);
            const int depth_blocks = (p.depth + BK - 1) / BK, col_blocks = (p.cols + BK - 1) / BK;
            constexpr int NL = SWAP ? 0 : LANES / 64;
            constexpr int NC = !COLUMN_SCALES ? 0 : NT < 64 ? 1 : NT / 64;
            const float *lanes[NL > 0 ? NL : 1], *columns[NC > 0 ? NC : 1], *tile = nullptr;
            int tile_step = 0;
            int ft = unit, left = -1;  // the tile whose scales are asked for, its blocks left
            uint32_t fslot = 0;
            auto fetch = [&]() {
                while (left <= 0 && ft < tiles) {  // the next tile that has blocks
                    if (left == 0)
                        ft += units;
                    if (ft >= tiles)
                        break;
                    const Tile x = plan.at(ft);
                    const Blocks b = blocks_of(x, S, rank);
                    left = b.count;
                    const int lane0 = (SWAP ? x.c0 : x.r0) + half, col0 = SWAP ? x.r0 : x.c0;
                    if constexpr (MODE == kF8Weight) {
                        const int64_t block = x.d0 / BK + b.first;
#pragma unroll
                        for (int j = 0; j < NL; ++j)
                            lanes[j] = p.a_scales + block * p.rows + min(lane0 + id + 64 * j, p.rows - 1);
#pragma unroll
                        for (int j = 0; j < NC; ++j)
                            columns[j] = p.b_scales + block * p.cols + min(col0 + id + 64 * j, p.cols - 1);
                    } else {
                        // W's tiles: forward depth x columns, input columns x depth.
                        const int cb = min((SWAP ? lane0 : col0 + (warp - 2) * BK) / BK, col_blocks - 1);
                        tile = p.b_scales + (int64_t)x.group * depth_blocks * col_blocks +
                               (MODE == kF8Forward ? (int64_t)b.first * col_blocks + cb
                                                   : (int64_t)cb * depth_blocks + b.first);
                        tile_step = MODE == kF8Forward ? col_blocks : 1;
#pragma unroll
                        for (int j = 0; j < (SWAP ? NC : NL); ++j)
                            (SWAP ? columns : lanes)[j] =
                                p.a_scales + b.first +
                                (int64_t)min((SWAP ? col0 : lane0) + id + 64 * j, x.row_end - 1) * depth_blocks;
                    }
                }
                if (left > 0) {
                    const uint32_t slot = ring + fslot * (Cf::SCALE_PITCH * 4);
#pragma unroll
                    for (int j = 0; j < NL; ++j) {
                        cp_async_4_full(slot + (id + 64 * j) * 4, lanes[j]);
                        lanes[j] += MODE == kF8Weight ? p.rows : 1;
                    }
#pragma unroll
                    for (int j = 0; j < NC; ++j) {
                        if (NT >= 64 || id < NT)
                            cp_async_4_full(slot + (Cf::SCALE_COLUMNS + id + 64 * j) * 4, columns[j]);
                        columns[j] += MODE == kF8Weight ? p.cols : 1;
                    }
                    if constexpr (MODE != kF8Weight) {
                        if (lane == 0 && (PAIR || warp == 2))
                            cp_async_4_full(slot + (Cf::SCALE_TILE + warp - 2) * 4, tile);
                        tile += tile_step;
                    }
                    fslot = (fslot + 1) % SCALE_SLOTS;
                    --left;
                }
                cp_async_commit();
            };
#pragma unroll 1
            for (int i = 0; i < SCALE_AHEAD; ++i)
                fetch();
            Place<Cf::SETS> set;
#pragma unroll 1
            for (int t = unit; t < tiles; t += units) {
                const int blocks = blocks_of(plan.at(t), S, rank).count;
#pragma unroll 1
                for (int i = 0; i < blocks; ++i) {
                    // In step with the sets: an arrival counts for the set's present phase.
                    wait_on(tfull_at + set.at * 8, set.phase ^ 1, p.limit_ns, p.err, abort);
                    fetch();
                    cp_async_wait<SCALE_AHEAD>();
                    __syncwarp();
                    if (lane == 0)
                        arrive(tfull_at + set.at * 8);
                    set.advance();
                }
            }
            cp_async_wait<0>();
        }
    } else {
        // ------------------------------------------------ promote and store
        if constexpr (PAIR)
            regs_inc<Cf::R_PROMOTE>();
        const int pw = wg - 1, quarter = warp & 3;
        const int row = quarter * 32 + lane;  // TMEM lane
        constexpr uint32_t SLOT_BYTES = Cf::SCALE_PITCH * 4;
        uint32_t scales = smem_u32(smem + Cf::OFF_SCALE), slot = 0;
        const uint32_t tfull_at = smem_u32(tfull);
        const uint32_t tempty_at = PAIR ? mapa_shared(smem_u32(tempty), leader) : smem_u32(tempty);
        Place<Cf::SETS> set;
        float acc[Cf::CPT];
        bool seen = false;  // what the look ahead said
        // (The loop's bounds are read again: every register here is a sum's.)
#pragma unroll 1
        for (int t = unit; t < plan.total(); t += (int)gridDim.x / (S * CTAS)) {
            const int blocks = blocks_of(plan.at(t), S, rank).count;
#pragma unroll
            for (int j = 0; j < Cf::CPT; ++j)
                acc[j] = 0.f;
#pragma unroll 1
            for (int i = 0; i < blocks; ++i) {
                if (FRAGMENTS || !seen)
                    wait_on(tfull_at + set.at * 8, set.phase, p.limit_ns, p.err, abort);
                __syncwarp();  // the lanes left the wait each for itself; the load is the warp's
                tc_fence_after();
                const uint32_t taddr = tmem_base + ((uint32_t)(quarter * 32) << 16) + set.at * NT +
                                       (uint32_t)(pw * Cf::CPT);
                Place<Cf::SETS> next = set;
                next.advance();
                if constexpr (FRAGMENTS) {
                    // acc: 32 columns c, lanes of half q, 8 columns k, lane t / 4 (+ 8 e).
                    constexpr int C32 = Cf::CPT / 32;
                    const uint32_t row_scales = scales + (quarter * 32 + (lane >> 2)) * 4;
                    float2 cs[COLUMN_SCALES ? 4 : 1];
                    float rs[2];
#pragma unroll
                    for (int n = 0; n < 2 * C32; ++n) {
                        // A weight gradient keeps the columns' scales over both halves of the
                        // lanes, the others the lanes' over the columns.
                        const int c = COLUMN_SCALES ? n / 2 : n % C32, q = COLUMN_SCALES ? n % 2 : n / C32;
                        uint32_t v[16];
                        tmem_ld_16x256b_x4(taddr + ((uint32_t)(q * 16) << 16) + c * 32, v);
                        if constexpr (COLUMN_SCALES) {
                            if (q == 0)
#pragma unroll
                                for (int k = 0; k < 4; ++k)
                                    cs[k] = lds_f32x2(scales + (Cf::SCALE_COLUMNS + pw * Cf::CPT + c * 32 +
                                                                8 * k + 2 * (lane & 3)) * 4);
                        }
                        if (COLUMN_SCALES || c == 0) {
                            rs[0] = lds_f32(row_scales + q * 64);
                            rs[1] = lds_f32(row_scales + q * 64 + 32);
                            if constexpr (!COLUMN_SCALES) {
                                const float tile = lds_f32(scales + (Cf::SCALE_TILE + (PAIR ? pw : 0)) * 4);
                                rs[0] *= tile;
                                rs[1] *= tile;
                            }
                        }
                        tmem_arrived<16>(v);
                        if (n == 2 * C32 - 1) {
                            tc_fence_before();
                            __syncwarp();
                            if (lane == 0)
                                arrive_set<PAIR>(tempty_at + set.at * 8);
                        }
#pragma unroll
                        for (int k = 0; k < 4; ++k)
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                float f0 = __uint_as_float(v[4 * k + 2 * e]);
                                float f1 = __uint_as_float(v[4 * k + 2 * e + 1]);
                                float *t = acc + ((c * 2 + q) * 4 + k) * 4 + 2 * e;
                                if constexpr (COLUMN_SCALES) {
                                    mul2(f0, f1, rs[e]);
                                    fma2_each(t[0], t[1], f0, f1, cs[k].x, cs[k].y);
                                } else {
                                    fma2(t[0], t[1], rs[e], f0, f1);
                                }
                            }
                    }
                } else {
                    constexpr int CH = Cf::CH;
                    float ls = 0.f;  // the tile's scale, and the lane's
#pragma unroll
                    for (int c = 0; c < Cf::CPT; c += CH) {
                        uint32_t v[CH];
                        tmem_load<CH>(taddr + c, v);
                        if (c == 0) {  // while the first load is under way
                            seen = peek(tfull_at + next.at * 8, next.phase);
                            ls = lds_f32(scales + (Cf::SCALE_TILE + pw) * 4);
                            if constexpr (!SWAP)
                                ls *= lds_f32(scales + row * 4);
                        }
                        tmem_arrived<CH>(v);
                        if (c + CH == Cf::CPT) {
                            tc_fence_before();
                            __syncwarp();
                            if (lane == 0)
                                arrive_set<PAIR>(tempty_at + set.at * 8);
                        }
#pragma unroll
                        for (int j = 0; j < CH; j += 4) {
                            float f[4];
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                f[e] = __uint_as_float(v[j + e]);
                            float *a = acc + c + j;
                            if constexpr (SWAP) {
                                const uint4 s = lds128(scales + (Cf::SCALE_COLUMNS + c + j) * 4);
                                mul2(f[0], f[1], ls);
                                mul2(f[2], f[3], ls);
                                fma2_each(a[0], a[1], f[0], f[1], __uint_as_float(s.x), __uint_as_float(s.y));
                                fma2_each(a[2], a[3], f[2], f[3], __uint_as_float(s.z), __uint_as_float(s.w));
                            } else {
                                fma2(a[0], a[1], ls, f[0], f[1]);
                                fma2(a[2], a[3], ls, f[2], f[3]);
                            }
                        }
                    }
                }
                set = next;
                scales += SLOT_BYTES;
                if (++slot == SCALE_SLOTS) {
                    slot = 0;
                    scales -= SCALE_SLOTS * SLOT_BYTES;
                }
            }
            const Tile x = plan.at(t);  // looked up again: its registers are the sums' meanwhile
            const int lane0 = (SWAP ? x.c0 : x.r0) + half;
            const int col0 = (SWAP ? x.r0 : x.c0) + pw * Cf::CPT;
            // Of fragments: f(lane of the tile's half, column, the two values from it).
            auto each_fragment = [&](auto f) {
#pragma unroll
                for (int i = 0; i < Cf::CPT / 2; ++i)  // c, q, k, e as above
                    f(quarter * 32 + (i / 8 % 2) * 16 + (i % 2) * 8 + (lane >> 2),
                      pw * Cf::CPT + (i / 16) * 32 + (i / 2 % 4) * 8 + 2 * (lane & 3), acc + 2 * i);
            };
            if (S > 1) {
                if constexpr (FRAGMENTS) {
                    each_fragment([&](int l, int c, const float *v) {
                        sts_f32x2(smem_u32(smem) + (uint32_t)(l * Cf::PITCH + c) * 4u, v[0], v[1]);
                    });
                    break;
                }
                const uint32_t part =
                    smem_u32(smem) + (uint32_t)(row * Cf::PITCH + pw * Cf::CPT) * 4u;
#pragma unroll
                for (int j = 0; j < Cf::CPT; j += 4)
                    sts128(part + 4 * j,
                           make_uint4(__float_as_uint(acc[j]), __float_as_uint(acc[j + 1]),
                                      __float_as_uint(acc[j + 2]), __float_as_uint(acc[j + 3])));
                break;
            }
            float *C = p.C + (MODE == kF8Weight ? (int64_t)x.group * p.rows * p.cols : 0);
            const int gl = lane0 + row;
            if constexpr (PAIR) {
                // 16 columns of the warp's 32 rows at a time through shared memory (64-byte
                // swizzle, two boxes in turn), stored by the tensor-memory-access unit; by the
                // warp, 64 bytes of two rows at a time, where rows of C are off its 16-byte
                // boundaries or the box ends in another expert's rows. Straight from registers,
                // in pieces of 8 to 32 bytes of 8 to 32 rows at a time: 8192 x 8192 x 2048
                // 157 us (142 this way), the gradient of W of 4097 x 4091 x 4001 120 (97), and
                // 8192 x 8191 x 8192, whose rows are off the boundaries, 423 (450).
                // Rows behind the last end the loop in the forward and input products, where an
                // expert's last tile can have many; in the gradient of W, where only the
                // matrix's last tile has any, the same test costs a tenth (8192^3 546, 494).
                const int r0 = lane0 + quarter * 32;
                const uint32_t boxes = smem_u32(smem + Cf::OFF_BOXES) +
                                       (uint32_t)(pw * 4 + quarter) * (2 * Cf::BOX_BYTES);
                const bool boxed = p.c_boxes && (x.row_end == p.rows || r0 + 32 <= x.row_end);
#pragma unroll
                for (int j = 0; j < Cf::CPT; j += 16) {
                    if (MODE != kF8Weight && r0 >= x.row_end)
                        break;
                    const uint32_t box = boxes + (uint32_t)(j / 16 & 1) * Cf::BOX_BYTES;
                    if (lane == 0)
                        bulk_wait_group_read<1>();  // what this box held has been read
                    __syncwarp();
                    if constexpr (FRAGMENTS) {
#pragma unroll
                        for (int i = 0; i < 8; ++i) {  // q, k, e
                            const int q = i / 4, k = i / 2 % 2, e = i % 2;
                            const int l = q * 16 + e * 8 + (lane >> 2);
                            const float *v = acc + ((j / 32 * 2 + q) * 4 + j / 16 % 2 * 2 + k) * 4 + 2 * e;
                            const uint32_t chunk = (uint32_t)(2 * k + ((lane & 3) >> 1));
                            sts_f32x2(box + (uint32_t)l * 64 + ((chunk ^ (l >> 1 & 3)) << 4) + (lane & 1) * 8,
                                      v[0], v[1]);
                        }
                    } else {
#pragma unroll
                        for (int c = 0; c < 4; ++c)
                            sts128(box + (uint32_t)lane * 64 + ((c ^ (lane >> 1 & 3)) << 4),
                                   make_uint4(__float_as_uint(acc[j + 4 * c]), __float_as_uint(acc[j + 4 * c + 1]),
                                              __float_as_uint(acc[j + 4 * c + 2]),
                                              __float_as_uint(acc[j + 4 * c + 3])));
                    }
                    const int c0 = col0 + j;
                    if (boxed) {
                        fence_proxy_async_shared();
                        __syncwarp();
                        if (lane == 0) {
                            if ((MODE != kF8Weight || r0 < x.row_end) && c0 < p.cols)
                                tma_store_3d(&tm_c, box, c0, r0, MODE == kF8Weight ? x.group : 0);
                            bulk_commit_group();
                        }
                    } else {
                        __syncwarp();
                        const int c = lane & 15, hi = lane >> 4;
                        const int rows = x.row_end - r0 - hi;
                        float *to = C + (int64_t)(r0 + hi) * p.cols + c0 + c;
#pragma unroll
                        for (int i = 0; i < 16; ++i, to += 2u * (uint32_t)p.cols) {  // below 2^32, not 2^31
                            const float v = lds_f32(box + (uint32_t)(2 * i + hi) * 64 +
                                                    (((c >> 2) ^ (i & 3)) << 4) + (c & 3) * 4);
                            if (2 * i < rows && c0 + c < p.cols)
                                *to = v;
                        }
                        if (lane == 0)
                            bulk_commit_group();  // an empty one: the wait above counts groups
                    }
                }
            } else if constexpr (FRAGMENTS) {
                each_fragment([&](int l, int c, const float *v) {
                    const int r = lane0 + l, at = x.c0 + c;
                    float *to = C + (int64_t)r * p.cols + at;
                    if (r >= x.row_end)
                        return;
                    if (p.c_vec && at + 1 < p.cols) {
                        *reinterpret_cast<float2 *>(to) = make_float2(v[0], v[1]);
                    } else {
                        if (at < p.cols)
                            to[0] = v[0];
                        if (at + 1 < p.cols)
                            to[1] = v[1];
                    }
                });
            } else {  // a warp's lanes: 32 consecutive floats of a row of C
                if (gl < p.cols) {
                    float *c = C + (int64_t)col0 * p.cols + gl;
                    const int n = x.row_end - col0;
#pragma unroll
                    for (int j = 0; j < Cf::CPT; ++j, c += p.cols)
                        if (j < n)
                            *c = acc[j];
                }
            }
        }
        if (PAIR && lane == 0)
            bulk_wait_group<0>();  // no store reads shared memory that is no longer this CTA's
    }
    __syncwarp();  // the barriers below are the whole warp's

    // Read again rather than held through the roles, whose registers are the sums'.
    const int tid = (int)special_tid_x();
    if (S > 1) {
        cluster_sync();  // every partial tile of the cluster is in shared memory
        const uint32_t cta = cluster_ctarank();
        const int rank = cta / CTAS, half = cta % CTAS == 0 ? 0 : LANES;
        if (tid >= 128 && unit < plan.total()) {
            const Tile x = plan.at(unit);
            // Neighbouring threads take neighbours in a row of C: columns of the tile, or lanes.
            const int cols = NT / S, first = rank * cols;
            const int lane0 = (SWAP ? x.c0 : x.r0) + half, col0 = SWAP ? x.r0 : x.c0;
            float *C = p.C + (MODE == kF8Weight ? (int64_t)x.group * p.rows * p.cols : 0);
            for (int i = tid - 128; i < LANES * cols / 2; i += 128 * Cf::PW) {
                const int l = SWAP ? i % LANES : i / (cols / 2);
                const int cc = first + 2 * (SWAP ? i / LANES : i % (cols / 2));
                const uint32_t at = smem_u32(smem) + (uint32_t)(l * Cf::PITCH + cc) * 4u;
                float2 sum = ld_shared_cluster_v2(mapa_shared(at, cta % CTAS));
                for (int q = 1; q < S; ++q) {
                    const float2 v =
                        ld_shared_cluster_v2(mapa_shared(at, (uint32_t)q * CTAS + cta % CTAS));
                    sum.x += v.x;
                    sum.y += v.y;
                }
                const int gl = lane0 + l, gc = col0 + cc;
                if constexpr (SWAP) {
                    if (gl < p.cols && gc < x.row_end)
                        C[(int64_t)gc * p.cols + gl] = sum.x;
                    if (gl < p.cols && gc + 1 < x.row_end)
                        C[(int64_t)(gc + 1) * p.cols + gl] = sum.y;
                } else if (gl < x.row_end) {
                    float *c = C + (int64_t)gl * p.cols + gc;
                    if (p.c_vec && gc + 1 < p.cols) {
                        *reinterpret_cast<float2 *>(c) = sum;
                    } else {
                        if (gc < p.cols)
                            c[0] = sum.x;
                        if (gc + 1 < p.cols)
                            c[1] = sum.y;
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
    if (tid == 0 && *abort) {
        const uint64_t t0 = globaltimer_ns();
        while (globaltimer_ns() - t0 < p.limit_ns) {
        }
    }
    __syncwarp();
    if constexpr (PAIR)
        cluster_sync();  // no CTA leaves while its peer may still signal or read it
    if (tid >> 5 == 1) {
        const uint32_t tmem_base = lds32(smem_u32(tmem_slot));
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

// batch x rows x cols codes, rows ld and matrices rows * ld bytes apart; boxes of box_rows x 128.
static bool encode_codes(EncodeTiledFn fn, CUtensorMap *map, const void *base, uint64_t batch,
                         uint64_t rows, uint64_t cols, uint64_t ld, uint32_t box_rows)
{
    cuuint64_t dims[3] = {cols, rows, batch};
    cuuint64_t strides[2] = {ld, batch > 1 ? rows * ld : ld};
    cuuint32_t box[3] = {128, box_rows, 1};
    cuuint32_t estr[3] = {1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void *>(base), dims, strides, box,
              estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// batch x rows x cols floats of C in boxes of 32 x 16.
static bool encode_result(EncodeTiledFn fn, CUtensorMap *map, float *base, uint64_t batch,
                          uint64_t rows, uint64_t cols)
{
    cuuint64_t dims[3] = {cols, rows, batch};
    cuuint64_t strides[2] = {cols * 4, batch > 1 ? rows * cols * 4 : cols * 4};
    cuuint32_t box[3] = {16, 32, 1};
    cuuint32_t estr[3] = {1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3, base, dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_64B,
              CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Most tiles that any offsets can make.
static int64_t most_tiles(const F8Launch &L, int rows, int cols)
{
    const int64_t tc = (L.cols + cols - 1) / cols, tr = (L.rows + rows - 1) / rows;
    if (L.mode == kF8Weight)
        return tr * tc * L.experts;
    if (!L.offsets)
        return tr * tc;
    return (L.rows / rows + (L.experts < L.rows ? L.experts : L.rows)) * tc;
}

template <int MODE, int NT, bool SWAP>
static cudaError_t launch_cfg(const F8Launch &L, const DeviceContext &d, bool mute, cudaStream_t stream)
{
    using Cf = Cfg<NT, SWAP>;
    auto fn = reinterpret_cast<EncodeTiledFn>(d.encode_tiled);
    if (!fn)
        return cudaErrorNotSupported;
    const uint64_t E = (uint64_t)L.experts;
    CUtensorMap lanes, cols;
    bool ok;
    if constexpr (MODE == kF8Weight) {
        ok = encode_codes(fn, &lanes, L.a, 1, L.depth, L.rows, L.lda, BK) &&
             encode_codes(fn, &cols, L.b, 1, L.depth, L.cols, L.ldb, BK);
    } else {
        CUtensorMap &am = SWAP ? cols : lanes, &wm = SWAP ? lanes : cols;
        ok = encode_codes(fn, &am, L.a, 1, L.rows, L.depth, L.lda, SWAP ? NT : LANES);
        if constexpr (MODE == kF8Forward)
            ok = ok && encode_codes(fn, &wm, L.b, E, L.depth, L.cols, L.ldb, BK);
        else
            ok = ok && encode_codes(fn, &wm, L.b, E, L.cols, L.depth, L.ldb, SWAP ? LANES : Cf::BN);
    }
    CUtensorMap result = {};
    const bool boxes = Cf::PAIR && L.cols % 4 == 0 && (reinterpret_cast<uintptr_t>(L.C) & 15) == 0;
    if (boxes)
        ok = ok && encode_result(fn, &result, L.C, MODE == kF8Weight ? E : 1, L.rows, L.cols);
    if (!ok)
        return cudaErrorInvalidValue;
    auto kernel = f8_tc_kernel<MODE, NT, SWAP>;
    static std::atomic<uint64_t> done{0};
    const cudaError_t e = set_smem_limit_once(kernel, (int)Cf::SMEM_BYTES, done);
    if (e != cudaSuccess)
        return e;
    const int64_t tiles = most_tiles(L, Cf::ROWS, Cf::COLS);
    if (tiles > 0x1fffffff)
        return cudaErrorInvalidValue;
    Params p = {};
    p.rows = (int)L.rows;
    p.cols = (int)L.cols;
    p.depth = (int)L.depth;
    p.groups = L.experts;
    p.offsets = L.offsets;
    p.a_scales = L.a_scales;
    p.b_scales = L.b_scales;
    p.C = L.C;
    p.err = d.err;
    p.limit_ns = d.wait_limit_ns;
    p.mute = mute ? 1 : 0;
    p.c_boxes = boxes ? 1 : 0;
    p.c_vec = L.cols % 2 == 0 && (reinterpret_cast<uintptr_t>(L.C) & 7) == 0;
    // Few tiles: split the depth while every CTA keeps at least two blocks (a pair four) and
    // all clusters (of at most 8 CTAs) are resident at once. (With one block a CTA 1 x 1024 x 1024
    // takes 13.4 us instead of 11.4, with at least eight 128 x 1024 x 2048 17.6 instead of 15.5;
    // four instead of two are the same but for 1 x 512 x 512, 9.4 against 11.4.)
    constexpr int CTAS = Cf::CTAS, LEAST = Cf::PAIR ? 4 : 2;
    const int64_t blocks = f8_blocks(L.depth) / (MODE == kF8Weight && L.offsets ? L.experts : 1);
    int splits = 1;
    while (splits * CTAS < 8 && tiles * splits * CTAS * 2 <= d.sms && blocks >= splits * 2 * LEAST)
        splits *= 2;
    static std::atomic<int> resident[4][64] = {};  // clusters of 1, 2, 4, 8
    int fit = d.sms;
    for (; splits * CTAS > 1; splits /= 2) {
        const int size = splits * CTAS;
        fit = resident_clusters(kernel, size, Cf::THREADS, Cf::SMEM_BYTES,
                                resident[size == 2 ? 1 : size == 4 ? 2 : 3]);
        if (fit <= 0)
            fit = d.sms / size;
        if (tiles <= fit || splits == 1)
            break;
    }
    if (splits * CTAS == 1)
        fit = d.sms;
    p.splits = splits;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((tiles < fit ? tiles : fit) * splits * CTAS), 1, 1);
    cfg.blockDim = dim3(Cf::THREADS, 1, 1);
    cfg.dynamicSmemBytes = Cf::SMEM_BYTES;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)(splits * CTAS);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, lanes, cols, result, p);
}

template <int MODE>
static cudaError_t launch_mode(const F8Launch &L, const DeviceContext &d, bool mute, cudaStream_t stream)
{
    if constexpr (MODE != kF8Weight) {
        // Up to 64 rows (of an expert, on average; the ends of the parts count as rows): W's columns
        // on the lanes, as few of the accumulator's as hold the rows (16 x 8192 x 8192 25.8 us,
        // with 64 columns 27.8; 33 rows in 16 columns 37.0, in 64 28.8). With more, 128 x 128 tiles
        // read W as often and give every lane a row (65 x 4096 x 4096 18.6 us, 128 swapped columns
        // 25.7; 129 x 8192 x 8192 31.9, in 64 swapped columns 42.1).
        const int64_t rows = L.offsets ? (L.rows + L.experts - 1) / L.experts : L.rows;
        if (rows <= 16)
            return launch_cfg<MODE, 16, true>(L, d, mute, stream);
        if (rows <= 32)
            return launch_cfg<MODE, 32, true>(L, d, mute, stream);
        if (rows <= 64)
            return launch_cfg<MODE, 64, true>(L, d, mute, stream);
        if (rows <= 128)
            return launch_cfg<MODE, 128, false>(L, d, mute, stream);
    }
    // Pairs from half as many tiles as there are pairs on: the tiles of 128 are then more than the
    // SMs, two rounds of them. Depth 4096, us in pairs and in tiles of 128: 40 tiles of pairs 25.8
    // and 33.9 (the gradient of W 29.9, 38.0), 72 tiles 27.8 and 33.9; below, where tiles of 128
    // are one round, 36 tiles 30.8 and 21.7 (31.9, 23.7), 16 tiles 28.8 and 20.6.
    if (most_tiles(L, 256, 256) * 4 >= d.sms)
        return launch_cfg<MODE, 256, false>(L, d, mute, stream);
    return launch_cfg<MODE, 128, false>(L, d, mute, stream);
}

} // namespace f8t

cudaError_t launch_f8_tc(const F8Launch &L, const DeviceContext &d, bool mute, cudaStream_t stream)
{
    return L.mode == kF8Forward ? f8t::launch_mode<kF8Forward>(L, d, mute, stream)
           : L.mode == kF8Input ? f8t::launch_mode<kF8Input>(L, d, mute, stream)
                                : f8t::launch_mode<kF8Weight>(L, d, mute, stream);
}

} // namespace rtm
