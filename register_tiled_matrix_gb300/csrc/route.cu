// Routing of tokens to experts, and the sum of the experts' products.
//
//     s = softmax(z) or sigmoid(z) over a token's E logits, in real numbers
//     chosen: the k largest of s + bias (of the experts in the top_groups groups whose two
//             largest sum highest), ties to the lowest index
//     w_j = scale * s_j / (sum of the chosen s + 1e-20), or scale * s_j
//     slots t * k + j ordered by expert, each expert's part padded to a multiple of align
//
// A warp owns a token, a lane every 32nd expert; maxima meet in warp reductions of the values'
// ordered bits. Which experts are chosen must not hang on rounding. Without bias and groups the
// logits decide (both scores rise with them). Otherwise fp32 scores decide while each gap that
// matters exceeds what their rounding can move; a token with a closer one (of random ones with a
// bias 1 in 1000 for sigmoids, 6 for softmax) is decided again in fp64.
//
// The order by expert is a stable counting sort without atomics on positions: a block owns a
// run of tokens and counts its slots by expert, a second launch adds the counts of the blocks
// before it and places its slots, each warp a run of them in order. Up to kOneBlock tokens one
// block does both in one launch: a decoded token's call is bound by its launch.
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <type_traits>

#include "f8.h"
#include "kernels.h"

namespace rtm {
namespace route {

constexpr uint32_t kAll = 0xffffffffu;
// Tokens that one block chooses for and orders: 16 of 256 grouped experts 14.5 us, in two launches
// 16.5; 32 19.6 and 17.5 in a graph, where a launch costs no host time.
constexpr int kOneBlock = 32;
constexpr int kMaxRuns = 152;    // blocks of the two-launch form: one an SM
// Warps of a block: as many as its registers and shared memory allow; eight for at most as many
// tokens (one token of 256 experts: 11.5 us, 13.4 with 32, where most only take part in the order;
// 12 tokens 13.5 with 32, 15.6 with eight).
__host__ __device__ constexpr int warps_of(int V, bool few) { return few ? 8 : V <= 8 ? 32 : 16; }
constexpr float kNil = 1e-20f;
constexpr uint32_t kNegInfKey = 0x007fffffu;

__device__ __forceinline__ float load(const void *p, int type, int64_t i)
{
    return type == kF32    ? __ldg(static_cast<const float *>(p) + i)
           : type == kBf16 ? __bfloat162float(static_cast<const __nv_bfloat16 *>(p)[i])
                           : __half2float(static_cast<const __half *>(p)[i]);
}

// Bits whose unsigned order is the values'; NaN counts as -inf, -0 as 0.
__device__ __forceinline__ uint32_t key_of(float f)
{
    const uint32_t u = __float_as_uint(f + 0.f);
    return f != f ? kNegInfKey : (int32_t)u < 0 ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float of_key(uint32_t k)
{
    return __uint_as_float((int32_t)k < 0 ? k & 0x7fffffffu : ~k);
}

// What a selection compares: ordered bits, of fp32 or of fp64 (the GPU has few fp64 units;
// comparing bits needs none). A key is never 0.
struct Single {
    using Key = uint32_t;
    using Value = float;
    static __device__ __forceinline__ Value value(Key k) { return of_key(k); }
    static __device__ __forceinline__ Key key(Value f) { return key_of(f); }
};
struct Double {
    using Key = uint64_t;
    using Value = double;
    static __device__ __forceinline__ Value value(Key k)
    {
        return __longlong_as_double((int64_t)k < 0 ? k & 0x7fffffffffffffffull : ~k);
    }
    static __device__ __forceinline__ Key key(Value f)
    {
        const uint64_t u = (uint64_t)__double_as_longlong(f + 0.0);
        return f != f ? 0x000fffffffffffffull : (int64_t)u < 0 ? ~u : u | 0x8000000000000000ull;
    }
};

constexpr int kNone = 0x7fffffff;

// The largest of the lanes' keys.
__device__ __forceinline__ uint32_t warp_max(uint32_t mine) { return __reduce_max_sync(kAll, mine); }
__device__ __forceinline__ uint64_t warp_max(uint64_t mine)
{
    const uint32_t hi = __reduce_max_sync(kAll, (uint32_t)(mine >> 32));
    const uint32_t lo =
        __reduce_max_sync(kAll, (uint32_t)(mine >> 32) == hi ? (uint32_t)mine : 0u);
    return (uint64_t)hi << 32 | lo;
}

// The largest key v[i] of expert i * 32 + lane and its expert, the lowest on a tie, whose key
// becomes 0. kNone where all are.
template <int V, class Key>
__device__ __forceinline__ int take_best(Key (&v)[V], int lane, Key &top)
{
    Key mine = v[0];
#pragma unroll
    for (int i = 1; i < V; ++i)
        mine = v[i] > mine ? v[i] : mine;
    top = warp_max(mine);
    uint32_t at = kNone;
#pragma unroll
    for (int i = V - 1; i >= 0; --i)
        at = v[i] == top ? i * 32 + lane : at;
    at = __reduce_min_sync(kAll, at);
    if (top == 0)
        return kNone;
#pragma unroll
    for (int i = 0; i < V; ++i)
        if (at == i * 32 + lane)
            v[i] = 0;
    return (int)at;
}

// Whether a's lead over b, scores + bias, is beyond what fp32 can have moved. A sigmoid is within
// 2.5e-7 of the real one and 1e-6 of itself, a softmax score within 1e-6, and 6e-6 of itself while
// it is above 1e-30 (the exponent's rounding, 2^-24 of at most 70, and the sum's); adding the bias
// rounds once more, 2^-24 of the sum. What is below b is then certain too: value + error rises
// with the value.
__device__ __forceinline__ bool leads(float a, float b, const RouteLaunch &L)
{
    const float size = fabsf(a) + fabsf(b);
    if (L.bias)
        return a - b > (L.sigmoid ? 1e-6f : 4e-6f) + 2.5e-7f * size;
    return a - b > (L.sigmoid ? 2.5e-6f : 1.3e-5f) * size + 1e-30f;
}
__device__ __forceinline__ bool leads(double, double, const RouteLaunch &) { return true; }

// What fp32 can have moved a group's sum of two scores + bias by, whose magnitudes add up to
// `wide`: each rounds, 2^-24 of itself, and so does their sum. The sum's own magnitude bounds
// nothing: biases of opposite sign cancel in it, their roundings do not.
__device__ __forceinline__ float group_error(float wide, const RouteLaunch &L)
{
    if (L.bias)
        return (L.sigmoid ? 5e-7f : 2e-6f) + 2.5e-7f * wide;
    return (L.sigmoid ? 2.5e-6f : 1.3e-5f) * wide + 1e-30f;
}

struct Args {
    RouteLaunch L;
    int runs;        // blocks, each a run of tokens
    int64_t per;     // tokens of a run
};

// The k chosen experts, lane j the j-th. `scored`: v are scores whose gaps count; returns
// whether all of them were wide enough. scratch: V * 32 keys of the warp's own.
template <class S, int V>
__device__ __forceinline__ bool select(typename S::Key (&v)[V], const RouteLaunch &L, int lane,
                                       bool scored, typename S::Key *scratch, int &mine)
{
    using Key = typename S::Key;
    using Value = typename S::Value;
    bool sure = true;
    if (L.groups > 1) {
        // 32 / groups lanes (a power of two) find the two largest of a group.
        const int size = L.E / L.groups, share = 1 << (31 - __clz(32 / L.groups));
        const int group = lane / share;
#pragma unroll
        for (int i = 0; i < V; ++i)
            scratch[i * 32 + lane] = v[i];
        __syncwarp();
        Key one = 0, two = 0;
        if (group < L.groups)
            for (int i = lane % share; i < size; i += share) {
                const Key x = scratch[group * size + i];
                two = x > one ? one : x > two ? x : two;
                one = x > one ? x : one;
            }
        for (int o = 1; o < share; o *= 2) {
            const Key x = __shfl_xor_sync(kAll, one, o), y = __shfl_xor_sync(kAll, two, o);
            const Key low = one < x ? one : x, high = two > y ? two : y;
            one = one > x ? one : x;
            two = low > high ? low : high;
        }
        __syncwarp();
        const Value first = S::value(one), second = size > 1 ? S::value(two) : Value(0);
        const int from = min(lane, L.groups - 1) * share;  // lane g: group g's
        const Key total = __shfl_sync(kAll, S::key(first + second), from);
        Key sum[1] = {lane < L.groups ? total : 0};
        uint32_t chosen = 0;
#pragma unroll 1
        for (int j = 0; j < L.top_groups; ++j) {
            Key top;
            chosen |= 1u << take_best<1>(sum, lane, top);
        }
        // Certain where every group taken leads every other one, each with an error of its own.
        // (Neighbours in the order do not tell: a sum far from another can have the larger one.)
        if (sizeof(Key) == 4 && L.top_groups < L.groups) {
            const float wide = __shfl_sync(kAll, fabsf(first) + fabsf(second), from);
            const float error = group_error(wide, L);
            const bool taken = chosen >> lane & 1, other = lane < L.groups && !taken;
            const uint32_t least = __reduce_min_sync(kAll, taken ? key_of(S::value(total) - error) : kAll);
            sure = least > warp_max(other ? key_of(S::value(total) + error) : 0u);
        }
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (!(chosen >> min((i * 32 + lane) / size, 31) & 1))
                v[i] = 0;
    }
    Value last = 0;
    const int rounds = scored ? L.k + 1 : L.k;
#pragma unroll 1
    for (int j = 0; j < rounds; ++j) {
        Key top;
        const int at = take_best<V>(v, lane, top);
        if (at == kNone)
            break;
        if (scored && j > 0 && !leads(last, S::value(top), L))
            sure = false;
        last = S::value(top);
        if (lane == j && j < L.k)
            mine = at;
    }
    return sure;
}

// The same from scores in fp64; z: the token's logits in the warp's shared memory.
template <int V>
__device__ __forceinline__ int select_exactly(const RouteLaunch &L, const float *z, int lane,
                                              uint64_t *scratch)
{
    float top = -INFINITY;
    bool nan = false;
#pragma unroll 1
    for (int i = 0; i < V; ++i) {
        nan = nan || z[i * 32 + lane] != z[i * 32 + lane];
        top = fmaxf(top, z[i * 32 + lane]);
    }
    nan = __any_sync(kAll, nan);
#pragma unroll
    for (int o = 16; o > 0; o /= 2)
        top = fmaxf(top, __shfl_xor_sync(kAll, top, o));
    const bool nothing = top == -INFINITY && !nan;
    double sum = 0;
    constexpr int TOGETHER = V < 4 ? V : 4;  // fp64 instructions are slow to answer
#pragma unroll TOGETHER
    for (int i = 0; i < V; ++i) {
        const double x = (double)z[i * 32 + lane];
        const double w = exp(L.sigmoid ? -x : x - (double)top);
        const double s = L.sigmoid ? 1.0 / (1.0 + w) : nothing ? 0.0 : w;
        scratch[i * 32 + lane] = (uint64_t)__double_as_longlong(s);
        sum += s;
    }
#pragma unroll
    for (int o = 16; o > 0; o /= 2)
        sum += __shfl_xor_sync(kAll, sum, o);
    if (L.sigmoid || nothing)
        sum = 1.0;
    const double part = 1.0 / sum;
    uint64_t v[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int e = i * 32 + lane;
        const double s = __longlong_as_double((int64_t)scratch[e]) * part;
        v[i] = e < L.E ? Double::key(s + (L.bias ? (double)__ldg(L.bias + e) : 0.0)) : 0;
    }
    __syncwarp();
    int mine = 0;
    select<Double, V>(v, L, lane, false, scratch, mine);
    return mine;
}

__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int o = 16; o > 0; o /= 2)
        v += __shfl_xor_sync(kAll, v, o);
    return v;
}

// What a token's scores are made with: s = exp(z - top) * part, or the sigmoid.
struct Shift {
    float top, part;
    bool nothing;  // every logit is -inf: softmax scores are 0
};
__device__ __forceinline__ float score_of(const RouteLaunch &L, const Shift &f, float z)
{
    if (L.sigmoid)
        return __fdividef(1.f, 1.f + expf(-z));  // 0 where the score is below 2^-126
    return f.nothing ? 0.f : expf(z - f.top) * f.part;
}

// z[i]: the logit of expert i * 32 + lane, -inf behind the last.
template <int V>
__device__ __forceinline__ void read_token(const RouteLaunch &L, int64_t t, int lane, float (&z)[V])
{
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int e = i * 32 + lane;
        z[i] = e < L.E ? load(L.logits, L.type, t * L.E + e) : -INFINITY;
    }
}

template <int V>
__device__ __forceinline__ Shift shift_of(const RouteLaunch &L, const float (&z)[V])
{
    Shift f = {0.f, 1.f, false};
    if (L.sigmoid)
        return f;
    float top = -INFINITY;
    bool nan = false;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        nan = nan || z[i] != z[i];
        top = fmaxf(top, z[i]);
    }
    f.top = of_key(warp_max(key_of(top)));
    nan = __any_sync(kAll, nan);
    f.nothing = f.top == -INFINITY && !nan;
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i)
        sum += f.nothing ? 0.f : expf(z[i] - f.top);
    f.part = f.nothing ? 0.f : 1.f / warp_sum(sum);  // NaN where a logit is
    return f;
}

// The experts and weights of the token with logits z; bias: the experts' (0 without one). At
// `chosen` (shared memory; may be null) too. In shared memory of the warp's own: scratch, V * 32
// keys of 64 bits, and held, V * 32 logits.
template <int V>
__device__ __forceinline__ void choose_token(const RouteLaunch &L, int64_t t, int lane,
                                             const float (&z)[V], const float (&bias)[V],
                                             uint64_t *scratch, float *held, int32_t *chosen)
{
#pragma unroll
    for (int i = 0; i < V; ++i)
        held[i * 32 + lane] = z[i];
    const Shift f = shift_of<V>(L, z);
    const bool by_logit = !L.bias && L.groups == 1;
    uint32_t keys[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        float x = z[i];
        if (!by_logit)
            x = score_of(L, f, x) + bias[i];
        keys[i] = i * 32 + lane < L.E ? key_of(x) : 0;
    }
    int mine = 0;
    if (!select<Single, V>(keys, L, lane, !by_logit, reinterpret_cast<uint32_t *>(scratch), mine))
        mine = select_exactly<V>(L, held, lane, scratch);
    __syncwarp();
    float p = 0.f;
    if (lane < L.k)
        p = score_of(L, f, held[mine]);
    const float total = warp_sum(p) + kNil;
    if (lane < L.k) {
        L.experts[t * L.k + lane] = mine;
        L.weights[t * L.k + lane] = L.scale * (L.renormalise ? p / total : p);
        if (chosen)
            chosen[lane] = mine;
    }
    __syncwarp();
}

// ---------------------------------------------------------------- order by expert

// Adds this warp's slots [from, to) to its counts by expert.
__device__ __forceinline__ void count_slots(const int32_t *experts, int64_t from, int64_t to,
                                            int32_t *counts, int lane)
{
    for (int64_t i = from; i < to; i += 32) {
        const bool in = i + lane < to;
        const int e = in ? experts[i + lane] : -1;
        const uint32_t same = __match_any_sync(kAll, e);
        if (in && (same & ((1u << lane) - 1)) == 0)
            counts[e] += __popc(same);
        __syncwarp();
    }
}

// Places the block's slots [from, to) with the experts that `experts` holds from `from` on. In
// shared memory: counts (kWarps x E, each warp's own), sums (E), scan (E + 1), warps (kWarps).
// With more than one run the other runs' counts are in L.counts.
template <int kWarps>
__device__ __forceinline__ void place_block(const Args &a, const int32_t *experts, int32_t *counts,
                                            int32_t *sums, int32_t *scan, int32_t *warps,
                                            int64_t from, int64_t to)
{
    const RouteLaunch &L = a.L;
    constexpr int threads = kWarps * 32;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, run = blockIdx.x;
    const int64_t n = to - from, each = (n + kWarps - 1) / kWarps;
    const int64_t first = min(n, warp * each), last = min(n, first + each);
    for (int i = threadIdx.x; i < kWarps * L.E; i += threads)
        counts[i] = 0;
    for (int e = threadIdx.x; e < L.E; e += threads) {
        sums[e] = 0;
        scan[e] = 0;
    }
    __syncthreads();
    count_slots(experts, first, last, counts + warp * L.E, lane);
    // Every expert's slots in all runs (sums) and in those before (scan). Whole numbers: the
    // order of these additions changes nothing.
    if (a.runs > 1) {
        const int parts = max(1, threads / L.E), each_run = (a.runs + parts - 1) / parts;
        for (int i = threadIdx.x; i < parts * L.E; i += threads) {
            const int part = i / L.E, e = i - part * L.E;
            const int r0 = part * each_run, r1 = min(a.runs, r0 + each_run);
            int32_t before = 0, total = 0;
#pragma unroll 16
            for (int r = r0; r < r1; ++r) {
                const int32_t c = __ldg(L.counts + r * L.E + e);
                before += r < run ? c : 0;
                total += c;
            }
            atomicAdd(sums + e, total);
            atomicAdd(scan + e, before);
        }
    }
    __syncthreads();
    // A thread has `own` neighbouring experts: the warps' first places among an expert's slots,
    // and the padded length of its part, whose exclusive sum is the part's start.
    constexpr int OWN = (kRouteMaxExperts + threads - 1) / threads;
    const int own = (L.E + threads - 1) / threads;
    int32_t length[OWN], sum = 0;
#pragma unroll
    for (int i = 0; i < OWN; ++i) {
        length[i] = 0;
        const int e = threadIdx.x * own + i;
        if (i < own && e < L.E) {
            int32_t at = scan[e];
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const int32_t c = counts[w * L.E + e];
                counts[w * L.E + e] = at;
                at += c;
            }
            if (a.runs == 1)
                sums[e] = at;
            length[i] = (sums[e] + L.align - 1) / L.align * L.align;
            sum += length[i];
        }
    }
    int32_t x = sum;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
        const int32_t y = __shfl_up_sync(kAll, x, o);
        if (lane >= o)
            x += y;
    }
    if (lane == 31)
        warps[warp] = x;
    __syncthreads();  // and every read of scan as the counts before
    int32_t start = x - sum;
#pragma unroll
    for (int w = 0; w < kWarps; ++w)
        start += w < warp ? warps[w] : 0;
#pragma unroll
    for (int i = 0; i < OWN; ++i) {
        const int e = threadIdx.x * own + i;
        if (i < own && e < L.E) {
            scan[e] = start;
            start += length[i];
            if (e == L.E - 1)
                scan[L.E] = start;
        }
    }
    __syncthreads();
    if (run == 0)
        for (int e = threadIdx.x; e <= L.E; e += threads)
            L.offsets[e] = scan[e];
    // Slots in order: this warp's run of them.
    for (int64_t i = first; i < last; i += 32) {
        const bool in = i + lane < last;
        const int e = in ? experts[i + lane] : -1;
        const uint32_t same = __match_any_sync(kAll, e);
        const int rank = __popc(same & ((1u << lane) - 1));
        int32_t at = 0;
        if (in)
            at = counts[warp * L.E + e] + rank;
        __syncwarp();
        if (in) {
            if (rank == 0)
                counts[warp * L.E + e] += __popc(same);
            const int32_t to_row = scan[e] + at;
            L.rows[to_row] = (int32_t)(from + i + lane);
            L.slots[from + i + lane] = to_row;
        }
        __syncwarp();
    }
    // Rows that no slot takes: the ends of the parts, and what lies behind the last.
    if (L.align > 1)
        for (int e = run * kWarps + warp; e < L.E; e += a.runs * kWarps)
            for (int32_t i = scan[e] + sums[e] + lane; i < scan[e + 1]; i += 32)
                L.rows[i] = -1;
    for (int64_t i = scan[L.E] + (int64_t)run * threads + threadIdx.x; i < L.R;
         i += (int64_t)a.runs * threads)
        L.rows[i] = -1;
}

// Words of shared memory of place_block.
__host__ __device__ constexpr int place_words(int warps, int E) { return (warps + 2) * E + 1 + warps; }

template <int kWarps>
__device__ __forceinline__ void place_in(const Args &a, const int32_t *experts, int32_t *words,
                                         int64_t from, int64_t to)
{
    const int E = a.L.E;
    place_block<kWarps>(a, experts, words, words + kWarps * E, words + (kWarps + 1) * E,
                words + (kWarps + 2) * E + 1, from, to);
}

// Experts and weights of a run of tokens, and the run's slots counted by expert; a single run
// places them, too.
template <int V, bool FEW>
__global__ void __launch_bounds__(warps_of(V, FEW) * 32, 1) choose_kernel(const Args a)
{
    constexpr int kWarps = warps_of(V, FEW);
    extern __shared__ __align__(8) int32_t shared[];
    __shared__ int32_t chosen[kOneBlock * kRouteMaxChosen];
    const RouteLaunch &L = a.L;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t from = min(L.T, blockIdx.x * a.per), to = min(L.T, from + a.per);
    uint64_t *scratch = reinterpret_cast<uint64_t *>(shared) + warp * V * 32;
    float *held = reinterpret_cast<float *>(shared) + (kWarps * 2 + warp) * V * 32;
    constexpr bool AHEAD = V <= 4;  // the next token's logits are read while this one is chosen for
    float bias[V], z[V], next[V];
    auto read_bias = [&]() {
#pragma unroll
        for (int i = 0; i < V; ++i)
            bias[i] = L.bias && i * 32 + lane < L.E ? __ldg(L.bias + i * 32 + lane) : 0.f;
    };
    if constexpr (AHEAD) {
        read_bias();
        if (from + warp < to)
            read_token<V>(L, from + warp, lane, next);
    }
    for (int64_t t = from + warp; t < to; t += kWarps) {
        if constexpr (AHEAD) {
#pragma unroll
            for (int i = 0; i < V; ++i)
                z[i] = next[i];
            if (t + kWarps < to)
                read_token<V>(L, t + kWarps, lane, next);
        } else {
            read_token<V>(L, t, lane, z);
            read_bias();
        }
        choose_token<V>(L, t, lane, z, bias, scratch, held, a.runs == 1 ? chosen + t * L.k : nullptr);
    }
    __syncthreads();
    if (a.runs == 1) {
        place_in<kWarps>(a, chosen, shared, from * L.k, to * L.k);
        return;
    }
    for (int e = threadIdx.x; e < L.E; e += kWarps * 32)
        shared[e] = 0;
    __syncthreads();
    // Whole numbers: the order of these additions changes nothing.
    for (int64_t i = from * L.k + threadIdx.x; i < to * L.k; i += kWarps * 32)
        atomicAdd(shared + L.experts[i], 1);
    __syncthreads();
    for (int e = threadIdx.x; e < L.E; e += kWarps * 32)
        L.counts[(int64_t)blockIdx.x * L.E + e] = shared[e];
}

constexpr int kPlaceWarps = 32;
__global__ void __launch_bounds__(kPlaceWarps * 32) place_kernel(const Args a)
{
    extern __shared__ int32_t shared[];
    const RouteLaunch &L = a.L;
    const int64_t from = min(L.T, blockIdx.x * a.per), to = min(L.T, from + a.per);
    place_in<kPlaceWarps>(a, L.experts + from * L.k, shared, from * L.k, to * L.k);
}

// The value of the lane whose weight (not negative) is largest; w: that weight.
__device__ __forceinline__ float of_heaviest(float v, float weight, float &w)
{
    const uint32_t most = __reduce_max_sync(kAll, __float_as_uint(weight));
    w = __uint_as_float(most);
    return __shfl_sync(kAll, v, __ffs(__ballot_sync(kAll, __float_as_uint(weight) == most)) - 1);
}

// dz from dw, a warp a token: with g_j = ds of the chosen, softmax: dz = s * (g - sum_j g_j s_j);
// sigmoid: dz = g * s * (1 - s). A softmax's difference is sum_e s_e (g - g_e) over all experts,
// g_e 0 of those that are not chosen. Without renormalisation (PLAIN) it is taken as g - c less
// sum_e s_e (g_e - c), c the g of the largest of the chosen scores and of the others' sum: where
// one score is nearly 1 the plain difference is rounding.
// Of renormalised weights, with P = sum_j s_j, S = P + 1e-20,
//     g_j = (sum_i s_i (dw_j - dw_i) + 1e-20 dw_j) / S^2,  sum_j g_j s_j = 1e-20 sum_j s_j dw_j / S^2
// where the sum is P (dw_j - c) - sum_i s_i (dw_i - c), c the dw of the largest s_i. (c = 0, dw_j
// less the weighted mean, leaves the mean's rounding where the dw are alike, one s_i outweighs
// the others or k is 1: 1e-8 of dw / S where the gradient is 1e-20 of it.) `scale` comes last:
// differences of the g are those of the dw.
template <int V, bool PLAIN>
__global__ void __launch_bounds__(256)
    route_backward_kernel(const RouteLaunch L, const int32_t *experts, const float *dweights,
                          float *dlogits)
{
    const int lane = threadIdx.x & 31;
    const int64_t t = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    if (t >= L.T)
        return;
    float z[V];
    read_token<V>(L, t, lane, z);
    const Shift f = shift_of<V>(L, z);
    int mine = -1;
    float dw = 0.f, p = 0.f, rest = 0.f;  // rest: 1 - p of a sigmoid, which p itself no longer tells
    if (lane < L.k) {
        const int e = experts[t * L.k + lane];
        if (e >= 0 && e < L.E) {
            mine = e;
            dw = dweights[t * L.k + lane];
            const float x = load(L.logits, L.type, t * L.E + e);
            p = score_of(L, f, x);
            rest = score_of(L, f, -x);
        }
    }
    float g = dw, inner = 0.f;
    if (L.renormalise) {
        float w;
        const float c = of_heaviest(dw, p, w), off = warp_sum(p * (dw - c));
        const float total = warp_sum(p), part = 1.f / (total + kNil), nil = kNil * part;
        g = mine >= 0 ? fmaf(fmaf(dw - c, total, -off), part, nil * dw) * part : 0.f;
        inner = nil * (fmaf(c, total, off) * part);
    }
    // The chosen experts' own terms; one that is named twice gets both.
    float all = 0.f;
    bool first = mine >= 0;  // of the slots that name this expert
    auto add_up = [&]() {
        all = 0.f;
        for (int j = 0; j < L.k; ++j) {
            const int e = __shfl_sync(kAll, mine, j);
            const float x = __shfl_sync(kAll, g, j);
            all += e == mine ? x : 0.f;
            first = first && (e != mine || j >= lane);
        }
    };
    float own = 0.f;
    if constexpr (PLAIN) {
        float others = 0.f, w;  // the scores of the experts that are not chosen
        int named = 0;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            z[i] = score_of(L, f, z[i]);  // 0 behind the last expert
            const uint32_t taken = __reduce_or_sync(kAll, mine >> 5 == i ? 1u << (mine & 31) : 0u);
            others += taken >> lane & 1 ? 0.f : z[i];
            named += __popc(taken);
        }
        others = warp_sum(others);
        all = g;
        if (named != __popc(__ballot_sync(kAll, mine >= 0)))
            add_up();
        const float heaviest = of_heaviest(all, first ? p : 0.f, w), c = others > w ? 0.f : heaviest;
        const float off = fmaf(-c, others, warp_sum(first ? p * (all - c) : 0.f));
        own = all - c - off;
        inner = c + off;
    }
    float *out = dlogits + t * L.E;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int e = i * 32 + lane;
        if (e < L.E)
            out[e] = L.sigmoid ? 0.f : -L.scale * (inner * (PLAIN ? z[i] : score_of(L, f, z[i])));
    }
    __syncwarp();
    if constexpr (!PLAIN) {
        add_up();
        own = L.sigmoid ? all * rest : all - inner;
    }
    if (mine >= 0)
        out[mine] = L.scale * (p * own);
}

// ---------------------------------------------------------------- joining

// Four columns a thread, a row in chunks of 256; four rows of C are asked for at once. Bound by the
// bytes of C. (Blocks of 256 threads, chunks of 1024: one token the same, 16384 tokens of 128 and
// four experts 21.6 us against 16.5, 8192 of 2047 and six 96 against 87, 16384 of 4096 291 and 285.)
constexpr int kJoinThreads = 64;
template <bool VEC>
__global__ void __launch_bounds__(kJoinThreads)
    join_kernel(int64_t T, int64_t N, int k, int64_t R, const float *C, const int32_t *slots,
                const float *weights, float *Y, int64_t chunks)
{
    const int64_t t = blockIdx.x / chunks, width = kJoinThreads * 4;
    const int64_t n = (blockIdx.x - t * chunks) * width + (VEC ? threadIdx.x * 4 : threadIdx.x);
    float acc[4] = {0.f, 0.f, 0.f, 0.f};
    if (n >= N)
        return;
    for (int j0 = 0; j0 < k; j0 += 4) {
        float v[4][4], w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            w[j] = 0.f;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                v[j][i] = 0.f;
            if (j0 + j >= k)
                continue;
            const int64_t r = __ldg(slots + t * k + j0 + j);
            if (r < 0 || r >= R)
                continue;
            w[j] = weights ? __ldg(weights + t * k + j0 + j) : 1.f;
            const float *c = C + r * N + n;
            if constexpr (VEC) {
                const float4 x = __ldg(reinterpret_cast<const float4 *>(c));
                v[j][0] = x.x, v[j][1] = x.y, v[j][2] = x.z, v[j][3] = x.w;
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (n + kJoinThreads * i < N)
                        v[j][i] = __ldg(c + kJoinThreads * i);
            }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (j0 + j < k)
                    acc[i] = fmaf(w[j], v[j][i], acc[i]);
    }
    float *y = Y + t * N + n;
    if constexpr (VEC) {
        *reinterpret_cast<float4 *>(y) = make_float4(acc[0], acc[1], acc[2], acc[3]);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (n + kJoinThreads * i < N)
                y[kJoinThreads * i] = acc[i];
    }
}

// Four values of dY from i on, their address on 8 (fp32: 16) bytes.
__device__ __forceinline__ float4 load4(const void *p, int type, int64_t i)
{
    if (type == kF32)
        return __ldg(reinterpret_cast<const float4 *>(static_cast<const float *>(p) + i));
    const uint2 b = __ldg(reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(p) + i));
    if (type == kBf16)
        return make_float4(__uint_as_float(b.x << 16), __uint_as_float(b.x & 0xffff0000u),
                           __uint_as_float(b.y << 16), __uint_as_float(b.y & 0xffff0000u));
    const float2 lo = __half22float2(*reinterpret_cast<const __half2 *>(&b.x));
    const float2 hi = __half22float2(*reinterpret_cast<const __half2 *>(&b.y));
    return make_float4(lo.x, lo.y, hi.x, hi.y);
}

// A slot's product is summed by the threads of a block of 128 (many slots: by a warp each), four
// columns at a time and four of those loads under way; then warps are added in order.
// (A kernel for each of dY's types: a choice in the loop kept the loads apart, 77 us against 64
// for 32768 slots of 2048 and bf16.)
template <int TYPE, bool VEC, int WARPS>
__global__ void __launch_bounds__(128)
    join_backward_kernel(int64_t count, int64_t N, int k, int64_t R, const void *dY,
                         const float *C, const int32_t *slots, float *dweights)
{
    __shared__ float part[4];
    constexpr int THREADS = WARPS * 32;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t i = (int64_t)blockIdx.x * (4 / WARPS) + (WARPS == 4 ? 0 : warp);
    const int id = WARPS == 4 ? threadIdx.x : lane;
    float sum[4] = {0.f, 0.f, 0.f, 0.f};
    const int64_t r = i < count ? slots[i] : -1, t = i / k;
    if (r >= 0 && r < R) {
        const float *c = C + r * N;
        if constexpr (VEC) {
#pragma unroll 4
            for (int64_t n = id * 4; n < N; n += THREADS * 4) {
                const float4 v = __ldg(reinterpret_cast<const float4 *>(c + n));
                const float4 d = load4(dY, TYPE, t * N + n);
                sum[0] = fmaf(d.x, v.x, sum[0]);
                sum[1] = fmaf(d.y, v.y, sum[1]);
                sum[2] = fmaf(d.z, v.z, sum[2]);
                sum[3] = fmaf(d.w, v.w, sum[3]);
            }
        } else {
#pragma unroll 4
            for (int64_t n = id; n < N; n += THREADS)
                sum[0] = fmaf(load(dY, TYPE, t * N + n), __ldg(c + n), sum[0]);
        }
    }
    float all = warp_sum((sum[0] + sum[1]) + (sum[2] + sum[3]));
    if constexpr (WARPS == 4) {
        if (lane == 0)
            part[warp] = all;
        __syncthreads();
        all = (part[0] + part[1]) + (part[2] + part[3]);
        if (threadIdx.x == 0)
            dweights[i] = all;
    } else if (lane == 0 && i < count) {
        dweights[i] = all;
    }
}

// Blocks, each a run of tokens: two tokens a block until there is a block on every SM.
static int runs_of(int64_t T) { return T <= kOneBlock ? 1 : (int)(T < kMaxRuns * 2 ? (T + 1) / 2 : kMaxRuns); }

constexpr size_t place_bytes(int warps, int E) { return (size_t)place_words(warps, E) * 4; }

template <int V, bool FEW>
static cudaError_t launch_choose(const Args &a, cudaStream_t stream)
{
    constexpr int warps = warps_of(V, FEW);
    constexpr size_t scratch = (size_t)warps * V * 32 * 12;  // the warps' keys and logits
    constexpr size_t most = place_bytes(warps, V * 32);
    static std::atomic<uint64_t> done{0};
    const cudaError_t e =
        set_smem_limit_once(choose_kernel<V, FEW>, (int)(scratch > most ? scratch : most), done);
    if (e != cudaSuccess)
        return e;
    const size_t place = place_bytes(warps, a.L.E), smem = place > scratch ? place : scratch;
    choose_kernel<V, FEW><<<a.runs, warps * 32, smem, stream>>>(a);
    return cudaGetLastError();
}

template <int V>
static cudaError_t launch_choose(const Args &a, cudaStream_t stream)
{
    return a.L.T <= warps_of(V, true) ? launch_choose<V, true>(a, stream)
                                      : launch_choose<V, false>(a, stream);
}

template <int V>
static cudaError_t launch_backward(const RouteLaunch &L, const int32_t *experts,
                                   const float *dweights, float *dlogits, cudaStream_t stream)
{
    const int64_t blocks = (L.T + 7) / 8;
    if (blocks > 0x7fffffff)
        return cudaErrorInvalidValue;
    if (!L.sigmoid && !L.renormalise)
        route_backward_kernel<V, true><<<(unsigned)blocks, 256, 0, stream>>>(L, experts, dweights, dlogits);
    else
        route_backward_kernel<V, false><<<(unsigned)blocks, 256, 0, stream>>>(L, experts, dweights, dlogits);
    return cudaGetLastError();
}

} // namespace route

int64_t route_rows(int64_t T, int E, int k, int align)
{
    const int64_t slots = T * k;
    return slots + (slots < E ? slots : E) * (align - 1);
}

int64_t route_workspace_ints(int64_t T, int E)
{
    const int runs = route::runs_of(T);
    return runs == 1 ? 0 : (int64_t)runs * E;
}

cudaError_t launch_route(const RouteLaunch &L, cudaStream_t stream)
{
    using namespace route;
    Args a;
    a.L = L;
    a.runs = runs_of(L.T);
    a.per = (L.T + a.runs - 1) / a.runs;
    const cudaError_t e = L.E <= 32    ? launch_choose<1>(a, stream)
                          : L.E <= 64  ? launch_choose<2>(a, stream)
                          : L.E <= 128 ? launch_choose<4>(a, stream)
                          : L.E <= 256 ? launch_choose<8>(a, stream)
                          : L.E <= 512 ? launch_choose<16>(a, stream)
                                       : launch_choose<32>(a, stream);
    if (e != cudaSuccess || a.runs == 1)
        return e;
    static std::atomic<uint64_t> done{0};
    const cudaError_t f = set_smem_limit_once(place_kernel, (int)place_bytes(kPlaceWarps, kRouteMaxExperts), done);
    if (f != cudaSuccess)
        return f;
    place_kernel<<<a.runs, kPlaceWarps * 32, place_bytes(kPlaceWarps, L.E), stream>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_route_backward(const RouteLaunch &L, const int32_t *experts,
                                  const float *dweights, float *dlogits, cudaStream_t stream)
{
    using namespace route;
    return L.E <= 32    ? launch_backward<1>(L, experts, dweights, dlogits, stream)
           : L.E <= 64  ? launch_backward<2>(L, experts, dweights, dlogits, stream)
           : L.E <= 128 ? launch_backward<4>(L, experts, dweights, dlogits, stream)
           : L.E <= 256 ? launch_backward<8>(L, experts, dweights, dlogits, stream)
           : L.E <= 512 ? launch_backward<16>(L, experts, dweights, dlogits, stream)
                        : launch_backward<32>(L, experts, dweights, dlogits, stream);
}

cudaError_t launch_experts_join(int64_t T, int64_t N, int k, int64_t R, const float *C,
                                const int32_t *slots, const float *weights, float *Y,
                                cudaStream_t stream)
{
    constexpr int threads = route::kJoinThreads;
    const int64_t chunks = (N + threads * 4 - 1) / (threads * 4);
    if (T * chunks > 0x7fffffff)
        return cudaErrorInvalidValue;
    const unsigned grid = (unsigned)(T * chunks);
    if (N % 4 == 0 && ((reinterpret_cast<uintptr_t>(C) | reinterpret_cast<uintptr_t>(Y)) & 15) == 0)
        route::join_kernel<true><<<grid, threads, 0, stream>>>(T, N, k, R, C, slots, weights, Y, chunks);
    else
        route::join_kernel<false><<<grid, threads, 0, stream>>>(T, N, k, R, C, slots, weights, Y, chunks);
    return cudaGetLastError();
}

template <int TYPE, bool VEC>
static cudaError_t launch_join_backward(int64_t T, int64_t N, int k, int64_t R,
                                        const void *dY, const float *C, const int32_t *slots,
                                        float *dweights, cudaStream_t stream)
{
    // A block a slot while that leaves SMs idle: 1024 slots of 4096 11.4 us, a warp each 17.6; 4096
    // of 512 11.4 and 10.4, 131072 of 512 96 and 64.
    const int64_t count = T * k;
    const bool few = count < 152 * 16;
    const int64_t blocks = few ? count : (count + 3) / 4;
    if (blocks > 0x7fffffff)
        return cudaErrorInvalidValue;
    if (few)
        route::join_backward_kernel<TYPE, VEC, 4><<<(unsigned)blocks, 128, 0, stream>>>(
            count, N, k, R, dY, C, slots, dweights);
    else
        route::join_backward_kernel<TYPE, VEC, 1><<<(unsigned)blocks, 128, 0, stream>>>(
            count, N, k, R, dY, C, slots, dweights);
    return cudaGetLastError();
}

cudaError_t launch_experts_join_backward(int64_t T, int64_t N, int k, int64_t R, int type,
                                         const void *dY, const float *C, const int32_t *slots,
                                         float *dweights, cudaStream_t stream)
{
    const bool vec =
        N % 4 == 0 && ((reinterpret_cast<uintptr_t>(C) | reinterpret_cast<uintptr_t>(dY)) & 15) == 0;
    auto launch = [&](auto one) {
        constexpr int TYPE = decltype(one)::value;
        return vec ? launch_join_backward<TYPE, true>(T, N, k, R, dY, C, slots, dweights, stream)
                   : launch_join_backward<TYPE, false>(T, N, k, R, dY, C, slots, dweights, stream);
    };
    return type == kF32    ? launch(std::integral_constant<int, kF32>{})
           : type == kBf16 ? launch(std::integral_constant<int, kBf16>{})
                           : launch(std::integral_constant<int, kF16>{});
}

} // namespace rtm
