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
// matters exceeds what their rounding can move; a token with a closer one (2 in 1000 of random
// ones) is decided again in fp64.
//
// The order by expert is a stable counting sort without atomics on positions: a block owns a
// run of tokens and counts its slots by expert, a second launch adds the counts of the blocks
// before it and places its slots, each warp a run of them in order. Up to kOneBlock tokens one
// block does both in one launch: a decoded token's call is bound by its launch.
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "f8.h"
#include "kernels.h"

namespace rtm {
namespace route {

constexpr uint32_t kAll = 0xffffffffu;
constexpr int kOneBlock = 128;   // tokens
constexpr int kMaxRuns = 152;    // blocks of the two-launch form: one an SM
constexpr int kWarps = 16;       // of a block
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

// The values that a selection runs on, a lane's i-th, as ordered bits: of fp32 in registers, of
// fp64 in the warp's shared memory (the GPU has few fp64 units; comparing bits needs none).
template <int V>
struct Keys {
    using Type = uint32_t;
    using Value = float;
    uint32_t v[V];
    __device__ __forceinline__ Type at(int i, int) const { return v[i]; }
    static __device__ __forceinline__ Value value(Type k) { return of_key(k); }
    static __device__ __forceinline__ Type key(Value f) { return key_of(f); }
};
struct DoubleKeys {
    using Type = uint64_t;
    using Value = double;
    const uint64_t *v;
    __device__ __forceinline__ Type at(int i, int lane) const { return v[i * 32 + lane]; }
    static __device__ __forceinline__ Value value(Type k)
    {
        return __longlong_as_double((int64_t)k < 0 ? k & 0x7fffffffffffffffull : ~k);
    }
    static __device__ __forceinline__ Type key(Value f)
    {
        const uint64_t u = (uint64_t)__double_as_longlong(f + 0.0);
        return f != f ? 0x000fffffffffffffull : (int64_t)u < 0 ? ~u : u | 0x8000000000000000ull;
    }
};

constexpr int kNone = 0x7fffffff;

// The largest of the lanes' keys and the index that came with it, the lowest on a tie; kNone
// where no lane has one. Keys are never 0.
__device__ __forceinline__ int best_of(uint32_t mine, int at, uint32_t &top)
{
    const uint32_t m = __reduce_max_sync(kAll, mine);
    top = m;
    return (int)__reduce_min_sync(kAll, mine == m ? (uint32_t)at : (uint32_t)kNone);
}
__device__ __forceinline__ int best_of(uint64_t mine, int at, uint64_t &top)
{
    const uint32_t hi = __reduce_max_sync(kAll, (uint32_t)(mine >> 32));
    const bool in = (uint32_t)(mine >> 32) == hi;
    const uint32_t lo = __reduce_max_sync(kAll, in ? (uint32_t)mine : 0u);
    top = (uint64_t)hi << 32 | lo;
    return (int)__reduce_min_sync(kAll, mine == top ? (uint32_t)at : (uint32_t)kNone);
}

// The largest of the lanes' open values (bit i of `open`: the i-th takes part) and its index
// i * 32 + lane.
template <int V, class S>
__device__ __forceinline__ int best(const S &v, uint32_t open, int lane, typename S::Type &top)
{
    typename S::Type mine = 0;
    int at = kNone;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const typename S::Type x = (open >> i & 1) ? v.at(i, lane) : 0;
        if (x > mine) {
            mine = x;
            at = i * 32 + lane;
        }
    }
    return best_of(mine, at, top);
}

// Whether a's lead over b is beyond what fp32 can have moved. A sigmoid is within 2e-7 of the
// real one and 1e-6 of itself, a softmax score within 1e-6, and 6e-6 of itself while it is above
// 1e-30 (the exponent's rounding, 2^-24 of at most 70, and the sum's); adding the bias or two
// scores rounds once more, 2^-24 of the sum.
__device__ __forceinline__ bool leads(float a, float b, const RouteLaunch &L)
{
    const float size = fabsf(a) + fabsf(b);
    if (L.bias)
        return a - b > (L.sigmoid ? 1e-6f : 4e-6f) + 2.5e-7f * size;
    return a - b > (L.sigmoid ? 2.5e-6f : 1.3e-5f) * size + 1e-30f;
}
__device__ __forceinline__ bool leads(double, double, const RouteLaunch &) { return true; }

struct Args {
    RouteLaunch L;
    int runs;        // blocks, each a run of tokens
    int64_t per;     // tokens of a run
};

// The k chosen experts, lane j the j-th. `scored`: v are scores whose gaps count; returns
// whether all of them were wide enough.
template <int V, class S>
__device__ __forceinline__ bool select(const S &v, const RouteLaunch &L, int lane, bool scored,
                                       int &mine)
{
    using Key = typename S::Type;
    using Value = typename S::Value;
    uint32_t open = 0;
#pragma unroll
    for (int i = 0; i < V; ++i)
        if (i * 32 + lane < L.E)
            open |= 1u << i;
    bool sure = true;
    if (L.groups > 1) {
        const int size = L.E / L.groups;
        Key sum = 0;  // lane g: group g's
#pragma unroll 1
        for (int g = 0; g < L.groups; ++g) {
            uint32_t in = 0;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int e = i * 32 + lane;
                if (e >= g * size && e < (g + 1) * size)
                    in |= 1u << i;
            }
            Key top;
            const int at = best<V>(v, in, lane, top);
            Value s = S::value(top);
            if (size > 1) {
                if ((at & 31) == lane)
                    in &= ~(1u << (at >> 5));
                best<V>(v, in, lane, top);
                s += S::value(top);
            }
            if (lane == g)
                sum = S::key(s);
        }
        uint32_t chosen = 0;
        Value last = 0;
        const int rounds = scored ? min(L.top_groups + 1, L.groups) : L.top_groups;
#pragma unroll 1
        for (int j = 0; j < rounds; ++j) {
            Key top;
            const int g = best_of(sum, lane, top);
            if (j == L.top_groups) {
                sure = leads(last, S::value(top), L);
            } else {
                chosen |= 1u << g;
                if (g == lane)
                    sum = 0;
            }
            last = S::value(top);
        }
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (!(chosen >> min((i * 32 + lane) / size, 31) & 1))
                open &= ~(1u << i);
    }
    Value last = 0;
#pragma unroll 1
    for (int j = 0; j <= L.k; ++j) {
        if (j == L.k && !scored)
            break;
        Key top;
        const int at = best<V>(v, open, lane, top);
        if (at == kNone)
            break;
        if (scored && j > 0 && !leads(last, S::value(top), L))
            sure = false;
        last = S::value(top);
        if (j < L.k) {
            if (lane == j)
                mine = at;
            if ((at & 31) == lane)
                open &= ~(1u << (at >> 5));
        }
    }
    return sure;
}

// The same from scores in fp64. v: V * 32 of the warp's own in shared memory.
template <int V>
__device__ __forceinline__ int select_exactly(const RouteLaunch &L, int64_t t, int lane, uint64_t *v)
{
    float top = -INFINITY;
    bool nan = false;
#pragma unroll 1
    for (int i = 0; i < V; ++i) {
        const int e = i * 32 + lane;
        const float z = e < L.E ? load(L.logits, L.type, t * L.E + e) : -INFINITY;
        nan = nan || z != z;
        top = fmaxf(top, z);
    }
    nan = __any_sync(kAll, nan);
#pragma unroll
    for (int o = 16; o > 0; o /= 2)
        top = fmaxf(top, __shfl_xor_sync(kAll, top, o));
    const bool nothing = top == -INFINITY && !nan;
    double sum = 0;
#pragma unroll 1
    for (int i = 0; i < V; ++i) {
        const int e = i * 32 + lane;
        const double z = e < L.E ? (double)load(L.logits, L.type, t * L.E + e) : -INFINITY;
        const double x = exp(L.sigmoid ? -z : z - (double)top);
        const double s = L.sigmoid ? 1.0 / (1.0 + x) : nothing ? 0.0 : x;
        v[e] = (uint64_t)__double_as_longlong(s);
        sum += s;
    }
#pragma unroll
    for (int o = 16; o > 0; o /= 2)
        sum += __shfl_xor_sync(kAll, sum, o);
    if (L.sigmoid || nothing)
        sum = 1.0;
#pragma unroll 1
    for (int i = 0; i < V; ++i) {
        const int e = i * 32 + lane;
        const double s = __longlong_as_double((int64_t)v[e]);
        v[e] = DoubleKeys::key(s / sum + (L.bias && e < L.E ? (double)__ldg(L.bias + e) : 0.0));
    }
    __syncwarp();
    int mine = 0;
    select<V>(DoubleKeys{v}, L, lane, false, mine);
    __syncwarp();
    return mine;
}

__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int o = 16; o > 0; o /= 2)
        v += __shfl_xor_sync(kAll, v, o);
    return v;
}

// What a token's scores are made with: s = exp(z - top) / whole, or the sigmoid.
struct Shift {
    float top, whole;
    bool nothing;  // every logit is -inf: softmax scores are 0
};
__device__ __forceinline__ float score_of(const RouteLaunch &L, const Shift &f, float z)
{
    if (L.sigmoid)
        return 1.f / (1.f + expf(-z));
    return f.nothing ? 0.f : expf(z - f.top) / f.whole;
}

// z[i]: the logit of expert i * 32 + lane, -inf behind the last.
template <int V>
__device__ __forceinline__ Shift read_token(const RouteLaunch &L, int64_t t, int lane, float (&z)[V])
{
    float top = -INFINITY;
    bool nan = false;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int e = i * 32 + lane;
        z[i] = e < L.E ? load(L.logits, L.type, t * L.E + e) : -INFINITY;
        nan = nan || z[i] != z[i];
        top = fmaxf(top, z[i]);
    }
    Shift f = {0.f, 1.f, false};
    if (L.sigmoid)
        return f;
#pragma unroll
    for (int o = 16; o > 0; o /= 2)
        top = fmaxf(top, __shfl_xor_sync(kAll, top, o));
    f.top = top;
    nan = __any_sync(kAll, nan);
    f.nothing = top == -INFINITY && !nan;
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i)
        sum += f.nothing ? 0.f : expf(z[i] - top);
    f.whole = warp_sum(sum);  // NaN where a logit is
    return f;
}

template <int V>
__device__ __forceinline__ void choose_token(const RouteLaunch &L, int64_t t, int lane, uint64_t *exact)
{
    float z[V];
    const Shift f = read_token<V>(L, t, lane, z);
    const bool by_logit = !L.bias && L.groups == 1;
    Keys<V> keys;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int e = i * 32 + lane;
        float x = z[i];
        if (!by_logit)
            x = score_of(L, f, x) + (L.bias && e < L.E ? __ldg(L.bias + e) : 0.f);
        keys.v[i] = key_of(x);
    }
    int mine = 0;
    if (!select<V>(keys, L, lane, !by_logit, mine))
        mine = select_exactly<V>(L, t, lane, exact);
    float p = 0.f;
    if (lane < L.k)
        p = score_of(L, f, load(L.logits, L.type, t * L.E + mine));
    const float total = warp_sum(p) + kNil;
    if (lane < L.k) {
        L.experts[t * L.k + lane] = mine;
        L.weights[t * L.k + lane] = L.scale * (L.renormalise ? p / total : p);
    }
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

// Places the block's slots. counts: kWarps x E in shared memory, each warp's own; `sums`: E
// and one more. With more than one run the other runs' counts are in L.counts.
__device__ __forceinline__ void place_block(const Args &a, int32_t *counts, int32_t *sums,
                                            int32_t *scan, int64_t from, int64_t to)
{
    const RouteLaunch &L = a.L;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, threads = kWarps * 32;
    const int run = blockIdx.x;
    const int64_t n = to - from, each = (n + kWarps - 1) / kWarps;
    const int64_t first = min(to, from + warp * each), last = min(to, first + each);
    for (int i = threadIdx.x; i < kWarps * L.E; i += threads)
        counts[i] = 0;
    __syncthreads();
    count_slots(L.experts, first, last, counts + warp * L.E, lane);
    __syncthreads();
    // Every expert's slots in all runs (sums) and in those before (scan). Whole numbers: the
    // order of these additions changes nothing.
    for (int e = threadIdx.x; e < L.E; e += threads) {
        int32_t total = 0;
        if (a.runs == 1)
            for (int w = 0; w < kWarps; ++w)
                total += counts[w * L.E + e];
        sums[e] = total;
        scan[e] = 0;
    }
    if (a.runs > 1) {
        __syncthreads();
        const int parts = max(1, threads / L.E), each_run = (a.runs + parts - 1) / parts;
        for (int i = threadIdx.x; i < parts * L.E; i += threads) {
            const int part = i / L.E, e = i - part * L.E;
            const int r0 = part * each_run, r1 = min(a.runs, r0 + each_run);
            int32_t before = 0, total = 0;
#pragma unroll 8
            for (int r = r0; r < r1; ++r) {
                const int32_t c = __ldg(L.counts + r * L.E + e);
                before += r < run ? c : 0;
                total += c;
            }
            atomicAdd(sums + e, total);
            atomicAdd(scan + e, before);
        }
        __syncthreads();
    }
    for (int e = threadIdx.x; e < L.E; e += threads) {
        int32_t at = scan[e];
        for (int w = 0; w < kWarps; ++w) {
            const int32_t c = counts[w * L.E + e];
            counts[w * L.E + e] = at;
            at += c;
        }
    }
    __syncthreads();
    // Starts of the experts' parts: an exclusive scan of the padded lengths by one warp.
    if (warp == 0) {
        int32_t carry = 0;
        for (int b = 0; b < L.E; b += 32) {
            const int e = b + lane;
            const int32_t c = e < L.E ? (sums[e] + L.align - 1) / L.align * L.align : 0;
            int32_t x = c;
#pragma unroll
            for (int o = 1; o < 32; o *= 2) {
                const int32_t y = __shfl_up_sync(kAll, x, o);
                if (lane >= o)
                    x += y;
            }
            if (e < L.E)
                scan[e] = carry + x - c;
            carry += __shfl_sync(kAll, x, 31);
        }
        if (lane == 0)
            scan[L.E] = carry;
    }
    __syncthreads();
    if (run == 0)
        for (int e = threadIdx.x; e <= L.E; e += threads)
            L.offsets[e] = scan[e];
    // Slots in order: this warp's run of them.
    for (int64_t i = first; i < last; i += 32) {
        const bool in = i + lane < last;
        const int e = in ? L.experts[i + lane] : -1;
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
            L.rows[to_row] = (int32_t)(i + lane);
            L.slots[i + lane] = to_row;
        }
        __syncwarp();
    }
    // Rows that no slot takes: the ends of the parts, and what lies behind the last.
    for (int e = run * kWarps + warp; e < L.E; e += a.runs * kWarps)
        for (int32_t i = scan[e] + sums[e] + lane; i < scan[e + 1]; i += 32)
            L.rows[i] = -1;
    for (int64_t i = scan[L.E] + (int64_t)run * threads + threadIdx.x; i < L.R;
         i += (int64_t)a.runs * threads)
        L.rows[i] = -1;
}

// Experts and weights of a run of tokens, and the run's slots counted by expert.
template <int V>
__global__ void __launch_bounds__(kWarps * 32, V <= 8 ? 2 : 1) choose_kernel(const Args a)
{
    extern __shared__ __align__(8) int32_t shared[];
    const RouteLaunch &L = a.L;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t from = min(L.T, blockIdx.x * a.per), to = min(L.T, from + a.per);
    for (int64_t t = from + warp; t < to; t += kWarps)
        choose_token<V>(L, t, lane, reinterpret_cast<uint64_t *>(shared) + warp * V * 32);
    __syncthreads();
    if (a.runs == 1) {
        place_block(a, shared, shared + kWarps * L.E, shared + (kWarps + 1) * L.E + 1, from * L.k,
                    to * L.k);
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

__global__ void __launch_bounds__(kWarps * 32) place_kernel(const Args a)
{
    extern __shared__ int32_t shared[];
    const RouteLaunch &L = a.L;
    const int64_t from = min(L.T, blockIdx.x * a.per), to = min(L.T, from + a.per);
    place_block(a, shared, shared + kWarps * L.E, shared + (kWarps + 1) * L.E + 1, from * L.k,
                to * L.k);
}

// dz from dw, a warp a token: with g_j = ds of the chosen (through the renormalisation where
// there is one), softmax: dz = s * (g - sum_j g_j s_j); sigmoid: dz = g * s * (1 - s).
template <int V>
__global__ void __launch_bounds__(256)
    route_backward_kernel(const RouteLaunch L, const int32_t *experts, const float *dweights,
                          float *dlogits)
{
    const int lane = threadIdx.x & 31;
    const int64_t t = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    if (t >= L.T)
        return;
    float z[V];
    const Shift f = read_token<V>(L, t, lane, z);
    int mine = -1;
    float dw = 0.f, p = 0.f;
    if (lane < L.k) {
        const int e = experts[t * L.k + lane];
        if (e >= 0 && e < L.E) {
            mine = e;
            dw = dweights[t * L.k + lane];
            p = score_of(L, f, load(L.logits, L.type, t * L.E + e));
        }
    }
    float g = L.scale * dw;
    if (L.renormalise) {
        const float total = warp_sum(p) + kNil, mean = warp_sum(dw * p) / total;
        g = mine >= 0 ? L.scale * (dw - mean) / total : 0.f;
    }
    const float inner = L.sigmoid ? 0.f : warp_sum(g * p);
    float *out = dlogits + t * L.E;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int e = i * 32 + lane;
        if (e < L.E)
            out[e] = L.sigmoid ? 0.f : -inner * score_of(L, f, z[i]);
    }
    __syncwarp();
    // The chosen experts' own terms; one that is named twice gets both.
    float all = 0.f;
    for (int j = 0; j < L.k; ++j) {
        const int e = __shfl_sync(kAll, mine, j);
        const float x = __shfl_sync(kAll, g, j);
        all += e == mine ? x : 0.f;
    }
    if (mine >= 0)
        out[mine] = L.sigmoid ? all * p * (1.f - p) : p * (all - inner);
}

// ---------------------------------------------------------------- joining

// Four columns a thread, a row in chunks of 1024 (or 256 of few tokens, whose call is bound by
// latency); four rows of C are asked for at once. Bound by the bytes of C.
template <bool VEC>
__global__ void __launch_bounds__(256)
    join_kernel(int64_t T, int64_t N, int k, int64_t R, const float *C, const int32_t *slots,
                const float *weights, float *Y, int64_t chunks)
{
    const int64_t t = blockIdx.x / chunks, width = blockDim.x * 4;
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
                    if (n + blockDim.x * i < N)
                        v[j][i] = __ldg(c + blockDim.x * i);
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
            if (n + blockDim.x * i < N)
                y[blockDim.x * i] = acc[i];
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
template <bool VEC, int WARPS>
__global__ void __launch_bounds__(128)
    join_backward_kernel(int64_t count, int64_t N, int k, int64_t R, int type, const void *dY,
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
                const float4 d = load4(dY, type, t * N + n);
                sum[0] = fmaf(d.x, v.x, sum[0]);
                sum[1] = fmaf(d.y, v.y, sum[1]);
                sum[2] = fmaf(d.z, v.z, sum[2]);
                sum[3] = fmaf(d.w, v.w, sum[3]);
            }
        } else {
#pragma unroll 4
            for (int64_t n = id; n < N; n += THREADS)
                sum[0] = fmaf(load(dY, type, t * N + n), __ldg(c + n), sum[0]);
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

static int runs_of(int64_t T) { return T <= kOneBlock ? 1 : (int)(T < kMaxRuns * 2 ? (T + 1) / 2 : kMaxRuns); }

constexpr size_t place_bytes(int E) { return ((size_t)(kWarps + 2) * E + 2) * 4; }

template <int V>
static cudaError_t launch_choose(const Args &a, cudaStream_t stream)
{
    constexpr size_t exact = (size_t)kWarps * V * 32 * 8;  // select_exactly's scores
    constexpr size_t most = place_bytes(V * 32);
    static std::atomic<uint64_t> done{0};
    const cudaError_t e =
        set_smem_limit_once(choose_kernel<V>, (int)(exact > most ? exact : most), done);
    if (e != cudaSuccess)
        return e;
    const size_t place = place_bytes(a.L.E), smem = place > exact ? place : exact;
    choose_kernel<V><<<a.runs, kWarps * 32, smem, stream>>>(a);
    return cudaGetLastError();
}

template <int V>
static cudaError_t launch_backward(const RouteLaunch &L, const int32_t *experts,
                                   const float *dweights, float *dlogits, cudaStream_t stream)
{
    const int64_t blocks = (L.T + 7) / 8;
    if (blocks > 0x7fffffff)
        return cudaErrorInvalidValue;
    route_backward_kernel<V><<<(unsigned)blocks, 256, 0, stream>>>(L, experts, dweights, dlogits);
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
    const cudaError_t f = set_smem_limit_once(place_kernel, (int)place_bytes(kRouteMaxExperts), done);
    if (f != cudaSuccess)
        return f;
    place_kernel<<<a.runs, kWarps * 32, place_bytes(L.E), stream>>>(a);
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
    const int threads = T * N < 152 * 4096 ? 64 : 256;
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

template <bool VEC>
static cudaError_t launch_join_backward(int64_t T, int64_t N, int k, int64_t R, int type,
                                        const void *dY, const float *C, const int32_t *slots,
                                        float *dweights, cudaStream_t stream)
{
    // A block a slot while that leaves SMs idle.
    const int64_t count = T * k;
    const bool few = count < 152 * 16;
    const int64_t blocks = few ? count : (count + 3) / 4;
    if (blocks > 0x7fffffff)
        return cudaErrorInvalidValue;
    if (few)
        route::join_backward_kernel<VEC, 4><<<(unsigned)blocks, 128, 0, stream>>>(
            count, N, k, R, type, dY, C, slots, dweights);
    else
        route::join_backward_kernel<VEC, 1><<<(unsigned)blocks, 128, 0, stream>>>(
            count, N, k, R, type, dY, C, slots, dweights);
    return cudaGetLastError();
}

cudaError_t launch_experts_join_backward(int64_t T, int64_t N, int k, int64_t R, int type,
                                         const void *dY, const float *C, const int32_t *slots,
                                         float *dweights, cudaStream_t stream)
{
    const bool vec =
        N % 4 == 0 && ((reinterpret_cast<uintptr_t>(C) | reinterpret_cast<uintptr_t>(dY)) & 15) == 0;
    return vec ? launch_join_backward<true>(T, N, k, R, type, dY, C, slots, dweights, stream)
               : launch_join_backward<false>(T, N, k, R, type, dY, C, slots, dweights, stream);
}

} // namespace rtm
