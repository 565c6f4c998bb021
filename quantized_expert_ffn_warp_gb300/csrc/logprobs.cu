// Log probabilities of given tokens, the entropy of their distribution, and the
// likeliest tokens, from rows of logits l [V]; and the gradient of the first two.
//   m = max l,  s = sum_v e^(l_v - m),  logsum = log s
//   logp    = (l_target - m) - logsum
//   entropy = logsum - (1/s) sum_v e^(l_v - m) (l_v - m)     (a sum of terms >= 0)
//   dl_v    = g_logp (1[v = target] - p_v) - g_ent p_v (log p_v + entropy)
// m and logsum are kept apart: their sum could not hold logsum next to a large m.
//
// One pass over the row: each thread holds the running max of its values and the two
// sums against it.  The likeliest tokens cost that pass nothing: behind it, the k-th
// largest of the threads' maxima bounds the k-th value, and the few threads whose
// maximum reaches it are gone through again.  Candidates go into lists of 32, sorted
// over a warp's lanes; a key is the value's order and the complement of its index, so
// that ties go to the lowest index in whatever order they are met.
// Bound by HBM in fp32 (2000 x 131072 with 20 alternatives 168 us, 92% of the measured
// copy rate).  In 16 bits a value has half the bytes and the same arithmetic: 4096 x
// 32003 bf16 take 48 us (81%) without alternatives, half of the issue slots used, 61 us
// with 5 and 69 us with 32, whose search no loads of the block's own cover.  3 x 131072
// fp32 with 20 alternatives: 9 us in two launches.  The gradient of 4096 x 131072 bf16
// with an entropy term: 322 us (98% of the measured copy rate).
#include <algorithm>

#include "args.cuh"
#include "vec.cuh"

namespace qe {

namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kRowWarps = 4;            // of a forward block for one row, or 1
constexpr int kMaxTokens = 1 << 26, kMaxVocab = 1 << 20, kMaxTop = 32;
constexpr int kWordsPerThread = 4;      // 16-byte loads that a thread has under way
constexpr int kMaxSplits = 64;          // blocks of one row
constexpr float kFar = -220.f;          // 2^kFar and e^kFar are 0 in fp32, kFar is finite

// fp32 values as unsigned numbers in their order; a NaN like -inf, -0 like 0.
__device__ __forceinline__ unsigned order_of(float x)
{
    x = x == x ? x + 0.f : -INFINITY;
    const unsigned u = __float_as_uint(x);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float value_of(unsigned o)
{
    return __uint_as_float(o & 0x80000000u ? o ^ 0x80000000u : ~o);
}
using Key = unsigned long long;
__device__ __forceinline__ Key key_of(float x, int i)
{
    return (Key)order_of(x) << 32 | (unsigned)~i;
}

// Running max and the sums against it.
struct Sums {
    float m, s, sd;     // max, sum e^(l - m), sum e^(l - m) (l - m)

    // Sums against a max of at least m.
    __device__ __forceinline__ void raise(float max)
    {
        const float d = fmaxf(m - (max == -INFINITY ? 0.f : max), kFar);
        const float f = ex2(d * kLog2E);
        sd = f * (sd + s * d);
        s *= f;
        m = max;
    }
    // Sums over the lanes, in all of them.
    __device__ __forceinline__ void join_lanes()
    {
        raise(max_warp(m));
        s = sum_warp(s);
        sd = sum_warp(sd);
    }
};

// Values that a chunk of a row may be raised to without a change of its sums, and the
// maxima against which that holds: e^(kLow - m) is 0 for |m| <= kMost.  Products with
// log2 e stay finite, and `rest` below, half a step of m log2 e at most, stays below 1 / 8:
// it is an exponent of 2, and one of 128 has no fp32 power (a row of -1e10 has 440).
template <typename T>
constexpr float kLow = std::is_same_v<T, __half> ? -65504.f : -0x1p120f;
template <typename T>
constexpr float kMost = std::is_same_v<T, __half> ? 32768.f : 0x1p20f;

// Adds the values of U words to the sums; `top` is their largest.
//   e^(l - m) = 2^(l log2 e - c) 2^-rest,  c + rest = m log2 e:
// l log2 e - c is one fused operation, rounded at the size of the difference, on pairs of
// values; a -inf is first raised to a finite number, whose product with its
// exponential, 0, is 0.
template <typename T, int U>
__device__ __forceinline__ void add_words(Sums &u, const uint4 (&q)[U], float top)
{
    constexpr int N = Vec<T>::N;
    if (top > u.m)
        u.raise(top);
    if (fabsf(u.m) <= kMost<T>) {
        const float c = u.m * kLog2E, rest = fmaf(u.m, kLog2E, -c), f = ex2(-rest);
        const F2 l2e = f2(kLog2E), mc = f2(-c);
        F2 s[2] = {f2(0.f), f2(0.f)}, sd[2] = {f2(0.f), f2(0.f)};
#pragma unroll
        for (int i = 0; i < U; i++) {
            F2 x[N / 2];
            unpack<T>(word_raise<T>(q[i], kLow<T>), x);
#pragma unroll
            for (int e = 0; e < N / 2; e++) {
                const F2 a = fma(x[e], l2e, mc);
                const float2 d = split(a);
                const F2 p = f2(ex2(d.x), ex2(d.y));
                s[e & 1] = add(s[e & 1], p);
                sd[e & 1] = fma(p, a, sd[e & 1]);
            }
        }
        const float sum_s = sum(add(s[0], s[1])), sum_sd = sum(add(sd[0], sd[1]));
        u.s = fmaf(f, sum_s, u.s);
        u.sd = fmaf(f * kLn2, fmaf(-rest, sum_s, sum_sd), u.sd);
        return;
    }
    // nothing but -inf or a mask's fill yet, large logits, or no number: m is subtracted first
    const float m = u.m == -INFINITY ? 0.f : u.m;
#pragma unroll
    for (int i = 0; i < U; i++) {
        float x[N];
        unpack<T>(q[i], x);
#pragma unroll
        for (int e = 0; e < N; e++) {
            const float d = max_nan(x[e] - m, kFar), p = ex2(d * kLog2E);
            u.s += p;
            u.sd = fmaf(p, d, u.sd);
        }
    }
}

__device__ __forceinline__ Key shfl_key(Key k, int src)
{
    return __shfl_sync(0xffffffffu, k, src);
}

// Puts c into the warp's list, sorted in falling order over its lanes.
__device__ __forceinline__ void insert(Key &list, Key c)
{
    const int lane = threadIdx.x & 31;
    const int at = __popc(__ballot_sync(0xffffffffu, list > c));
    const Key up = __shfl_up_sync(0xffffffffu, list, 1);
    list = lane < at ? list : lane == at ? c : up;
}

// The best 32 of two sorted lists, sorted: the larger of each value and its
// mirror image are a bitonic sequence.
template <typename V>
__device__ __forceinline__ V merge(V a, V b)
{
    const int lane = threadIdx.x & 31;
    const V r = __shfl_sync(0xffffffffu, b, 31 - lane);
    a = a > r ? a : r;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
        const V o = __shfl_xor_sync(0xffffffffu, a, d);
        a = ((lane & d) == 0) == (a > o) ? a : o;
    }
    return a;
}

// The lanes' values in falling order (a bitonic sort).
__device__ __forceinline__ float sort_lanes(float v)
{
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int size = 2; size <= 32; size <<= 1)
#pragma unroll
        for (int d = size / 2; d > 0; d >>= 1) {
            const float o = __shfl_xor_sync(0xffffffffu, v, d);
            const bool larger = ((lane & d) == 0) == ((lane & size) == 0);
            v = larger ? fmaxf(v, o) : fminf(v, o);
        }
    return v;
}

struct LogprobArgs {
    const void *logits;
    long long ld;
    int n, V, top;
    int splits, per;        // blocks of a row, words of one
    const int32_t *targets;
    float *logp, *entropy;
    float2 *stats;
    int32_t *top_ids;
    float *top_logp;
    float4 *part;           // [n][splits] sums of the blocks
    Key *part_keys;         // [n][splits][32]
};

// A thread's values are cut into at most kGroups groups of 4 words, 8, 16 .., whose
// largest values are kept until the row's bound is known.
constexpr int kGroups = 32, kBatch = 8;     // groups whose words are gone through at once

template <int W>
struct Block {
    float4 sums[W];
    Key keys[W][32];
};
template <int W>
struct Candidates {
    float most[W][32];              // the threads' largest values, sorted
    float group[kGroups][32 * W];   // the groups'
    int queued;
    int queue[kBatch * 32 * W];     // group * threads + thread
};

// Joins the W warps' sums and lists; warp 0 gets the result.
template <bool TOP, int W>
__device__ __forceinline__ void join_warps(Block<W> &sm, Sums &t, Key &list)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    t.join_lanes();
    if (lane == 0)
        sm.sums[warp] = make_float4(t.m, t.s, t.sd, 0.f);
    if (TOP)
        sm.keys[warp][lane] = list;
    __syncthreads();
    if (warp == 0) {
        const float4 q = lane < W ? sm.sums[lane] : make_float4(-INFINITY, 0.f, 0.f, 0.f);
        t = {q.x, q.y, q.z};
        t.join_lanes();
    }
    if (TOP) {
#pragma unroll
        for (int half = W / 2; half > 0; half >>= 1) {
            if (warp < half) {
                list = merge(list, sm.keys[warp + half][lane]);
                sm.keys[warp][lane] = list;
            }
            __syncthreads();
        }
    }
}

// A row's results, by warp 0; `given` is the target's logit.
template <bool TOP>
__device__ __forceinline__ void finish_row(const LogprobArgs &a, long long t, const Sums &u,
                                           Key list, int target, float given)
{
    const int lane = threadIdx.x & 31;
    const bool empty = u.m == -INFINITY && u.s == 0.f;  // nothing but -inf
    const float logsum = empty ? 0.f : logf(u.s);
    if (lane == 0) {
        a.stats[t] = make_float2(u.m, logsum);
        a.entropy[t] = empty ? 0.f : logsum - u.sd / u.s;
        if (a.targets)
            a.logp[t] = target < 0 || target >= a.V ? 0.f
                        : empty                     ? -INFINITY
                                                    : (given - u.m) - logsum;
    }
    if (TOP && lane < a.top) {
        a.top_ids[t * a.top + lane] = ~(unsigned)list;
        a.top_logp[t * a.top + lane] =
            empty ? -INFINITY : (value_of((unsigned)(list >> 32)) - u.m) - logsum;
    }
}

// The warp's list of the block's likeliest tokens.  The k-th largest of the threads'
// largest values bounds the block's k-th largest value from below, and few groups hold a
// value that reaches it: their words are queued and read again.
template <typename T, int W>
__device__ __forceinline__ Key collect(Candidates<W> &sm, const RowWords<T> &row, int lo, int hi,
                                       float most, int groups, int words, int top)
{
    constexpr int N = Vec<T>::N, threads = 32 * W;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    float best = sort_lanes(most);
    if (W > 1) {
        sm.most[warp][lane] = best;
        __syncthreads();
        best = sm.most[0][lane];
#pragma unroll
        for (int w = 1; w < W; w++)
            best = merge(best, sm.most[w][lane]);
    }
    const float bound = __shfl_sync(0xffffffffu, best, top - 1);
    Key list = 0, kth = 0;
    for (int g0 = 0; g0 < groups; g0 += kBatch) {
        if (threadIdx.x == 0)
            sm.queued = 0;
        __syncthreads();
        if (most >= bound)
            for (int g = g0; g < min(groups, g0 + kBatch); g++)
                if (sm.group[g][threadIdx.x] >= bound)
                    sm.queue[atomicAdd(&sm.queued, 1)] = g * threads + threadIdx.x;
        __syncthreads();
        const int count = sm.queued * words;
        for (int i0 = warp * 32; i0 < count; i0 += threads) {
            unsigned mask = 0;
            int first = 0;
            float x[N];
            if (i0 + lane < count) {
                const int e = sm.queue[(i0 + lane) / words], j = (i0 + lane) % words;
                const int v = lo + (e / threads * words + j) * threads + e % threads;
                first = row.first(v);
                if (v < hi) {
                    unpack<T>(row.load(v, -INFINITY), x);
#pragma unroll
                    for (int n = 0; n < N; n++)     // not below it: a NaN counts as -inf
                        mask |= !(x[n] < bound) && first + n >= 0 && first + n < row.len ? 1u << n
                                                                                         : 0u;
                }
            }
            while (__any_sync(0xffffffffu, mask != 0)) {
                Key c = 0;
                if (mask) {
                    const int n = __ffs(mask) - 1;
                    float v = x[0];
#pragma unroll
                    for (int k = 1; k < N; k++)
                        v = n == k ? x[k] : v;
                    c = key_of(v, first + n);
                    mask &= mask - 1;
                }
                unsigned offers = __ballot_sync(0xffffffffu, c > kth);
                while (offers) {
                    const Key k = shfl_key(c, __ffs(offers) - 1);
                    if (k > kth) {
                        insert(list, k);
                        kth = shfl_key(list, top - 1);
                    }
                    offers &= offers - 1;
                }
            }
        }
        __syncthreads();        // the queue is gone through
    }
    return list;
}

// W warps a row.
template <typename T, bool TOP, int W>
__global__ void __launch_bounds__(32 * W, 32 / W) logprobs_kernel(LogprobArgs a)
{
    constexpr int N = Vec<T>::N, U = kWordsPerThread, threads = 32 * W;
    __shared__ Block<W> sm;
    __shared__ std::conditional_t<TOP, Candidates<W>, int> cand;
    pdl_enter();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    float low[N];
#pragma unroll
    for (int e = 0; e < N; e++)
        low[e] = -INFINITY;
    const uint4 none = pack<T>(low);
    uint4 next[U];
    // words at + threadIdx.x + i threads
    const auto load = [&](const RowWords<T> &row, int at, int hi) {
        if (at + U * threads <= hi && row.inner(at, U * threads)) {
            const T *src = row.row + row.first(at + threadIdx.x);
#pragma unroll
            for (int i = 0; i < U; i++)
                next[i] = load_stream(src + i * (threads * N));
        } else {
#pragma unroll
            for (int i = 0; i < U; i++) {
                const int v = at + threadIdx.x + i * threads;
                next[i] = v < hi ? row.load(v, -INFINITY) : none;
            }
        }
    };
    // chunks of a group
    int per_group = 1;
    while (per_group * kGroups * U * threads < a.per)
        per_group *= 2;
    for (long long t = blockIdx.y; t < a.n; t += gridDim.y) {
        const RowWords<T> row(static_cast<const T *>(a.logits) + t * a.ld, a.V);
        const int lo = blockIdx.x * a.per, hi = min(row.count, lo + a.per);
        load(row, lo, hi);
        // the target's logit is under way behind them
        const int target = a.targets ? a.targets[t] : -1;
        const float given = target >= 0 && target < a.V ? to_float<T>(row.row[target]) : 0.f;
        Sums u = {-INFINITY, 0.f, 0.f};
        float most = -INFINITY;
        int chunk = 0, group = 0;
        for (int at = lo; at < hi; at += U * threads) {
            uint4 q[U];
            float top = -INFINITY;
#pragma unroll
            for (int i = 0; i < U; i++) {
                q[i] = next[i];
                top = fmaxf(top, word_max<T>(q[i]));
            }
            if (at + U * threads < hi)
                load(row, at + U * threads, hi);
            if constexpr (TOP) {
                most = fmaxf(most, top);
                if (++chunk == per_group || at + U * threads >= hi) {
                    cand.group[group++][threadIdx.x] = most;
                    most = -INFINITY;
                    chunk = 0;
                }
            }
            add_words<T, U>(u, q, top);
        }
        Key list = 0;
        if constexpr (TOP)
            list = collect<T, W>(cand, row, lo, hi, u.m, group, per_group * U, a.top);
        join_warps<TOP, W>(sm, u, list);
        if (warp == 0) {
            if (a.splits == 1) {
                finish_row<TOP>(a, t, u, list, target, given);
            } else {
                const long long at = t * a.splits + blockIdx.x;
                if (lane == 0)
                    a.part[at] = make_float4(u.m, u.s, u.sd, 0.f);
                if (TOP)
                    a.part_keys[at * 32 + lane] = list;
            }
        }
        __syncthreads();        // the next row's sums go into the same memory
    }
}

// Joins the blocks of each row.
template <typename T, bool TOP>
__global__ void __launch_bounds__(kThreads) logprobs_join_kernel(LogprobArgs a)
{
    __shared__ Block<kWarps> sm;
    pdl_enter();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const long long t = blockIdx.x, at = t * a.splits;
    const int target = a.targets ? a.targets[t] : -1;
    const float given = target >= 0 && target < a.V
                            ? to_float<T>(static_cast<const T *>(a.logits)[t * a.ld + target])
                            : 0.f;
    Sums u = {-INFINITY, 0.f, 0.f};
    if (threadIdx.x < a.splits) {       // at most kMaxSplits of them
        const float4 q = a.part[at + threadIdx.x];
        u = {q.x, q.y, q.z};
    }
    Key list = 0;
    if (TOP)
        for (int i = warp; i < a.splits; i += kWarps)
            list = merge(list, a.part_keys[(at + i) * 32 + lane]);
    join_warps<TOP, kWarps>(sm, u, list);
    if (warp == 0)
        finish_row<TOP>(a, t, u, list, target, given);
}

// Words of the longest row, whatever its address.
int most_words(int V, int per) { return (V + per - 1 + per - 1) / per; }

// Rows of at most eight chunks of words for every lane of a warp.
bool short_row(int V, int size)
{
    return most_words(V, 16 / size) <= 32 * kWordsPerThread * 8;
}
// Warps of a row: one for short rows, whose joins are the warp's own then (16000 x 4000
// bf16 with 20 alternatives 145 to 59 us), unless there are too few to fill the SMs.
int row_warps(int n, int V, int size) { return short_row(V, size) && n >= 4 * 152 ? 1 : kRowWarps; }

// Blocks of a row: enough for a block on every SM four times over, each with a
// load of kWordsPerThread words per thread.  Asks no device, since the workspace's size
// follows from it.
int row_splits(int n, int V, int size)
{
    const int words = most_words(V, 16 / size), step = 32 * kRowWarps * kWordsPerThread;
    const int want = 4 * 152 / std::min(n, 4 * 152);
    const int most = (words + step - 1) / step;
    return short_row(V, size) ? 1 : std::max(1, std::min({want, most, kMaxSplits}));
}

size_t key_offset(int n, int splits) { return ((size_t)n * splits * sizeof(float4) + 255) / 256 * 256; }

size_t logprob_ws(int n, int V, int size, int top)
{
    const int splits = row_splits(n, V, size);
    if (splits == 1)
        return 0;
    return key_offset(n, splits) + (top ? (size_t)n * splits * 32 * sizeof(Key) : 0);
}

template <typename T, bool TOP, int W>
cudaError_t launch_rows(const LogprobArgs &a, cudaStream_t st)
{
    return launch_pdl(logprobs_kernel<T, TOP, W>, dim3(a.splits, std::min(a.n, 65535)), dim3(32 * W), 0, st, a);
}
template <typename T, bool TOP>
cudaError_t launch_top(const LogprobArgs &a, cudaStream_t st)
{
    cudaError_t e = row_warps(a.n, a.V, sizeof(T)) == 1 ? launch_rows<T, TOP, 1>(a, st)
                                                   : launch_rows<T, TOP, kRowWarps>(a, st);
    if (e == cudaSuccess && a.splits > 1)
        e = launch_pdl(logprobs_join_kernel<T, TOP>, dim3(a.n), dim3(kThreads), 0, st, a);
    return e;
}
template <typename T>
cudaError_t launch_logprobs(const LogprobArgs &a, cudaStream_t st)
{
    return a.top ? launch_top<T, true>(a, st) : launch_top<T, false>(a, st);
}

struct LogprobGradArgs {
    const void *logits;
    long long ld;
    int n, V;
    const int32_t *targets;
    const float2 *stats;
    const float *entropy, *dlogp, *dent;
    void *out;
    long long ldo;
    bool aligned;       // the rows of both lie alike in their 16-byte words
};

// p_v = 2^(l_v log2 e - c) with c = (m + logsum) log2 e as a pair: l_v log2 e - c_hi is
// one fused operation, rounded at the size of the difference, and 2^-c_lo is a factor of
// the row's coefficients.  The constant's rounding scales l - m alone: logsum is multiplied
// by its two parts.  (An error of c_lo is one of all the row's p: the sum in one direction
// alone left up to half a step of logsum log2 e, 14 x 2^-24 of p in flat rows of 160001.)
template <typename T, bool ENT>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 2 ? 5 : 6) logprobs_grad_kernel(LogprobGradArgs a)
{
    constexpr int N = Vec<T>::N, U = kWordsPerThread;
    pdl_enter();
    const int v0 = blockIdx.x * (U * kThreads) + threadIdx.x;
    for (long long t = blockIdx.y; t < a.n; t += gridDim.y) {
        const RowWords<T> row(static_cast<const T *>(a.logits) + t * a.ld, a.V);
        T *out = static_cast<T *>(a.out) + t * a.ldo;
        int target = a.targets ? a.targets[t] : -1;
        if (target < 0 || target >= a.V)
            target = -1 - 2 * N;
        const float gl = target >= 0 ? a.dlogp[t] : 0.f;
        const float2 st = a.stats[t];
        // a token that takes no part, or a row of nothing but -inf
        const bool none = (!ENT && target < 0) || (st.x == -INFINITY && st.y == 0.f);
        if (none) {
            const float zero[N] = {};
#pragma unroll
            for (int i = 0; i < U; i++)
                if (v0 + i * kThreads < row.count)
                    row.store(out, v0 + i * kThreads, pack<T>(zero), a.aligned);
            continue;
        }
        uint4 q[U];
        // the block's words lie inside the row: no checks
        const bool inside = a.aligned && row.inner(blockIdx.x * (U * kThreads), U * kThreads);
        const T *src = row.row + row.first(v0);
#pragma unroll
        for (int i = 0; i < U; i++) {
            if (inside)
                q[i] = load_stream(src + i * (kThreads * N));
            else if (v0 + i * kThreads < row.count)
                q[i] = row.load(v0 + i * kThreads, 0.f);
        }
        // where `rest` could leave the exponents' range: m is subtracted first
        const bool far = fabsf(st.x) > 0x1p20f;
        const float m = far ? 0.f : st.x;
        // a two-sum of the rounded products, whichever is the larger; none is fused into it
        const float hi = __fmul_rn(m, kLog2E), ls = __fmul_rn(st.y, kLog2E), c = __fadd_rn(hi, ls);
        const float back = __fsub_rn(c, hi);
        const float err = __fadd_rn(__fsub_rn(hi, __fsub_rn(c, back)), __fsub_rn(ls, back));
        const float rest = fmaf(m, kLog2E, -hi) + fmaf(st.y, kLog2E, -ls) + err + st.y * kLog2ELow;
        const float f = ex2(-rest);
        const float ge = ENT ? a.dent[t] : 0.f, ent = ENT ? a.entropy[t] : 0.f;
        // -p (gl + ge (log p + entropy)), log p = (arg - rest) ln 2
        const F2 l2e = f2(kLog2E), mc = f2(-c);
        const F2 slope = f2(-f * ge * kLn2), level = f2(-f * (gl + ge * (ent - rest * kLn2)));
#pragma unroll
        for (int i = 0; i < U; i++) {
            const int v = v0 + i * kThreads;
            if (!inside && v >= row.count)
                break;
            F2 x[N / 2];
            unpack<T>(q[i], x);
            if (far) {
#pragma unroll
                for (int e = 0; e < N / 2; e++) {
                    const float2 w = split(x[e]);
                    x[e] = f2(w.x - st.x, w.y - st.x);
                }
            }
#pragma unroll
            for (int e = 0; e < N / 2; e++) {
                float2 d = split(fma(x[e], l2e, mc));
                if (ENT) {      // a finite number for a logit of -inf
                    d.x = max_nan(d.x, kFar);
                    d.y = max_nan(d.y, kFar);
                }
                const F2 p = f2(ex2(d.x), ex2(d.y));
                x[e] = mul(p, ENT ? fma(f2(d.x, d.y), slope, level) : level);
            }
            const unsigned at = target - row.first(v);
            if (at < N) {
#pragma unroll
                for (int e = 0; e < N / 2; e++)
                    x[e] = add(x[e], f2(at == 2u * e ? gl : 0.f, at == 2u * e + 1 ? gl : 0.f));
            }
            if (inside)
                *reinterpret_cast<uint4 *>(out + row.first(v)) = pack<T>(x);
            else
                row.store(out, v, pack<T>(x), a.aligned);
        }
    }
}

template <typename T>
cudaError_t launch_logprobs_grad(const LogprobGradArgs &a, cudaStream_t st)
{
    constexpr int per = kThreads * kWordsPerThread;
    const int words = most_words(a.V, Vec<T>::N);
    const dim3 grid((words + per - 1) / per, std::min(a.n, 65535));
    return a.dent ? launch_pdl(logprobs_grad_kernel<T, true>, grid, dim3(kThreads), 0, st, a)
                  : launch_pdl(logprobs_grad_kernel<T, false>, grid, dim3(kThreads), 0, st, a);
}

int check_sizes(int dtype, int n, int V)
{
    if (dtype != MOE_FP16 && dtype != MOE_BF16 && dtype != MOE_FP32)
        return record_failure(MOE_ERR_UNSUPPORTED, "dtype must be MOE_FP16, MOE_BF16 or MOE_FP32");
    if (n < 1 || n > kMaxTokens)
        return record_failure(MOE_ERR_INVALID_ARG, "n_tokens must be in 1..67108864");
    if (V < 1 || V > kMaxVocab)
        return record_failure(MOE_ERR_INVALID_ARG, "vocab must be in 1..1048576");
    return MOE_OK;
}

int size_of(int dtype) { return dtype == MOE_FP32 ? 4 : 2; }

}  // namespace

}  // namespace qe

extern "C" size_t moe_token_logprobs_workspace(int n_tokens, int vocab, int dtype, int top)
{
    using namespace qe;
    if (n_tokens < 1 || n_tokens > kMaxTokens || vocab < 1 || vocab > kMaxVocab || top < 0 ||
        top > kMaxTop || dtype < MOE_FP16 || dtype > MOE_FP32)
        return 0;
    return logprob_ws(n_tokens, vocab, size_of(dtype), top);
}

extern "C" int moe_token_logprobs(const void *logits, int dtype, long long ld, int n_tokens,
                                  int vocab, const int32_t *targets, int top, float *logp,
                                  float *entropy, float *stats, int32_t *top_ids, float *top_logp,
                                  void *workspace, size_t workspace_bytes, void *stream)
{
    using namespace qe;
    const int rc = check_sizes(dtype, n_tokens, vocab);
    if (rc)
        return rc;
    if (top < 0 || top > kMaxTop || top > vocab)
        return record_failure(MOE_ERR_INVALID_ARG, "top must be in 0..min(32, vocab)");
    if (!logits || !entropy || !stats || (targets && !logp) || (top && (!top_ids || !top_logp)))
        return record_failure(MOE_ERR_INVALID_ARG, "null pointer argument");
    const int size = size_of(dtype);
    const size_t need = logprob_ws(n_tokens, vocab, size, top), n = n_tokens;
    if (need && (!workspace || workspace_bytes < need))
        return record_failure(MOE_ERR_INVALID_ARG,
                              "workspace below moe_token_logprobs_workspace(...)");
    const Arg args[] = {rows_arg(logits, ld, vocab, n_tokens, size, size),
                        flat_arg(targets, n, 4),
                        flat_arg(targets ? logp : nullptr, n, 4, true),
                        flat_arg(entropy, n, 4, true),
                        flat_arg(stats, n, 8, true),
                        flat_arg(top ? top_ids : nullptr, n * top, 4, true),
                        flat_arg(top ? top_logp : nullptr, n * top, 4, true),
                        flat_arg(need ? workspace : nullptr, (need + 255) / 256, 256, true)};
    int dev, sms;
    if (const int bad = check_args(args, sizeof(args) / sizeof(args[0]), &dev, &sms))
        return bad;
    LogprobArgs a{};
    a.logits = logits;
    a.ld = ld;
    a.n = n_tokens;
    a.V = vocab;
    a.top = top;
    a.splits = row_splits(n_tokens, vocab, size);
    a.per = (most_words(vocab, 16 / size) + a.splits - 1) / a.splits;
    a.targets = targets;
    a.logp = logp;
    a.entropy = entropy;
    a.stats = reinterpret_cast<float2 *>(stats);
    a.top_ids = top_ids;
    a.top_logp = top_logp;
    a.part = static_cast<float4 *>(workspace);
    a.part_keys = reinterpret_cast<Key *>(static_cast<char *>(workspace) +
                                          key_offset(n_tokens, a.splits));
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return launch_result(dtype == MOE_FP32   ? launch_logprobs<float>(a, st)
                         : dtype == MOE_FP16 ? launch_logprobs<__half>(a, st)
                                             : launch_logprobs<__nv_bfloat16>(a, st));
}

extern "C" int moe_token_logprobs_grad(const void *logits, int dtype, long long ld, int n_tokens,
                                       int vocab, const int32_t *targets, const float *stats,
                                       const float *entropy, const float *dlogp,
                                       const float *dentropy, void *dlogits, long long ldd,
                                       void *stream)
{
    using namespace qe;
    const int rc = check_sizes(dtype, n_tokens, vocab);
    if (rc)
        return rc;
    if (!logits || !stats || !dlogits || (dentropy && !entropy) || (dlogp && !targets))
        return record_failure(MOE_ERR_INVALID_ARG, "null pointer argument");
    if (!dlogp && !dentropy)
        return record_failure(MOE_ERR_INVALID_ARG, "need dlogp or dentropy");
    const int size = size_of(dtype);
    const size_t n = n_tokens;
    const Arg args[] = {rows_arg(logits, ld, vocab, n_tokens, size, size),
                        flat_arg(dlogp ? targets : nullptr, n, 4),
                        flat_arg(stats, n, 8),
                        flat_arg(dentropy ? entropy : nullptr, n, 4),
                        flat_arg(dlogp, n, 4),
                        flat_arg(dentropy, n, 4),
                        rows_arg(dlogits, ldd, vocab, n_tokens, size, size, true, logits)};
    int dev, sms;
    if (const int bad = check_args(args, sizeof(args) / sizeof(args[0]), &dev, &sms))
        return bad;
    LogprobGradArgs a{};
    a.logits = logits;
    a.ld = ld;
    a.n = n_tokens;
    a.V = vocab;
    a.targets = dlogp ? targets : nullptr;
    a.stats = reinterpret_cast<const float2 *>(stats);
    a.entropy = entropy;
    a.dlogp = dlogp;
    a.dent = dentropy;
    a.out = dlogits;
    a.ldo = ldd;
    a.aligned = ((uintptr_t)logits - (uintptr_t)dlogits) % 16 == 0 &&
                (n_tokens == 1 || (ld - ldd) * size % 16 == 0);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return launch_result(dtype == MOE_FP32   ? launch_logprobs_grad<float>(a, st)
                         : dtype == MOE_FP16 ? launch_logprobs_grad<__half>(a, st)
                                             : launch_logprobs_grad<__nv_bfloat16>(a, st));
}
