// Routing losses of a batch and their gradient in the router logits.
//
// For the tokens t of segment s (valid ones, T_s of them) with p = softmax(l_t):
//   f[s][e] = E / (k T_s) * counts[s][e],   P[s][e] = 1/T_s sum_t p[t][e]
//   balance = mean over segments with T_s > 0 of sum_e f[s][e] P[s][e]
//   z       = sum_t lse_t^2 / sum_s T_s,    lse_t = log sum_e exp(l[t][e])
// counts is a constant of the gradient (it does not move with the logits):
//   dl[t][e] = g_b / (S' T_s) p_e (f_e - sum_j f_j p_j) + g_z 2 lse_t / T p_e
// and, with the top-k weights w = softmax of the selected logits,
//   dl[t][idx_j] += w_j (dw_j - sum_i w_i dw_i).
//
// Everything is a stream over the logits, one warp per token, its row in
// registers, the next token's row already under way (a token's arithmetic is
// shorter than a load).  The forward sums p over the tokens of a block in
// registers and writes one partial row per (block of tokens, segment); a
// second kernel adds the partial rows in block order, so a result never depends
// on timing.  A batch that one CTA handles needs neither partial rows nor the
// second kernel.
// Measured in a replayed graph: losses of 64 tokens x 64 experts 4.0 us (one
// CTA, latency), of 32768 x 256 fp32 18.8 us (two thirds of the issue slots used,
// then the second kernel's latency); gradient of 65521 x 256 with top-8 weights in bf16
// 29.8 us (70% of the issue slots used), in fp32 45.5 us (55%, with 29% of the
// warps an SM holds: loads and shared memory are waited for); without weights
// 21.2 and 35.4 us.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <cstring>

#include "internal.cuh"

namespace qe {

namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kFinalThreads = 1024;
constexpr int kMaxTokens = 1 << 26;
constexpr int kMaxSegments = 65535;     // a grid dimension

__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int d = 16; d > 0; d >>= 1)
        v += __shfl_xor_sync(0xffffffffu, v, d);
    return v;
}

// A pair of values as one word (or two), so that it is loaded and stored whole.
template <typename T>
struct Pair {
    uint32_t u;
};
template <>
struct Pair<float> {
    float2 u;
};
__device__ __forceinline__ float2 unpair(const Pair<float> &p) { return p.u; }
__device__ __forceinline__ float2 unpair(const Pair<__half> &p)
{
    return __half22float2(*reinterpret_cast<const __half2 *>(&p.u));
}
__device__ __forceinline__ float2 unpair(const Pair<__nv_bfloat16> &p)
{
    return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&p.u));
}
__device__ __forceinline__ void pair(Pair<float> &p, float a, float b) { p.u = make_float2(a, b); }
__device__ __forceinline__ void pair(Pair<__half> &p, float a, float b)
{
    const __half2 h = __floats2half2_rn(a, b);
    p.u = *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ void pair(Pair<__nv_bfloat16> &p, float a, float b)
{
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    p.u = *reinterpret_cast<const uint32_t *>(&h);
}

// exp(x), documented within 2 + floor(1.173 |x|) ulp: a relative error of at most
// (4 + 2.35 |x|) 2^-24.  x may exceed 0 by a rounding of lse.
__device__ __forceinline__ float exp_neg(float x) { return __expf(x); }

// The hardware's 2^x.
__device__ __forceinline__ float exp2_fast(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// A lane's part of a row of E values, as loaded: V of them, pairs side by side
// (V = 1: one value, the pair's first).  The same values in the same lane
// whether or not the rows allow pair loads (`wide`: E and the stride even, the
// base on a pair), so that sums do not depend on the stride.
template <typename T, int V>
struct Row {
    static constexpr int W = V > 1 ? 2 : 1, N = V / W;
    Pair<T> q[N];
    static __device__ __forceinline__ int at(int i, int lane)
    {
        return (i / W) * 32 * W + lane * W + i % W;
    }
    // values past the row read -inf
    __device__ __forceinline__ void load(const T *row, int E, int lane, bool wide)
    {
        if (wide && E == 32 * V) {
#pragma unroll
            for (int n = 0; n < N; n++)
                if (W == 2)
                    q[n] = *reinterpret_cast<const Pair<T> *>(row + at(n * W, lane));
            if (W == 2)
                return;
        }
#pragma unroll
        for (int n = 0; n < N; n++) {
            const int e = at(n * W, lane);
            pair(q[n], -INFINITY, -INFINITY);
            if (W == 2 && wide) {
                if (e < E)
                    q[n] = *reinterpret_cast<const Pair<T> *>(row + e);
            } else {
                T v[2];
                memcpy(v, &q[n], sizeof(v));
                if (e < E)
                    v[0] = row[e];
                if (W == 2 && e + 1 < E)
                    v[1] = row[e + 1];
                memcpy(&q[n], v, sizeof(v));
            }
        }
    }
    __device__ __forceinline__ void get(float (&d)[V]) const
    {
#pragma unroll
        for (int n = 0; n < N; n++) {
            const float2 f = unpair(q[n]);
            d[n * W] = f.x;
            if (W == 2)
                d[n * W + W - 1] = f.y;
        }
    }
    static __device__ __forceinline__ void store(T *row, const float (&d)[V], int E, int lane,
                                                 bool wide)
    {
#pragma unroll
        for (int n = 0; n < N; n++) {
            const int e = at(n * W, lane);
            Pair<T> p;
            pair(p, d[n * W], d[n * W + W - 1]);
            if (W == 2 && wide) {
                if (e < E)
                    *reinterpret_cast<Pair<T> *>(row + e) = p;
            } else {
                T v[2];
                memcpy(v, &p, sizeof(p));
                if (e < E)
                    row[e] = v[0];
                if (W == 2 && e + 1 < E)
                    row[e + 1] = v[1];
            }
        }
    }
};

// Segment bounds as the kernels use them: inside [0, n] whatever the array holds.
struct Segs {
    const int32_t *off;     // [S + 1] or null: one segment of all tokens
    int S, n;
    __device__ __forceinline__ int begin(int s) const
    {
        return off ? min(max(off[s], 0), n) : 0;
    }
    __device__ __forceinline__ int end(int s) const
    {
        return off ? min(max(off[s + 1], 0), n) : n;
    }
    // first segment that ends after token t (S: none)
    __device__ __forceinline__ int first_after(int t) const
    {
        if (!off)
            return 0;
        int lo = 0, hi = S;
        while (lo < hi) {
            const int mid = (lo + hi) / 2;
            if (off[mid + 1] > t)
                hi = mid;
            else
                lo = mid + 1;
        }
        return lo;
    }
};

// Sums are fp32 (64-bit arithmetic is slow on this GPU) in chains whose length
// does not grow with the batch: kChain tokens in a warp's registers, folded into
// pairs (sum, rounding errors); the warps of a block; the blocks of a segment, at
// most 20 in each of 32 chains or, with more than 150 segments, 153 in each of 4;
// pairs again over the segments.  A sum of non-negative terms is off by at most
// 64 + 8 + 157 fp32 roundings and a few more at any size.
constexpr int kChain = 64;

// Adds v to the pair (sum, err) without loss: the rounding of each addition goes
// into err (two-sum).
__device__ __forceinline__ void fold(float &sum, float &err, float v)
{
    const float s = __fadd_rn(sum, v), b = __fsub_rn(s, sum);
    err += __fadd_rn(__fsub_rn(sum, __fsub_rn(s, b)), __fsub_rn(v, b));
    sum = s;
}
// The pair's value (behind an infinity the errors are NaN).
__device__ __forceinline__ float unfold(float sum, float err)
{
    return err == err ? sum + err : sum;
}

// Workspace: [ticket, 256 B][loss parts f32 [S][ceil(E/32)]][z sums f32 [slots]]
// [z sums f32 [S]][valid tokens int [slots]][prob sums f32 [slots][E]][counts int [slots][E]]
struct BalanceWs {
    unsigned *ticket;
    float *part;
    float *z;
    float *zseg;
    int *valid;
    float *prob;
    int *counts;
    size_t bytes;
};

// Tokens of a block: as many blocks as run at once on 152 SMs (four per SM, two
// and one for the widest rows), and at least one token per warp.  The workspace's
// size follows from it, so it asks no device.
int block_tokens(int n, int E)
{
    const int blocks = 152 * (E <= 256 ? 4 : E <= 512 ? 2 : 1);
    return ((n + blocks - 1) / blocks + kWarps - 1) / kWarps * kWarps;
}

// Whether one CTA of kOneWarps warps handles the whole batch: it takes about a
// microsecond per 64 tokens and per segment, two dependent kernels about five
// more than that.
constexpr int kOneWarps = 32;
bool one_block(int n, int E, int S) { return n <= 8 * kOneWarps && E <= 512 && S <= 4; }

BalanceWs balance_ws(void *base, int n, int E, int S)
{
    const int C = block_tokens(n, E);
    const size_t slots = (size_t)(n + C - 1) / C + S;
    BalanceWs w{};
    char *b = static_cast<char *>(base);
    size_t at = 0;
    const auto take = [&](size_t bytes) {
        char *p = b + at;
        at += (bytes + 255) / 256 * 256;
        return p;
    };
    w.ticket = reinterpret_cast<unsigned *>(take(4));
    w.part = reinterpret_cast<float *>(take(4 * (size_t)S * ((E + 31) / 32)));
    w.z = reinterpret_cast<float *>(take(4 * slots));
    w.zseg = reinterpret_cast<float *>(take(4 * (size_t)S));
    w.valid = reinterpret_cast<int *>(take(4 * slots));
    w.prob = reinterpret_cast<float *>(take(4 * slots * E));
    w.counts = reinterpret_cast<int *>(take(4 * slots * E));
    w.bytes = at;
    return w;
}

struct FwdArgs {
    const void *logits;
    long long ld;
    const int32_t *idx;
    const uint8_t *mask;
    Segs segs;
    int n, E, k, C;
    bool wide;              // rows allow pair loads
    BalanceWs ws;
    float *loss, *prob, *lse;
    int32_t *counts, *tokens;
};

// Per block of C tokens: lse of every token, and per segment that the block
// meets the partial sums at slot (block + segment): both only ever grow along
// the tokens, so a slot belongs to one pair.  ONE: the block is the batch and
// writes the results themselves.
template <typename T, int V, bool ONE>
__global__ void __launch_bounds__(ONE ? 32 * kOneWarps : kThreads, ONE ? 1 : V <= 8 ? 4 : V <= 16 ? 2 : 1)
    balance_stats_kernel(FwdArgs a)
{
    constexpr int NW = ONE ? kOneWarps : kWarps, NT = 32 * NW;
    using R = Row<T, V>;
    // prob [NW][E], counts int [E], and in long blocks the prob sums' errors [NW][E]
    extern __shared__ float sm[];
    __shared__ float zred[NW], zerr[NW];
    __shared__ int vred[NW];
    __shared__ float lred[NW];
    pdl_enter();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int E = a.E, t_lo = blockIdx.x * a.C, t_hi = min(a.n, t_lo + a.C);
    int *hist = reinterpret_cast<int *>(sm + NW * E);
    const T *logits = static_cast<const T *>(a.logits);
    if (!ONE && blockIdx.x == 0 && threadIdx.x == 0)
        *a.ws.ticket = 0;
    float bal = 0.f, zall = 0.f;        // ONE: sums over the segments
    int all = 0, segs = 0;

    // U tokens at a time: one's reductions run in the other's shadow
    constexpr int U = V <= (ONE ? 8 : 16) ? 2 : 1;
    struct Token {
        R row;
        int id;
        bool on;
    };
    const auto load = [&](int tok, int end, Token &k) {
        k.on = false;
        k.id = -1;
        if (tok < end) {
            k.row.load(logits + tok * a.ld, E, lane, a.wide);
            k.on = !a.mask || a.mask[tok];
            if (lane < a.k)
                k.id = a.idx[(long long)tok * a.k + lane];
        }
    };

    int t = t_lo;       // next token without a segment
    // ONE writes every segment's results, the empty ones in front of token 0 too
    for (int s = ONE ? 0 : a.segs.first_after(t_lo); s < a.segs.S && (t < t_hi || ONE); s++) {
        const int b = min(max(a.segs.begin(s), t), t_hi), e = min(a.segs.end(s), t_hi);
        for (int i = t + threadIdx.x; i < b; i += NT)
            a.lse[i] = 0.f;             // tokens in front of the first segment
        t = max(t, b);
        if (e <= b && !ONE)
            continue;
        t = max(t, e);
        Token next[U];
#pragma unroll
        for (int i = 0; i < U; i++)
            load(b + warp + i * NW, e, next[i]);
        for (int i = threadIdx.x; i < E; i += NT)
            hist[i] = 0;
        __syncthreads();
        float psum[V];
#pragma unroll
        for (int i = 0; i < V; i++)
            psum[i] = 0.f;
        float zsum = 0.f;
        int valid = 0;
        // A long block's tokens in spans of kChain per warp; behind each span the
        // warp's sums go into its shared row and zred.
        constexpr int kSpan = kChain * NW;
        const auto fold_all = [&](bool first) {
            float *sum = sm + warp * E + lane, *err = sum + (NW + 1) * E;
#pragma unroll
            for (int i = 0; i < V; i++) {
                const int x = R::at(i, lane) - lane;
                if (x + lane < E) {
                    if (first)
                        sum[x] = err[x] = 0.f;
                    fold(sum[x], err[x], psum[i]);
                }
                psum[i] = 0.f;
            }
            if (lane == 0) {
                if (first)
                    zred[warp] = zerr[warp] = 0.f;
                fold(zred[warp], zerr[warp], zsum);
            }
            zsum = 0.f;
        };
        int tok = b + warp;
        for (int stop = ONE ? e : min(e, b + kSpan);; stop = min(e, stop + kSpan)) {
            for (; tok < stop; tok += U * NW) {
                float l[U][V], m[U], sum[U];
                bool on[U];
#pragma unroll
                for (int u = 0; u < U; u++) {
                    on[u] = next[u].on;
                    valid += on[u];
                    if (on[u] && next[u].id >= 0 && next[u].id < E)
                        atomicAdd(hist + next[u].id, 1);
                    next[u].row.get(l[u]);
                    m[u] = -INFINITY;
                    if (!on[u]) {   // a row of -inf: p = 0
#pragma unroll
                        for (int i = 0; i < V; i++)
                            l[u][i] = -INFINITY;
                    }
#pragma unroll
                    for (int i = 0; i < V; i++)
                        m[u] = fmaxf(m[u], l[u][i]);
                    load(tok + (U + u) * NW, e, next[u]);
                }
#pragma unroll
                for (int d = 16; d > 0; d >>= 1)
#pragma unroll
                    for (int u = 0; u < U; u++)
                        m[u] = fmaxf(m[u], __shfl_xor_sync(0xffffffffu, m[u], d));
#pragma unroll
                for (int u = 0; u < U; u++) {
                    // exp(l - m) = 2^(l log2 e - m log2 e): the rounding of m log2 e is a
                    // common factor of the row, which p does not see and lse, about m
                    // itself, holds to an fp32 step
                    constexpr float kLog2e = 1.4426950408889634f;
                    m[u] = m[u] == -INFINITY ? 0.f : m[u];
                    float ml = -m[u] * kLog2e;
                    // beyond 2^16 (rows of a mask's lowest value) that factor, or
                    // m log2 e itself, could overflow: m is subtracted first
                    if (fabsf(m[u]) > 65536.f) {
                        ml = 0.f;
#pragma unroll
                        for (int i = 0; i < V; i++)
                            l[u][i] -= m[u];
                    }
                    sum[u] = 0.f;
#pragma unroll
                    for (int i = 0; i < V; i++) {
                        l[u][i] = exp2_fast(fmaf(l[u][i], kLog2e, ml));
                        sum[u] += l[u][i];
                    }
                }
#pragma unroll
                for (int d = 16; d > 0; d >>= 1)
#pragma unroll
                    for (int u = 0; u < U; u++)
                        sum[u] += __shfl_xor_sync(0xffffffffu, sum[u], d);
#pragma unroll
                for (int u = 0; u < U; u++) {
                    // a row of -inf (every expert masked) has no distribution: p = 0
                    const float inv = sum[u] == 0.f ? 0.f : __fdividef(1.0f, sum[u]);
#pragma unroll
                    for (int i = 0; i < V; i++)
                        psum[i] = fmaf(l[u][i], inv, psum[i]);
                    const float lse = m[u] + __logf(sum[u]);
                    if (sum[u] != 0.f)
                        zsum = fmaf(lse, lse, zsum);
                    if (lane == 0 && tok + u * NW < e)
                        a.lse[tok + u * NW] = on[u] ? lse : 0.f;
                }
            }
            if (ONE || stop == e)
                break;
            fold_all(stop == b + kSpan);
        }
        if (!ONE && e - b > kSpan) {
            fold_all(false);
#pragma unroll
            for (int i = 0; i < V; i++)
                if (R::at(i, lane) < E) {
                    float *sum = sm + warp * E + R::at(i, lane);
                    *sum = unfold(*sum, sum[(NW + 1) * E]);
                }
            if (lane == 0)
                zred[warp] = unfold(zred[warp], zerr[warp]);
        } else {
#pragma unroll
            for (int i = 0; i < V; i++)
                if (R::at(i, lane) < E)
                    sm[warp * E + R::at(i, lane)] = psum[i];
            if (lane == 0)
                zred[warp] = zsum;
        }
        if (lane == 0)
            vred[warp] = valid;
        __syncthreads();
        int v = 0;
        float z = 0.f;
        if (ONE || threadIdx.x == 0) {
#pragma unroll 8
            for (int w = 0; w < NW; w++) {
                z += zred[w];
                v += vred[w];
            }
        }
        float part = 0.f;
        const long long slot = (long long)blockIdx.x + s;
        for (int i = threadIdx.x; i < E; i += NT) {
            float p = sm[i];
#pragma unroll 8
            for (int w = 1; w < NW; w++)
                p += sm[w * E + i];
            if (ONE) {
                a.counts[(long long)s * E + i] = hist[i];
                a.prob[(long long)s * E + i] = v > 0 ? p / (float)v : 0.f;
                part += (float)hist[i] * p;
            } else {
                a.ws.prob[slot * E + i] = p;
                a.ws.counts[slot * E + i] = hist[i];
            }
        }
        if (ONE) {
#pragma unroll
            for (int d = 16; d > 0; d >>= 1)
                part += __shfl_xor_sync(0xffffffffu, part, d);
            if (lane == 0)
                lred[warp] = part;
            if (v > 0) {
                zall += z;
                all += v;
                segs++;
            }
            if (threadIdx.x == 0)
                a.tokens[s] = v;
        } else if (threadIdx.x == 0) {
            a.ws.z[slot] = z;
            a.ws.valid[slot] = v;
        }
        __syncthreads();
        if (ONE && v > 0) {
            part = 0.f;
#pragma unroll 8
            for (int w = 0; w < NW; w++)
                part += lred[w];
            bal += part / (float)v * ((float)E / ((float)a.k * (float)v));
        }
    }
    for (int i = t + threadIdx.x; i < t_hi; i += NT)
        a.lse[i] = 0.f;                 // tokens behind the last segment
    if (ONE && threadIdx.x == 0) {
        a.loss[0] = segs ? bal / (float)segs : 0.f;
        a.loss[1] = all ? zall / (float)all : 0.f;
    }
}

// One CTA per (32 experts, segment): the partial rows in block order, counts,
// mean probabilities and the CTA's part of the loss; the last CTA of the grid
// adds the parts in a fixed order.
__global__ void __launch_bounds__(kFinalThreads) balance_final_kernel(FwdArgs a)
{
    constexpr int W = kFinalThreads / 32;
    __shared__ float sp[W][32];
    __shared__ int sc[W][32];
    __shared__ int sv[W];
    __shared__ float sz[W], sb[W];
    __shared__ int last;
    pdl_enter();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    const int s = blockIdx.y, e = blockIdx.x * 32 + lane, E = a.E;
    const int b = a.segs.begin(s), end = a.segs.end(s);
    const int b0 = b / a.C, b1 = end > b ? (end - 1) / a.C + 1 : b0;
    float p = 0.f, z = 0.f;
    int c = 0, v = 0;
#pragma unroll 4
    for (int i = b0 + warp; i < b1; i += warps) {
        const long long slot = (long long)i + s;
        if (e < E) {
            p += a.ws.prob[slot * E + e];
            c += a.ws.counts[slot * E + e];
        }
        v += a.ws.valid[slot];
        z += a.ws.z[slot];
    }
    sp[warp][lane] = p;
    sc[warp][lane] = c;
    if (lane == 0) {
        sv[warp] = v;
        sz[warp] = z;
    }
    __syncthreads();
    if (warp == 0) {
        p = z = 0.f;
        c = v = 0;
        for (int w = 0; w < warps; w++) {
            p += sp[w][lane];
            c += sc[w][lane];
            v += sv[w];
            z += sz[w];
        }
        float part = 0.f;
        if (v > 0 && e < E)
            part = (float)c * p / (float)v * ((float)E / ((float)a.k * (float)v));
        if (e < E) {
            a.counts[(long long)s * E + e] = c;
            a.prob[(long long)s * E + e] = v > 0 ? p / (float)v : 0.f;
        }
        part = warp_sum(part);
        if (lane == 0) {
            if (blockIdx.x == 0) {
                a.tokens[s] = v;
                a.ws.zseg[s] = z;
            }
            a.ws.part[(long long)s * gridDim.x + blockIdx.x] = part;
            __threadfence();
            last = atomicAdd(a.ws.ticket, 1u) + 1 == gridDim.x * gridDim.y;
        }
    }
    __syncthreads();
    if (!last)
        return;
    __threadfence();
    float bal = 0.f, bal_err = 0.f, z_err = 0.f;
    z = 0.f;
    int tokens = 0, live = 0;
    for (int i = threadIdx.x; i < (int)(gridDim.x * gridDim.y); i += blockDim.x)
        fold(bal, bal_err, __ldcg(a.ws.part + i));
    for (int q = threadIdx.x; q < a.segs.S; q += blockDim.x) {
        const int t = __ldcg(a.tokens + q);
        tokens += t;
        live += t > 0;
        fold(z, z_err, __ldcg(a.ws.zseg + q));
    }
    bal = unfold(bal, bal_err);
    z = unfold(z, z_err);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
        bal += __shfl_xor_sync(0xffffffffu, bal, d);
        z += __shfl_xor_sync(0xffffffffu, z, d);
        tokens += __shfl_xor_sync(0xffffffffu, tokens, d);
        live += __shfl_xor_sync(0xffffffffu, live, d);
    }
    if (lane == 0) {
        sb[warp] = bal;
        sz[warp] = z;
        sv[warp] = tokens;
        sc[warp][0] = live;
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        bal = z = 0.f;
        tokens = live = 0;
        for (int w = 0; w < warps; w++) {
            bal += sb[w];
            z += sz[w];
            tokens += sv[w];
            live += sc[w][0];
        }
        a.loss[0] = live ? bal / (float)live : 0.f;
        a.loss[1] = tokens ? z / (float)tokens : 0.f;
    }
}

struct BwdArgs {
    const void *logits;
    long long ld;
    const int32_t *idx;
    const uint8_t *mask;
    Segs segs;
    int n, E, k, per_warp;
    int half_k;             // k rounded up to a power of two, halved
    bool wide;              // rows allow pair loads and stores
    const float *lse;
    const int32_t *counts, *tokens;
    const float *dloss, *w, *dw;
    void *out;
    long long ldo;
};

// One warp per run of `per_warp` tokens, so that the row f of its segment
// mostly stays in registers.  The gradients of the top-k weights are computed
// for as many tokens as fill a warp, and reach their experts' lanes through two
// rows of shared memory in turn: a token writes one and clears what the token
// before it wrote in the other.  One warp barrier stands between that token's
// reads and the clearing, a second between this token's writes and its reads.
template <typename T, int V>
__global__ void __launch_bounds__(kThreads) balance_grad_kernel(BwdArgs a)
{
    using R = Row<T, V>;
    extern __shared__ float sm[];       // with dw: [kWarps][2][32 V], zero between tokens
    __shared__ int red_t[kWarps], red_l[kWarps];
    pdl_enter();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, E = a.E;
    float *add = sm + warp * 64 * V;
    if (a.dw)
        for (int i = lane; i < 64 * V; i += 32)
            add[i] = 0.f;
    // valid tokens and segments with any, over the batch
    int tokens = 0, live = 0;
    for (int s = threadIdx.x; s < a.segs.S; s += kThreads) {
        const int v = a.tokens[s];
        tokens += v;
        live += v > 0;
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
        tokens += __shfl_xor_sync(0xffffffffu, tokens, d);
        live += __shfl_xor_sync(0xffffffffu, live, d);
    }
    if (lane == 0) {
        red_t[warp] = tokens;
        red_l[warp] = live;
    }

    const T *logits = static_cast<const T *>(a.logits);
    T *out = static_cast<T *>(a.out);
    const long long t_lo = ((long long)blockIdx.x * kWarps + warp) * a.per_warp;
    const int t_hi = (int)min((long long)a.n, t_lo + a.per_warp);
    struct Token {
        R row;
        float lse;
        bool on;
    };
    const auto load = [&](int tok, int end, Token &k) {
        k.on = false;
        if (tok < end) {
            k.row.load(logits + tok * a.ld, E, lane, a.wide);
            k.lse = a.lse[tok];
            k.on = !a.mask || a.mask[tok];
        }
    };
    // the top-k weights of 32 / kp tokens at once, kp lanes each
    const int kp = 2 * a.half_k > 0 ? 2 * a.half_k : 1, batch = 32 / kp;
    float w = 0.f, dw = 0.f;
    int id = -1;
    const auto load_w = [&](int tok) {
        const int tk = tok + lane / kp, j = lane % kp;
        w = dw = 0.f;
        id = -1;
        if (tk < t_hi && j < a.k) {
            const long long at = (long long)tk * a.k + j;
            w = a.w[at];
            dw = a.dw[at];
            id = a.idx[at];
        }
    };
    Token next;
    load((int)min((long long)a.n, t_lo), t_hi, next);
    if (a.dw)
        load_w((int)min((long long)a.n, t_lo));
    __syncthreads();
    tokens = live = 0;
    for (int i = 0; i < kWarps; i++) {
        tokens += red_t[i];
        live += red_l[i];
    }
    const float gb = live > 0 ? a.dloss[0] / (float)live : 0.f;
    const float gz = tokens > 0 ? 2.0f * a.dloss[1] / (float)tokens : 0.f;
    if (t_lo >= a.n)
        return;

    int batch0 = (int)t_lo - batch;     // first token of the batch in v, to
    float v = 0.f;                      // gradient in this lane's selected logit
    int to = -1, was = -1;              // its expert; the entry to clear
    int row = 0;                        // the two shared rows take turns
    // this token's contributions into shared row `row`; clears the other row
    const auto scatter = [&](int tok) {
        if (tok >= batch0 + batch) {
            batch0 = tok;
            float wd = w * dw;
            for (int o = a.half_k; o > 0; o >>= 1)
                wd += __shfl_xor_sync(0xffffffffu, wd, o);
            v = w * (dw - wd);
            const bool real = id >= 0 && id < E;
            // an expert twice in a token: its first slot adds them all, in order
            const int key = real ? id * 32 + lane / kp : -1 - lane;
            const unsigned same = __match_any_sync(0xffffffffu, key);
            if (__any_sync(0xffffffffu, same & (same - 1))) {
                float total = 0.f;
                for (int j = 0; j < 32; j++) {
                    const float o = __shfl_sync(0xffffffffu, v, j);
                    total += same >> j & 1 ? o : 0.f;
                }
                v = total;
            }
            to = real && (same & ((1u << lane) - 1)) == 0 ? id : -1;
            load_w(tok + batch);
        }
        const int mine = lane / kp == tok - batch0 ? to : -1;
        __syncwarp();
        if (was >= 0)
            add[(row ^ 1) * 32 * V + was] = 0.f;
        if (mine >= 0)
            add[row * 32 * V + mine] = v;
        was = mine;
        __syncwarp();
    };

    int s = a.segs.first_after((int)t_lo), tok = (int)t_lo;
    while (tok < t_hi) {
        // a run of tokens inside one segment, or between two
        const bool seg = s < a.segs.S;
        const int sb = seg ? a.segs.begin(s) : a.n, se = seg ? a.segs.end(s) : a.n;
        const bool in = seg && tok >= sb;
        const int stop = min(t_hi, in ? max(se, tok + 1) : max(sb, tok + 1));
        const int ts = in ? a.tokens[s] : 0;
        const float scale = ts > 0 ? (float)E / ((float)a.k * (float)ts) * (gb / (float)ts) : 0.f;
        float f[V];         // g_b / (S' T_s) f_e of this lane's experts
#pragma unroll
        for (int i = 0; i < V; i++) {
            const int x = R::at(i, lane);
            f[i] = in && x < E ? (float)a.counts[(long long)s * E + x] * scale : 0.f;
        }
        for (; tok < stop; tok++) {
            const bool on = in && next.on;
            // a row of -inf has no distribution, and a token that takes no part no
            // gradient
            const bool none = !on || next.lse == -INFINITY;
            const float lse = none ? 0.f : next.lse;
            float d[V], dot = 0.f;
            next.row.get(d);
            load(tok + 1, t_hi, next);
            if (none) {
#pragma unroll
                for (int i = 0; i < V; i++)
                    d[i] = -INFINITY;
            }
#pragma unroll
            for (int i = 0; i < V; i++) {
                d[i] = exp_neg(d[i] - lse);
                dot = fmaf(f[i], d[i], dot);
            }
            dot = warp_sum(dot);
            // lse holds log(sum) to an fp32 step of lse only: rows of large
            // logits are normalised again (p is off by at most a factor E)
            if (fabsf(lse) > 64.f) {
                float sum = 0.f;
#pragma unroll
                for (int i = 0; i < V; i++)
                    sum += d[i];
                const float inv = 1.f / warp_sum(sum);
                dot *= inv;
#pragma unroll
                for (int i = 0; i < V; i++)
                    d[i] *= inv;
            }
            const float all = gz * lse - dot;
#pragma unroll
            for (int i = 0; i < V; i++)
                d[i] *= f[i] + all;
            if (none) {     // 0 whatever dloss holds (0 times its infinity is not)
#pragma unroll
                for (int i = 0; i < V; i++)
                    d[i] = 0.f;
            }
            if (a.dw) {
                scatter(tok);
                if (on) {
#pragma unroll
                    for (int i = 0; i < V; i += R::W) {
                        const float *p = add + row * 32 * V + R::at(i, lane);
                        if (R::W == 2) {
                            const float2 v2 = *reinterpret_cast<const float2 *>(p);
                            d[i] += v2.x;
                            d[i + R::W - 1] += v2.y;
                        } else {
                            d[i] += *p;
                        }
                    }
                }
                row ^= 1;
            }
            R::store(out + tok * a.ldo, d, E, lane, a.wide);
        }
        if (in)
            s = max(s + 1, a.segs.first_after(tok));
    }
}

template <typename T, int V>
cudaError_t launch_stats(const FwdArgs &a, cudaStream_t st)
{
    if (V <= 16 && one_block(a.n, a.E, a.segs.S)) {
        constexpr int VO = V <= 16 ? V : 16;
        auto kernel = balance_stats_kernel<T, VO, true>;
        const size_t smem = sizeof(float) * (kOneWarps + 1) * a.E;
        // the kernel's largest, whatever this call needs: a smaller value set
        // by one call would fail a larger one on another thread
        constexpr size_t most = sizeof(float) * (kOneWarps + 1) * 32 * VO;
        if (most > 48 * 1024) {
            const cudaError_t e = cudaFuncSetAttribute(
                kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most);
            if (e != cudaSuccess)
                return e;
        }
        return launch_pdl(kernel, dim3(1), dim3(32 * kOneWarps), smem, st, a);
    }
    cudaError_t e = cudaSuccess;
    const int rows = a.C > kChain * kWarps ? 2 * kWarps + 1 : kWarps + 1;
    constexpr size_t most = sizeof(float) * (2 * kWarps + 1) * 32 * V;
    if (most > 48 * 1024)
        e = cudaFuncSetAttribute(balance_stats_kernel<T, V, false>,
                                 cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most);
    if (e == cudaSuccess)
        e = launch_pdl(balance_stats_kernel<T, V, false>, dim3((a.n + a.C - 1) / a.C),
                       dim3(kThreads), sizeof(float) * rows * a.E, st, a);
    if (e != cudaSuccess)
        return e;
    // a warp for each block that a segment meets on average, up to 32
    const int per = (int)((a.n + a.C - 1) / a.C / a.segs.S) + 1;
    const int warps = per >= 16 ? 32 : per >= 8 ? 16 : per >= 4 ? 8 : 4;
    return launch_pdl(balance_final_kernel, dim3((a.E + 31) / 32, a.segs.S), dim3(32 * warps), 0, st,
                      a);
}

template <typename T, int V>
cudaError_t launch_grad(const BwdArgs &a, cudaStream_t st)
{
    const long long warps = (a.n + a.per_warp - 1) / a.per_warp;
    const size_t smem = a.dw ? sizeof(float) * kWarps * 64 * V : 0;
    if (smem > 48 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(
            balance_grad_kernel<T, V>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess)
            return e;
    }
    return launch_pdl(balance_grad_kernel<T, V>, dim3((unsigned)((warps + kWarps - 1) / kWarps)),
                      dim3(kThreads), smem, st, a);
}

// V = ceil(E / 32) rounded up to a power of two: a row's registers per lane.
template <typename T>
cudaError_t stats(const FwdArgs &a, cudaStream_t st)
{
    return a.E <= 32    ? launch_stats<T, 1>(a, st)
           : a.E <= 64  ? launch_stats<T, 2>(a, st)
           : a.E <= 128 ? launch_stats<T, 4>(a, st)
           : a.E <= 256 ? launch_stats<T, 8>(a, st)
           : a.E <= 512 ? launch_stats<T, 16>(a, st)
                        : launch_stats<T, 32>(a, st);
}

template <typename T>
cudaError_t grad(const BwdArgs &a, cudaStream_t st)
{
    return a.E <= 32    ? launch_grad<T, 1>(a, st)
           : a.E <= 64  ? launch_grad<T, 2>(a, st)
           : a.E <= 128 ? launch_grad<T, 4>(a, st)
           : a.E <= 256 ? launch_grad<T, 8>(a, st)
           : a.E <= 512 ? launch_grad<T, 16>(a, st)
                        : launch_grad<T, 32>(a, st);
}

// Whether every row starts on a boundary of two values of `size` bytes.
bool pairs(const void *p, long long ld, int E, size_t size)
{
    return E % 2 == 0 && ld % 2 == 0 && reinterpret_cast<uintptr_t>(p) % (2 * size) == 0;
}

}  // namespace

bool rows_overlap(const void *a, long long lda, int wa, const void *b, long long ldb, int wb, int n,
                  int size);
bool rows_meet(const void *p, long long ld, int w, int n, int size, const void *q, size_t bytes);
bool ranges_meet(const void *p, size_t n, const void *q, size_t m);
bool device_pointer_here(const void *p, int dev);
int record_failure(int code, const char *msg);
int record_success();

namespace {

// Checks that both calls share; 0 or a recorded failure.
int check_batch(int dtype, long long ld, int n, int E, int k, int S, const void *seq)
{
    if (dtype != MOE_FP16 && dtype != MOE_BF16 && dtype != MOE_FP32)
        return record_failure(MOE_ERR_UNSUPPORTED, "dtype must be MOE_FP16, MOE_BF16 or MOE_FP32");
    if (n < 1 || n > kMaxTokens)
        return record_failure(MOE_ERR_INVALID_ARG, "n_tokens must be in 1..67108864");
    if (E < 1 || E > kMaxExperts)
        return record_failure(MOE_ERR_INVALID_ARG, "n_experts must be in 1..1024");
    if (k < 1 || k > kMaxTopK || k > E)
        return record_failure(MOE_ERR_INVALID_ARG, "top_k must be in 1..min(32, n_experts)");
    if (ld < E || ld > (1LL << 31))
        return record_failure(MOE_ERR_INVALID_ARG,
                              "a row stride is below n_experts or above 2^31");
    if (S < 1 || S > kMaxSegments || (!seq && S != 1))
        return record_failure(MOE_ERR_INVALID_ARG,
                              "n_segments must be in 1..65535, and 1 without seq_offsets");
    return MOE_OK;
}

bool misaligned(const void *p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) != 0; }

int current_device()
{
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) {
        cudaGetLastError();
        return -1;
    }
    return dev;
}

uintptr_t size_of(int dtype) { return dtype == MOE_FP32 ? 4 : 2; }

int launched(cudaError_t e)
{
    if (e != cudaSuccess) {
        cudaGetLastError();
        return record_failure(MOE_ERR_CUDA, cudaGetErrorString(e));
    }
    return record_success();
}

}  // namespace

}  // namespace qe

extern "C" size_t moe_balance_workspace(int n_tokens, int n_experts, int n_segments)
{
    if (n_tokens < 1 || n_tokens > qe::kMaxTokens || n_experts < 1 || n_experts > qe::kMaxExperts ||
        n_segments < 1 || n_segments > qe::kMaxSegments)
        return 0;
    return qe::balance_ws(nullptr, n_tokens, n_experts, n_segments).bytes;
}

extern "C" int moe_balance_loss(const void *logits, int dtype, long long ld, int n_tokens,
                                int n_experts, const int32_t *topk_idx, int top_k,
                                const int32_t *seq_offsets, int n_segments, const uint8_t *mask,
                                float *loss, int32_t *counts, int32_t *tokens, float *prob,
                                float *lse, void *workspace, size_t workspace_bytes, void *stream)
{
    using namespace qe;
    if (!logits || !topk_idx || !loss || !counts || !tokens || !prob || !lse || !workspace)
        return record_failure(MOE_ERR_INVALID_ARG, "null pointer argument");
    const int rc = check_batch(dtype, ld, n_tokens, n_experts, top_k, n_segments, seq_offsets);
    if (rc)
        return rc;
    if (misaligned(logits, size_of(dtype)) || misaligned(topk_idx, 4) ||
        misaligned(seq_offsets, 4) || misaligned(loss, 4) || misaligned(counts, 4) ||
        misaligned(tokens, 4) || misaligned(prob, 4) || misaligned(lse, 4) ||
        misaligned(workspace, 256))
        return record_failure(MOE_ERR_INVALID_ARG,
                              "misaligned pointer (workspace needs 256 bytes)");
    FwdArgs a{};
    a.ws = balance_ws(workspace, n_tokens, n_experts, n_segments);
    if (workspace_bytes < a.ws.bytes)
        return record_failure(MOE_ERR_INVALID_ARG,
                              "workspace below moe_balance_workspace(n, n_experts, n_segments)");
    // what the call writes against everything else
    const size_t n = n_tokens, S = n_segments;
    const struct {
        const void *p;
        size_t bytes;
    } range[] = {{workspace, a.ws.bytes}, {loss, 8}, {counts, 4 * S * n_experts}, {tokens, 4 * S},
                 {prob, 4 * S * n_experts}, {lse, 4 * n}, {topk_idx, 4 * n * top_k},
                 {seq_offsets, seq_offsets ? 4 * (S + 1) : 0}, {mask, mask ? n : 0}};
    constexpr int kWritten = 6, kRanges = sizeof(range) / sizeof(range[0]);
    for (int i = 0; i < kWritten; i++) {
        bool meet = rows_meet(logits, ld, n_experts, n_tokens, (int)size_of(dtype), range[i].p,
                              range[i].bytes);
        for (int j = i + 1; j < kRanges; j++)
            meet = meet || ranges_meet(range[i].p, range[i].bytes, range[j].p, range[j].bytes);
        if (meet)
            return record_failure(MOE_ERR_INVALID_ARG,
                                  "an output or the workspace overlaps another argument");
    }
    const int dev = current_device();
    if (dev < 0)
        return record_failure(MOE_ERR_CUDA, "no usable current CUDA device");
    const void *all[] = {logits, topk_idx, seq_offsets, mask, loss, counts, tokens, prob, lse, workspace};
    for (const void *p : all)
        if (p && !device_pointer_here(p, dev))
            return record_failure(MOE_ERR_INVALID_ARG,
                                  "arguments must be device pointers of the current device");
    a.logits = logits;
    a.ld = ld;
    a.idx = topk_idx;
    a.mask = mask;
    a.segs = {seq_offsets, n_segments, n_tokens};
    a.n = n_tokens;
    a.E = n_experts;
    a.k = top_k;
    a.C = one_block(n_tokens, n_experts, n_segments) ? n_tokens : block_tokens(n_tokens, n_experts);
    a.wide = pairs(logits, ld, n_experts, size_of(dtype));
    a.loss = loss;
    a.counts = counts;
    a.tokens = tokens;
    a.prob = prob;
    a.lse = lse;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return launched(dtype == MOE_FP32   ? stats<float>(a, st)
                    : dtype == MOE_FP16 ? stats<__half>(a, st)
                                        : stats<__nv_bfloat16>(a, st));
}

extern "C" int moe_balance_loss_grad(const void *logits, int dtype, long long ld, int n_tokens,
                                     int n_experts, const int32_t *topk_idx, int top_k,
                                     const int32_t *seq_offsets, int n_segments,
                                     const uint8_t *mask, const float *lse, const int32_t *counts,
                                     const int32_t *tokens, const float *dloss,
                                     const float *topk_w, const float *dtopk_w, void *dlogits,
                                     long long ldd, void *stream)
{
    using namespace qe;
    if (!logits || !lse || !counts || !tokens || !dloss || !dlogits)
        return record_failure(MOE_ERR_INVALID_ARG, "null pointer argument");
    if (dtopk_w && (!topk_w || !topk_idx))
        return record_failure(MOE_ERR_INVALID_ARG, "dtopk_w needs topk_w and topk_idx");
    const int rc = check_batch(dtype, std::min(ld, ldd), n_tokens, n_experts, top_k, n_segments,
                               seq_offsets);
    if (rc)
        return rc;
    if (std::max(ld, ldd) > (1LL << 31))
        return record_failure(MOE_ERR_INVALID_ARG, "a row stride is above 2^31");
    if (misaligned(logits, size_of(dtype)) || misaligned(dlogits, size_of(dtype)) ||
        misaligned(topk_idx, 4) || misaligned(seq_offsets, 4) || misaligned(lse, 4) ||
        misaligned(counts, 4) || misaligned(tokens, 4) || misaligned(dloss, 4) ||
        misaligned(topk_w, 4) || misaligned(dtopk_w, 4))
        return record_failure(MOE_ERR_INVALID_ARG, "misaligned pointer");
    if (!(logits == dlogits && ld == ldd) &&
        rows_overlap(logits, ld, n_experts, dlogits, ldd, n_experts, n_tokens, (int)size_of(dtype)))
        return record_failure(MOE_ERR_INVALID_ARG,
                              "dlogits overlaps logits (it may be logits itself)");
    const int dev = current_device();
    int sms = 0;
    if (dev < 0 || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return record_failure(MOE_ERR_CUDA, "no usable current CUDA device");
    const void *all[] = {logits, topk_idx, seq_offsets, mask, lse, counts, tokens, dloss,
                         topk_w, dtopk_w, dlogits};
    for (const void *p : all)
        if (p && !device_pointer_here(p, dev))
            return record_failure(MOE_ERR_INVALID_ARG,
                                  "arguments must be device pointers of the current device");
    BwdArgs a{};
    a.logits = logits;
    a.ld = ld;
    a.idx = topk_idx;
    a.mask = mask;
    a.segs = {seq_offsets, n_segments, n_tokens};
    a.n = n_tokens;
    a.E = n_experts;
    a.k = top_k;
    a.lse = lse;
    a.counts = counts;
    a.tokens = tokens;
    a.dloss = dloss;
    a.w = topk_w;
    a.dw = dtopk_w;
    a.out = dlogits;
    a.ldo = ldd;
    while (2 * a.half_k < top_k)
        a.half_k = std::max(1, 2 * a.half_k);
    a.wide = pairs(logits, ld, n_experts, size_of(dtype)) &&
             pairs(dlogits, ldd, n_experts, size_of(dtype));
    // Four CTAs per SM, two for wide rows.  They run at once where an instance has
    // the registers for it; fp32 rows of 129 to 256 experts (74 registers) run
    // three and of 513 to 1024 (181) one, the rest behind them.
    const long long warps = (n_experts > 256 ? 2LL : 4LL) * sms * kWarps;
    a.per_warp = (int)((n_tokens + warps - 1) / warps);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return launched(dtype == MOE_FP32   ? grad<float>(a, st)
                    : dtype == MOE_FP16 ? grad<__half>(a, st)
                                        : grad<__nv_bfloat16>(a, st));
}
