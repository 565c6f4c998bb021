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
// registers.  The forward sums p over the tokens of a block in registers and
// writes one partial row per (block of tokens, segment); a second kernel adds
// the partial rows in block order, so a result never depends on timing.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>

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

__device__ __forceinline__ float warp_max(float v)
{
#pragma unroll
    for (int d = 16; d > 0; d >>= 1)
        v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, d));
    return v;
}

__device__ __forceinline__ float ldf(const float *p) { return *p; }
__device__ __forceinline__ float ldf(const __half *p) { return __half2float(*p); }
__device__ __forceinline__ float ldf(const __nv_bfloat16 *p) { return __bfloat162float(*p); }
__device__ __forceinline__ void stf(float *p, float v) { *p = v; }
__device__ __forceinline__ void stf(__half *p, float v) { *p = __float2half_rn(v); }
__device__ __forceinline__ void stf(__nv_bfloat16 *p, float v) { *p = __float2bfloat16_rn(v); }

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

// Workspace: [ticket, 256 B][loss parts f64 [S][ceil(E/32)]][z sums f64 [slots]]
// [valid tokens int [slots]][prob sums f32 [slots][E]][counts int [slots][E]]
struct BalanceWs {
    unsigned *ticket;
    double *part;
    double *z;
    int *valid;
    float *prob;
    int *counts;
    size_t bytes;
};

// Tokens of a block: enough blocks for two per SM of the largest parts, and
// at least one token per warp.
int block_tokens(int n)
{
    const int per = (n + 303) / 304;
    return (std::max(per, 1) + kWarps - 1) / kWarps * kWarps;
}

BalanceWs balance_ws(void *base, int n, int E, int S)
{
    const int C = block_tokens(n);
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
    w.part = reinterpret_cast<double *>(take(8 * (size_t)S * ((E + 31) / 32)));
    w.z = reinterpret_cast<double *>(take(8 * slots));
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
    BalanceWs ws;
    float *loss, *prob, *lse;
    int32_t *counts, *tokens;
};

// Per block of C tokens: lse of every token, and per segment that the block
// meets the partial sums at slot (block + segment): both only ever grow along
// the tokens, so a slot belongs to one pair.
template <typename T, int V>
__global__ void __launch_bounds__(kThreads) balance_stats_kernel(FwdArgs a)
{
    extern __shared__ float sm[];       // prob [kWarps][E], then counts int [E]
    __shared__ double zred[kWarps];
    __shared__ int vred[kWarps];
    pdl_enter();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int E = a.E, t_lo = blockIdx.x * a.C, t_hi = min(a.n, t_lo + a.C);
    int *hist = reinterpret_cast<int *>(sm + kWarps * E);
    const T *logits = static_cast<const T *>(a.logits);
    if (blockIdx.x == 0 && threadIdx.x == 0)
        *a.ws.ticket = 0;

    int t = t_lo;       // next token without a segment
    for (int s = a.segs.first_after(t_lo); s < a.segs.S && t < t_hi; s++) {
        const int b = min(max(a.segs.begin(s), t), t_hi), e = min(a.segs.end(s), t_hi);
        for (int i = t + threadIdx.x; i < b; i += kThreads)
            a.lse[i] = 0.f;             // tokens in front of the first segment
        t = max(t, b);
        if (e <= b)
            continue;
        t = e;
        for (int i = threadIdx.x; i < E; i += kThreads)
            hist[i] = 0;
        __syncthreads();
        float psum[V];
#pragma unroll
        for (int i = 0; i < V; i++)
            psum[i] = 0.f;
        float zsum = 0.f;
        int valid = 0;
        for (int tok = b + warp; tok < e; tok += kWarps) {
            if (a.mask && !a.mask[tok]) {
                if (lane == 0)
                    a.lse[tok] = 0.f;
                continue;
            }
            valid++;
            if (lane < a.k) {
                const int id = a.idx[(long long)tok * a.k + lane];
                if (id >= 0 && id < E)
                    atomicAdd(hist + id, 1);
            }
            const T *row = logits + tok * a.ld;
            float l[V];
            float m = -INFINITY;
#pragma unroll
            for (int i = 0; i < V; i++) {
                const int x = i * 32 + lane;
                l[i] = x < E ? ldf(row + x) : -INFINITY;
            }
#pragma unroll
            for (int i = 0; i < V; i++)
                m = fmaxf(m, l[i]);
            m = warp_max(m);
            const float base = m == -INFINITY ? 0.f : m;
            float sum = 0.f;
#pragma unroll
            for (int i = 0; i < V; i++) {
                l[i] = expf(l[i] - base);
                sum += l[i];
            }
            sum = warp_sum(sum);
            // a row of -inf (every expert masked) has no distribution: p = 0
            const float inv = sum == 0.f ? 0.f : 1.0f / sum;
#pragma unroll
            for (int i = 0; i < V; i++)
                psum[i] = fmaf(l[i], inv, psum[i]);
            const float lse = base + logf(sum);
            if (sum != 0.f)
                zsum = fmaf(lse, lse, zsum);
            if (lane == 0)
                a.lse[tok] = lse;
        }
#pragma unroll
        for (int i = 0; i < V; i++)
            if (i * 32 + lane < E)
                sm[warp * E + i * 32 + lane] = psum[i];
        if (lane == 0) {
            zred[warp] = zsum;
            vred[warp] = valid;
        }
        __syncthreads();
        const long long slot = (long long)blockIdx.x + s;
        for (int i = threadIdx.x; i < E; i += kThreads) {
            float p = sm[i];
#pragma unroll
            for (int w = 1; w < kWarps; w++)
                p += sm[w * E + i];
            a.ws.prob[slot * E + i] = p;
            a.ws.counts[slot * E + i] = hist[i];
        }
        if (threadIdx.x == 0) {
            double z = 0;
            int v = 0;
            for (int w = 0; w < kWarps; w++) {
                z += zred[w];
                v += vred[w];
            }
            a.ws.z[slot] = z;
            a.ws.valid[slot] = v;
        }
        __syncthreads();
    }
    for (int i = t + threadIdx.x; i < t_hi; i += kThreads)
        a.lse[i] = 0.f;                 // tokens behind the last segment
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
    __shared__ double dred[W], zred[W];
    __shared__ long long tred[W], lred[W];
    __shared__ int last;
    pdl_enter();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int s = blockIdx.y, e = blockIdx.x * 32 + lane, E = a.E;
    const int b = a.segs.begin(s), end = a.segs.end(s);
    const int b0 = b / a.C, b1 = end > b ? (end - 1) / a.C + 1 : b0;
    float p = 0.f;
    int c = 0, v = 0;
    for (int i = b0 + warp; i < b1; i += W) {
        const long long slot = (long long)i + s;
        if (e < E) {
            p += a.ws.prob[slot * E + e];
            c += a.ws.counts[slot * E + e];
        }
        v += a.ws.valid[slot];
    }
    sp[warp][lane] = p;
    sc[warp][lane] = c;
    if (lane == 0)
        sv[warp] = v;
    __syncthreads();
    if (warp == 0) {
        p = 0.f;
        c = 0;
        v = 0;
        for (int w = 0; w < W; w++) {
            p += sp[w][lane];
            c += sc[w][lane];
            v += sv[w];
        }
        double part = 0;
        if (v > 0)
            part = (double)c * (double)p * ((double)E / ((double)a.k * v * v));
        if (e < E) {
            a.counts[(long long)s * E + e] = c;
            a.prob[(long long)s * E + e] = v > 0 ? p / (float)v : 0.f;
        } else {
            part = 0;
        }
#pragma unroll
        for (int d = 16; d > 0; d >>= 1)
            part += __shfl_xor_sync(0xffffffffu, part, d);
        if (lane == 0) {
            if (blockIdx.x == 0)
                a.tokens[s] = v;
            a.ws.part[(long long)s * gridDim.x + blockIdx.x] = part;
            __threadfence();
            last = atomicAdd(a.ws.ticket, 1u) + 1 == gridDim.x * gridDim.y;
        }
    }
    __syncthreads();
    if (!last)
        return;
    __threadfence();
    double bal = 0, z = 0;
    long long tokens = 0, live = 0;
    for (int i = threadIdx.x; i < (int)(gridDim.x * gridDim.y); i += kFinalThreads)
        bal += __ldcg(a.ws.part + i);
    // the z sums of the slots in use: walk the segments' block ranges
    for (int q = threadIdx.x; q < a.segs.S; q += kFinalThreads) {
        const int v = __ldcg(a.tokens + q);
        tokens += v;
        live += v > 0;
    }
    for (int q = a.segs.S > W ? warp : 0; q < a.segs.S; q += a.segs.S > W ? W : 1) {
        const int qb = a.segs.begin(q), qe = a.segs.end(q);
        if (qe <= qb)
            continue;
        const int i1 = (qe - 1) / a.C + 1;
        // few segments: all threads share each one's blocks; many: a warp each
        for (int i = qb / a.C + (a.segs.S > W ? lane : (int)threadIdx.x); i < i1;
             i += a.segs.S > W ? 32 : kFinalThreads)
            z += a.ws.z[(long long)i + q];
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
        bal += __shfl_xor_sync(0xffffffffu, bal, d);
        z += __shfl_xor_sync(0xffffffffu, z, d);
        tokens += __shfl_xor_sync(0xffffffffu, tokens, d);
        live += __shfl_xor_sync(0xffffffffu, live, d);
    }
    if (lane == 0) {
        dred[warp] = bal;
        zred[warp] = z;
        tred[warp] = tokens;
        lred[warp] = live;
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        bal = z = 0;
        tokens = live = 0;
        for (int w = 0; w < W; w++) {
            bal += dred[w];
            z += zred[w];
            tokens += tred[w];
            live += lred[w];
        }
        a.loss[0] = live ? (float)(bal / (double)live) : 0.f;
        a.loss[1] = tokens ? (float)(z / (double)tokens) : 0.f;
    }
}

struct BwdArgs {
    const void *logits;
    long long ld;
    const int32_t *idx;
    const uint8_t *mask;
    Segs segs;
    int n, E, k, per_warp;
    const float *lse;
    const int32_t *counts, *tokens;
    const float *dloss, *w, *dw;
    void *out;
    long long ldo;
};

// One warp per run of `per_warp` tokens, so that the row f of its segment
// mostly stays in registers.
template <typename T, int V>
__global__ void __launch_bounds__(kThreads) balance_grad_kernel(BwdArgs a)
{
    __shared__ int red_t[kWarps], red_l[kWarps];
    pdl_enter();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, E = a.E;
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
    __syncthreads();
    tokens = live = 0;
    for (int w = 0; w < kWarps; w++) {
        tokens += red_t[w];
        live += red_l[w];
    }
    const float gb = live > 0 ? a.dloss[0] / (float)live : 0.f;
    const float gz = tokens > 0 ? 2.0f * a.dloss[1] / (float)tokens : 0.f;

    const T *logits = static_cast<const T *>(a.logits);
    T *out = static_cast<T *>(a.out);
    const long long t_lo = ((long long)blockIdx.x * kWarps + warp) * a.per_warp;
    const int t_hi = (int)min((long long)a.n, t_lo + a.per_warp);
    if (t_lo >= a.n)
        return;
    int s = a.segs.first_after((int)t_lo), s_end = -1, s_begin = 0;
    float f[V];
    float gs = 0.f;
    for (int tok = (int)t_lo; tok < t_hi; tok++) {
        if (tok >= s_end) {             // the next segment that holds or follows tok
            if (s_end >= 0)
                s = max(s, a.segs.first_after(tok));
            s_begin = s < a.segs.S ? a.segs.begin(s) : a.n;
            s_end = s < a.segs.S ? a.segs.end(s) : a.n;
            const int ts = s < a.segs.S ? a.tokens[s] : 0;
            const float scale = ts > 0 ? (float)E / ((float)a.k * (float)ts) : 0.f;
            gs = ts > 0 ? gb / (float)ts : 0.f;
#pragma unroll
            for (int i = 0; i < V; i++) {
                const int x = i * 32 + lane;
                f[i] = s < a.segs.S && x < E ? (float)a.counts[(long long)s * E + x] * scale : 0.f;
            }
        }
        T *orow = out + tok * a.ldo;
        const bool in = tok >= s_begin && s < a.segs.S && (!a.mask || a.mask[tok]);
        float d[V];
#pragma unroll
        for (int i = 0; i < V; i++)
            d[i] = 0.f;
        if (in) {
            const T *row = logits + tok * a.ld;
            const float lse = a.lse[tok];
            // a row of -inf has no distribution: no gradient through p
            if (lse != -INFINITY) {
                float dot = 0.f;
#pragma unroll
                for (int i = 0; i < V; i++) {
                    const int x = i * 32 + lane;
                    d[i] = x < E ? ldf(row + x) : -INFINITY;
                }
#pragma unroll
                for (int i = 0; i < V; i++) {
                    d[i] = expf(d[i] - lse);
                    dot = fmaf(f[i], d[i], dot);
                }
                dot = warp_sum(dot);
                const float cz = gz * lse;
#pragma unroll
                for (int i = 0; i < V; i++)
                    d[i] *= fmaf(gs, f[i] - dot, cz);
            }
            if (a.dw) {
                const long long at = (long long)tok * a.k + lane;
                const float w = lane < a.k ? a.w[at] : 0.f, dw = lane < a.k ? a.dw[at] : 0.f;
                const int id = lane < a.k ? a.idx[at] : -1;
                const float dot = warp_sum(w * dw);
                const float v = w * (dw - dot);
                for (int j = 0; j < a.k; j++) {
                    const int e = __shfl_sync(0xffffffffu, id, j);
                    const float add = __shfl_sync(0xffffffffu, v, j);
                    const int at_i = e >= 0 && (e & 31) == lane ? e >> 5 : -1;
#pragma unroll
                    for (int i = 0; i < V; i++)
                        if (at_i == i)
                            d[i] += add;
                }
            }
        }
#pragma unroll
        for (int i = 0; i < V; i++) {
            const int x = i * 32 + lane;
            if (x < E)
                stf(orow + x, d[i]);
        }
    }
}

template <typename T, int V>
cudaError_t launch_stats(const FwdArgs &a, cudaStream_t st)
{
    const size_t smem = sizeof(float) * (kWarps + 1) * a.E;
    return launch_pdl(balance_stats_kernel<T, V>, dim3((a.n + a.C - 1) / a.C), dim3(kThreads),
                      smem, st, a);
}

template <typename T, int V>
cudaError_t launch_grad(const BwdArgs &a, cudaStream_t st)
{
    const long long warps = (a.n + a.per_warp - 1) / a.per_warp;
    return launch_pdl(balance_grad_kernel<T, V>, dim3((unsigned)((warps + kWarps - 1) / kWarps)),
                      dim3(kThreads), 0, st, a);
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

}  // namespace

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
    a.C = block_tokens(n_tokens);
    a.loss = loss;
    a.counts = counts;
    a.tokens = tokens;
    a.prob = prob;
    a.lse = lse;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaError_t e = dtype == MOE_FP32   ? stats<float>(a, st)
                    : dtype == MOE_FP16 ? stats<__half>(a, st)
                                        : stats<__nv_bfloat16>(a, st);
    if (e == cudaSuccess)
        e = launch_pdl(balance_final_kernel, dim3((n_experts + 31) / 32, n_segments),
                       dim3(kFinalThreads), 0, st, a);
    return launched(e);
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
    {
        const char *p = static_cast<const char *>(logits), *q = static_cast<const char *>(dlogits);
        const long long np = (long long)size_of(dtype) * ((n_tokens - 1) * ld + n_experts);
        const long long nq = (long long)size_of(dtype) * ((n_tokens - 1) * ldd + n_experts);
        if (!(p == q && ld == ldd) && p < q + nq && q < p + np)
            return record_failure(MOE_ERR_INVALID_ARG,
                                  "dlogits overlaps logits (it may be logits itself)");
    }
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
    a.per_warp = (int)std::max(1LL, (long long)n_tokens / ((long long)sms * 6 * kWarps));
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return launched(dtype == MOE_FP32   ? grad<float>(a, st)
                    : dtype == MOE_FP16 ? grad<__half>(a, st)
                                        : grad<__nv_bfloat16>(a, st));
}
