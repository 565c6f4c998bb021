// The norm behind a block, its gate, the scaled residual stream and the norm in
// front of the next block, in one pass over a row, and their gradients.
//   r1 = 1 / sqrt(mean(y^2) + eps), v = gain * y * r1     (without gain: r1 = 1, v = y)
//   out = c * resid + gate * v
//   r2 = 1 / sqrt(mean(out^2) + eps), xn = next_gain * out * r2
// Backward, with the gradients dout and dxn that arrive at out and xn:
//   dn = dxn * next_gain, n = out * r2, do = dout + r2 (dn - n mean(dn n))
//   dresid = c * do,  dnext_gain = sum_t dxn n
//   q = do * gate * gain, z = y * r1,  dy = r1 (q - z mean(q z))   (without gain: do * gate)
//   dgain = sum_t do gate z,  dgate = do . v over the row (a gate for each token) or
//   sum_t do v (a gate for each channel): all from the one column sum of do gate z,
//   and, for a gate for each token, from the one row sum that dy needs.
//
// Bound by HBM: four arrays of n x H are read or written forward, six backward.
// A CTA holds a row in registers, two reductions a row, and goes through rows with
// the vectors that all rows share in registers; the column sums stay there too, and
// leave as one partial row per kRun rows and CTA, added by a second kernel in a
// fixed order.
#include <algorithm>

#include "args.cuh"
#include "vec.cuh"

namespace qe {

namespace {

constexpr int kMaxTokens = 1 << 26, kMaxWidth = 16384;
constexpr int kMaxThreads = 512, kMaxWarps = kMaxThreads / 32;
// Rows whose column sums are one fp32 chain.
constexpr int kRun = 256;

struct NormArgs {
    const void *resid, *y, *gain, *gate, *next_gain;
    long long ld_resid, ld_y, ld_out, ld_xn;
    int n, H, vecs;
    float scale, eps, inv_h;
    bool token_gate;
    void *out, *xn;
    float2 *stats;
};

// Sum over the block in a fixed order; `part` is one of two buffers used in turn.
__device__ __forceinline__ float sum_block(float v, float *part, int warps)
{
    v = sum_warp(v);
    if (warps == 1)
        return v;
    if ((threadIdx.x & 31) == 0)
        part[threadIdx.x >> 5] = v;
    __syncthreads();
    float s = 0.f;
    for (int w = 0; w < warps; w++)
        s += part[w];
    return s;
}

template <typename T>
__device__ __forceinline__ uint4 ones()
{
    const float d[8] = {1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f};
    return pack<T>(d);
}

template <typename T, int V>
__device__ __forceinline__ void load_row(uint4 (&q)[V], const void *base, long long at, int vecs)
{
    const T *row = static_cast<const T *>(base) + at;
#pragma unroll
    for (int i = 0; i < V; i++) {
        const int v = threadIdx.x + i * blockDim.x;
        q[i] = v < vecs ? load_stream(row + 8 * v) : make_uint4(0, 0, 0, 0);
    }
}

// The vector that all rows share, 1 where there is none.
template <typename T, int V>
__device__ __forceinline__ void load_shared(uint4 (&q)[V], const void *base, int vecs)
{
#pragma unroll
    for (int i = 0; i < V; i++) {
        const int v = threadIdx.x + i * blockDim.x;
        q[i] = base && v < vecs ? *(reinterpret_cast<const uint4 *>(base) + v) : ones<T>();
    }
}

template <typename T, int V>
__global__ void __launch_bounds__(kMaxThreads, 1) residual_norm_kernel(NormArgs a)
{
    constexpr bool kAhead = V <= 2;     // the next row's loads under way
    __shared__ float part[2][kMaxWarps];
    pdl_enter();
    const int warps = blockDim.x / 32;
    uint4 gain[V], gate[V], next_gain[V], rq[V], yq[V];
    load_shared<T, V>(gain, a.gain, a.vecs);
    load_shared<T, V>(gate, a.token_gate ? nullptr : a.gate, a.vecs);
    load_shared<T, V>(next_gain, a.next_gain, a.vecs);
    const T *token_gate = a.token_gate ? static_cast<const T *>(a.gate) : nullptr;
    const auto load = [&](long long t) {
        load_row<T, V>(rq, a.resid, t * a.ld_resid, a.vecs);
        load_row<T, V>(yq, a.y, t * a.ld_y, a.vecs);
    };
    long long t = blockIdx.x;
    if (t < a.n)
        load(t);
    for (; t < a.n; t += gridDim.x) {
        float o[V][8], r[V][8];
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < V; i++) {
            unpack<T>(yq[i], o[i]);
            unpack<T>(rq[i], r[i]);
#pragma unroll
            for (int e = 0; e < 8; e++)
                ss = fmaf(o[i][e], o[i][e], ss);
        }
        const float tg = token_gate ? to_float<T>(token_gate[t]) : 1.f;
        if (kAhead && t + gridDim.x < a.n)
            load(t + gridDim.x);
        float r1 = 1.f, r2 = 1.f;
        if (a.gain)
            r1 = __frsqrt_rn(fmaf(sum_block(ss, part[0], warps), a.inv_h, a.eps));
        const float f = r1 * tg;
        ss = 0.f;
#pragma unroll
        for (int i = 0; i < V; i++) {
            float g[8], c[8];
            unpack<T>(gain[i], g);
            unpack<T>(gate[i], c);
#pragma unroll
            for (int e = 0; e < 8; e++) {
                o[i][e] = fmaf(a.scale, r[i][e], o[i][e] * f * (g[e] * c[e]));
                ss = fmaf(o[i][e], o[i][e], ss);
            }
            const int v = threadIdx.x + i * blockDim.x;
            if (v < a.vecs)
                *reinterpret_cast<uint4 *>(static_cast<T *>(a.out) + t * a.ld_out + 8 * v) =
                    pack<T>(o[i]);
        }
        if (a.xn) {
            r2 = __frsqrt_rn(fmaf(sum_block(ss, part[1], warps), a.inv_h, a.eps));
#pragma unroll
            for (int i = 0; i < V; i++) {
                float g[8];
                unpack<T>(next_gain[i], g);
#pragma unroll
                for (int e = 0; e < 8; e++)
                    g[e] *= o[i][e] * r2;
                const int v = threadIdx.x + i * blockDim.x;
                if (v < a.vecs)
                    *reinterpret_cast<uint4 *>(static_cast<T *>(a.xn) + t * a.ld_xn + 8 * v) =
                        pack<T>(g);
            }
        }
        if (threadIdx.x == 0)
            a.stats[t] = make_float2(r1, r2);
        if (!kAhead && t + gridDim.x < a.n)
            load(t + gridDim.x);
        // a row with one reduction alone writes the buffer that it reads next time
        if (warps > 1 && !(a.gain && a.xn))
            __syncthreads();
    }
}

struct NormGradArgs {
    const void *dout, *dxn, *out, *y, *gain, *gate, *next_gain;
    long long ld_dout, ld_dxn, ld_out, ld_y, ld_dresid, ld_dy;
    const float2 *stats;
    int n, H, vecs;
    float scale, inv_h;
    bool token_gate, sums;
    int runs;               // partial rows of a CTA
    void *dresid, *dy;
    float *dgate;           // token gates
    float *part;            // [2][slots][H] column sums of do gate z and of dxn n
    float *dgain, *dgate_ch, *dnext_gain;
};

// Column sums of V = 4 lie in shared memory: registers hold no more than two words.
template <typename T, int V>
__global__ void __launch_bounds__(kMaxThreads, 1) residual_norm_grad_kernel(NormGradArgs a)
{
    constexpr bool kAhead = V <= 2;
    extern __shared__ float4 sums_sm[];     // V = 4: [2][V][2][threads]
    __shared__ float part[2][kMaxWarps];
    pdl_enter();
    const int warps = blockDim.x / 32;
    uint4 gain[V], gate[V], next_gain[V];
    load_shared<T, V>(gain, a.gain, a.vecs);
    load_shared<T, V>(gate, a.token_gate ? nullptr : a.gate, a.vecs);
    load_shared<T, V>(next_gain, a.next_gain, a.vecs);
    const T *token_gate = a.token_gate ? static_cast<const T *>(a.gate) : nullptr;
    uint4 dq[V], nq[V], oq[V], yq[V];
#pragma unroll
    for (int i = 0; i < V; i++)
        dq[i] = nq[i] = oq[i] = make_uint4(0, 0, 0, 0);
    const auto load = [&](long long t) {
        if (a.dout)
            load_row<T, V>(dq, a.dout, t * a.ld_dout, a.vecs);
        if (a.dxn) {
            load_row<T, V>(nq, a.dxn, t * a.ld_dxn, a.vecs);
            load_row<T, V>(oq, a.out, t * a.ld_out, a.vecs);
        }
        load_row<T, V>(yq, a.y, t * a.ld_y, a.vecs);
    };
    constexpr int R = V <= 2 ? V : 1;
    float s1[R][8], s2[R][8];       // V <= 2: the column sums
    const auto clear = [&]() {
#pragma unroll
        for (int i = 0; i < V; i++)
            if constexpr (V <= 2) {
#pragma unroll
                for (int e = 0; e < 8; e++)
                    s1[i][e] = s2[i][e] = 0.f;
            } else if (a.sums) {
#pragma unroll
                for (int j = 0; j < 4; j++)
                    sums_sm[(4 * i + j) * blockDim.x + threadIdx.x] = make_float4(0.f, 0.f, 0.f, 0.f);
            }
    };
    clear();
    const auto flush = [&](int run) {
        float *p = a.part + ((long long)blockIdx.x * a.runs + run) * a.H;
        float *q = p + (long long)gridDim.x * a.runs * a.H;
#pragma unroll
        for (int i = 0; i < V; i++) {
            const int v = threadIdx.x + i * blockDim.x;
            if (v >= a.vecs)
                continue;
            float4 w[4];
#pragma unroll
            for (int j = 0; j < 4; j++)
                if constexpr (V <= 2) {
                    const float *s = j < 2 ? s1[i] + 4 * j : s2[i] + 4 * (j - 2);
                    w[j] = make_float4(s[0], s[1], s[2], s[3]);
                } else {
                    w[j] = sums_sm[(4 * i + j) * blockDim.x + threadIdx.x];
                }
            *reinterpret_cast<float4 *>(p + 8 * v) = w[0];
            *reinterpret_cast<float4 *>(p + 8 * v + 4) = w[1];
            *reinterpret_cast<float4 *>(q + 8 * v) = w[2];
            *reinterpret_cast<float4 *>(q + 8 * v + 4) = w[3];
        }
        clear();
    };
    long long t = blockIdx.x;
    if (t < a.n)
        load(t);
    int rows = 0, run = 0;
    for (; t < a.n; t += gridDim.x) {
        const float2 st = a.stats[t];
        const float tg = token_gate ? to_float<T>(token_gate[t]) : 1.f;
        float d[V][8], z[V][8], n[V][8];
        float m = 0.f;
#pragma unroll
        for (int i = 0; i < V; i++) {
            float g[8];
            unpack<T>(dq[i], d[i]);
            unpack<T>(oq[i], n[i]);
            unpack<T>(yq[i], z[i]);
            unpack<T>(next_gain[i], g);
            float x[8];
            unpack<T>(nq[i], x);
            float c[8];
#pragma unroll
            for (int e = 0; e < 8; e++) {
                n[i][e] *= st.y;
                z[i][e] *= st.x;
                c[e] = x[e] * n[i][e];
                m = fmaf(c[e], g[e], m);
                // do without its mean's part
                d[i][e] = fmaf(st.y, x[e] * g[e], d[i][e]);
            }
            if constexpr (V <= 2) {
#pragma unroll
                for (int e = 0; e < 8; e++)
                    s2[i][e] += c[e];
            } else if (a.sums) {
#pragma unroll
                for (int j = 0; j < 2; j++) {
                    float4 &s = sums_sm[(4 * i + 2 + j) * blockDim.x + threadIdx.x];
                    s = make_float4(s.x + c[4 * j], s.y + c[4 * j + 1], s.z + c[4 * j + 2],
                                    s.w + c[4 * j + 3]);
                }
            }
        }
        if (kAhead && t + gridDim.x < a.n)
            load(t + gridDim.x);
        const float mean = a.dxn ? sum_block(m, part[0], warps) * a.inv_h * st.y : 0.f;
        m = 0.f;
#pragma unroll
        for (int i = 0; i < V; i++) {
            float g[8], c[8], w[8];
            unpack<T>(gain[i], g);
            unpack<T>(gate[i], c);
#pragma unroll
            for (int e = 0; e < 8; e++) {
                d[i][e] = fmaf(-n[i][e], mean, d[i][e]);
                w[e] = d[i][e] * z[i][e];
                m = fmaf(w[e], g[e] * c[e], m);
                w[e] *= tg;
            }
            if constexpr (V <= 2) {
#pragma unroll
                for (int e = 0; e < 8; e++)
                    s1[i][e] += w[e];
            } else if (a.sums) {
#pragma unroll
                for (int j = 0; j < 2; j++) {
                    float4 &s = sums_sm[(4 * i + j) * blockDim.x + threadIdx.x];
                    s = make_float4(s.x + w[4 * j], s.y + w[4 * j + 1], s.z + w[4 * j + 2],
                                    s.w + w[4 * j + 3]);
                }
            }
#pragma unroll
            for (int e = 0; e < 8; e++)
                w[e] = a.scale * d[i][e];
            const int v = threadIdx.x + i * blockDim.x;
            if (v < a.vecs)
                *reinterpret_cast<uint4 *>(static_cast<T *>(a.dresid) + t * a.ld_dresid + 8 * v) =
                    pack<T>(w);
        }
        // sum of do gain gate z, the gate of a token left out
        const float dot = sum_block(m, part[1], warps);
        const float back = a.gain ? dot * tg * a.inv_h : 0.f, f = a.gain ? st.x : 1.f;
#pragma unroll
        for (int i = 0; i < V; i++) {
            float g[8], c[8];
            unpack<T>(gain[i], g);
            unpack<T>(gate[i], c);
#pragma unroll
            for (int e = 0; e < 8; e++)
                g[e] = f * fmaf(-z[i][e], back, d[i][e] * tg * (g[e] * c[e]));
            const int v = threadIdx.x + i * blockDim.x;
            if (v < a.vecs)
                *reinterpret_cast<uint4 *>(static_cast<T *>(a.dy) + t * a.ld_dy + 8 * v) =
                    pack<T>(g);
        }
        if (token_gate && a.dgate && threadIdx.x == 0)
            a.dgate[t] = dot;
        if (a.sums && ++rows == kRun) {
            flush(run++);
            rows = 0;
        }
        if (!kAhead && t + gridDim.x < a.n)
            load(t + gridDim.x);
        if (warps > 1 && !a.dxn)
            __syncthreads();        // one buffer alone is in use
    }
    // runs that this CTA has no rows for are zeros
    if (a.sums)
        for (; run < a.runs; run++)
            flush(run);
}

// Column sums over the partial rows: 32 columns a CTA, 32 chains each.
template <typename T>
__global__ void __launch_bounds__(1024) residual_norm_sums_kernel(NormGradArgs a, int slots)
{
    __shared__ float sm[32][33];
    pdl_enter();
    const int c = threadIdx.x & 31, j = threadIdx.x >> 5, h = blockIdx.x * 32 + c;
    const bool next = blockIdx.y != 0;
    const float *p = a.part + (next ? (long long)slots * a.H : 0) + h;
    float s = 0.f, err = 0.f;
    if (h < a.H)
        for (int i = j; i < slots; i += 32) {
            // two-sum: the chain's length costs nothing
            const float v = p[(long long)i * a.H], x = __fadd_rn(s, v), b = __fsub_rn(x, s);
            err += __fadd_rn(__fsub_rn(s, __fsub_rn(x, b)), __fsub_rn(v, b));
            s = x;
        }
    sm[j][c] = err == err ? s + err : s;
    __syncthreads();
    s = sum_warp(sm[c][j]);
    const int col = blockIdx.x * 32 + j;
    if (c != 0 || col >= a.H)
        return;
    if (next) {
        if (a.dnext_gain)
            a.dnext_gain[col] = s;
        return;
    }
    const T *gate = a.token_gate ? nullptr : static_cast<const T *>(a.gate);
    if (a.dgain)
        a.dgain[col] = gate ? s * to_float<T>(gate[col]) : s;
    if (a.dgate_ch)
        a.dgate_ch[col] = a.gain ? s * to_float<T>(static_cast<const T *>(a.gain)[col]) : s;
}

// Threads of a row: two words each, four for the widest.
int row_words(int H) { return H > 16 * kMaxThreads ? 4 : 2; }
int row_threads(int H)
{
    const int per = 8 * row_words(H);
    return ((H + per - 1) / per + 31) / 32 * 32;
}

// CTAs of the gradient: as many as run at once on 152 SMs with 128 registers a
// thread.  The workspace's size follows from it, so it asks no device.
int grad_blocks(int n, int H) { return std::min(n, 152 * std::max(1, 512 / row_threads(H))); }
int grad_runs(int n, int H)
{
    const int rows = (n + grad_blocks(n, H) - 1) / grad_blocks(n, H);
    return (rows + kRun - 1) / kRun;
}
size_t grad_ws(int n, int H)
{
    return 2 * sizeof(float) * (size_t)grad_blocks(n, H) * grad_runs(n, H) * H;
}

template <typename T>
cudaError_t launch_norm(const NormArgs &a, int sms, cudaStream_t st)
{
    const int threads = row_threads(a.H);
    const dim3 grid(std::min(a.n, sms * std::max(1, 1024 / threads)));
    return row_words(a.H) == 2
               ? launch_pdl(residual_norm_kernel<T, 2>, grid, dim3(threads), 0, st, a)
               : launch_pdl(residual_norm_kernel<T, 4>, grid, dim3(threads), 0, st, a);
}

template <typename T>
cudaError_t launch_norm_grad(const NormGradArgs &a, cudaStream_t st)
{
    const int threads = row_threads(a.H);
    const dim3 grid(grad_blocks(a.n, a.H));
    cudaError_t e = cudaSuccess;
    if (row_words(a.H) == 2) {
        e = launch_pdl(residual_norm_grad_kernel<T, 2>, grid, dim3(threads), 0, st, a);
    } else {
        const size_t smem = a.sums ? sizeof(float4) * 16 * threads : 0;
        e = cudaFuncSetAttribute(residual_norm_grad_kernel<T, 4>,
                                 cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (int)sizeof(float4) * 16 * kMaxThreads);
        if (e == cudaSuccess)
            e = launch_pdl(residual_norm_grad_kernel<T, 4>, grid, dim3(threads), smem, st, a);
    }
    if (e == cudaSuccess && a.sums)
        e = launch_pdl(residual_norm_sums_kernel<T>, dim3((a.H + 31) / 32, a.dnext_gain ? 2 : 1),
                       dim3(1024), 0, st, a, (int)grid.x * a.runs);
    return e;
}

int check_sizes(int dtype, int n, int H)
{
    if (dtype != MOE_FP16 && dtype != MOE_BF16)
        return record_failure(MOE_ERR_UNSUPPORTED, "dtype must be MOE_FP16 or MOE_BF16");
    if (n < 1 || n > kMaxTokens)
        return record_failure(MOE_ERR_INVALID_ARG, "n_tokens must be in 1..67108864");
    if (H < 8 || H > kMaxWidth || H % 8)
        return record_failure(MOE_ERR_INVALID_ARG, "hidden must be a multiple of 8 in 8..16384");
    return MOE_OK;
}

}  // namespace

}  // namespace qe

extern "C" int moe_residual_norm(const void *resid, long long ld_resid, const void *y,
                                 long long ld_y, int dtype, int n_tokens, int hidden,
                                 const void *gain, const void *gate, int gate_per_token,
                                 float scale, const void *next_gain, float eps, void *out,
                                 long long ld_out, void *xn, long long ld_xn, float *stats,
                                 void *stream)
{
    using namespace qe;
    const int rc = check_sizes(dtype, n_tokens, hidden);
    if (rc)
        return rc;
    if (!resid || !y || !out || !stats || (xn && !next_gain))
        return record_failure(MOE_ERR_INVALID_ARG, "null pointer argument");
    if (!(eps >= 0.f) || eps > 3.4028235e38f || !(scale - scale == 0.f))
        return record_failure(MOE_ERR_INVALID_ARG, "eps must be finite and >= 0, scale finite");
    const size_t n = n_tokens, H = hidden;
    const Arg wide[] = {rows_arg(gain, 0, hidden, 1, 2, 16),
                        rows_arg(gate_per_token ? nullptr : gate, 0, hidden, 1, 2, 16),
                        rows_arg(xn ? next_gain : nullptr, 0, hidden, 1, 2, 16)};
    const Arg args[] = {wide[0], wide[1], wide[2],
                        flat_arg(gate_per_token ? gate : nullptr, n, 2),
                        rows_arg(resid, ld_resid, hidden, n_tokens, 2, 16),
                        rows_arg(y, ld_y, hidden, n_tokens, 2, 16),
                        rows_arg(out, ld_out, hidden, n_tokens, 2, 16, true, resid),
                        rows_arg(xn, ld_xn, hidden, n_tokens, 2, 16, true),
                        flat_arg(stats, n, 8, true)};
    int dev, sms;
    if (const int bad = check_args(args, sizeof(args) / sizeof(args[0]), &dev, &sms))
        return bad;
    NormArgs a{};
    a.resid = resid;
    a.y = y;
    a.gain = gain;
    a.gate = gate;
    a.next_gain = xn ? next_gain : nullptr;
    a.ld_resid = ld_resid;
    a.ld_y = ld_y;
    a.ld_out = ld_out;
    a.ld_xn = ld_xn;
    a.n = n_tokens;
    a.H = hidden;
    a.vecs = hidden / 8;
    a.scale = scale;
    a.eps = eps;
    a.inv_h = 1.f / (float)H;
    a.token_gate = gate && gate_per_token;
    a.out = out;
    a.xn = xn;
    a.stats = reinterpret_cast<float2 *>(stats);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return launch_result(dtype == MOE_FP16 ? launch_norm<__half>(a, sms, st)
                                           : launch_norm<__nv_bfloat16>(a, sms, st));
}

extern "C" size_t moe_residual_norm_grad_workspace(int n_tokens, int hidden)
{
    using namespace qe;
    if (n_tokens < 1 || n_tokens > kMaxTokens || hidden < 8 || hidden > kMaxWidth || hidden % 8)
        return 0;
    return grad_ws(n_tokens, hidden);
}

extern "C" int moe_residual_norm_grad(const void *dout, long long ld_dout, const void *dxn,
                                      long long ld_dxn, const void *out, long long ld_out,
                                      const void *y, long long ld_y, const float *stats, int dtype,
                                      int n_tokens, int hidden, const void *gain, const void *gate,
                                      int gate_per_token, float scale, const void *next_gain,
                                      void *dresid, long long ld_dresid, void *dy, long long ld_dy,
                                      float *dgain, float *dgate, float *dnext_gain,
                                      void *workspace, size_t workspace_bytes, void *stream)
{
    using namespace qe;
    const int rc = check_sizes(dtype, n_tokens, hidden);
    if (rc)
        return rc;
    if (!y || !stats || !dresid || !dy || (dxn && (!out || !next_gain)))
        return record_failure(MOE_ERR_INVALID_ARG, "null pointer argument");
    if (!dout && !dxn)
        return record_failure(MOE_ERR_INVALID_ARG, "need dout or dxn");
    if ((dgain && !gain) || (dgate && !gate) || (dnext_gain && !dxn))
        return record_failure(MOE_ERR_INVALID_ARG,
                              "dgain needs gain, dgate needs gate, dnext_gain needs dxn");
    if (!(scale - scale == 0.f))
        return record_failure(MOE_ERR_INVALID_ARG, "scale must be finite");
    const size_t n = n_tokens, H = hidden;
    const bool sums = dgain || dnext_gain || (dgate && !gate_per_token);
    const size_t need = sums ? grad_ws(n_tokens, hidden) : 0;
    if (need && (!workspace || workspace_bytes < need))
        return record_failure(MOE_ERR_INVALID_ARG,
                              "workspace below moe_residual_norm_grad_workspace(n, hidden)");
    const Arg args[] = {rows_arg(gain, 0, hidden, 1, 2, 16),
                        rows_arg(gate_per_token ? nullptr : gate, 0, hidden, 1, 2, 16),
                        flat_arg(gate_per_token ? gate : nullptr, n, 2),
                        rows_arg(dxn ? next_gain : nullptr, 0, hidden, 1, 2, 16),
                        rows_arg(dout, ld_dout, hidden, n_tokens, 2, 16),
                        rows_arg(dxn, ld_dxn, hidden, n_tokens, 2, 16),
                        rows_arg(dxn ? out : nullptr, ld_out, hidden, n_tokens, 2, 16),
                        rows_arg(y, ld_y, hidden, n_tokens, 2, 16),
                        flat_arg(stats, n, 8),
                        rows_arg(dresid, ld_dresid, hidden, n_tokens, 2, 16, true, dout),
                        rows_arg(dy, ld_dy, hidden, n_tokens, 2, 16, true),
                        flat_arg(dgain, H, 4, true),
                        flat_arg(dgate, gate_per_token ? n : H, 4, true),
                        flat_arg(dnext_gain, H, 4, true),
                        rows_arg(need ? workspace : nullptr, 0, need / 4, 1, 4, 16, true)};
    int dev, sms;
    if (const int bad = check_args(args, sizeof(args) / sizeof(args[0]), &dev, &sms))
        return bad;
    NormGradArgs a{};
    a.dout = dout;
    a.dxn = dxn;
    a.out = out;
    a.y = y;
    a.gain = gain;
    a.gate = gate;
    a.next_gain = dxn ? next_gain : nullptr;
    a.ld_dout = ld_dout;
    a.ld_dxn = ld_dxn;
    a.ld_out = ld_out;
    a.ld_y = ld_y;
    a.ld_dresid = ld_dresid;
    a.ld_dy = ld_dy;
    a.stats = reinterpret_cast<const float2 *>(stats);
    a.n = n_tokens;
    a.H = hidden;
    a.vecs = hidden / 8;
    a.scale = scale;
    a.inv_h = 1.f / (float)H;
    a.token_gate = gate && gate_per_token;
    a.sums = sums;
    a.runs = grad_runs(n_tokens, hidden);
    a.dresid = dresid;
    a.dy = dy;
    a.dgate = a.token_gate ? dgate : nullptr;
    a.dgate_ch = a.token_gate ? nullptr : dgate;
    a.part = static_cast<float *>(workspace);
    a.dgain = dgain;
    a.dnext_gain = dnext_gain;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return launch_result(dtype == MOE_FP16 ? launch_norm_grad<__half>(a, st)
                                           : launch_norm_grad<__nv_bfloat16>(a, st));
}
