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
// A CTA goes through rows, one in registers and the next one's loads under way, two
// reductions a row.  The vectors that all rows share lie in shared memory as fp32, each
// thread's part by itself (no barriers).  The column sums stay in registers and leave as
// one partial row per kRun rows and CTA, added by a second kernel in a fixed order.
// Measured: 16001 x 4096 bf16 with a gate per token 84 us (92% of the measured copy rate),
// its gradients for 16384 x 4096 139 us (86%, half of the issue slots used); 4000 x 16384
// 82 and 163 us (94% and 71%).  More than 8192 columns of the gradient take a cluster of two
// CTAs.  One CTA of four words a thread, its sums in shared memory and no row ahead: 269 us.
// Every thread adding all warps' sums: 97 and 184 us; and with a cluster's barrier in place
// of the counted stores, which waits for dresid's stores too, 240 us; four CTAs of 256
// threads: 310 us.
#include <algorithm>

#include "args.cuh"
#include "vec.cuh"
#include "w4.cuh"

namespace qe {

namespace {

constexpr int kMaxTokens = 1 << 26, kMaxWidth = 16384;
constexpr int kMaxThreads = 512, kMaxWarps = 1024 / 32;
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
__device__ __forceinline__ float sum_block(float v, float4 *part, int warps)
{
    v = sum_warp(v);
    if (warps == 1)
        return v;
    if ((threadIdx.x & 31) == 0)
        reinterpret_cast<float *>(part)[threadIdx.x >> 5] = v;
    __syncthreads();
    if (warps > 8) {        // a lane for each: fewer instructions, a longer chain
        const int lane = threadIdx.x & 31;
        return sum_warp(lane < warps ? reinterpret_cast<const float *>(part)[lane] : 0.f);
    }
    float s = 0.f;
    for (int w = 0; w < warps; w += 4) {
        const float4 q = part[w / 4];
        s += (q.x + (w + 1 < warps ? q.y : 0.f)) +
             ((w + 2 < warps ? q.z : 0.f) + (w + 3 < warps ? q.w : 0.f));
    }
    return s;
}

template <int V>
__device__ __forceinline__ void load_row(uint4 (&q)[V], const void *base, long long at, int vecs)
{
    const uint16_t *row = static_cast<const uint16_t *>(base) + at;
#pragma unroll
    for (int i = 0; i < V; i++) {
        const int v = threadIdx.x + i * blockDim.x;
        if (v < vecs)
            q[i] = load_stream(row + 8 * v);
    }
}

// A vector that all rows share, as fp32 in shared memory: word 2 i + j of a thread holds
// four of its values.  `by` multiplies it; 1 where there is none.
struct Shared {
    float4 *mine;

    __device__ __forceinline__ void put(int word, const float *d)
    {
        mine[word * blockDim.x] = make_float4(d[0], d[1], d[2], d[3]);
    }
    template <typename T, int V>
    __device__ __forceinline__ void load(const void *base, const void *by, int vecs)
    {
#pragma unroll
        for (int i = 0; i < V; i++) {
            const int v = threadIdx.x + i * blockDim.x;
            float d[8], f[8];
#pragma unroll
            for (int e = 0; e < 8; e++)
                d[e] = f[e] = 1.f;
            if (base && v < vecs)
                unpack<T>(*(static_cast<const uint4 *>(base) + v), d);
            if (by && v < vecs)
                unpack<T>(*(static_cast<const uint4 *>(by) + v), f);
#pragma unroll
            for (int e = 0; e < 8; e++)
                d[e] *= f[e];
            put(2 * i, d);
            put(2 * i + 1, d + 4);
        }
    }
    // the eight values of the thread's word i, in pairs
    __device__ __forceinline__ void get(int i, F2 (&d)[4]) const
    {
        const ulonglong2 a = *reinterpret_cast<const ulonglong2 *>(mine + 2 * i * blockDim.x);
        const ulonglong2 b = *reinterpret_cast<const ulonglong2 *>(mine + (2 * i + 1) * blockDim.x);
        d[0].v = a.x, d[1].v = a.y, d[2].v = b.x, d[3].v = b.y;
    }
};

// Two words of a row for each of at most MAX threads.
template <typename T, int MAX>
__global__ void __launch_bounds__(MAX, 1024 / MAX) residual_norm_kernel(NormArgs a)
{
    constexpr int V = 2;
    extern __shared__ float4 shared[];  // [2][2 V][threads]
    __shared__ float4 part[2][kMaxWarps / 4];
    pdl_enter();
    const int warps = blockDim.x / 32;
    Shared weight{shared + threadIdx.x}, next_gain{shared + 2 * V * blockDim.x + threadIdx.x};
    uint4 rq[V], yq[V];
#pragma unroll
    for (int i = 0; i < V; i++)
        rq[i] = yq[i] = make_uint4(0, 0, 0, 0);
    const auto load = [&](long long t) {
        load_row<V>(rq, a.resid, t * a.ld_resid, a.vecs);
        load_row<V>(yq, a.y, t * a.ld_y, a.vecs);
    };
    long long t = blockIdx.x;
    load(t);
    weight.load<T, V>(a.gain, a.token_gate ? nullptr : a.gate, a.vecs);
    next_gain.load<T, V>(a.next_gain, nullptr, a.vecs);
    const T *token_gate = a.token_gate ? static_cast<const T *>(a.gate) : nullptr;
    const F2 scale = f2(a.scale);
    for (; t < a.n; t += gridDim.x) {
        const float tg = token_gate ? to_float<T>(token_gate[t]) : 1.f;
        F2 o[V][4], r[V][4];
        F2 ss = f2(0.f);
#pragma unroll
        for (int i = 0; i < V; i++) {
            unpack<T>(yq[i], o[i]);
            unpack<T>(rq[i], r[i]);
#pragma unroll
            for (int e = 0; e < 4; e++) {
                ss = fma(o[i][e], o[i][e], ss);
                r[i][e] = mul(r[i][e], scale);
            }
        }
        if (t + gridDim.x < a.n)        // the next row's loads are under way
            load(t + gridDim.x);
        float r1 = 1.f, r2 = 1.f;
        if (a.gain)
            r1 = __frsqrt_rn(fmaf(sum_block(sum(ss), part[0], warps), a.inv_h, a.eps));
        const F2 f = f2(r1 * tg);
        ss = f2(0.f);
#pragma unroll
        for (int i = 0; i < V; i++) {
            F2 w[4];
            weight.get(i, w);
#pragma unroll
            for (int e = 0; e < 4; e++) {
                o[i][e] = fma(mul(o[i][e], f), w[e], r[i][e]);
                ss = fma(o[i][e], o[i][e], ss);
            }
            const int v = threadIdx.x + i * blockDim.x;
            if (v < a.vecs)
                *reinterpret_cast<uint4 *>(static_cast<T *>(a.out) + t * a.ld_out + 8 * v) =
                    pack<T>(o[i]);
        }
        if (a.xn) {
            r2 = __frsqrt_rn(fmaf(sum_block(sum(ss), part[1], warps), a.inv_h, a.eps));
            const F2 f2nd = f2(r2);
#pragma unroll
            for (int i = 0; i < V; i++) {
                F2 g[4];
                next_gain.get(i, g);
#pragma unroll
                for (int e = 0; e < 4; e++)
                    g[e] = mul(mul(o[i][e], f2nd), g[e]);
                const int v = threadIdx.x + i * blockDim.x;
                if (v < a.vecs)
                    *reinterpret_cast<uint4 *>(static_cast<T *>(a.xn) + t * a.ld_xn + 8 * v) =
                        pack<T>(g);
            }
        }
        if (threadIdx.x == 0)
            a.stats[t] = make_float2(r1, r2);
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

// A row's columns belong to CTAS of a cluster, two words for each thread: a wide row's column
// sums, shared vectors and next loads would not fit one CTA's registers.
struct RowSums {
    float4 part[2][kMaxWarps / 4];
    unsigned long long bar[2];
    int gave_up;
};
// Sum over the cluster, number `turn`, a row's first or second, in the same order in all
// CTAs.  Each warp sends its sum to every CTA and goes on when all of them have arrived.  The
// two buffers take turns: a warp that sends sum i + 2 has sum i + 1 of every warp, which read
// sum i before.
template <int CTAS>
__device__ __forceinline__ float sum_row(float v, RowSums &sm, bool second, int turn, int warps,
                                         int rank)
{
    if constexpr (CTAS == 1)
        return sum_block(v, sm.part[second], warps);
    float4 *part = sm.part[turn & 1];
    constexpr int kEach = kMaxWarps / CTAS;
    const uint32_t bar = saddr(&sm.bar[turn & 1]);
    const int lane = threadIdx.x & 31;
    v = sum_warp(v);
    if (threadIdx.x == 0)
        bar_expect_tx(bar, CTAS * warps * sizeof(float));
    if (lane < CTAS) {      // each lane to one of the CTAs
        const float *mine = reinterpret_cast<float *>(part) + rank * kEach + (threadIdx.x >> 5);
        st_async(cluster_addr(saddr(mine), lane), v, cluster_addr(bar, lane));
    }
    if (!__all_sync(0xffffffffu, bar_wait(bar, turn >> 1 & 1, &sm.gave_up))) {
        sm.gave_up = 1;     // a wait that gives up makes the rest of the rows NaN
        return NAN;
    }
    return sum_warp(lane % kEach < warps ? reinterpret_cast<const float *>(part)[lane] : 0.f);
}

// The statistics' products out r2 and y r1 are formed again after each reduction, since
// their packed words take a quarter of the registers.
template <typename T, int CTAS>
__global__ void __launch_bounds__(kMaxThreads, 1) residual_norm_grad_kernel(NormGradArgs a)
{
    constexpr int V = 2;
    extern __shared__ float4 shared[];  // [2][2 V][threads]
    __shared__ RowSums sums;
    pdl_enter();
    const int warps = blockDim.x / 32, rank = blockIdx.x % CTAS;
    const int share = (a.vecs + CTAS - 1) / CTAS, vec0 = rank * share;
    const int vecs = min(share, a.vecs - vec0), col0 = 8 * vec0;
    const long long step = gridDim.x / CTAS;
    Shared weight{shared + threadIdx.x}, next_gain{shared + 2 * V * blockDim.x + threadIdx.x};
    const T *token_gate = a.token_gate ? static_cast<const T *>(a.gate) : nullptr;
    uint4 dq[V], nq[V], oq[V], yq[V];
#pragma unroll
    for (int i = 0; i < V; i++)
        dq[i] = nq[i] = oq[i] = yq[i] = make_uint4(0, 0, 0, 0);
    const auto load = [&](long long t) {
        if (a.dout)
            load_row<V>(dq, a.dout, t * a.ld_dout + col0, vecs);
        if (a.dxn) {
            load_row<V>(nq, a.dxn, t * a.ld_dxn + col0, vecs);
            load_row<V>(oq, a.out, t * a.ld_out + col0, vecs);
        }
        load_row<V>(yq, a.y, t * a.ld_y + col0, vecs);
    };
    long long t = blockIdx.x / CTAS;
    load(t);
    const auto columns = [&](const void *base) {
        return base ? static_cast<const T *>(base) + col0 : nullptr;
    };
    weight.load<T, V>(columns(a.gain), columns(a.token_gate ? nullptr : a.gate), vecs);
    next_gain.load<T, V>(columns(a.next_gain), nullptr, vecs);
    if constexpr (CTAS > 1) {       // the other CTAs run: their memory may be written
        if (threadIdx.x == 0) {
            sums.gave_up = 0;
            bar_init(saddr(&sums.bar[0]), 1);
            bar_init(saddr(&sums.bar[1]), 1);
            asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        }
        __syncwarp();
        cluster_arrive();
        cluster_wait();
    }
    F2 s1[V][4], s2[V][4];      // the column sums
    const auto clear = [&]() {
#pragma unroll
        for (int i = 0; i < V; i++)
#pragma unroll
            for (int e = 0; e < 4; e++)
                s1[i][e] = s2[i][e] = f2(0.f);
    };
    clear();
    const auto flush = [&](int run) {
        float *p = a.part + (blockIdx.x / CTAS * (long long)a.runs + run) * a.H + col0;
        float *q = p + step * a.runs * a.H;
#pragma unroll
        for (int i = 0; i < V; i++) {
            const int v = threadIdx.x + i * blockDim.x;
            if (v >= vecs)
                continue;
#pragma unroll
            for (int j = 0; j < 2; j++) {
                *reinterpret_cast<ulonglong2 *>(p + 8 * v + 4 * j) =
                    make_ulonglong2(s1[i][2 * j].v, s1[i][2 * j + 1].v);
                *reinterpret_cast<ulonglong2 *>(q + 8 * v + 4 * j) =
                    make_ulonglong2(s2[i][2 * j].v, s2[i][2 * j + 1].v);
            }
        }
        clear();
    };
    const F2 scale = f2(a.scale);
    int rows = 0, run = 0, turn = 0;
    for (; t < a.n; t += step) {
        float2 st = a.stats[t];
        if (!a.dxn)             // out alone: the second factor, whatever it is, takes no part
            st.y = 0.f;
        const float tg = token_gate ? to_float<T>(token_gate[t]) : 1.f;
        const F2 r1 = f2(st.x), r2 = f2(st.y);
        F2 d[V][4];
        uint4 ok[V], yk[V];
        F2 m = f2(0.f);
#pragma unroll
        for (int i = 0; i < V; i++) {
            F2 x[4], n[4], g[4];
            unpack<T>(dq[i], d[i]);
            unpack<T>(oq[i], n);
            unpack<T>(nq[i], x);
            next_gain.get(i, g);
            ok[i] = oq[i];
            yk[i] = yq[i];
#pragma unroll
            for (int e = 0; e < 4; e++) {
                const F2 c = mul(x[e], mul(n[e], r2));
                m = fma(c, g[e], m);
                // do without its mean's part
                d[i][e] = fma(r2, mul(x[e], g[e]), d[i][e]);
                s2[i][e] = add(s2[i][e], c);
            }
        }
        if (t + step < a.n)
            load(t + step);
        const float mean =
            a.dxn ? sum_row<CTAS>(sum(m), sums, false, turn++, warps, rank) * a.inv_h * st.y : 0.f;
        const F2 minus = f2(-mean), gate = f2(tg);
        m = f2(0.f);
#pragma unroll
        for (int i = 0; i < V; i++) {
            F2 n[4], z[4], w[4];
            unpack<T>(ok[i], n);
            unpack<T>(yk[i], z);
            weight.get(i, w);
#pragma unroll
            for (int e = 0; e < 4; e++) {
                d[i][e] = fma(mul(n[e], r2), minus, d[i][e]);
                z[e] = mul(d[i][e], mul(z[e], r1));
                m = fma(z[e], w[e], m);
                s1[i][e] = fma(z[e], gate, s1[i][e]);
                n[e] = mul(d[i][e], scale);
            }
            const int v = threadIdx.x + i * blockDim.x;
            if (v < vecs)
                *reinterpret_cast<uint4 *>(static_cast<T *>(a.dresid) + t * a.ld_dresid + col0 +
                                           8 * v) = pack<T>(n);
        }
        // sum of do gain gate z, the gate of a token left out
        const float dot = sum_row<CTAS>(sum(m), sums, true, turn++, warps, rank);
        const F2 back = f2(-dot * tg * a.inv_h * st.x), f = f2(st.x * tg);
#pragma unroll
        for (int i = 0; i < V; i++) {
            F2 z[4], w[4];
            unpack<T>(yk[i], z);
            weight.get(i, w);
#pragma unroll
            for (int e = 0; e < 4; e++)
                z[e] = a.gain ? fma(mul(z[e], r1), back, mul(mul(d[i][e], f), w[e]))
                              : mul(mul(d[i][e], f), w[e]);
            const int v = threadIdx.x + i * blockDim.x;
            if (v < vecs)
                *reinterpret_cast<uint4 *>(static_cast<T *>(a.dy) + t * a.ld_dy + col0 + 8 * v) =
                    pack<T>(z);
        }
        if (token_gate && a.dgate && rank == 0 && threadIdx.x == 0)
            a.dgate[t] = dot;
        if (a.sums && ++rows == kRun) {
            flush(run++);
            rows = 0;
        }
        if (CTAS == 1 && warps > 1 && !a.dxn)
            __syncthreads();        // one buffer alone is in use
    }
    // runs that this CTA has no rows for are zeros
    if (a.sums)
        for (; run < a.runs; run++)
            flush(run);
    if constexpr (CTAS > 1) {       // no CTA ends before the others' last sums have left
        __syncwarp();
        cluster_arrive();
        cluster_wait();
    }
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

// CTAs of a row of the gradient, and threads of each, with two words a thread.
int row_ctas(int H) { return H > 16 * kMaxThreads ? 2 : 1; }
int row_threads(int H)
{
    const int per = 16 * row_ctas(H);
    return ((H + per - 1) / per + 31) / 32 * 32;
}

// Rows of the gradient at once: as many as run on 152 SMs with 128 registers a
// thread.  The workspace's size follows from it, so it asks no device.
int grad_blocks(int n, int H)
{
    return std::min(n, 152 * std::max(1, 512 / row_threads(H)) / row_ctas(H));
}
int grad_runs(int n, int H)
{
    const int rows = (n + grad_blocks(n, H) - 1) / grad_blocks(n, H);
    return (rows + kRun - 1) / kRun;
}
size_t grad_ws(int n, int H)
{
    return 2 * sizeof(float) * (size_t)grad_blocks(n, H) * grad_runs(n, H) * H;
}

// Shared memory of a thread: its part of two vectors.
constexpr int kThreadBytes = 2 * 4 * (int)sizeof(float4);

template <typename T, int MAX>
cudaError_t launch_norm_as(const NormArgs &a, int sms, cudaStream_t st)
{
    const int threads = ((a.H + 15) / 16 + 31) / 32 * 32;   // two words a thread
    const cudaError_t e = cudaFuncSetAttribute(residual_norm_kernel<T, MAX>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               kThreadBytes * MAX);
    if (e != cudaSuccess)
        return e;
    // as many CTAs as run at once
    const dim3 grid(std::min(a.n, sms * std::max(1, 1024 / threads)));
    return launch_pdl(residual_norm_kernel<T, MAX>, grid, dim3(threads), kThreadBytes * threads,
                      st, a);
}
template <typename T>
cudaError_t launch_norm(const NormArgs &a, int sms, cudaStream_t st)
{
    return a.H <= 16 * kMaxThreads ? launch_norm_as<T, kMaxThreads>(a, sms, st)
                                   : launch_norm_as<T, 1024>(a, sms, st);
}

template <typename T, int CTAS>
cudaError_t launch_norm_grad_as(const NormGradArgs &a, cudaStream_t st)
{
    const cudaError_t e = cudaFuncSetAttribute(residual_norm_grad_kernel<T, CTAS>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               kThreadBytes * kMaxThreads);
    if (e != cudaSuccess)
        return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(CTAS * grad_blocks(a.n, a.H));
    cfg.blockDim = dim3(row_threads(a.H));
    cfg.dynamicSmemBytes = kThreadBytes * row_threads(a.H);
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = CTAS;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = CTAS > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, residual_norm_grad_kernel<T, CTAS>, a);
}
template <typename T>
cudaError_t launch_norm_grad(const NormGradArgs &a, cudaStream_t st)
{
    cudaError_t e = row_ctas(a.H) == 1 ? launch_norm_grad_as<T, 1>(a, st)
                                       : launch_norm_grad_as<T, 2>(a, st);
    if (e == cudaSuccess && a.sums)
        e = launch_pdl(residual_norm_sums_kernel<T>, dim3((a.H + 31) / 32, a.dnext_gain ? 2 : 1),
                       dim3(1024), 0, st, a, grad_blocks(a.n, a.H) * a.runs);
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
                        flat_arg(need ? workspace : nullptr, need / 16, 16, true)};
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
