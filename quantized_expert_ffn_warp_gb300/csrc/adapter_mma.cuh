// The adapters' products (see adapter.cu), for one type of activations.
#pragma once
#include <algorithm>

#include "adapter.cuh"
#include "tcgen05.cuh"
#include "vec.cuh"

namespace qe {

namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kTile = kAdapterTile, kCols = kAdapterCols, kBlk = kAdapterStep;

// Copy of 16 bytes into shared memory; 0 behind the `bytes` that are there.
__device__ __forceinline__ void copy16(uint32_t dst, const void *src, int bytes)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
                 : "memory");
}
__device__ __forceinline__ void commit_copies() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// All but the last N groups of the thread's copies are there.
template <int N>
__device__ __forceinline__ void wait_copies()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Values i .. i + 7 of a row of `len` 2-byte values into a slot, 0 behind its end.
__device__ __forceinline__ void fetch8(uint32_t dst, const uint16_t *row, int i, int len,
                                       bool aligned)
{
    if (aligned) {
        copy16(dst, i < len ? row + i : row, min(max(2 * (len - i), 0), 16));
        return;
    }
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; e++) {
        const uint32_t a = i + 2 * e < len ? row[i + 2 * e] : 0;
        const uint32_t b = i + 2 * e + 1 < len ? row[i + 2 * e + 1] : 0;
        w[e] = a | b << 16;
    }
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(dst), "r"(w[0]), "r"(w[1]),
                 "r"(w[2]), "r"(w[3])
                 : "memory");
}

// Copies of ROWS rows of CH chunks of 16 bytes each into rows of 128 bytes (blocks of
// eight chunks, `block` bytes apart), by the whole CTA: a thread has one chunk of every
// kPass-th row, its places a constant number of bytes apart.
template <int CH, int ROWS, int THREADS = kThreads>
struct Rows {
    static constexpr int kPass = THREADS / CH;
    static constexpr int kPasses = (ROWS + kPass - 1) / kPass;
    int row, chunk;
    uint32_t at;
    bool on;

    __device__ __forceinline__ explicit Rows(uint32_t block)
        : row(threadIdx.x / CH), chunk(threadIdx.x % CH),
          at((chunk >> 3) * block + sw128_at(row, chunk & 7)), on(kPass <= ROWS || row < ROWS)
    {
    }
    static constexpr uint32_t kNext = kPass * 128;
};

// ---------------------------------------------------------------- the tensor core

// What a CTA needs around its products.
struct Tensor {
    uint32_t bars;          // barriers, one for each stage
    uint32_t tmem;
    volatile int *gave_up;
};
constexpr int kStages = 5;      // at most
struct TensorSmem {
    uint64_t bar[kStages];
    uint32_t tmem;
    int gave_up;
};

// Lets the next kernel launch when the CTA has its tensor memory, not before: one that
// takes all of it and then waits for this kernel would never let it finish.
__device__ __forceinline__ Tensor tensor_begin(TensorSmem &sm, uint32_t cols)
{
    if (threadIdx.x < 32)
        tmem_alloc(&sm.tmem, cols);
    if (threadIdx.x == 32) {
        sm.gave_up = 0;
        for (int i = 0; i < kStages; i++)
            bar_init(saddr(&sm.bar[i]), 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    pdl_launch();
    return {saddr(sm.bar), sm.tmem, &sm.gave_up};
}
__device__ __forceinline__ void tensor_end(const Tensor &t, uint32_t cols)
{
    tc_fence_before();
    __syncthreads();
    if (threadIdx.x < 32)
        tmem_free(t.tmem, cols);
}
// Waits for the products of use `use` of barrier i.  A wait that gives up makes the CTA's
// results NaN; its threads go on, so that all of them meet the CTA's barriers.
__device__ __forceinline__ void tensor_wait(const Tensor &t, int i, int use)
{
    if (!bar_wait(t.bars + 8 * i, use & 1, t.gave_up))
        *t.gave_up = 1;
}

__host__ __device__ constexpr uint32_t tmem_cols(int n)
{
    return n <= 32 ? 32 : n <= 64 ? 64 : n <= 128 ? 128 : n <= 256 ? 256 : 512;
}
// 128-byte rows that hold `r` values.
__host__ __device__ constexpr int row_blocks(int r) { return (r + kBlk - 1) / kBlk; }

// A multi-stage contraction: fetch(i, stage) starts the copies of step i, multiply(stage,
// first) issues its products in one elected thread.  Copies of the steps ahead are under
// way while a step is multiplied; a stage is filled again when its products are done.
// Bit s of `uses` counts the waits for stage s over the CTA's contractions, by their parity:
// none is left out if the CTA goes on to `another`.
template <int S, typename F, typename M>
__device__ __forceinline__ void contract(const Tensor &t, int steps, uint32_t &uses, bool another,
                                         F fetch, M multiply)
{
    const auto wait = [&](int s) {
        tensor_wait(t, s, uses >> s);
        uses ^= 1u << s;
    };
#pragma unroll
    for (int i = 0; i < S - 1; i++) {
        if (i < steps)
            fetch(i, i);
        commit_copies();
    }
    int stage = 0;
    for (int i = 0; i < steps; i++) {
        wait_copies<S - 2>();
        fence_async_shared();
        __syncthreads();
        if (threadIdx.x < 32) {
            tc_fence_after();
            if (elect_one()) {
                multiply(stage, i == 0);
                umma_commit(t.bars + 8 * stage);
            }
            __syncwarp();
        }
        const int before = stage == 0 ? S - 1 : stage - 1;
        if (i + S - 1 < steps) {
            if (i > 0)
                wait(before);
            fetch(i + S - 1, before);
        }
        commit_copies();
        stage = stage + 1 == S ? 0 : stage + 1;
    }
    wait_copies<0>();
    // the last step first: those in front of it are done then, and cost no wait
    for (int i = another ? min(steps, S) : min(steps, 1); i > 0; i--) {
        stage = stage == 0 ? S - 1 : stage - 1;
        wait(stage);
    }
    tc_fence_after();
}
// A LONG contraction, of more than kOneChain terms, is cut into chains of kChain, whose sums are
// added in fp32: the tensor cores cut what a chain adds to a step of its sum, always towards 0
// (0.4% of a sum of 2^20 terms of one sign in one chain).  kOneChain terms are 1024 sums of 16,
// off by 2^-13 of the terms at most.  A variant of its own, since the code for chains costs
// every CTA 0.3 us although it is not run (8192 tokens of 64 adapters 138 to 142 us).
constexpr int kChain = 4096, kOneChain = 16384;

// Sixteen sums, with those that an earlier chain left at `kept`.
__device__ __forceinline__ void add_kept(float (&v)[16], uint32_t kept, bool any)
{
    if (!any)
        return;
    float w[16];
    tmem_ld16(kept, w);
#pragma unroll
    for (int e = 0; e < 16; e++)
        v[e] += w[e];
}

// A call's dynamic shared memory from a 1024-byte boundary on, as the swizzle needs.
extern __shared__ uint8_t adapter_smem[];
__device__ __forceinline__ uint32_t smem_base() { return (saddr(adapter_smem) + 1023) & ~1023u; }
__device__ __forceinline__ uint8_t *smem_at(uint32_t address)
{
    return adapter_smem + (address - saddr(adapter_smem));
}
constexpr int kSmemSlack = 1024;

// ---------------------------------------------------------------- shrink

struct ShrinkArgs {
    AdapterPlan p;
    const uint16_t *x;      // [n][K]
    long long ldx;
    const uint16_t *w;      // [L][r][K], or (BY_ROW) [L][K][r]
    int n, L, K, r, slices;
    bool vec_x, vec_w;
    float *part;            // [slices][n][PAD] partial sums
    float *mid;             // [n][PAD], kLifted types
    uint16_t *parts;        // [n][kParts][PAD], others
    uint16_t *h;            // [n][r], or null
    bool most;              // keep the largest of each adapter
};

template <typename T>
__device__ __forceinline__ uint16_t bits(T v)
{
    return *reinterpret_cast<const uint16_t *>(&v);
}

// An fp32 value of h or u is multiplied as the sum of kParts values of T: 24 bits in bf16,
// 22 in fp16.
template <typename T>
constexpr int kParts = std::is_same_v<T, __nv_bfloat16> ? 3 : 2;
// The type's own exponents do not reach all fp32 values: 2^e of them are split.
template <typename T>
constexpr bool kLifted = std::is_same_v<T, __half>;
// In the sums over tokens, of a part of u to the one in front of it: lifted, what the first
// lacks fills the same range, so that a token's u has its 22 bits down to 2^-28 of the
// adapter's largest.
template <typename T>
constexpr float kNext = kLifted<T> ? 2048.f : 1.f;

// (2^e, 2^-e) with 2^e most in [2^14, 2^15); both are normal numbers for any most.
__device__ __forceinline__ float2 lift_of(float most)
{
    const int e = min(141 - (int)(__float_as_uint(most) >> 23), 100);
    return make_float2(__uint_as_float((uint32_t)(127 + e) << 23),
                       __uint_as_float((uint32_t)(127 - e) << 23));
}
// The parts of N values; each is what those in front of it lack, times `next` for each.
template <typename T, int P, int N>
__device__ __forceinline__ void split(float (&v)[N], float next, uint32_t (&q)[P][N / 2])
{
#pragma unroll
    for (int p = 0; p < P; p++)
#pragma unroll
        for (int e = 0; e < N; e += 2) {
            q[p][e / 2] = pack2<T>(v[e], v[e + 1]);
            const float2 f = unpack2<T>(q[p][e / 2]);
            // an infinity or a NaN has no remainder
            v[e] = fabsf(f.x) <= 3.4e38f ? (v[e] - f.x) * next : 0.f;
            v[e + 1] = fabsf(f.y) <= 3.4e38f ? (v[e + 1] - f.y) * next : 0.f;
        }
}
__device__ __forceinline__ void store_shared(uint32_t at, const uint32_t (&q)[4])
{
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(q[0]), "r"(q[1]),
                 "r"(q[2]), "r"(q[3])
                 : "memory");
}
__device__ __forceinline__ void load8(float (&v)[8], const float *p, bool in)
{
    const float4 a = in ? *reinterpret_cast<const float4 *>(p) : make_float4(0.f, 0.f, 0.f, 0.f);
    const float4 b =
        in ? *reinterpret_cast<const float4 *>(p + 4) : make_float4(0.f, 0.f, 0.f, 0.f);
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
    v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}

// The parts of an adapter's u for the sums over its tokens: eight ranks of a place.
template <typename T, int PAD>
__device__ __forceinline__ void put_lifted(uint16_t *parts, long long place, int k,
                                           const float (&u)[8], float lift)
{
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; e++)
        v[e] = u[e] * lift;
    uint32_t q[kParts<T>][4];
    split<T>(v, kNext<T>, q);
#pragma unroll
    for (int p = 0; p < kParts<T>; p++)
        *reinterpret_cast<uint4 *>(parts + (place * kParts<T> + p) * PAD + k) =
            make_uint4(q[p][0], q[p][1], q[p][2], q[p][3]);
}

// Four of a token's results from rank k on, at its place and in h; those behind the last rank
// are 0: the product's are 0 times x, a NaN where x is not finite.  `most` takes their size.
template <typename T, int PAD>
__device__ __forceinline__ void put_results(const ShrinkArgs &a, int place, int token, int k,
                                            const float (&sums)[4], float &most)
{
    float v[4];
#pragma unroll
    for (int e = 0; e < 4; e++)
        v[e] = k < a.r ? sums[e] : 0.f;
    if (a.h && k < a.r)
        *reinterpret_cast<uint2 *>(a.h + (long long)token * a.r + k) =
            make_uint2(pack2<T>(v[0], v[1]), pack2<T>(v[2], v[3]));
    if constexpr (kLifted<T>) {
        *reinterpret_cast<float4 *>(a.mid + (long long)place * PAD + k) =
            make_float4(v[0], v[1], v[2], v[3]);
#pragma unroll
        for (int e = 0; e < 4; e++)
            most = fmaxf(most, fabsf(v[e]));
    } else {
        uint32_t q[kParts<T>][2];
        split<T>(v, 1.f, q);
#pragma unroll
        for (int p = 0; p < kParts<T>; p++)
            *reinterpret_cast<uint2 *>(a.parts + ((long long)place * kParts<T> + p) * PAD + k) =
                make_uint2(q[p][0], q[p][1]);
    }
}
// The warp's largest result to its adapter's, whatever the order: a NaN is passed over.
__device__ __forceinline__ void put_most(const ShrinkArgs &a, int adapter, float most)
{
    most = max_warp(most);
    if ((threadIdx.x & 31) == 0 && most > 0.f)
        atomicMax(a.p.most + adapter, __float_as_uint(most));
}

constexpr int kShrinkStages = 4;
template <bool BY_ROW, int PAD>
constexpr int kShrinkStage = 128 * kTile + (BY_ROW ? 128 * kBlk * row_blocks(PAD) : 128 * PAD);

// A tile's tokens (the product's rows) times all ranks.  The slices' sums are added by
// whichever CTA of a tile arrives last, in the slices' order.
template <typename T, bool BY_ROW, int PAD, bool LONG>
__global__ void __launch_bounds__(kThreads, PAD <= 64 ? 2 : 1) adapter_shrink_kernel(ShrinkArgs a)
{
    __shared__ TensorSmem ts;
    __shared__ int last;
    pdl_wait();
    if ((int)blockIdx.x >= *a.p.n_tiles)
        return;
    const int4 tile = a.p.tiles[blockIdx.x];
    const int slice = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (tile.x == a.L) {        // no adapter
        if (slice == 0 && a.h)
            for (int i = threadIdx.x; i < tile.z * a.r; i += kThreads)
                a.h[(long long)a.p.perm[tile.y + i / a.r] * a.r + i % a.r] = 0;
        return;
    }
    constexpr uint32_t cols = tmem_cols(LONG ? 2 * PAD : PAD);
    const Tensor t = tensor_begin(ts, cols);
    const int blocks = (a.K + kBlk - 1) / kBlk;
    const int begin = (int)((long long)blocks * slice / a.slices);
    const int end = (int)((long long)blocks * (slice + 1) / a.slices);
    const uint32_t smem = smem_base();
    constexpr int stage_bytes = kShrinkStage<BY_ROW, PAD>;
    // a thread's chunks of the tokens, and of the matrix: rows of ranks, or (BY_ROW) of K
    using X = Rows<8, kTile>;
    using W = std::conditional_t<BY_ROW, Rows<PAD / 8, kBlk>, Rows<8, PAD>>;
    const X xr(0);
    const W wr(128 * kBlk);
    const uint16_t *w = a.w + (long long)tile.x * a.r * a.K;
    const uint16_t *src[X::kPasses];
    bool there[X::kPasses];
#pragma unroll
    for (int j = 0; j < X::kPasses; j++) {
        const int at = xr.row + X::kPass * j;
        there[j] = at < tile.z;
        src[j] = a.x + (long long)a.p.perm[tile.y + (there[j] ? at : 0)] * a.ldx;
    }
    const uint16_t *mat0 = BY_ROW ? w + (long long)wr.row * a.r + 8 * wr.chunk
                                  : w + (long long)wr.row * a.K + 8 * wr.chunk;
    const long long mat_pass = (long long)W::kPass * (BY_ROW ? a.r : a.K);
    const auto fetch = [&](int i, int stage) {
        const int k0 = (begin + i) * kBlk;
        const uint32_t xs = smem + stage * stage_bytes + xr.at;
        const uint32_t ws = smem + stage * stage_bytes + 128 * kTile + wr.at;
        if (a.vec_x && a.vec_w && k0 + kBlk <= a.K) {
#pragma unroll
            for (int j = 0; j < X::kPasses; j++)
                if (there[j])
                    copy16(xs + X::kNext * j, src[j] + k0 + 8 * xr.chunk, 16);
            const uint16_t *m = mat0 + (BY_ROW ? (long long)k0 * a.r : k0);
#pragma unroll
            for (int j = 0; j < W::kPasses; j++) {      // 0 for the ranks behind the last
                const bool in = BY_ROW ? 8 * wr.chunk < a.r : wr.row + W::kPass * j < a.r;
                if (wr.on)
                    copy16(ws + W::kNext * j, in ? m + mat_pass * j : w, in ? 16 : 0);
            }
            return;
        }
#pragma unroll 1
        for (int j = 0; j < X::kPasses; j++) {
            const int at = xr.row + X::kPass * j;
            if (at < tile.z)
                fetch8(xs + X::kNext * j, a.x + (long long)a.p.perm[tile.y + at] * a.ldx,
                       k0 + 8 * xr.chunk, a.K, a.vec_x);
        }
#pragma unroll 1
        for (int j = 0; j < W::kPasses && wr.on; j++) {
            const int row = wr.row + W::kPass * j;
            if constexpr (BY_ROW) {
                const bool in = k0 + row < a.K && 8 * wr.chunk < a.r;
                copy16(ws + W::kNext * j,
                       in ? w + (long long)(k0 + row) * a.r + 8 * wr.chunk : w, in ? 16 : 0);
            } else {
                fetch8(ws + W::kNext * j, row < a.r ? w + (long long)row * a.K : w,
                       k0 + 8 * wr.chunk, row < a.r ? a.K : 0, a.vec_w);
            }
        }
    };
    constexpr uint32_t idesc =
        (1u << 4) | (std::is_same_v<T, __nv_bfloat16> ? (1u << 7 | 1u << 10) : 0u) |
        ((uint32_t)(PAD >> 3) << 17) | (8u << 24) | (BY_ROW ? kMnMajorB : 0u);
    const auto multiply = [&](int stage, bool first) {
        const uint32_t at = smem + stage * stage_bytes, mat = at + 128 * kTile;
        const uint64_t da = sw128_desc(at);
        const uint64_t db = BY_ROW ? sw128_desc_mn(mat, 128 * kBlk) : sw128_desc(mat);
#pragma unroll
        for (int k = 0; k < 4; k++)
            umma_ss(t.tmem, da + 2 * k, db + (BY_ROW ? 128 : 2) * k, idesc, !first || k);
    };
    const uint32_t sums = t.tmem + ((uint32_t)(32 * (warp & 3)) << 16), kept = sums + PAD;
    const int at = 32 * warp + lane, place = tile.y + at;
    const int token = at < tile.z ? a.p.perm[place] : 0;
    uint32_t uses = 0;
    float most = 0.f;
    constexpr int chain = kChain / kBlk;
    int s0 = begin;
    do {
        const bool more = LONG && s0 + chain < end;
        const auto fetch_from = [&](int i, int stage) { fetch(s0 - begin + i, stage); };
        contract<kShrinkStages>(t, more ? chain : end - s0, uses, more, fetch_from, multiply);
        const bool failed = *t.gave_up;
        if (warp < 4)
#pragma unroll 1
            for (int c = 0; c < PAD; c += 16) {
                float v[16];
                tmem_ld16(sums + c, v);
                add_kept(v, kept + c, LONG && s0 > begin);
                if (more) {
                    tmem_st16(kept + c, v);
                    continue;
                }
                if (at < tile.z) {
#pragma unroll
                    for (int q = 0; q < 4; q++) {
                        float d[4];
#pragma unroll
                        for (int e = 0; e < 4; e++)
                            d[e] = failed ? NAN : v[4 * q + e];
                        if (a.slices == 1)
                            put_results<T, PAD>(a, place, token, c + 4 * q, d, most);
                        else
                            *reinterpret_cast<float4 *>(
                                a.part + ((long long)slice * a.n + place) * PAD + c + 4 * q) =
                                make_float4(d[0], d[1], d[2], d[3]);
                    }
                }
                __syncwarp();       // the next load is the whole warp's
            }
        tc_fence_before();          // the next chain's products write where this one's were read
        s0 += chain;
    } while (LONG && s0 < end);
    if (a.most && a.slices == 1 && warp < 4)
        put_most(a, tile.x, most);
    tensor_end(t, cols);
    if (a.slices == 1)
        return;
    __threadfence();
    __syncthreads();
    if (threadIdx.x == 0)
        last = atomicAdd(a.p.tickets + blockIdx.x, 1u) == a.slices - 1u;
    __syncthreads();
    if (!last)
        return;
    __threadfence();
    constexpr int I = 4, U = 4;     // places and slices whose loads are under way together
    const int items = tile.z * (PAD / 4);
    const long long next = (long long)a.n * PAD;
    for (int i0 = threadIdx.x; i0 < items; i0 += I * kThreads) {
        float v[I][4] = {};
        int token[I];
#pragma unroll
        for (int j = 0; j < I; j++) {
            const int i = i0 + j * kThreads;
            token[j] = i < items ? a.p.perm[tile.y + i / (PAD / 4)] : 0;
        }
        for (int s0 = 0; s0 < a.slices; s0 += U) {
            float4 q[I][U];
#pragma unroll
            for (int j = 0; j < I; j++) {
                const int i = i0 + j * kThreads;
                const float *from = a.part + (s0 * (long long)a.n + tile.y) * PAD + 4 * (long long)i;
#pragma unroll
                for (int s = 0; s < U; s++)
                    if (i < items && s0 + s < a.slices)
                        q[j][s] = __ldcg(reinterpret_cast<const float4 *>(from + s * next));
            }
#pragma unroll
            for (int j = 0; j < I; j++)
#pragma unroll
                for (int s = 0; s < U; s++)
                    if (s0 + s < a.slices)
                        v[j][0] += q[j][s].x, v[j][1] += q[j][s].y, v[j][2] += q[j][s].z,
                            v[j][3] += q[j][s].w;
        }
#pragma unroll
        for (int j = 0; j < I; j++) {
            const int i = i0 + j * kThreads;
            if (i < items)
                put_results<T, PAD>(a, tile.y + i / (PAD / 4), token[j], i % (PAD / 4) * 4, v[j],
                                    most);
        }
    }
    __syncwarp();
    if (a.most)
        put_most(a, tile.x, most);
}

// ---------------------------------------------------------------- expand

struct ExpandArgs {
    AdapterPlan p;
    const float *mid;       // [n][PAD], kLifted types
    uint16_t *parts;        // [n][kParts][PAD]: read; kLifted, written (or null)
    const uint16_t *w;      // [L][N][r], or (BY_ROW) [L][r][N]
    const float *scale;     // [L] or null
    const uint16_t *base;   // [n][N] or null
    long long ldb;
    uint16_t *out;          // [n][N]
    long long ldo;
    int L, N, r;
    bool vec_w, vec_b, vec_o;
};

// Values i .. i + 7 of a row of `len` 2-byte values, 0 behind its end; and back.
__device__ __forceinline__ uint4 load8(const uint16_t *row, int i, int len, bool aligned)
{
    if (aligned && i + 8 <= len)
        return load_stream(row + i);
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; e++) {
        const uint32_t a = i + 2 * e < len ? row[i + 2 * e] : 0;
        const uint32_t b = i + 2 * e + 1 < len ? row[i + 2 * e + 1] : 0;
        w[e] = a | b << 16;
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void store8(uint16_t *row, int i, int len, bool aligned, const uint4 &q)
{
    if (aligned && i + 8 <= len) {
        *reinterpret_cast<uint4 *>(row + i) = q;
        return;
    }
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int e = 0; e < 8; e++)
        if (i + e < len)
            row[i + e] = (uint16_t)(w[e / 2] >> (16 * (e & 1)));
}

// h in 128-byte rows, part after part.
template <typename T, int PAD>
constexpr int kPartBlocks = row_blocks(kParts<T> * PAD);
template <bool BY_ROW, int PAD>
constexpr int kMatrix = BY_ROW ? 2 * kCols * PAD : 128 * kCols * row_blocks(PAD);
// A tile's rows of base, then of out, for one block of columns: rows 16 bytes longer than
// their values lie in different banks at equal columns.
constexpr int kExpandThreads = 512;
constexpr int kPitch = 2 * kCols + 16, kRowsBytes = kTile * kPitch;
// Blocks of columns whose copies are under way ahead; one more buffer of rows for the
// block at hand.
template <int PAD>
constexpr int kAhead = PAD <= 64 ? 2 : 1;
template <int PAD>
constexpr int kRowBuffers = kAhead<PAD> + 1;
// One block ahead, a block's matrix is copied when the last product is done with its own.
template <int PAD>
constexpr int kMatrices = kAhead<PAD>;
template <typename T, bool BY_ROW, int PAD>
constexpr int kExpandSmem = 128 * kTile * kPartBlocks<T, PAD> + kMatrices<PAD> * kMatrix<BY_ROW, PAD> +
                            kRowBuffers<PAD> * kRowsBytes + kSmemSlack;

// Tiles of tokens (the product's rows) times blocks of columns: a CTA takes an equal share
// of the cost of all (tile, block) pairs, tile after tile.  While a block's sums leave tensor memory,
// the next block is multiplied beside it, and the matrix and base of the one behind that
// are copied.  A thread has a quarter of a token's row and adds the sums to base where base
// lies in shared memory; then the warp stores 64 bytes of every row.
template <typename T, bool BY_ROW, int PAD>
__global__ void __launch_bounds__(kExpandThreads, 1) adapter_expand_kernel(ExpandArgs a)
{
    __shared__ TensorSmem ts;
    __shared__ int toks[kTile];
    __shared__ float undo[kLifted<T> ? kTile : 1];      // a row's 2^-e
    pdl_wait();
    const int blocks = (a.N + kCols - 1) / kCols;
    const int n_tiles = a.p.n_tiles[0];
    const long long cost = (long long)a.p.n_tiles[1] * blocks;
    // the (tile, block) pairs at which the share of the cost begins and ends: the tiles in
    // front are counted by all threads at once
    const long long from_cost = cost * blockIdx.x / gridDim.x;
    const long long to_cost = cost * (blockIdx.x + 1) / gridDim.x;
    int tile0 = -1, tile1 = -1;
    // (few pairs are shared out by number: the search takes 2 us)
    const long long total = (long long)n_tiles * blocks;
    const bool few = total <= 2 * (long long)gridDim.x;
    for (int k = 0; k < n_tiles && !few; k += blockDim.x) {
        const int i = k + threadIdx.x;
        const long long before = i < n_tiles ? (long long)a.p.tiles[i].w * blocks : cost + 1;
        tile0 += __syncthreads_count(before <= from_cost);
        tile1 += __syncthreads_count(before <= to_cost);
    }
    const auto place = [&](int tile, long long to) {
        const int4 q = a.p.tiles[tile];
        const unsigned block =
            (unsigned)(to - (long long)q.w * blocks) / (unsigned)tile_cost(q.x == a.L, q.z);
        return (long long)tile * blocks + min(block, (unsigned)blocks);
    };
    long long at = few ? total * blockIdx.x / gridDim.x : place(tile0, from_cost);
    const long long end = few ? total * (blockIdx.x + 1) / gridDim.x : place(tile1, to_cost);
    if (at >= end)
        return;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const Tensor t = tensor_begin(ts, 2 * kCols);
    constexpr int parts = kParts<T>, matrix = kMatrix<BY_ROW, PAD>;
    constexpr int ahead = kAhead<PAD>, buffers = kRowBuffers<PAD>;
    const uint32_t hs = smem_base(), mats = hs + 128 * kTile * kPartBlocks<T, PAD>;
    const uint32_t rows = mats + kMatrices<PAD> * matrix;
    // the matrix: rows of ranks (0 behind the last), or (BY_ROW) of columns for each rank
    using W = std::conditional_t<BY_ROW, Rows<kCols / 8, PAD, kExpandThreads>,
                                 Rows<PAD / 8, kCols, kExpandThreads>>;
    const W wr(BY_ROW ? 128 * PAD : 128 * kCols);
    const long long mat_pass = (long long)W::kPass * (BY_ROW ? a.N : a.r);
    constexpr uint32_t idesc =
        (1u << 4) | (std::is_same_v<T, __nv_bfloat16> ? (1u << 7 | 1u << 10) : 0u) |
        ((uint32_t)(kCols >> 3) << 17) | (8u << 24) | (BY_ROW ? kMnMajorB : 0u);
    // the thread's row and 32 of its columns; its chunk of base in every 32nd row
    const int row = 32 * (warp & 3) + lane, col = 32 * (warp >> 2);
    const int base_row = threadIdx.x / 16, base_chunk = threadIdx.x % 16;
    constexpr int kBasePass = kExpandThreads / 16;
    // its eight values of h in every kMidPass-th row
    constexpr int kMidRow = PAD / 8, kMidPass = kExpandThreads / kMidRow;
    constexpr int kMidPasses = (kTile + kMidPass - 1) / kMidPass;
    const int mid_row = threadIdx.x / kMidRow, mid_chunk = threadIdx.x % kMidRow;
    int done = 0;       // products so far: their tensor memory and barrier alternate
    while (at < end) {
        const int4 tile = a.p.tiles[at / blocks];
        const int first = (int)(at % blocks), steps = (int)min(end - at, (long long)blocks - first);
        at += steps;
        if (tile.x == a.L) {        // no adapter: base, or 0
            if (a.out == a.base)
                continue;
            const int begin = first * kCols, stop = min(a.N, (first + steps) * kCols);
            const int wide = (stop - begin + 7) / 8;
            constexpr int U = 8;        // loads of a thread under way
            for (int i0 = threadIdx.x; i0 < tile.z * wide; i0 += U * kExpandThreads) {
                uint4 q[U];
                long long tok[U];
                int c[U];
#pragma unroll
                for (int u = 0; u < U; u++) {
                    const int i = i0 + u * kExpandThreads;
                    q[u] = make_uint4(0, 0, 0, 0);
                    tok[u] = -1;
                    if (i < tile.z * wide) {
                        tok[u] = a.p.perm[tile.y + i / wide];
                        c[u] = begin + i % wide * 8;
                    }
                }
#pragma unroll
                for (int u = 0; u < U; u++)
                    if (a.base && tok[u] >= 0)
                        q[u] = load8(a.base + tok[u] * a.ldb, c[u], stop, a.vec_b);
#pragma unroll
                for (int u = 0; u < U; u++)
                    if (tok[u] >= 0)
                        store8(a.out + tok[u] * a.ldo, c[u], stop, a.vec_o, q[u]);
            }
            continue;
        }
        __syncthreads();        // the last tile's rows have left
        if (threadIdx.x < kTile)
            toks[threadIdx.x] =
                a.p.perm[tile.y + ((int)threadIdx.x < tile.z ? threadIdx.x : 0)];
        float mid[kMidPasses][8];
        if constexpr (kLifted<T>) {
#pragma unroll
            for (int j = 0; j < kMidPasses; j++) {
                const int r = mid_row + kMidPass * j;
                load8(mid[j], a.mid + (long long)(tile.y + r) * PAD + 8 * mid_chunk, r < tile.z);
            }
        } else {
#pragma unroll
            for (int j = 0; j < kMidPasses; j++) {
                const int r = mid_row + kMidPass * j;
#pragma unroll
                for (int p = 0; p < parts; p++) {
                    const int c = p * kMidRow + mid_chunk;
                    if (r < tile.z)
                        copy16(hs + (c >> 3) * (128 * kTile) + sw128_at(r, c & 7),
                               a.parts + (long long)(tile.y + r) * parts * PAD + 8 * c, 16);
                }
            }
        }
        __syncthreads();
        const uint16_t *w = a.w + (long long)tile.x * a.r * a.N;
        const uint16_t *mat0 = BY_ROW ? w + (long long)wr.row * a.N + 8 * wr.chunk
                                      : w + (long long)wr.row * a.r + 8 * wr.chunk;
        const float scale = a.scale ? a.scale[tile.x] : 1.f;
        // what the thread stores: 8 columns of rows lane / 4, + 8, .. of the warp's 32
        uint16_t *to[4];
        bool on[4];
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const int r = 32 * (warp & 3) + 8 * i + lane / 4;
            on[i] = r < tile.z;
            to[i] = a.out + (long long)toks[r] * a.ldo + col + 8 * (lane & 3);
        }
        const uint16_t *from[kTile / kBasePass];
#pragma unroll
        for (int j = 0; j < kTile / kBasePass; j++)
            from[j] = a.base + (long long)toks[base_row + kBasePass * j] * a.ldb + 8 * base_chunk;
        const auto fetch = [&](int step) {
            const int c0 = (first + step) * kCols;
            const uint32_t ws = mats + step % kMatrices<PAD> * matrix + wr.at;
            const bool whole = c0 + kCols <= a.N;
            if (step >= steps) {
                commit_copies();
                return;
            }
            if (a.vec_w && whole) {
                const uint16_t *m = mat0 + (BY_ROW ? c0 : (long long)c0 * a.r);
#pragma unroll
                for (int j = 0; j < W::kPasses; j++) {
                    const bool in = BY_ROW ? wr.row + W::kPass * j < a.r : 8 * wr.chunk < a.r;
                    if (wr.on)
                        copy16(ws + W::kNext * j, in ? m + mat_pass * j : w, in ? 16 : 0);
                }
            } else {
#pragma unroll 1
                for (int j = 0; j < W::kPasses && wr.on; j++) {
                    const int r = wr.row + W::kPass * j;
                    if constexpr (BY_ROW) {
                        fetch8(ws + W::kNext * j, r < a.r ? w + (long long)r * a.N : w,
                               c0 + 8 * wr.chunk, r < a.r ? a.N : 0, a.vec_w);
                    } else {
                        const bool in = c0 + r < a.N && 8 * wr.chunk < a.r;
                        copy16(ws + W::kNext * j,
                               in ? w + (long long)(c0 + r) * a.r + 8 * wr.chunk : w, in ? 16 : 0);
                    }
                }
            }
            if (a.base) {
                const uint32_t bs =
                    rows + step % buffers * kRowsBytes + base_row * kPitch + 16 * base_chunk;
                if (a.vec_b && whole) {
#pragma unroll
                    for (int j = 0; j < kTile / kBasePass; j++)
                        if (base_row + kBasePass * j < tile.z)
                            copy16(bs + kBasePass * kPitch * j, from[j] + c0, 16);
                } else if (a.vec_b) {
#pragma unroll 1
                    for (int r = base_row; r < tile.z; r += kBasePass)
                        fetch8(bs + (r - base_row) * kPitch, a.base + toks[r] * a.ldb,
                               c0 + 8 * base_chunk, a.N, true);
                } else {        // odd rows: a warp a row, neighbours side by side
                    constexpr int kWarpsHere = kExpandThreads / 32, E = kCols / 32;
#pragma unroll 2
                    for (int r = warp; r < tile.z; r += kWarpsHere) {
                        const uint16_t *src = a.base + toks[r] * a.ldb + c0;
                        uint16_t *dst = reinterpret_cast<uint16_t *>(
                            smem_at(rows + step % buffers * kRowsBytes + r * kPitch));
                        uint16_t v[E];
#pragma unroll
                        for (int e = 0; e < E; e++)
                            v[e] = c0 + 32 * e + lane < a.N ? src[32 * e + lane] : 0;
#pragma unroll
                        for (int e = 0; e < E; e++)
                            dst[32 * e + lane] = v[e];
                    }
                }
            }
            commit_copies();
        };
        const auto multiply = [&](int step) {
            if (warp == 0 && step < steps) {
                tc_fence_after();
                if (elect_one()) {
                    const uint32_t mat = mats + step % kMatrices<PAD> * matrix;
                    const int buffer = (done + step) & 1;
#pragma unroll
                    for (int part = 0; part < parts; part++)
#pragma unroll
                        for (int k = 0; k < PAD / 16; k++) {
                            const int ka = part * (PAD / 16) + k;
                            const uint64_t da =
                                sw128_desc(hs + (ka >> 2) * (128 * kTile)) + 2 * (ka & 3);
                            const uint64_t db =
                                BY_ROW ? sw128_desc_mn(mat, 128 * PAD) + 128 * k
                                       : sw128_desc(mat + (k >> 2) * (128 * kCols)) + 2 * (k & 3);
                            umma_ss(t.tmem + kCols * buffer, da, db, idesc, part || k);
                        }
                    umma_commit(t.bars + 8 * buffer);
                }
                __syncwarp();
            }
        };
        fetch(0);
        if (ahead == 2)
            fetch(1);
        if constexpr (kLifted<T>) {
            // whoever has a tile's first block leaves its parts for the sums over tokens
            const bool leave = a.parts && first == 0;
            const float all =
                leave ? lift_of(__uint_as_float(a.p.most[tile.x])).x : 0.f;
#pragma unroll
            for (int j = 0; j < kMidPasses; j++) {
                const int r = mid_row + kMidPass * j;
                if (leave && r < tile.z)
                    put_lifted<T, PAD>(a.parts, tile.y + r, 8 * mid_chunk, mid[j], all);
                float most = 0.f;
#pragma unroll
                for (int e = 0; e < 8; e++)
                    most = fmaxf(most, fabsf(mid[j][e]));
#pragma unroll
                for (int d = 1; d < kMidRow; d <<= 1)
                    most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, d));
                const float2 lift = lift_of(most);
#pragma unroll
                for (int e = 0; e < 8; e++)
                    mid[j][e] *= lift.x;
                if (mid_chunk == 0 && r < tile.z)
                    undo[r] = lift.y;
                uint32_t q[parts][4];
                split<T>(mid[j], 1.f, q);
#pragma unroll
                for (int p = 0; p < parts; p++) {
                    const int c = p * kMidRow + mid_chunk;
                    if (r < tile.z)
                        store_shared(hs + (c >> 3) * (128 * kTile) + sw128_at(r, c & 7), q[p]);
                }
            }
        }
        if (ahead == 2) {
            wait_copies<1>();
            fence_async_shared();
            __syncthreads();
            multiply(0);
        }
        for (int step = 0; step < steps; step++) {
            const int c0 = (first + step) * kCols, buffer = (done + step) & 1;
            // the copies of the next product are through, and the last block's rows have left
            wait_copies<0>();
            fence_async_shared();
            tc_fence_before();
            __syncthreads();
            multiply(step + ahead - 1);
            tensor_wait(t, buffer, (done + step) >> 1);
            tc_fence_after();
            fetch(step + ahead);
            const F2 factor = f2(*t.gave_up ? NAN : kLifted<T> ? scale * undo[row] : scale);
            uint8_t *const block = smem_at(rows + step % buffers * kRowsBytes + 2 * col);
            uint4 *const mine = reinterpret_cast<uint4 *>(block + row * kPitch);
            const uint8_t *const theirs =
                block + (32 * (warp & 3) + lane / 4) * kPitch + 16 * (lane & 3);
            if (32 * (warp & 3) < tile.z && c0 + col < a.N) {
                uint4 q[4];
#pragma unroll
                for (int i = 0; i < 4; i++)
                    q[i] = a.base ? mine[i] : make_uint4(0, 0, 0, 0);
                float v[32];
                tmem_ld32(t.tmem + ((uint32_t)(32 * (warp & 3)) << 16) + kCols * buffer + col, v);
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    F2 d[4];
                    unpack<T>(q[i], d);
#pragma unroll
                    for (int e = 0; e < 4; e++)
                        d[e] = fma(factor, f2(v[8 * i + 2 * e], v[8 * i + 2 * e + 1]), d[e]);
                    q[i] = pack<T>(d);
                }
#pragma unroll
                for (int i = 0; i < 4; i++)
                    mine[i] = q[i];
                __syncwarp();
                const int c = c0 + col + 8 * (lane & 3);
                if (!a.vec_o) {         // odd rows: neighbours side by side
                    const uint16_t *from = reinterpret_cast<const uint16_t *>(
                                               block + 32 * (warp & 3) * kPitch) + lane;
                    const int many = c0 + col + lane < a.N ? min(32, tile.z - 32 * (warp & 3)) : 0;
#pragma unroll 4
                    for (int r = 0; r < many; r++)
                        a.out[(long long)toks[32 * (warp & 3) + r] * a.ldo + c0 + col + lane] =
                            from[r * (kPitch / 2)];
                    continue;
                }
#pragma unroll
                for (int i = 0; i < 4; i++)
                    q[i] = *reinterpret_cast<const uint4 *>(theirs + 8 * kPitch * i);
                if (c0 + kCols <= a.N) {
#pragma unroll
                    for (int i = 0; i < 4; i++)
                        if (on[i])
                            *reinterpret_cast<uint4 *>(to[i] + c0) = q[i];
                } else {
#pragma unroll
                    for (int i = 0; i < 4; i++)
                        if (on[i])
                            store8(to[i] - (col + 8 * (lane & 3)), c, a.N, a.vec_o, q[i]);
                }
            }
        }
        done += steps;
        tc_fence_before();
    }
    wait_copies<0>();
    tensor_end(t, 2 * kCols);
}

// ---------------------------------------------------------------- outer

struct OuterSide {
    const uint16_t *src;    // [n][C] by token
    long long ld;
    bool vec;
    int C, blocks;          // columns, blocks of kCols of them
    uint16_t *out;
};
struct OuterArgs {
    AdapterPlan p;
    OuterSide a, b;         // dA [L][r][K] from x and u, dB [L][N][r] from dy and h
    const uint16_t *u;      // [n][kParts][PAD] by place
    const uint16_t *h;      // [n][r] by token
    const float *scale;
    int L, r, splits, turns;    // turns: blocks of a CTA, one after another
    float *part;            // [splits][L][blocks of both][kCols][PAD]
    unsigned *tickets;      // [L][blocks of both]
};
constexpr int kOuterList = 16;      // steps whose tokens are at hand
// Tokens of a step, and steps: two CTAs an SM, each with two steps of 64 tokens on their way,
// or four of 32 where three parts of 64 ranks leave no room for three stages of 64.
template <typename T, int PAD>
constexpr int kOuterTokens = PAD == 64 && kParts<T> == 3 ? 32 : 64;
template <typename T, int PAD>
constexpr int kOuterStage = 128 * kOuterTokens<T, PAD> * (kCols / kBlk + kPartBlocks<T, PAD>);
template <typename T, int PAD>
constexpr int kOuterStages = kOuterTokens<T, PAD> == 32 ? 5 : 3;

// Sixteen ranks of a column from rank k on, at the end of a sum over tokens.
template <typename T>
__device__ __forceinline__ void put_outer(const OuterArgs &a, const OuterSide &o, bool of_a,
                                          int adapter, int c, int k, const float (&v)[16])
{
    uint16_t *out = o.out + (long long)adapter * a.r * o.C;
    if (c >= o.C)
        return;
    if (of_a) {     // lanes are neighbours in c
#pragma unroll
        for (int e = 0; e < 16; e++)
            if (k + e < a.r)
                out[(long long)(k + e) * o.C + c] = bits(from_float<T>(v[e]));
        return;
    }
#pragma unroll
    for (int e = 0; e < 16; e += 8)
        if (k + e < a.r)
            *reinterpret_cast<uint4 *>(out + (long long)c * a.r + k + e) =
                make_uint4(pack2<T>(v[e], v[e + 1]), pack2<T>(v[e + 2], v[e + 3]),
                           pack2<T>(v[e + 4], v[e + 5]), pack2<T>(v[e + 6], v[e + 7]));
}

// The sum over an adapter's tokens of kCols columns (the product's rows) times all ranks.
// Both operands are read along their rows: the tokens are the contraction.
template <typename T, int PAD, bool LONG>
__global__ void __launch_bounds__(kThreads, PAD <= 64 ? 2 : 1) adapter_outer_kernel(OuterArgs a)
{
    __shared__ TensorSmem ts;
    constexpr int tokens = kOuterTokens<T, PAD>;
    __shared__ int toks[kOuterList * tokens];
    __shared__ int last;
    pdl_wait();
    const int adapter = blockIdx.y, split = blockIdx.z, all_blocks = a.a.blocks + a.b.blocks;
    const int first = blockIdx.x * a.turns, stop = min(first + a.turns, all_blocks);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int lo = a.p.off[adapter], count = a.p.off[adapter + 1] - lo;
    const int all = (count + tokens - 1) / tokens;
    const int begin = (int)((long long)all * split / a.splits);
    const int steps = (int)((long long)all * (split + 1) / a.splits) - begin;
    const int c = 32 * warp + lane;
    const float scale = a.scale ? a.scale[adapter] : 1.f;
    if (count == 0) {
        const float zero[16] = {};
        for (int blk = first; blk < stop && split == 0 && warp < 4; blk++) {
            const bool of_a = blk < a.a.blocks;
            for (int k = 0; k < PAD; k += 16)
                put_outer<T>(a, of_a ? a.a : a.b, of_a, adapter,
                             kCols * (of_a ? blk : blk - a.a.blocks) + c, k, zero);
        }
        return;
    }
    constexpr int parts = kParts<T>;
    constexpr uint32_t cols = tmem_cols((LONG ? parts + 1 : parts) * PAD);
    const Tensor t = tensor_begin(ts, cols);
    const uint32_t smem = smem_base();
    constexpr int stage_bytes = kOuterStage<T, PAD>;
    using X = Rows<kCols / 8, tokens>;
    using V = Rows<PAD / 8, tokens>;
    const X xr(128 * tokens);
    const V vr(128 * tokens);
    uint32_t uses = 0;
    const float2 lift =
        kLifted<T> ? lift_of(__uint_as_float(a.p.most[adapter])) : make_float2(1.f, 1.f);
    for (int blk = first; blk < stop; blk++) {
        const bool of_a = blk < a.a.blocks;
        const OuterSide &o = of_a ? a.a : a.b;
        const int c0 = kCols * (of_a ? blk : blk - a.a.blocks);
        const uint16_t *src = o.src + c0 + 8 * xr.chunk;
        const bool whole = o.vec && c0 + kCols <= o.C;
        const int rank_bytes = 8 * vr.chunk < a.r ? 16 : 0;     // 0 for the ranks behind the last
        const uint16_t *ranks = rank_bytes ? a.h + 8 * vr.chunk : a.h;
        const auto fetch = [&](int i, int stage) {
            const int s0 = (begin + i) * tokens;
            if (i % kOuterList == 0) {      // the list that the next steps take their tokens from
                for (int j = threadIdx.x; j < kOuterList * tokens; j += kThreads)
                    toks[j] = s0 + j < count ? a.p.perm[lo + s0 + j] : -1;
                __syncthreads();
            }
            const int *list = toks + i % kOuterList * tokens;
            const uint32_t xs = smem + stage * stage_bytes + xr.at;
            const uint32_t vs = smem + stage * stage_bytes + 128 * tokens * (kCols / kBlk);
            if (whole && s0 + tokens <= count) {
#pragma unroll
                for (int j = 0; j < X::kPasses; j++)
                    copy16(xs + X::kNext * j, src + list[xr.row + X::kPass * j] * o.ld, 16);
            } else {                        // 0 behind the last token
#pragma unroll 1
                for (int j = 0; j < X::kPasses; j++) {
                    const int tok = list[xr.row + X::kPass * j];
                    fetch8(xs + X::kNext * j, o.src + max(tok, 0) * o.ld, c0 + 8 * xr.chunk,
                           tok >= 0 ? o.C : 0, o.vec);
                }
            }
            if (!vr.on)
                return;
            if (of_a) {                     // u in its parts, side by side
                const uint16_t *from = a.u + (long long)(lo + s0 + vr.row) * parts * PAD + 8 * vr.chunk;
#pragma unroll
                for (int j = 0; j < V::kPasses; j++) {
                    const bool in = s0 + vr.row + V::kPass * j < count;
#pragma unroll
                    for (int p = 0; p < parts; p++) {
                        const int chunk = p * (PAD / 8) + vr.chunk;
                        copy16(vs + (chunk >> 3) * (128 * tokens) +
                                   sw128_at(vr.row + V::kPass * j, chunk & 7),
                               in ? from + (V::kPass * j * parts + p) * PAD : a.u, in ? 16 : 0);
                    }
                }
            } else {
#pragma unroll
                for (int j = 0; j < V::kPasses; j++) {
                    const int tok = list[vr.row + V::kPass * j];
                    copy16(vs + vr.at + V::kNext * j, ranks + (long long)max(tok, 0) * a.r,
                           tok >= 0 ? rank_bytes : 0);
                }
            }
        };
        // the parts' sums lie side by side too, at most 256 columns an instruction
        const auto multiply = [&](int stage, bool first) {
            const uint32_t at = smem + stage * stage_bytes, vs = at + 128 * tokens * (kCols / kBlk);
            const uint64_t da = sw128_desc_mn(at, 128 * tokens);
            for (int n0 = 0, all = of_a ? parts * PAD : PAD; n0 < all; n0 += 256) {
                const uint32_t idesc =
                    (1u << 4) | (std::is_same_v<T, __nv_bfloat16> ? (1u << 7 | 1u << 10) : 0u) |
                    ((uint32_t)(min(all - n0, 256) >> 3) << 17) | (8u << 24) | kMnMajorA | kMnMajorB;
                const uint64_t db = sw128_desc_mn(vs + n0 / kBlk * (128 * tokens), 128 * tokens);
#pragma unroll
                for (int k = 0; k < tokens / 16; k++)
                    umma_ss(t.tmem + n0, da + 128 * k, db + 128 * k, idesc, !first || k);
            }
        };
        if (blk > first)
            __syncthreads();        // the list of tokens is taken again
        const uint32_t sums = t.tmem + ((uint32_t)(32 * (warp & 3)) << 16);
        const uint32_t kept = sums + parts * PAD;
        const int block = adapter * all_blocks + blk;
        const long long slots = (long long)a.L * all_blocks;
        constexpr int chain = kChain / tokens;
        int s0 = 0;
        do {                        // once without steps: 0
            if (LONG && s0 > 0)
                __syncthreads();    // the list of tokens is taken again
            const bool more = LONG && s0 + chain < steps;
            const auto fetch_from = [&](int i, int stage) { fetch(s0 + i, stage); };
            contract<kOuterStages<T, PAD>>(t, more ? chain : steps - s0, uses,
                                           more || blk + 1 < stop, fetch_from, multiply);
            const bool failed = *t.gave_up;
            if (warp < 4)
#pragma unroll 1
                for (int k = 0; k < PAD; k += 16) {
                    float v[16];
                    tmem_ld16(sums + k, v);
                    if (of_a) {
                        float weight = lift.y;
#pragma unroll
                        for (int e = 0; e < 16; e++)
                            v[e] *= weight;
#pragma unroll
                        for (int p = 1; p < parts; p++) {
                            float rest[16];
                            tmem_ld16(sums + p * PAD + k, rest);
                            weight /= kNext<T>;
#pragma unroll
                            for (int e = 0; e < 16; e++)
                                v[e] = fmaf(rest[e], weight, v[e]);
                        }
                    }
                    add_kept(v, kept + k, LONG && s0 > 0);
                    if (more) {
                        tmem_st16(kept + k, v);
                        continue;
                    }
#pragma unroll
                    for (int e = 0; e < 16; e++)
                        v[e] = failed ? NAN : steps > 0 ? v[e] : 0.f;
                    if (a.splits == 1) {
#pragma unroll
                        for (int e = 0; e < 16; e++)
                            v[e] *= scale;
                        put_outer<T>(a, o, of_a, adapter, c0 + c, k, v);
                        __syncwarp();       // the next load is the whole warp's
                        continue;
                    }
                    float4 *p = reinterpret_cast<float4 *>(
                        a.part + ((split * slots + block) * kCols + c) * PAD + k);
#pragma unroll
                    for (int q = 0; q < 4; q++)
                        p[q] = make_float4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
                }
            tc_fence_before();      // the next chain's products write where this one's were read
            s0 += chain;
        } while (LONG && s0 < steps);
        if (a.splits == 1)
            continue;
        __threadfence();
        __syncthreads();
        if (threadIdx.x == 0)
            last = atomicAdd(a.tickets + block, 1u) == a.splits - 1u;
        __syncthreads();
        if (!last)
            continue;
        __threadfence();
        for (int i = threadIdx.x; i < kCols * (PAD / 16); i += kThreads) {
            const int col = i % kCols, k = i / kCols * 16;
            float v[16] = {};
            for (int s = 0; s < a.splits; s++) {
                const float4 *p = reinterpret_cast<const float4 *>(
                    a.part + ((s * slots + block) * kCols + col) * PAD + k);
#pragma unroll
                for (int q = 0; q < 4; q++) {
                    const float4 d = __ldcg(p + q);
                    v[4 * q] += d.x, v[4 * q + 1] += d.y, v[4 * q + 2] += d.z, v[4 * q + 3] += d.w;
                }
            }
#pragma unroll
            for (int e = 0; e < 16; e++)
                v[e] *= scale;
            put_outer<T>(a, o, of_a, adapter, c0 + col, k, v);
        }
    }
    tensor_end(t, cols);
}

// What the expansion leaves of u, where none is asked for: a CTA has a tile.
template <typename T, int PAD>
__global__ void __launch_bounds__(kThreads) adapter_split_kernel(AdapterPlan p, int L,
                                                                 const float *mid, uint16_t *parts)
{
    pdl_enter();
    if ((int)blockIdx.x >= *p.n_tiles)
        return;
    const int4 tile = p.tiles[blockIdx.x];
    if (tile.x == L)
        return;
    const float lift = lift_of(__uint_as_float(p.most[tile.x])).x;
    for (int i = threadIdx.x; i < tile.z * (PAD / 8); i += kThreads) {
        const long long place = tile.y + i / (PAD / 8);
        const int k = 8 * (i % (PAD / 8));
        float u[8];
        load8(u, mid + place * PAD + k, true);
        put_lifted<T, PAD>(parts, place, k, u, lift);
    }
}

// ---------------------------------------------------------------- host

// A kernel with more dynamic shared memory than the default.
template <typename... P, typename A>
cudaError_t launch_wide(void (*kernel)(P...), dim3 grid, int smem, cudaStream_t st, const A &a,
                        int threads = kThreads)
{
    const cudaError_t e =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    return e != cudaSuccess ? e : launch_pdl(kernel, grid, dim3(threads), smem, st, a);
}

template <typename T, bool BY_ROW, int PAD>
cudaError_t launch_shrink(const ShrinkArgs &a, int tiles, cudaStream_t st)
{
    const bool chains = a.K > (long long)kOneChain * a.slices;
    return launch_wide(chains ? adapter_shrink_kernel<T, BY_ROW, PAD, true>
                              : adapter_shrink_kernel<T, BY_ROW, PAD, false>,
                       dim3(tiles, a.slices),
                       kShrinkStages * kShrinkStage<BY_ROW, PAD> + kSmemSlack, st, a);
}

template <typename T, bool BY_ROW, int PAD>
cudaError_t launch_expand(const ExpandArgs &a, int tiles, int sms, cudaStream_t st)
{
    const long long total = (long long)((a.N + kCols - 1) / kCols) * tiles;
    // as many CTAs as run at once
    return launch_wide(adapter_expand_kernel<T, BY_ROW, PAD>,
                       dim3((unsigned)std::min(total, (long long)sms)),
                       kExpandSmem<T, BY_ROW, PAD>, st, a, kExpandThreads);
}

bool vec_rows(const void *p, long long ld, int n)
{
    return (uintptr_t)p % 16 == 0 && (n == 1 || ld % 8 == 0);
}

const uint16_t *half_words(const void *p) { return static_cast<const uint16_t *>(p); }

// Where the parts lie: behind fp32 values where those are kept.
template <typename T, int PAD>
uint16_t *parts_of(const AdapterWorkspace &w, int n)
{
    return reinterpret_cast<uint16_t *>(w.mid + (kLifted<T> ? (size_t)n * PAD : 0));
}

template <typename T, int PAD>
cudaError_t run_adapter(const AdapterCall &c, cudaStream_t st)
{
    const int tiles = adapter_tiles(c.n, c.L);
    const ShrinkArgs s = {c.w.p, half_words(c.x), c.ldx, half_words(c.A), c.n, c.L, c.K, c.r,
                          c.w.slices, vec_rows(c.x, c.ldx, c.n), c.K % 8 == 0, c.w.part, c.w.mid,
                          parts_of<T, PAD>(c.w, c.n), static_cast<uint16_t *>(c.h), false};
    const cudaError_t e = launch_shrink<T, false, PAD>(s, tiles, st);
    if (e != cudaSuccess)
        return e;
    const ExpandArgs x = {c.w.p, c.w.mid, kLifted<T> ? nullptr : s.parts, half_words(c.B), c.scale, half_words(c.base), c.ldb,
                          static_cast<uint16_t *>(c.out), c.ldo, c.L, c.N, c.r, true,
                          vec_rows(c.base, c.ldb, c.n), vec_rows(c.out, c.ldo, c.n)};
    return launch_expand<T, false, PAD>(x, tiles, c.sms, st);
}

template <typename T, int PAD>
cudaError_t run_adapter_grad(const AdapterGradCall &c, cudaStream_t st)
{
    const int tiles = adapter_tiles(c.n, c.L);
    uint16_t *parts = parts_of<T, PAD>(c.w, c.n);
    const ShrinkArgs s = {c.w.p, half_words(c.dy), c.lddy, half_words(c.B), c.n, c.L, c.N, c.r,
                          c.w.slices, vec_rows(c.dy, c.lddy, c.n), true, c.w.part, c.w.mid, parts,
                          nullptr, kLifted<T> && c.dA};
    cudaError_t e = launch_shrink<T, true, PAD>(s, tiles, st);
    if (e != cudaSuccess)
        return e;
    if (c.dx) {
        const ExpandArgs x = {c.w.p, c.w.mid, kLifted<T> && !c.dA ? nullptr : parts, half_words(c.A), c.scale, half_words(c.base), c.ldb,
                              static_cast<uint16_t *>(c.dx), c.lddx, c.L, c.K, c.r,
                              c.K % 8 == 0, vec_rows(c.base, c.ldb, c.n),
                              vec_rows(c.dx, c.lddx, c.n)};
        e = launch_expand<T, true, PAD>(x, tiles, c.sms, st);
        if (e != cudaSuccess)
            return e;
    }
    if (kLifted<T> && c.dA && !c.dx) {
        e = launch_pdl(adapter_split_kernel<T, PAD>, dim3(tiles), dim3(kThreads), 0, st, c.w.p, c.L,
                       c.w.mid, parts);
        if (e != cudaSuccess)
            return e;
    }
    if (!c.dA && !c.dB)
        return e;
    OuterArgs o{};
    o.p = c.w.p;
    o.scale = c.scale;
    o.L = c.L;
    o.r = c.r;
    o.splits = c.w.splits;
    o.part = c.w.outer_part;
    o.tickets = c.w.outer_tickets;
    o.u = parts;
    o.h = half_words(c.h);
    if (c.dA)
        o.a = {half_words(c.x), c.ldx, vec_rows(c.x, c.ldx, c.n), c.K, (c.K + kCols - 1) / kCols,
               static_cast<uint16_t *>(c.dA)};
    if (c.dB)
        o.b = {half_words(c.dy), c.lddy, vec_rows(c.dy, c.lddy, c.n), c.N,
               (c.N + kCols - 1) / kCols, static_cast<uint16_t *>(c.dB)};
    // Several blocks a CTA once they fill the SMs' two places eight times: few tokens each, so
    // that a CTA's start weighs.  Measured, one block a CTA against this: 64 adapters of 4096 x
    // 4096, 500 tokens (rank 16) 85 and 74 us, 8192 tokens (rank 32) 147 and 140; 256 adapters
    // of 2048 x 2048, 9000 tokens (rank 16) 170 and 141.  With fewer than eight, unequal
    // adapters end apart: the second took 148 where it took 137 with eight.
    const int blocks = o.a.blocks + o.b.blocks;
    o.turns = std::max(1, (int)std::min(8LL, (long long)blocks * c.L / (8 * c.sms)));
    return launch_wide(c.n > kOneChain * o.splits ? adapter_outer_kernel<T, PAD, true>
                                                  : adapter_outer_kernel<T, PAD, false>,
                       dim3((blocks + o.turns - 1) / o.turns, c.L, o.splits),
                       kOuterStages<T, PAD> * kOuterStage<T, PAD> + kSmemSlack, st, o);
}

template <typename T>
cudaError_t run_adapter(const AdapterCall &c, cudaStream_t st)
{
    switch (rank_pad(c.r)) {
    case 16: return run_adapter<T, 16>(c, st);
    case 32: return run_adapter<T, 32>(c, st);
    case 64: return run_adapter<T, 64>(c, st);
    default: return run_adapter<T, 128>(c, st);
    }
}
template <typename T>
cudaError_t run_adapter_grad(const AdapterGradCall &c, cudaStream_t st)
{
    switch (rank_pad(c.r)) {
    case 16: return run_adapter_grad<T, 16>(c, st);
    case 32: return run_adapter_grad<T, 32>(c, st);
    case 64: return run_adapter_grad<T, 64>(c, st);
    default: return run_adapter_grad<T, 128>(c, st);
    }
}

}  // namespace

}  // namespace qe
