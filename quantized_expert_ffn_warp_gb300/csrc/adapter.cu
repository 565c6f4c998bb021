// Low-rank adapters of many requests beside one projection, and their gradients.
// Token t has adapter a = ids[t] (A_a [r][K], B_a [N][r], scale s_a), or none:
//   h = A_a x,  out = base + s_a B_a h
//   u = B_a^T dy,  dx = base + s_a A_a^T u
//   dA_a = s_a sum_t u_t x_t^T,  dB_a = s_a sum_t dy_t h_t^T   over the adapter's tokens
//
// A plan kernel sorts the tokens by adapter (stably) and cuts each adapter's tokens
// into tiles of 128.  "Shrink" contracts a tile with the long side of a matrix, "expand"
// goes back to full width and adds base, "outer" sums over an adapter's tokens.  All
// three are bound by the activations' bytes (r operations per byte and less), so the
// products go to the tcgen05 tensor cores, which leave the warps to the copies: rows of
// 128 bytes are gathered token by token with asynchronous copies into the swizzled
// layout, and the descriptors take either side of a matrix as the contraction's, so that
// nothing is transposed.
// h and u are held as the sum of two values of the activations' type: one would add a
// rounding of 2^-9 (bf16) to the delta and to dA, and the second product is hidden
// behind the copies.
#include <algorithm>

#include "args.cuh"
#include "tcgen05.cuh"
#include "vec.cuh"

namespace qe {

namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kTile = 128;              // tokens of a tile
constexpr int kBlk = 64;                // values of a 128-byte row: the step of a contraction
constexpr int kMaxTokens = 1 << 20, kMaxAdapters = 1024, kMaxRank = 128, kMaxWidth = 1 << 20;
constexpr int kMaxSlices = 16;          // CTAs that share a tile's contraction

__host__ __device__ constexpr int rank_pad(int r) { return (r + 15) / 16 * 16; }

struct Plan {
    int *off;           // [L + 2] first token of an adapter in perm; then those without one
    int *perm;          // [n] tokens in the order of their adapters
    int4 *tiles;        // (adapter, first place in perm, tokens, -); L: none
    int *n_tiles;
    unsigned *tickets;  // parts that have arrived: of tiles, then of outer blocks
};

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

// ---------------------------------------------------------------- plan

// One CTA: a stable counting sort.  A warp owns a run of consecutive tokens.
__global__ void __launch_bounds__(1024) adapter_plan_kernel(const int32_t *__restrict__ ids, int n,
                                                           int L, Plan p, int max_tickets)
{
    extern __shared__ int sm[];
    const int G = L + 1;        // the last group has no adapter
    int *hist = sm, *first = sm + 32 * G, *tile0 = first + G + 1;
    pdl_enter();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int i = threadIdx.x; i < 32 * G; i += 1024)
        hist[i] = 0;
    for (int i = threadIdx.x; i < max_tickets; i += 1024)
        p.tickets[i] = 0;
    __syncthreads();
    const int per = ((n + 31) / 32 + 31) / 32 * 32;
    const int lo = min(n, warp * per), hi = min(n, lo + per);
    int *mine = hist + warp * G;
    constexpr int U = 8;
    // calls f(token, group, lanes of the same group) for the warp's tokens, 32 at a time
    const auto walk = [&](auto f) {
        for (int b = lo; b < hi; b += 32 * U) {
            int g[U];
#pragma unroll
            for (int i = 0; i < U; i++) {
                const int t = b + 32 * i + lane;
                g[i] = -1;
                if (t < hi) {
                    const int a = ids[t];
                    g[i] = a >= 0 && a < L ? a : L;
                }
            }
#pragma unroll
            for (int i = 0; i < U; i++)
                if (b + 32 * i < hi) {
                    f(b + 32 * i + lane, g[i], __match_any_sync(0xffffffffu, g[i]));
                    __syncwarp();
                }
        }
    };
    walk([&](int, int g, unsigned same) {
        if (g >= 0 && lane == __ffs(same) - 1)
            mine[g] += __popc(same);
    });
    __syncthreads();
    for (int g = threadIdx.x; g < G; g += 1024) {
        int run = 0;
        for (int w = 0; w < 32; w++) {
            const int c = hist[w * G + g];
            hist[w * G + g] = run;
            run += c;
        }
        first[g] = run;
    }
    __syncthreads();
    if (warp == 0) {
        int tok = 0, tile = 0;
        for (int b = 0; b < G; b += 32) {
            const int c = b + lane < G ? first[b + lane] : 0, k = (c + kTile - 1) / kTile;
            int sc = c, sk = k;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int uc = __shfl_up_sync(0xffffffffu, sc, d);
                const int uk = __shfl_up_sync(0xffffffffu, sk, d);
                if (lane >= d) {
                    sc += uc;
                    sk += uk;
                }
            }
            if (b + lane < G) {
                first[b + lane] = tok + sc - c;
                tile0[b + lane] = tile + sk - k;
            }
            tok += __shfl_sync(0xffffffffu, sc, 31);
            tile += __shfl_sync(0xffffffffu, sk, 31);
        }
        if (lane == 0) {
            first[G] = n;
            tile0[G] = tile;
            *p.n_tiles = tile;
        }
    }
    __syncthreads();
    for (int g = threadIdx.x; g <= G; g += 1024)
        p.off[g] = first[g];
    for (int i = threadIdx.x; i < tile0[G]; i += 1024) {
        int a = 0, b = G - 1;       // the last group whose tiles start at i or before
        while (a < b) {
            const int mid = (a + b + 1) / 2;
            if (tile0[mid] <= i)
                a = mid;
            else
                b = mid - 1;
        }
        const int start = first[a] + (i - tile0[a]) * kTile;
        p.tiles[i] = make_int4(a, start, min(kTile, first[a + 1] - start), 0);
    }
    walk([&](int t, int g, unsigned same) {
        if (g >= 0)
            p.perm[first[g] + mine[g] + __popc(same & ((1u << lane) - 1))] = t;
        __syncwarp();       // before the leaders count these tokens
        if (g >= 0 && lane == __ffs(same) - 1)
            mine[g] += __popc(same);
    });
}

// ---------------------------------------------------------------- the tensor core

// What a CTA needs around its products.
struct Tensor {
    uint32_t bars;          // barriers, one for each stage
    uint32_t tmem;
    volatile int *gave_up;
};
constexpr int kStages = 4;      // at most
struct TensorSmem {
    uint64_t bar[kStages];
    uint32_t tmem;
    int gave_up;
};

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
    return n <= 32 ? 32 : n <= 64 ? 64 : n <= 128 ? 128 : 256;
}
// 128-byte rows that hold `r` values.
__host__ __device__ constexpr int row_blocks(int r) { return (r + kBlk - 1) / kBlk; }

// A multi-stage contraction: fetch(i, stage) starts the copies of step i, multiply(stage,
// first) issues its products in one elected thread.  Copies of the steps ahead are under
// way while a step is multiplied; a stage is filled again when its products are done.
template <int S, typename F, typename M>
__device__ __forceinline__ void contract(const Tensor &t, int steps, F fetch, M multiply)
{
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
                tensor_wait(t, before, (i - 1) / S);
            fetch(i + S - 1, before);
        }
        commit_copies();
        stage = stage + 1 == S ? 0 : stage + 1;
    }
    wait_copies<0>();
    if (steps > 0)
        tensor_wait(t, (steps - 1) % S, (steps - 1) / S);
    tc_fence_after();
}

// A call's dynamic shared memory from a 1024-byte boundary on, as the swizzle needs.
__device__ __forceinline__ uint32_t smem_base()
{
    extern __shared__ uint8_t adapter_smem[];
    return (saddr(adapter_smem) + 1023) & ~1023u;
}
constexpr int kSmemSlack = 1024;

// ---------------------------------------------------------------- shrink

struct ShrinkArgs {
    Plan p;
    const uint16_t *x;      // [n][K]
    long long ldx;
    const uint16_t *w;      // [L][r][K], or (BY_ROW) [L][K][r]
    int n, L, K, r, slices;
    bool vec_x, vec_w;
    float *part;            // [slices][n][rank_pad] partial sums
    uint16_t *pair;         // [n][2][rank_pad] the result in two parts, in perm's order
    uint16_t *h;            // [n][r], or null
};

template <typename T>
__device__ __forceinline__ uint16_t bits(T v)
{
    return *reinterpret_cast<const uint16_t *>(&v);
}

// Four of a token's results from rank k on: two parts at its place, and h.
template <typename T>
__device__ __forceinline__ void put_results(const ShrinkArgs &a, int place, int token, int k,
                                            const float (&v)[4])
{
    const int pad = rank_pad(a.r);
    float rest[4];
#pragma unroll
    for (int e = 0; e < 4; e++) {
        const float f = to_float<T>(from_float<T>(v[e]));
        // an infinity or a NaN has no remainder
        rest[e] = fabsf(f) <= 3.4e38f ? v[e] - f : 0.f;
    }
    const uint2 hi = make_uint2(pack2<T>(v[0], v[1]), pack2<T>(v[2], v[3]));
    uint16_t *row = a.pair + (long long)place * 2 * pad + k;
    *reinterpret_cast<uint2 *>(row) = hi;
    *reinterpret_cast<uint2 *>(row + pad) =
        make_uint2(pack2<T>(rest[0], rest[1]), pack2<T>(rest[2], rest[3]));
    if (a.h && k < a.r)
        *reinterpret_cast<uint2 *>(a.h + (long long)token * a.r + k) = hi;
}

constexpr int kShrinkStages = 4;
template <bool BY_ROW>
__host__ __device__ constexpr int shrink_stage(int r)
{
    return 128 * kTile + (BY_ROW ? 128 * kBlk * row_blocks(rank_pad(r)) : 128 * rank_pad(r));
}

// A tile's tokens (the product's rows) times all ranks.  The slices' sums are added by
// whichever CTA of a tile arrives last, in the slices' order.
template <typename T, bool BY_ROW>
__global__ void __launch_bounds__(kThreads, 2) adapter_shrink_kernel(ShrinkArgs a)
{
    __shared__ TensorSmem ts;
    __shared__ int last;
    pdl_enter();
    if ((int)blockIdx.x >= *a.p.n_tiles)
        return;
    const int4 tile = a.p.tiles[blockIdx.x];
    const int slice = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int pad = rank_pad(a.r);
    if (tile.x == a.L) {        // no adapter
        if (slice == 0 && a.h)
            for (int i = threadIdx.x; i < tile.z * a.r; i += kThreads)
                a.h[(long long)a.p.perm[tile.y + i / a.r] * a.r + i % a.r] = 0;
        return;
    }
    const uint32_t cols = tmem_cols(pad);
    const Tensor t = tensor_begin(ts, cols);
    const uint16_t *w = a.w + (long long)tile.x * a.r * a.K;
    const int blocks = (a.K + kBlk - 1) / kBlk;
    const int begin = (int)((long long)blocks * slice / a.slices);
    const int end = (int)((long long)blocks * (slice + 1) / a.slices);
    const uint32_t smem = smem_base();
    const int stage_bytes = shrink_stage<BY_ROW>(a.r);
    // thread's chunk of eight values: of tokens threadIdx.x / 8, + 32, .., and of the matrix
    const int row = threadIdx.x >> 3, chunk = threadIdx.x & 7;
    const uint16_t *src[4];
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const int at = row + 32 * i;
        src[i] = a.x + (long long)a.p.perm[tile.y + (at < tile.z ? at : 0)] * a.ldx;
    }
    const int wide = pad / 8;       // BY_ROW: chunks of a row
    const auto fetch = [&](int i, int stage) {
        const int k0 = (begin + i) * kBlk, k = k0 + 8 * chunk;
        const uint32_t at = smem + stage * stage_bytes, mat = at + 128 * kTile;
#pragma unroll
        for (int j = 0; j < 4; j++)
            if (row + 32 * j < tile.z)
                fetch8(at + sw128_at(row + 32 * j, chunk), src[j], k, a.K, a.vec_x);
        if constexpr (!BY_ROW) {
            for (int rank = row; rank < pad; rank += 32)    // 0 for the ranks behind the last
                fetch8(mat + sw128_at(rank, chunk), rank < a.r ? w + (long long)rank * a.K : w, k,
                       rank < a.r ? a.K : 0, a.vec_w);
        } else {
            for (int j = threadIdx.x; j < kBlk * wide; j += kThreads) {
                const int kr = j / wide, c = j % wide;
                const bool in = k0 + kr < a.K && 8 * c < a.r;
                copy16(mat + (c >> 3) * (128 * kBlk) + sw128_at(kr, c & 7),
                       in ? w + (long long)(k0 + kr) * a.r + 8 * c : w, in ? 16 : 0);
            }
        }
    };
    const uint32_t idesc =
        idesc_f16(pad, std::is_same_v<T, __nv_bfloat16>) | (BY_ROW ? kMnMajorB : 0);
    const auto multiply = [&](int stage, bool first) {
        const uint32_t at = smem + stage * stage_bytes, mat = at + 128 * kTile;
        const uint64_t da = sw128_desc(at);
        const uint64_t db = BY_ROW ? sw128_desc_mn(mat, 128 * kBlk) : sw128_desc(mat);
#pragma unroll
        for (int k = 0; k < 4; k++)
            umma_ss(t.tmem, da + 2 * k, db + (BY_ROW ? 128 : 2) * k, idesc, !first || k);
    };
    contract<kShrinkStages>(t, end - begin, fetch, multiply);
    const bool failed = *t.gave_up;
    const int at = 32 * warp + lane, place = tile.y + at;
    if (warp < 4) {
        const int token = at < tile.z ? a.p.perm[place] : 0;
        for (int c = 0; c < pad; c += 16) {
            float v[16];
            tmem_ld16(t.tmem + ((uint32_t)(32 * warp) << 16) + c, v);
            if (at >= tile.z)
                continue;
#pragma unroll
            for (int q = 0; q < 4; q++) {
                float d[4];
#pragma unroll
                for (int e = 0; e < 4; e++)
                    d[e] = failed ? NAN : v[4 * q + e];
                if (a.slices == 1)
                    put_results<T>(a, place, token, c + 4 * q, d);
                else
                    *reinterpret_cast<float4 *>(
                        a.part + ((long long)slice * a.n + place) * pad + c + 4 * q) =
                        make_float4(d[0], d[1], d[2], d[3]);
            }
        }
    }
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
    for (int i = threadIdx.x; i < tile.z * (pad / 4); i += kThreads) {
        const int place = tile.y + i / (pad / 4), k = i % (pad / 4) * 4;
        float v[4] = {};
        for (int s = 0; s < a.slices; s++) {
            const float4 q = __ldcg(reinterpret_cast<const float4 *>(
                a.part + ((long long)s * a.n + place) * pad + k));
            v[0] += q.x, v[1] += q.y, v[2] += q.z, v[3] += q.w;
        }
        put_results<T>(a, place, a.p.perm[place], k, v);
    }
}

// ---------------------------------------------------------------- expand

struct ExpandArgs {
    Plan p;
    const uint16_t *pair;   // [n][2][rank_pad]
    const uint16_t *w;      // [L][N][r], or (BY_ROW) [L][r][N]
    const float *scale;     // [L] or null
    const uint16_t *base;   // [n][N] or null
    long long ldb;
    uint16_t *out;          // [n][N]
    long long ldo;
    int L, N, r, steps;     // steps: blocks of kCols columns of a CTA
    bool vec_w, vec_b, vec_o;
};
constexpr int kCols = 128;

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

// h in 128-byte rows, the upper parts and then the lower: side by side if both fit.
__host__ __device__ constexpr int pair_blocks(int pad)
{
    return 2 * pad <= kBlk ? 1 : 2 * row_blocks(pad);
}
template <bool BY_ROW>
__host__ __device__ constexpr int matrix_bytes(int pad)
{
    return BY_ROW ? 2 * kCols * pad : 128 * kCols * row_blocks(pad);
}
template <bool BY_ROW>
constexpr int expand_smem(int pad)
{
    return 128 * kTile * pair_blocks(pad) + 2 * matrix_bytes<BY_ROW>(pad) + 4096 * kWarps +
           kSmemSlack;
}

// A tile's tokens (the product's rows) times columns.  The next columns' matrix is copied
// while a block's sums leave tensor memory; these pass through a warp's shared memory,
// where a lane finds eight neighbours of a token's row, and meet base, loaded before
// the product is waited for.
template <typename T, bool BY_ROW>
__global__ void __launch_bounds__(kThreads, 2) adapter_expand_kernel(ExpandArgs a)
{
    __shared__ TensorSmem ts;
    pdl_enter();
    if ((int)blockIdx.x >= *a.p.n_tiles)
        return;
    const int4 tile = a.p.tiles[blockIdx.x];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int first = blockIdx.y * a.steps * kCols;
    const int stop = min(a.N, first + a.steps * kCols);
    if (tile.x == a.L) {        // no adapter: base, or 0
        if (a.out == a.base)
            return;
        for (int i = warp; i < tile.z; i += kWarps) {
            const long long tok = a.p.perm[tile.y + i];
            for (int c = first + 8 * lane; c < stop; c += 256)
                store8(a.out + tok * a.ldo, c, stop, a.vec_o,
                       a.base ? load8(a.base + tok * a.ldb, c, stop, a.vec_b)
                              : make_uint4(0, 0, 0, 0));
        }
        return;
    }
    const Tensor t = tensor_begin(ts, kCols);
    const int pad = rank_pad(a.r), wide = pad / 8, blocks = row_blocks(pad);
    const int chunks = a.r / 8;
    const bool side = 2 * pad <= kBlk;
    const uint32_t hs = smem_base(), mats = hs + 128 * kTile * pair_blocks(pad);
    const uint32_t mine = mats + 2 * matrix_bytes<BY_ROW>(pad) + 4096 * warp;
    // h: chunk c of part p of a row
    for (int i = threadIdx.x; i < tile.z * 2 * wide; i += kThreads) {
        const int row = i / (2 * wide), c = i % (2 * wide), part = c >= wide;
        const int at = side ? c : c - part * wide + part * 8 * blocks;
        copy16(hs + (at >> 3) * (128 * kTile) + sw128_at(row, at & 7),
               a.pair + (long long)(tile.y + row) * 2 * pad + 8 * c, 16);
    }
    const uint16_t *w = a.w + (long long)tile.x * a.r * a.N;
    const float scale = a.scale ? a.scale[tile.x] : 1.f;
    const auto fetch = [&](int c0, int buffer) {
        const uint32_t mat = mats + buffer * matrix_bytes<BY_ROW>(pad);
        if constexpr (!BY_ROW) {    // rows of ranks, 0 behind the last
            for (int i = threadIdx.x; i < kCols * wide; i += kThreads) {
                const int col = i / wide, c = i % wide;
                const bool in = c0 + col < a.N && c < chunks;
                copy16(mat + (c >> 3) * (128 * kCols) + sw128_at(col, c & 7),
                       in ? w + (long long)(c0 + col) * a.r + 8 * c : w, in ? 16 : 0);
            }
        } else {                    // a row of columns for each rank, two blocks of 64
            for (int i = threadIdx.x; i < pad * (kCols / 8); i += kThreads) {
                const int rank = i / (kCols / 8), c = i % (kCols / 8);
                fetch8(mat + (c >> 3) * (128 * pad) + sw128_at(rank, c & 7),
                       rank < a.r ? w + (long long)rank * a.N : w, c0 + 8 * c,
                       rank < a.r ? a.N : 0, a.vec_w);
            }
        }
        commit_copies();
    };
    const uint32_t idesc =
        idesc_f16(kCols, std::is_same_v<T, __nv_bfloat16>) | (BY_ROW ? kMnMajorB : 0);
    // rows of the warp's pass: 8 i + lane / 4 of its 32, columns 8 (lane % 4) .. of 32
    const int quad = warp & 3, half = warp >> 2;
    long long base_at[4], out_at[4];
    bool on[4];
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const int at = 32 * quad + 8 * i + lane / 4;
        on[i] = at < tile.z;
        const long long tok = on[i] ? a.p.perm[tile.y + at] : 0;
        base_at[i] = tok * a.ldb;
        out_at[i] = tok * a.ldo;
    }
    fetch(first, 0);
    int step = 0;
    for (int c0 = first; c0 < stop; c0 += kCols, step++) {
        wait_copies<0>();
        fence_async_shared();
        tc_fence_before();
        __syncthreads();
        if (warp == 0) {
            tc_fence_after();
            if (elect_one()) {
                const uint32_t mat = mats + (step & 1) * matrix_bytes<BY_ROW>(pad);
                for (int part = 0; part < 2; part++)
                    for (int k = 0; k < pad / 16; k++) {
                        const int ka = side ? part * (pad / 16) + k : part * 4 * blocks + k;
                        const uint64_t da =
                            sw128_desc(hs + (ka >> 2) * (128 * kTile)) + 2 * (ka & 3);
                        const uint64_t db =
                            BY_ROW ? sw128_desc_mn(mat, 128 * pad) + 128 * k
                                   : sw128_desc(mat + (k >> 2) * (128 * kCols)) + 2 * (k & 3);
                        umma_ss(t.tmem, da, db, idesc, part || k);
                    }
                umma_commit(t.bars);
            }
            __syncwarp();
        }
        if (c0 + kCols < stop)      // its buffer's products were waited for
            fetch(c0 + kCols, (step + 1) & 1);
        uint4 b[2][4];
#pragma unroll
        for (int p = 0; p < 2; p++) {
            const int c = c0 + 64 * half + 32 * p + 8 * (lane & 3);
#pragma unroll
            for (int i = 0; i < 4; i++) {
                b[p][i] = make_uint4(0, 0, 0, 0);
                if (a.base && on[i] && c < a.N)
                    b[p][i] = load8(a.base + base_at[i], c, a.N, a.vec_b);
            }
        }
        tensor_wait(t, 0, step);
        tc_fence_after();
        const float factor = *t.gave_up ? NAN : scale;
#pragma unroll
        for (int p = 0; p < 2; p++) {
            const int c = 64 * half + 32 * p;
            if (c0 + c >= a.N || 32 * quad >= tile.z)
                break;
#pragma unroll
            for (int j = 0; j < 2; j++) {
                float v[16];
                tmem_ld16(t.tmem + ((uint32_t)(32 * quad) << 16) + c + 16 * j, v);
#pragma unroll
                for (int q = 0; q < 4; q++)
                    asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(
                                     mine + sw128_at(lane, 4 * j + q)),
                                 "f"(v[4 * q]), "f"(v[4 * q + 1]), "f"(v[4 * q + 2]),
                                 "f"(v[4 * q + 3])
                                 : "memory");
            }
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 4; i++) {
                const int row = 8 * i + lane / 4;
                float v[8];
#pragma unroll
                for (int q = 0; q < 2; q++)
                    asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                                 : "=f"(v[4 * q]), "=f"(v[4 * q + 1]), "=f"(v[4 * q + 2]),
                                   "=f"(v[4 * q + 3])
                                 : "r"(mine + sw128_at(row, 2 * (lane & 3) + q))
                                 : "memory");
                if (!on[i])
                    continue;
                F2 d[4];
                unpack<T>(b[p][i], d);
#pragma unroll
                for (int e = 0; e < 4; e++)
                    d[e] = fma(f2(factor), f2(v[2 * e], v[2 * e + 1]), d[e]);
                store8(a.out + out_at[i], c0 + c + 8 * (lane & 3), a.N, a.vec_o, pack<T>(d));
            }
            __syncwarp();
        }
    }
    wait_copies<0>();
    tensor_end(t, kCols);
}

// ---------------------------------------------------------------- outer

struct OuterSide {
    const uint16_t *src;    // [n][C] by token
    long long ld;
    bool vec;
    int C, blocks;          // columns, blocks of kCols of them
    const uint16_t *v;      // ranks: of a token (h [n][r]), or of a place (pair)
    uint16_t *out;
};
struct OuterArgs {
    Plan p;
    OuterSide a, b;         // dA [L][r][K] from x and u, dB [L][N][r] from dy and h
    const float *scale;
    int L, r, splits;
    float *part;            // [splits][L][blocks of both][kCols][rank_pad]
    unsigned *tickets;      // [L][blocks of both]
};
constexpr int kOuterStages = 3, kOuterList = 16;    // steps whose tokens are at hand
__host__ __device__ constexpr int outer_stage(int pad)
{
    return 128 * kBlk * (kCols / kBlk + 2 * row_blocks(pad));
}

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
template <typename T>
__global__ void __launch_bounds__(kThreads, 2) adapter_outer_kernel(OuterArgs a)
{
    __shared__ TensorSmem ts;
    __shared__ int toks[kOuterList * kBlk];
    __shared__ int last;
    pdl_enter();
    const bool of_a = (int)blockIdx.x < a.a.blocks;
    const OuterSide &o = of_a ? a.a : a.b;
    const int c0 = kCols * (of_a ? blockIdx.x : blockIdx.x - a.a.blocks);
    const int adapter = blockIdx.y, split = blockIdx.z, pad = rank_pad(a.r), wide = pad / 8;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int lo = a.p.off[adapter], count = a.p.off[adapter + 1] - lo;
    const int all = (count + kBlk - 1) / kBlk;
    const int begin = (int)((long long)all * split / a.splits);
    const int steps = (int)((long long)all * (split + 1) / a.splits) - begin;
    const int c = 32 * warp + lane;
    const float scale = a.scale ? a.scale[adapter] : 1.f;
    if (count == 0) {
        const float zero[16] = {};
        if (split == 0 && warp < 4)
            for (int k = 0; k < pad; k += 16)
                put_outer<T>(a, o, of_a, adapter, c0 + c, k, zero);
        return;
    }
    const uint32_t cols = tmem_cols(pad);
    const Tensor t = tensor_begin(ts, cols);
    const uint32_t smem = smem_base();
    const int stage_bytes = outer_stage(pad), part_bytes = 128 * kBlk * row_blocks(pad);
    const int row = threadIdx.x >> 4, chunk = threadIdx.x & 15;
    const auto fetch = [&](int i, int stage) {
        const int s0 = (begin + i) * kBlk;
        if (i % kOuterList == 0) {      // the list that the next steps take their tokens from
            for (int j = threadIdx.x; j < kOuterList * kBlk; j += kThreads)
                toks[j] = s0 + j < count ? a.p.perm[lo + s0 + j] : -1;
            __syncthreads();
        }
        const int *list = toks + i % kOuterList * kBlk;
        const uint32_t at = smem + stage * stage_bytes, vs = at + 128 * kBlk * (kCols / kBlk);
#pragma unroll
        for (int j = 0; j < 4; j++) {   // 0 behind the last token
            const int r = row + 16 * j, tok = list[r];
            fetch8(at + (chunk >> 3) * (128 * kBlk) + sw128_at(r, chunk & 7),
                   o.src + max(tok, 0) * o.ld, c0 + 8 * chunk, tok >= 0 ? o.C : 0, o.vec);
        }
        for (int j = threadIdx.x; j < kBlk * wide; j += kThreads) {
            const int r = j / wide, c8 = j % wide, tok = list[r];
            const uint32_t dst = vs + (c8 >> 3) * (128 * kBlk) + sw128_at(r, c8 & 7);
            const bool in = tok >= 0 && 8 * c8 < a.r;
            if (of_a) {
                const uint16_t *v = in ? o.v + (long long)(lo + s0 + r) * 2 * pad + 8 * c8 : o.v;
                copy16(dst, v, in ? 16 : 0);
                copy16(dst + part_bytes, in ? v + pad : o.v, in ? 16 : 0);
            } else {
                copy16(dst, in ? o.v + (long long)tok * a.r + 8 * c8 : o.v, in ? 16 : 0);
            }
        }
    };
    const uint32_t idesc =
        idesc_f16(pad, std::is_same_v<T, __nv_bfloat16>) | kMnMajorA | kMnMajorB;
    const auto multiply = [&](int stage, bool first) {
        const uint32_t at = smem + stage * stage_bytes, vs = at + 128 * kBlk * (kCols / kBlk);
        const uint64_t da = sw128_desc_mn(at, 128 * kBlk);
        for (int part = 0; part < (of_a ? 2 : 1); part++) {
            const uint64_t db = sw128_desc_mn(vs + part * part_bytes, 128 * kBlk);
#pragma unroll
            for (int k = 0; k < kBlk / 16; k++)
                umma_ss(t.tmem, da + 128 * k, db + 128 * k, idesc, !first || part || k);
        }
    };
    contract<kOuterStages>(t, steps, fetch, multiply);
    const bool failed = *t.gave_up;
    const int block = adapter * (a.a.blocks + a.b.blocks) + blockIdx.x;
    const long long slots = (long long)a.L * (a.a.blocks + a.b.blocks);
    if (warp < 4)
        for (int k = 0; k < pad; k += 16) {
            float v[16];
            tmem_ld16(t.tmem + ((uint32_t)(32 * warp) << 16) + k, v);
#pragma unroll
            for (int e = 0; e < 16; e++)
                v[e] = failed ? NAN : steps > 0 ? v[e] : 0.f;
            if (a.splits == 1) {
#pragma unroll
                for (int e = 0; e < 16; e++)
                    v[e] *= scale;
                put_outer<T>(a, o, of_a, adapter, c0 + c, k, v);
                continue;
            }
            float4 *p = reinterpret_cast<float4 *>(
                a.part + ((split * slots + block) * kCols + c) * pad + k);
#pragma unroll
            for (int q = 0; q < 4; q++)
                p[q] = make_float4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
        }
    tensor_end(t, cols);
    if (a.splits == 1)
        return;
    __threadfence();
    __syncthreads();
    if (threadIdx.x == 0)
        last = atomicAdd(a.tickets + block, 1u) == a.splits - 1u;
    __syncthreads();
    if (!last)
        return;
    __threadfence();
    for (int i = threadIdx.x; i < kCols * (pad / 16); i += kThreads) {
        const int col = i % kCols, k = i / kCols * 16;
        float v[16] = {};
        for (int s = 0; s < a.splits; s++) {
            const float4 *p = reinterpret_cast<const float4 *>(
                a.part + ((s * slots + block) * kCols + col) * pad + k);
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

// ---------------------------------------------------------------- host

// Most tiles of n tokens: an adapter's tokens end with one that is not full.
int most_tiles(int n, int L) { return n / kTile + std::min(n, L + 1); }

// CTAs that share the contraction of a tile: two for each SM in all, each with two steps
// at least.  Asks no device, since the workspace depends on it.
int shrink_slices(int n, int L, int K)
{
    const int most = std::max(1, (K + kBlk - 1) / kBlk / 2);
    return std::max(1, std::min({304 / most_tiles(n, L), most, kMaxSlices}));
}
// CTAs that share an adapter's tokens, in the same way, each with four steps at least.
int outer_blocks(int K, int N) { return (K + kCols - 1) / kCols + (N + kCols - 1) / kCols; }
int outer_splits(int n, int L, int K, int N)
{
    const long long ctas = (long long)outer_blocks(K, N) * L;
    return (int)std::max(1LL, std::min({304 / ctas, (long long)n / (4 * kBlk), 8LL}));
}

struct Workspace {
    Plan p;
    int tickets;
    unsigned *outer_tickets;
    uint16_t *pair;
    float *part, *outer_part;
    size_t bytes;
};

Workspace adapter_ws(void *base, int n, int L, int r, int K, int N, bool grad)
{
    Workspace w{};
    size_t at = 0;
    const auto take = [&](size_t bytes) {
        char *p = static_cast<char *>(base) + at;
        at += (bytes + 255) / 256 * 256;
        return p;
    };
    const int slices = shrink_slices(n, L, grad ? N : K), splits = grad ? outer_splits(n, L, K, N) : 1;
    const int tiles = slices > 1 ? most_tiles(n, L) : 0;
    const int outer = splits > 1 ? L * outer_blocks(K, N) : 0;
    w.tickets = tiles + outer;
    w.p.n_tiles = reinterpret_cast<int *>(take(4));
    w.p.off = reinterpret_cast<int *>(take(4 * ((size_t)L + 2)));
    w.p.perm = reinterpret_cast<int *>(take(4 * (size_t)n));
    w.p.tiles = reinterpret_cast<int4 *>(take(16 * (size_t)most_tiles(n, L)));
    w.p.tickets = reinterpret_cast<unsigned *>(take(4 * (size_t)w.tickets));
    w.outer_tickets = w.p.tickets + tiles;
    w.pair = reinterpret_cast<uint16_t *>(take(4 * (size_t)n * rank_pad(r)));
    w.part = reinterpret_cast<float *>(
        take(slices > 1 ? 4 * (size_t)slices * n * rank_pad(r) : 0));
    w.outer_part = reinterpret_cast<float *>(
        take(4 * (size_t)splits * outer * kCols * rank_pad(r)));
    w.bytes = at;
    return w;
}

cudaError_t launch_plan(const int32_t *ids, int n, int L, const Workspace &w, cudaStream_t st)
{
    const size_t smem = sizeof(int) * (32 * ((size_t)L + 1) + 2 * ((size_t)L + 2));
    if (smem > 48 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(
            adapter_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
            (int)(sizeof(int) * (32 * (kMaxAdapters + 1) + 2 * (kMaxAdapters + 2))));
        if (e != cudaSuccess)
            return e;
    }
    return launch_pdl(adapter_plan_kernel, dim3(1), dim3(1024), smem, st, ids, n, L, w.p, w.tickets);
}

// A kernel with more dynamic shared memory than the default; `most` over all calls, since
// the attribute is shared by calls of other threads.
template <typename... P, typename A>
cudaError_t launch_wide(void (*kernel)(P...), dim3 grid, int smem, int most, cudaStream_t st,
                        const A &a)
{
    const cudaError_t e =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
    return e != cudaSuccess ? e : launch_pdl(kernel, grid, dim3(kThreads), smem, st, a);
}

template <typename T, bool BY_ROW>
cudaError_t launch_shrink(const ShrinkArgs &a, int tiles, cudaStream_t st)
{
    return launch_wide(adapter_shrink_kernel<T, BY_ROW>, dim3(tiles, a.slices),
                       kShrinkStages * shrink_stage<BY_ROW>(a.r) + kSmemSlack,
                       kShrinkStages * shrink_stage<BY_ROW>(kMaxRank) + kSmemSlack, st, a);
}

template <typename T, bool BY_ROW>
cudaError_t launch_expand(ExpandArgs a, int tiles, cudaStream_t st)
{
    const int blocks = (a.N + kCols - 1) / kCols;
    // four waves of CTAs and more; up to eight blocks of columns save reading h again
    a.steps = std::max(1, std::min(8, (int)((long long)blocks * tiles / 1216)));
    return launch_wide(adapter_expand_kernel<T, BY_ROW>,
                       dim3(tiles, (blocks + a.steps - 1) / a.steps),
                       expand_smem<BY_ROW>(rank_pad(a.r)), expand_smem<BY_ROW>(kMaxRank), st, a);
}

template <typename T>
cudaError_t launch_outer(const OuterArgs &a, cudaStream_t st)
{
    return launch_wide(adapter_outer_kernel<T>, dim3(a.a.blocks + a.b.blocks, a.L, a.splits),
                       kOuterStages * outer_stage(rank_pad(a.r)) + kSmemSlack,
                       kOuterStages * outer_stage(kMaxRank) + kSmemSlack, st, a);
}

int check_sizes(int dtype, int n, int L, int r, int K, int N)
{
    if (dtype != MOE_FP16 && dtype != MOE_BF16)
        return record_failure(MOE_ERR_UNSUPPORTED, "dtype must be MOE_FP16 or MOE_BF16");
    if (n < 1 || n > kMaxTokens)
        return record_failure(MOE_ERR_INVALID_ARG, "n_tokens must be in 1..1048576");
    if (L < 1 || L > kMaxAdapters)
        return record_failure(MOE_ERR_INVALID_ARG, "n_adapters must be in 1..1024");
    if (r < 8 || r > kMaxRank || r % 8)
        return record_failure(MOE_ERR_INVALID_ARG, "rank must be a multiple of 8 in 8..128");
    if (K < 1 || K > kMaxWidth || N < 1 || N > kMaxWidth)
        return record_failure(MOE_ERR_INVALID_ARG, "cols and rows must be in 1..1048576");
    return MOE_OK;
}

bool vec_rows(const void *p, long long ld, int n)
{
    return (uintptr_t)p % 16 == 0 && (n == 1 || ld % 8 == 0);
}

const uint16_t *half_words(const void *p) { return static_cast<const uint16_t *>(p); }

struct AdapterCall {
    const void *x;
    long long ldx;
    const int32_t *ids;
    const void *A, *B, *base;
    long long ldb;
    void *out;
    long long ldo;
    void *h;
    const float *scale;
    int n, L, r, K, N;
    Workspace w;
};

template <typename T>
cudaError_t run_adapter(const AdapterCall &c, cudaStream_t st)
{
    const int tiles = most_tiles(c.n, c.L);
    cudaError_t e = launch_plan(c.ids, c.n, c.L, c.w, st);
    if (e != cudaSuccess)
        return e;
    const ShrinkArgs s = {c.w.p, half_words(c.x), c.ldx, half_words(c.A), c.n, c.L, c.K, c.r,
                          shrink_slices(c.n, c.L, c.K),
                          vec_rows(c.x, c.ldx, c.n), c.K % 8 == 0, c.w.part, c.w.pair,
                          static_cast<uint16_t *>(c.h)};
    e = launch_shrink<T, false>(s, tiles, st);
    if (e != cudaSuccess)
        return e;
    const ExpandArgs x = {c.w.p, c.w.pair, half_words(c.B), c.scale, half_words(c.base), c.ldb,
                          static_cast<uint16_t *>(c.out), c.ldo, c.L, c.N, c.r, 0, true,
                          vec_rows(c.base, c.ldb, c.n), vec_rows(c.out, c.ldo, c.n)};
    return launch_expand<T, false>(x, tiles, st);
}

struct AdapterGradCall {
    const void *dy, *x;
    long long lddy, ldx;
    const void *h;
    const int32_t *ids;
    const void *A, *B, *base;
    long long ldb;
    void *dx;
    long long lddx;
    void *dA, *dB;
    const float *scale;
    int n, L, r, K, N;
    Workspace w;
};

template <typename T>
cudaError_t run_adapter_grad(const AdapterGradCall &c, cudaStream_t st)
{
    const int tiles = most_tiles(c.n, c.L);
    cudaError_t e = launch_plan(c.ids, c.n, c.L, c.w, st);
    if (e != cudaSuccess)
        return e;
    const ShrinkArgs s = {c.w.p, half_words(c.dy), c.lddy, half_words(c.B), c.n, c.L, c.N, c.r,
                          shrink_slices(c.n, c.L, c.N),
                          vec_rows(c.dy, c.lddy, c.n), true, c.w.part, c.w.pair, nullptr};
    e = launch_shrink<T, true>(s, tiles, st);
    if (e != cudaSuccess)
        return e;
    if (c.dx) {
        const ExpandArgs x = {c.w.p, c.w.pair, half_words(c.A), c.scale, half_words(c.base), c.ldb,
                              static_cast<uint16_t *>(c.dx), c.lddx, c.L, c.K, c.r, 0,
                              c.K % 8 == 0, vec_rows(c.base, c.ldb, c.n),
                              vec_rows(c.dx, c.lddx, c.n)};
        e = launch_expand<T, true>(x, tiles, st);
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
    o.splits = outer_splits(c.n, c.L, c.K, c.N);
    o.part = c.w.outer_part;
    o.tickets = c.w.outer_tickets;
    if (c.dA)
        o.a = {half_words(c.x), c.ldx, vec_rows(c.x, c.ldx, c.n), c.K, (c.K + kCols - 1) / kCols,
               c.w.pair, static_cast<uint16_t *>(c.dA)};
    if (c.dB)
        o.b = {half_words(c.dy), c.lddy, vec_rows(c.dy, c.lddy, c.n), c.N,
               (c.N + kCols - 1) / kCols, half_words(c.h), static_cast<uint16_t *>(c.dB)};
    return launch_outer<T>(o, st);
}

Arg weights_arg(const void *p, int L, int r, int width, bool written = false)
{
    Arg a = flat_arg(p, (size_t)L * r * width, 2, written);
    a.align = 16;
    return a;
}

}  // namespace

}  // namespace qe

extern "C" size_t moe_adapter_workspace(int n_tokens, int n_adapters, int rank, int cols, int rows)
{
    using namespace qe;
    if (n_tokens < 1 || n_tokens > kMaxTokens || n_adapters < 1 || n_adapters > kMaxAdapters ||
        rank < 8 || rank > kMaxRank || rank % 8 || cols < 1 || cols > kMaxWidth || rows < 1 ||
        rows > kMaxWidth)
        return 0;
    return std::max(adapter_ws(nullptr, n_tokens, n_adapters, rank, cols, rows, false).bytes,
                    adapter_ws(nullptr, n_tokens, n_adapters, rank, cols, rows, true).bytes);
}

extern "C" int moe_adapter(const void *x, long long ldx, int dtype, int n_tokens, int cols,
                           int rows, const int32_t *ids, int n_adapters, int rank, const void *A,
                           const void *B, const float *scale, const void *base, long long ldb,
                           void *out, long long ldo, void *h, void *workspace,
                           size_t workspace_bytes, void *stream)
{
    using namespace qe;
    const int rc = check_sizes(dtype, n_tokens, n_adapters, rank, cols, rows);
    if (rc)
        return rc;
    if (!x || !ids || !A || !B || !out || !workspace)
        return record_failure(MOE_ERR_INVALID_ARG, "null pointer argument");
    const size_t need = moe_adapter_workspace(n_tokens, n_adapters, rank, cols, rows);
    if (workspace_bytes < need)
        return record_failure(MOE_ERR_INVALID_ARG, "workspace below moe_adapter_workspace(...)");
    const size_t n = n_tokens;
    Arg hs = flat_arg(h, n * rank, 2, true);
    hs.align = 16;
    const Arg args[] = {rows_arg(x, ldx, cols, n_tokens, 2, 2),
                        flat_arg(ids, n, 4),
                        weights_arg(A, n_adapters, rank, cols),
                        weights_arg(B, n_adapters, rank, rows),
                        flat_arg(scale, n_adapters, 4),
                        rows_arg(base, ldb, rows, n_tokens, 2, 2),
                        rows_arg(out, ldo, rows, n_tokens, 2, 2, true, base),
                        hs,
                        flat_arg(workspace, need / 256, 256, true)};
    int dev, sms;
    if (const int bad = check_args(args, sizeof(args) / sizeof(args[0]), &dev, &sms))
        return bad;
    const AdapterCall c = {x, ldx, ids, A, B, base, ldb, out, ldo, h, scale, n_tokens, n_adapters,
                           rank, cols, rows,
                           adapter_ws(workspace, n_tokens, n_adapters, rank, cols, rows, false)};
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return launch_result(dtype == MOE_FP16 ? run_adapter<__half>(c, st)
                                           : run_adapter<__nv_bfloat16>(c, st));
}

extern "C" int moe_adapter_grad(const void *dy, long long lddy, const void *x, long long ldx,
                                const void *h, int dtype, int n_tokens, int cols, int rows,
                                const int32_t *ids, int n_adapters, int rank, const void *A,
                                const void *B, const float *scale, const void *base, long long ldb,
                                void *dx, long long lddx, void *dA, void *dB, void *workspace,
                                size_t workspace_bytes, void *stream)
{
    using namespace qe;
    const int rc = check_sizes(dtype, n_tokens, n_adapters, rank, cols, rows);
    if (rc)
        return rc;
    if (!dy || !ids || !A || !B || !workspace || (dA && !x) || (dB && !h))
        return record_failure(MOE_ERR_INVALID_ARG, "null pointer argument");
    if (!dx && !dA && !dB)
        return record_failure(MOE_ERR_INVALID_ARG, "need dx, dA or dB");
    const size_t need = moe_adapter_workspace(n_tokens, n_adapters, rank, cols, rows);
    if (workspace_bytes < need)
        return record_failure(MOE_ERR_INVALID_ARG, "workspace below moe_adapter_workspace(...)");
    const size_t n = n_tokens;
    Arg hs = flat_arg(dB ? h : nullptr, n * rank, 2);
    hs.align = 16;
    const void *in = dx ? base : nullptr;
    const Arg args[] = {rows_arg(dy, lddy, rows, n_tokens, 2, 2),
                        rows_arg(dA ? x : nullptr, ldx, cols, n_tokens, 2, 2),
                        hs,
                        flat_arg(ids, n, 4),
                        weights_arg(A, n_adapters, rank, cols),
                        weights_arg(B, n_adapters, rank, rows),
                        flat_arg(scale, n_adapters, 4),
                        rows_arg(in, ldb, cols, n_tokens, 2, 2),
                        rows_arg(dx, lddx, cols, n_tokens, 2, 2, true, in),
                        weights_arg(dA, n_adapters, rank, cols, true),
                        weights_arg(dB, n_adapters, rank, rows, true),
                        flat_arg(workspace, need / 256, 256, true)};
    int dev, sms;
    if (const int bad = check_args(args, sizeof(args) / sizeof(args[0]), &dev, &sms))
        return bad;
    const AdapterGradCall c = {dy, x, lddy, ldx, h, ids, A, B, in, ldb, dx, lddx, dA, dB, scale,
                               n_tokens, n_adapters, rank, cols, rows,
                               adapter_ws(workspace, n_tokens, n_adapters, rank, cols, rows, true)};
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return launch_result(dtype == MOE_FP16 ? run_adapter_grad<__half>(c, st)
                                           : run_adapter_grad<__nv_bfloat16>(c, st));
}
