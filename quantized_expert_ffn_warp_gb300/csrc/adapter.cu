// Low-rank adapters of many requests beside one projection, and their gradients.
// Token t has adapter a = ids[t] (A_a [r][K], B_a [N][r], scale s_a), or none:
//   h = A_a x,  out = base + s_a B_a h
//   u = B_a^T dy,  dx = base + s_a A_a^T u
//   dA_a = s_a sum_t u_t x_t^T,  dB_a = s_a sum_t dy_t h_t^T   over the adapter's tokens
//
// A plan kernel sorts the tokens by adapter (stably) and cuts each adapter's tokens
// into tiles of 64.  "Shrink" contracts a tile with the long side of a matrix, "expand"
// goes back to full width and adds base, "outer" sums over an adapter's tokens.  All
// three are bound by the activations' bytes (r operations per byte and less), so they
// feed warp MMAs straight from global memory: an MMA takes its contraction index, rows
// and columns in any order, as long as both operands agree, so that every load is a
// lane's 16, 8 or 4 contiguous bytes, and operands whose pairs lie in different rows are
// paired by byte permutes.
// h and u are held as the sum of two values of the activations' type: one would add a
// rounding of 2^-9 (bf16) to the delta and to dA, and the second product is hidden
// behind the loads.
#include <algorithm>

#include "args.cuh"
#include "vec.cuh"
#include "w4.cuh"

namespace qe {

namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kTile = 64;               // tokens of a tile
constexpr int kMaxTokens = 1 << 20, kMaxAdapters = 1024, kMaxRank = 128, kMaxWidth = 1 << 20;
constexpr int kMaxSlices = 16;          // CTAs that share a tile's contraction

__host__ __device__ constexpr int rank_pad(int r) { return (r + 15) / 16 * 16; }

struct Plan {
    int *off;           // [L + 2] first token of an adapter in perm; then those without one
    int *perm;          // [n] tokens in the order of their adapters
    int4 *tiles;        // (adapter, first place in perm, tokens, -); L: none
    int *n_tiles;
    unsigned *tickets;  // [tiles][passes] slices that have arrived
};

// Words [lo | hi halves] of two 32-bit words.
__device__ __forceinline__ uint32_t low_halves(uint32_t a, uint32_t b)
{
    return __byte_perm(a, b, 0x5410);
}
__device__ __forceinline__ uint32_t high_halves(uint32_t a, uint32_t b)
{
    return __byte_perm(a, b, 0x7632);
}

// Values i .. i + 7 of a row of `len` 2-byte values, 0 behind its end.
__device__ __forceinline__ uint4 load8(const uint16_t *row, int i, int len, bool aligned)
{
    if (aligned && i + 8 <= len)
        return *reinterpret_cast<const uint4 *>(row + i);
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; e++) {
        const uint32_t a = i + 2 * e < len ? row[i + 2 * e] : 0;
        const uint32_t b = i + 2 * e + 1 < len ? row[i + 2 * e + 1] : 0;
        w[e] = a | b << 16;
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
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

// ---------------------------------------------------------------- shrink

struct ShrinkArgs {
    Plan p;
    const uint16_t *x;      // [n][K]
    long long ldx;
    const uint16_t *w;      // [L][r][K], or (BY_ROW) [L][K][r]
    int n, L, K, r, slices, passes;
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

// The result at place `at` of perm, rank `k`.
template <typename T>
__device__ __forceinline__ void put_result(const ShrinkArgs &a, int at, int k, float v)
{
    const int pad = rank_pad(a.r);
    if (k >= pad)
        return;
    if (k >= a.r)
        v = 0.f;
    const T hi = from_float<T>(v);
    const float f = to_float<T>(hi);
    // an infinity or a NaN has no remainder
    const float rest = fabsf(f) <= 3.4e38f ? v - f : 0.f;
    uint16_t *row = a.pair + (long long)at * 2 * pad;
    row[k] = bits(hi);
    row[pad + k] = bits(from_float<T>(rest));
    if (a.h && k < a.r)
        a.h[(long long)a.p.perm[at] * a.r + k] = bits(hi);
}

// RB blocks of 16 ranks of a tile.  The ranks are the MMA's rows, the tokens its
// columns; warps take blocks of 32 of K in turn and their sums are added in shared
// memory, the slices' by whichever CTA of a tile arrives last, in the slices' order.
template <typename T, bool BY_ROW, int RB>
__global__ void __launch_bounds__(kThreads, 1) adapter_shrink_kernel(ShrinkArgs a)
{
    constexpr int NT = kTile / 8, R = 16 * RB, S = R + 4;
    extern __shared__ float red[];      // [warps][kTile][S]
    __shared__ int last;
    pdl_enter();
    if ((int)blockIdx.x >= *a.p.n_tiles)
        return;
    const int4 tile = a.p.tiles[blockIdx.x];
    const int slice = blockIdx.y, rank0 = blockIdx.z * R;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    if (tile.x == a.L) {        // no adapter
        if (slice == 0 && blockIdx.z == 0 && a.h)
            for (int i = threadIdx.x; i < tile.z * a.r; i += kThreads)
                a.h[(long long)a.p.perm[tile.y + i / a.r] * a.r + i % a.r] = 0;
        return;
    }
    const uint16_t *w = a.w + (long long)tile.x * a.r * a.K;
    const uint16_t *row[NT];
#pragma unroll
    for (int i = 0; i < NT; i++) {
        const int at = 8 * i + g;
        row[i] = a.x + (long long)a.p.perm[tile.y + (at < tile.z ? at : 0)] * a.ldx;
    }
    float acc[RB][NT][4];
#pragma unroll
    for (int b = 0; b < RB; b++)
#pragma unroll
        for (int i = 0; i < NT; i++)
#pragma unroll
            for (int e = 0; e < 4; e++)
                acc[b][i][e] = 0.f;
    const int blocks = (a.K + 31) / 32, per = (blocks + a.slices - 1) / a.slices;
    const int end = min(blocks, (slice + 1) * per);
    const int used = (tile.z + 7) / 8;
    for (int kb = slice * per + warp; kb < end; kb += kWarps) {
        const int k = 32 * kb + 8 * t;
        uint4 q[NT];
#pragma unroll
        for (int i = 0; i < NT; i++)
            q[i] = i < used ? load8(row[i], k, a.K, a.vec_x) : make_uint4(0, 0, 0, 0);
        // rows of A in two steps of 16 of K: lane t's words 0, 1 and 2, 3
        uint32_t f[RB][2][4];
        if constexpr (!BY_ROW) {
#pragma unroll
            for (int b = 0; b < RB; b++) {
                uint4 u[2];
#pragma unroll
                for (int half = 0; half < 2; half++) {
                    const int rank = rank0 + 16 * b + 8 * half + g;
                    u[half] = rank < a.r ? load8(w + (long long)rank * a.K, k, a.K, a.vec_w)
                                         : make_uint4(0, 0, 0, 0);
                }
                f[b][0][0] = u[0].x, f[b][0][1] = u[1].x, f[b][0][2] = u[0].y, f[b][0][3] = u[1].y;
                f[b][1][0] = u[0].z, f[b][1][1] = u[1].z, f[b][1][2] = u[0].w, f[b][1][3] = u[1].w;
            }
        } else {
            // a lane reads its 2 RB ranks of a row of the matrix: they are row g of the
            // MMA's upper and lower half of each block
            uint32_t v[8][RB];
            const int rank = rank0 + 2 * RB * g;
#pragma unroll
            for (int j = 0; j < 8; j++) {
#pragma unroll
                for (int b = 0; b < RB; b++)
                    v[j][b] = 0;
                if (k + j < a.K && rank < a.r) {
                    const uint16_t *src = w + (long long)(k + j) * a.r + rank;
                    if constexpr (RB == 1) {
                        v[j][0] = *reinterpret_cast<const uint32_t *>(src);
                    } else {
                        const uint2 d = *reinterpret_cast<const uint2 *>(src);
                        v[j][0] = d.x;
                        v[j][1] = d.y;
                    }
                }
            }
#pragma unroll
            for (int b = 0; b < RB; b++)
#pragma unroll
                for (int s = 0; s < 2; s++) {
                    f[b][s][0] = low_halves(v[4 * s][b], v[4 * s + 1][b]);
                    f[b][s][1] = high_halves(v[4 * s][b], v[4 * s + 1][b]);
                    f[b][s][2] = low_halves(v[4 * s + 2][b], v[4 * s + 3][b]);
                    f[b][s][3] = high_halves(v[4 * s + 2][b], v[4 * s + 3][b]);
                }
        }
#pragma unroll
        for (int b = 0; b < RB; b++)
#pragma unroll
            for (int i = 0; i < NT; i++) {
                if (i >= used)
                    break;
                mma16816<T>(acc[b][i], f[b][0][0], f[b][0][1], f[b][0][2], f[b][0][3], q[i].x, q[i].y);
                mma16816<T>(acc[b][i], f[b][1][0], f[b][1][1], f[b][1][2], f[b][1][3], q[i].z, q[i].w);
            }
    }
    float *mine = red + warp * kTile * S;
#pragma unroll
    for (int b = 0; b < RB; b++)
#pragma unroll
        for (int i = 0; i < NT; i++)
#pragma unroll
            for (int e = 0; e < 4; e++) {
                const int tok = 8 * i + 2 * t + (e & 1);
                const int rank = BY_ROW ? 2 * RB * g + 2 * b + (e >> 1) : 16 * b + 8 * (e >> 1) + g;
                mine[tok * S + rank] = acc[b][i][e];
            }
    __syncthreads();
    const int pad = rank_pad(a.r);
    for (int i = threadIdx.x; i < tile.z * R; i += kThreads) {
        const int tok = i / R, k = i % R;
        float v = 0.f;
#pragma unroll
        for (int w8 = 0; w8 < kWarps; w8++)
            v += red[(w8 * kTile + tok) * S + k];
        if (a.slices == 1)
            put_result<T>(a, tile.y + tok, rank0 + k, v);
        else if (rank0 + k < pad)
            a.part[((long long)slice * a.n + tile.y + tok) * pad + rank0 + k] = v;
    }
    if (a.slices == 1)
        return;
    __threadfence();
    __syncthreads();
    if (threadIdx.x == 0)
        last = atomicAdd(a.p.tickets + blockIdx.x * a.passes + blockIdx.z, 1u) == a.slices - 1u;
    __syncthreads();
    if (!last)
        return;
    __threadfence();
    for (int i = threadIdx.x; i < tile.z * R; i += kThreads) {
        const int at = tile.y + i / R, k = rank0 + i % R;
        if (k >= pad)
            continue;
        float v = 0.f;
        for (int s = 0; s < a.slices; s++)
            v += __ldcg(a.part + ((long long)s * a.n + at) * pad + k);
        put_result<T>(a, at, k, v);
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
    int L, N, r, steps;     // steps: blocks of 32 columns of a warp
    bool vec_w, vec_b, vec_o;
};

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

// A tile's columns.  The tokens are the MMA's rows; of 32 columns, lane t ends up
// with 8t .. 8t + 7 of its two tokens.  KS steps of 16 ranks.
template <typename T, bool BY_ROW, int KS>
__global__ void __launch_bounds__(kThreads, KS <= 4 ? 2 : 1) adapter_expand_kernel(ExpandArgs a)
{
    constexpr int R = 16 * KS, S = 2 * R + 8, MB = kTile / 16;
    __shared__ __align__(16) uint16_t hs[kTile][S];
    __shared__ int tok[kTile];
    pdl_enter();
    if ((int)blockIdx.x >= *a.p.n_tiles)
        return;
    const int4 tile = a.p.tiles[blockIdx.x];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    if (threadIdx.x < kTile)
        tok[threadIdx.x] = a.p.perm[tile.y + ((int)threadIdx.x < tile.z ? threadIdx.x : 0)];
    const bool none = tile.x == a.L;
    const int pad = rank_pad(a.r);
    if (!none)
        for (int i = threadIdx.x; i < kTile * 2 * R / 8; i += kThreads) {
            const int row = i / (2 * R / 8), c = i % (2 * R / 8) * 8, part = c / R, k = c % R;
            uint4 q = make_uint4(0, 0, 0, 0);
            if (row < tile.z && k < pad)
                q = *reinterpret_cast<const uint4 *>(
                    a.pair + ((long long)(tile.y + row) * 2 + part) * pad + k);
            *reinterpret_cast<uint4 *>(&hs[row][c]) = q;
        }
    __syncthreads();
    const uint16_t *w = a.w + (long long)(none ? 0 : tile.x) * a.r * a.N;
    const float scale = none ? 0.f : a.scale ? a.scale[tile.x] : 1.f;
    for (int s = 0; s < a.steps; s++) {
        const int c0 = 32 * ((blockIdx.y * a.steps + s) * kWarps + warp);
        if (c0 >= a.N)
            break;
        const int c = c0 + 8 * t;
        uint4 b[MB][2];
#pragma unroll
        for (int m = 0; m < MB; m++)
#pragma unroll
            for (int half = 0; half < 2; half++) {
                const int at = 16 * m + 8 * half + g;
                b[m][half] = make_uint4(0, 0, 0, 0);
                if (a.base && at < tile.z)
                    b[m][half] = load8(a.base + tok[at] * a.ldb, c, a.N, a.vec_b);
            }
        uint32_t f[KS][4][2];
        if (!none) {
#pragma unroll
            for (int k = 0; k < KS; k++) {
                const int rank = 16 * k + 4 * t;
                if constexpr (!BY_ROW) {
#pragma unroll
                    for (int j = 0; j < 4; j++) {
                        const int col = c0 + 8 * (g >> 1) + 2 * j + (g & 1);
                        uint2 u = make_uint2(0, 0);
                        if (col < a.N && rank < a.r)
                            u = *reinterpret_cast<const uint2 *>(w + (long long)col * a.r + rank);
                        f[k][j][0] = u.x;
                        f[k][j][1] = u.y;
                    }
                } else {
                    uint2 u[4];
#pragma unroll
                    for (int j = 0; j < 4; j++) {
                        u[j] = make_uint2(0, 0);
                        const int col = c0 + 4 * g;
                        if (rank + j >= a.r)
                            continue;
                        const uint16_t *src = w + (long long)(rank + j) * a.N + col;
                        if (a.vec_w && col + 4 <= a.N) {
                            u[j] = *reinterpret_cast<const uint2 *>(src);
                        } else {
                            uint32_t v[4];
#pragma unroll
                            for (int e = 0; e < 4; e++)
                                v[e] = col + e < a.N ? src[e] : 0;
                            u[j] = make_uint2(v[0] | v[1] << 16, v[2] | v[3] << 16);
                        }
                    }
#pragma unroll
                    for (int half = 0; half < 2; half++) {
                        f[k][0][half] = low_halves(u[2 * half].x, u[2 * half + 1].x);
                        f[k][1][half] = high_halves(u[2 * half].x, u[2 * half + 1].x);
                        f[k][2][half] = low_halves(u[2 * half].y, u[2 * half + 1].y);
                        f[k][3][half] = high_halves(u[2 * half].y, u[2 * half + 1].y);
                    }
                }
            }
        }
#pragma unroll
        for (int m = 0; m < MB; m++) {
            if (16 * m >= tile.z)
                break;
            float acc[4][4];
#pragma unroll
            for (int j = 0; j < 4; j++)
#pragma unroll
                for (int e = 0; e < 4; e++)
                    acc[j][e] = 0.f;
            if (!none) {
#pragma unroll
                for (int part = 1; part >= 0; part--)
#pragma unroll
                    for (int k = 0; k < KS; k++) {
                        const uint2 u = *reinterpret_cast<const uint2 *>(
                            &hs[16 * m + g][part * R + 16 * k + 4 * t]);
                        const uint2 v = *reinterpret_cast<const uint2 *>(
                            &hs[16 * m + 8 + g][part * R + 16 * k + 4 * t]);
#pragma unroll
                        for (int j = 0; j < 4; j++)
                            mma16816<T>(acc[j], u.x, v.x, u.y, v.y, f[k][j][0], f[k][j][1]);
                    }
            }
#pragma unroll
            for (int half = 0; half < 2; half++) {
                const int at = 16 * m + 8 * half + g;
                if (at >= tile.z)
                    continue;
                float d[8];
                unpack<T>(b[m][half], d);
#pragma unroll
                for (int e = 0; e < 8; e++) {
                    // block j's column n is column 8 (n / 2) + 2 j + n % 2, or (BY_ROW) 4 n + j
                    const float v = BY_ROW ? acc[e & 3][2 * half + (e >> 2)]
                                           : acc[e >> 1][2 * half + (e & 1)];
                    if (!none)
                        d[e] = fmaf(scale, v, d[e]);
                }
                store8(a.out + tok[at] * a.ldo, c, a.N, a.vec_o,
                          none ? b[m][half] : pack<T>(d));
            }
        }
    }
}

// ---------------------------------------------------------------- outer

struct OuterSide {
    const uint16_t *src;    // [n][C] by token
    long long ld;
    bool vec;
    int C, blocks;          // columns, blocks of 64 of them
    const uint16_t *v;      // ranks: of a token (h [n][r]), or of a place (pair)
    uint16_t *out;
};
struct OuterArgs {
    Plan p;
    OuterSide a, b;         // dA [L][r][K] from x and u, dB [L][N][r] from dy and h
    const float *scale;
    int r;
};

// The sum over an adapter's tokens of 64 columns times RN x 8 ranks.  The columns are
// the MMA's rows, warps take 16 tokens in turn.
template <typename T, int RN>
__global__ void __launch_bounds__(kThreads, RN <= 4 ? 2 : 1) adapter_outer_kernel(OuterArgs a)
{
    constexpr int R = 8 * RN, S = R + 1;
    extern __shared__ float red[];      // [4][64][S]
    pdl_enter();
    const bool of_a = (int)blockIdx.x < a.a.blocks;
    const OuterSide &o = of_a ? a.a : a.b;
    const int c0 = 64 * (of_a ? blockIdx.x : blockIdx.x - a.a.blocks);
    const int adapter = blockIdx.y, rank0 = blockIdx.z * R, pad = rank_pad(a.r);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int lo = a.p.off[adapter], count = a.p.off[adapter + 1] - lo;
    float acc[4][RN][4];
#pragma unroll
    for (int m = 0; m < 4; m++)
#pragma unroll
        for (int b = 0; b < RN; b++)
#pragma unroll
            for (int e = 0; e < 4; e++)
                acc[m][b][e] = 0.f;
    const int rank = rank0 + RN * g;
    for (int s = 16 * warp; s < count; s += 16 * kWarps) {
        uint32_t q[4][4], v[2][4][RN / 2];
#pragma unroll
        for (int j = 0; j < 4; j++) {
            const int at = s + 4 * t + j;
            uint4 u = make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int i = 0; i < RN / 2; i++)
                v[0][j][i] = v[1][j][i] = 0;
            if (at < count) {
                const int tok = a.p.perm[lo + at];
                u = load8(o.src + tok * o.ld, c0 + 8 * g, o.C, o.vec);
                const uint16_t *row = of_a ? o.v + (long long)(lo + at) * 2 * pad
                                           : o.v + (long long)tok * a.r;
                if (rank < a.r) {
#pragma unroll
                    for (int part = 0; part < 2; part++) {
                        if (part && !of_a)
                            continue;
                        const uint16_t *src = row + part * pad + rank;
                        if constexpr (RN == 2) {
                            v[part][j][0] = *reinterpret_cast<const uint32_t *>(src);
                        } else if constexpr (RN == 4) {
                            const uint2 d = *reinterpret_cast<const uint2 *>(src);
                            v[part][j][0] = d.x, v[part][j][1] = d.y;
                        } else {
                            const uint4 d = *reinterpret_cast<const uint4 *>(src);
                            v[part][j][0] = d.x, v[part][j][1] = d.y;
                            v[part][j][2] = d.z, v[part][j][3] = d.w;
                        }
                    }
                }
            }
            q[j][0] = u.x, q[j][1] = u.y, q[j][2] = u.z, q[j][3] = u.w;
        }
        uint32_t f[4][4];
#pragma unroll
        for (int m = 0; m < 4; m++) {
            f[m][0] = low_halves(q[0][m], q[1][m]);
            f[m][1] = high_halves(q[0][m], q[1][m]);
            f[m][2] = low_halves(q[2][m], q[3][m]);
            f[m][3] = high_halves(q[2][m], q[3][m]);
        }
#pragma unroll
        for (int part = 0; part < 2; part++) {
            if (part && !of_a)
                continue;
#pragma unroll
            for (int b = 0; b < RN; b++) {
                const uint32_t(&u)[4][RN / 2] = v[part];
                const uint32_t x = b & 1 ? high_halves(u[0][b / 2], u[1][b / 2])
                                         : low_halves(u[0][b / 2], u[1][b / 2]);
                const uint32_t y = b & 1 ? high_halves(u[2][b / 2], u[3][b / 2])
                                         : low_halves(u[2][b / 2], u[3][b / 2]);
#pragma unroll
                for (int m = 0; m < 4; m++)
                    mma16816<T>(acc[m][b], f[m][0], f[m][1], f[m][2], f[m][3], x, y);
            }
        }
    }
    // the upper four warps' sums, then the lower four's on top, then over the four
    float *mine = red + (warp & 3) * 64 * S;
#pragma unroll
    for (int round = 0; round < 2; round++) {
        if ((warp >> 2) == 1 - round) {
#pragma unroll
            for (int m = 0; m < 4; m++)
#pragma unroll
                for (int b = 0; b < RN; b++)
#pragma unroll
                    for (int e = 0; e < 4; e++) {
                        const int c = 8 * g + 2 * m + (e >> 1), k = RN * (2 * t + (e & 1)) + b;
                        float &d = mine[c * S + k];
                        d = round ? d + acc[m][b][e] : acc[m][b][e];
                    }
        }
        __syncthreads();
    }
    const float scale = a.scale ? a.scale[adapter] : 1.f;
    uint16_t *out = o.out + (long long)adapter * a.r * o.C;
    for (int i = threadIdx.x; i < 64 * R; i += kThreads) {
        const int c = of_a ? i % 64 : i / R, k = of_a ? i / 64 : i % R;
        if (c0 + c >= o.C || rank0 + k >= a.r)
            continue;
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < 4; w++)
            v += red[(w * 64 + c) * S + k];
        const long long at = of_a ? (long long)(rank0 + k) * o.C + c0 + c
                                  : (long long)(c0 + c) * a.r + rank0 + k;
        out[at] = bits(from_float<T>(scale * v));
    }
}

// ---------------------------------------------------------------- host

// Most tiles of n tokens: an adapter's tokens end with one that is not full.
int most_tiles(int n, int L) { return n / kTile + std::min(n, L + 1); }

int rank_passes(int r) { return r <= 16 ? 1 : (r + 31) / 32; }

// CTAs that share the contraction of a tile: two for each SM in all, each with 32
// columns for every warp at least.  Asks no device, since the workspace depends on it.
int shrink_slices(int n, int L, int K, int r)
{
    const int ctas = most_tiles(n, L) * rank_passes(r);
    const int most = std::max(1, K / (32 * kWarps));
    return std::max(1, std::min({304 / ctas, most, kMaxSlices}));
}

struct Workspace {
    Plan p;
    int tickets;
    uint16_t *pair;
    float *part;
    size_t bytes;
};

// For a contraction over K columns.
Workspace adapter_ws(void *base, int n, int L, int r, int K)
{
    Workspace w{};
    size_t at = 0;
    const auto take = [&](size_t bytes) {
        char *p = static_cast<char *>(base) + at;
        at += (bytes + 255) / 256 * 256;
        return p;
    };
    const int slices = shrink_slices(n, L, K, r);
    w.tickets = slices > 1 ? most_tiles(n, L) * rank_passes(r) : 0;
    w.p.n_tiles = reinterpret_cast<int *>(take(4));
    w.p.off = reinterpret_cast<int *>(take(4 * ((size_t)L + 2)));
    w.p.perm = reinterpret_cast<int *>(take(4 * (size_t)n));
    w.p.tiles = reinterpret_cast<int4 *>(take(16 * (size_t)most_tiles(n, L)));
    w.p.tickets = reinterpret_cast<unsigned *>(take(4 * (size_t)w.tickets));
    w.pair = reinterpret_cast<uint16_t *>(take(4 * (size_t)n * rank_pad(r)));
    w.part = reinterpret_cast<float *>(
        take(slices > 1 ? 4 * (size_t)slices * n * rank_pad(r) : 0));
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

template <typename T, bool BY_ROW, int RB>
cudaError_t launch_shrink_as(const ShrinkArgs &a, int tiles, cudaStream_t st)
{
    constexpr int smem = 4 * kWarps * kTile * (16 * RB + 4);
    const cudaError_t e = cudaFuncSetAttribute(
        adapter_shrink_kernel<T, BY_ROW, RB>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess)
        return e;
    return launch_pdl(adapter_shrink_kernel<T, BY_ROW, RB>, dim3(tiles, a.slices, a.passes),
                      dim3(kThreads), smem, st, a);
}
template <typename T, bool BY_ROW>
cudaError_t launch_shrink(const ShrinkArgs &a, int tiles, cudaStream_t st)
{
    return a.r <= 16 ? launch_shrink_as<T, BY_ROW, 1>(a, tiles, st)
                     : launch_shrink_as<T, BY_ROW, 2>(a, tiles, st);
}

template <typename T, bool BY_ROW>
cudaError_t launch_expand(ExpandArgs a, int tiles, cudaStream_t st)
{
    const int blocks = (a.N + 32 * kWarps - 1) / (32 * kWarps);
    // four CTAs for each SM and more; up to eight steps save reading h again
    a.steps = std::max(1, std::min(8, (int)((long long)blocks * tiles / 1216)));
    const dim3 grid(tiles, (blocks + a.steps - 1) / a.steps);
    return a.r <= 16   ? launch_pdl(adapter_expand_kernel<T, BY_ROW, 1>, grid, dim3(kThreads), 0, st, a)
           : a.r <= 32 ? launch_pdl(adapter_expand_kernel<T, BY_ROW, 2>, grid, dim3(kThreads), 0, st, a)
           : a.r <= 64 ? launch_pdl(adapter_expand_kernel<T, BY_ROW, 4>, grid, dim3(kThreads), 0, st, a)
                       : launch_pdl(adapter_expand_kernel<T, BY_ROW, 8>, grid, dim3(kThreads), 0, st, a);
}

template <typename T, int RN>
cudaError_t launch_outer_as(const OuterArgs &a, int L, cudaStream_t st)
{
    constexpr int R = 8 * RN, smem = 4 * 4 * 64 * (R + 1);
    const cudaError_t e = cudaFuncSetAttribute(
        adapter_outer_kernel<T, RN>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess)
        return e;
    return launch_pdl(adapter_outer_kernel<T, RN>, dim3(a.a.blocks + a.b.blocks, L, (a.r + R - 1) / R),
                      dim3(kThreads), smem, st, a);
}
template <typename T>
cudaError_t launch_outer(const OuterArgs &a, int L, cudaStream_t st)
{
    return a.r <= 16   ? launch_outer_as<T, 2>(a, L, st)
           : a.r <= 32 ? launch_outer_as<T, 4>(a, L, st)
                       : launch_outer_as<T, 8>(a, L, st);
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
                          shrink_slices(c.n, c.L, c.K, c.r), rank_passes(c.r),
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
                          shrink_slices(c.n, c.L, c.N, c.r), rank_passes(c.r),
                          vec_rows(c.dy, c.lddy, c.n), true, c.w.part, c.w.pair, nullptr};
    e = launch_shrink<T, true>(s, tiles, st);
    if (e != cudaSuccess)
        return e;
    if (c.dx) {
        const ExpandArgs x = {c.w.p, c.w.pair, half_words(c.A), c.scale, half_words(c.base), c.ldb,
                              static_cast<uint16_t *>(c.dx), c.lddx, c.L, c.K, c.r, 0,
                              c.K % 4 == 0, vec_rows(c.base, c.ldb, c.n),
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
    o.r = c.r;
    if (c.dA)
        o.a = {half_words(c.x), c.ldx, vec_rows(c.x, c.ldx, c.n), c.K, (c.K + 63) / 64, c.w.pair,
               static_cast<uint16_t *>(c.dA)};
    if (c.dB)
        o.b = {half_words(c.dy), c.lddy, vec_rows(c.dy, c.lddy, c.n), c.N, (c.N + 63) / 64,
               half_words(c.h), static_cast<uint16_t *>(c.dB)};
    return launch_outer<T>(o, c.L, st);
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
    return std::max(adapter_ws(nullptr, n_tokens, n_adapters, rank, cols).bytes,
                    adapter_ws(nullptr, n_tokens, n_adapters, rank, rows).bytes);
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
                           rank, cols, rows, adapter_ws(workspace, n_tokens, n_adapters, rank, cols)};
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
                               adapter_ws(workspace, n_tokens, n_adapters, rank, rows)};
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return launch_result(dtype == MOE_FP16 ? run_adapter_grad<__half>(c, st)
                                           : run_adapter_grad<__nv_bfloat16>(c, st));
}
