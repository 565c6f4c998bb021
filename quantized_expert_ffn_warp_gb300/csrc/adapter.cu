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
// Measured in a replayed graph: 4001 tokens of 9 requests through 4096 x 14336 at rank 64
// (bf16, with base) 89 us, of which the plan takes 5, the shrink and the join of its
// slices 20 and the expansion 59 (229 MB of base and out at 3.9 TB/s); the gradients of 8192
// tokens through 4096 x 4096 at rank 32 103 us: 6, 20, 35, and 34 for the weights'.  13
// tokens of 13 requests take 16.5 us, three launches of dependent loads.
// h and u are fp32 sums and are multiplied as sums of values of the activations' type, since
// the tensor cores take 16-bit operands: one would add a rounding of 2^-9 (bf16) to the
// delta and to dA.  bf16 takes three, all 24 bits; with two, 16 bits, dA differed from fp32
// products by 1.5e-4 of itself in place of 1.1e-4, all else the rounding of the result.
// The third costs 4 us of 89 in the first case and 7 us of 116 in the gradients at rank 64
// (8192 tokens, 4096 x 4096), and nothing up to rank 32.
// fp16 takes two, 22 bits of what lies near its largest number only (gradients' u are often
// below 2^-14, all of its range a subnormal's), so that they are 2^e h and 2^e u with the
// largest next to 2^15: e of a token where the token's own result is formed, of an adapter
// in the sums over its tokens, where the second value has 2^11 besides and sums of its own.
// The factors are undone in fp32.
#include <algorithm>

#include "adapter.cuh"
#include "args.cuh"

namespace qe {

namespace {

constexpr int kMaxTokens = 1 << 20, kMaxWidth = 1 << 20;
constexpr int kMaxSlices = 16;          // CTAs that share a tile's contraction

// ---------------------------------------------------------------- plan

// One CTA: a stable counting sort.  A warp owns a run of consecutive tokens.
__global__ void __launch_bounds__(1024) adapter_plan_kernel(const int32_t *__restrict__ ids, int n,
                                                           int L, AdapterPlan p, int max_tickets)
{
    extern __shared__ int sm[];
    const int G = L + 1;        // the last group has no adapter
    int *hist = sm, *first = sm + 32 * G, *tile0 = first + G + 1, *cost0 = tile0 + G + 1;
    pdl_enter();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int i = threadIdx.x; i < 32 * G; i += 1024)
        hist[i] = 0;
    for (int i = threadIdx.x; i < max_tickets; i += 1024)
        p.tickets[i] = 0;
    for (int i = threadIdx.x; i < L; i += 1024)
        p.most[i] = 0;
    __syncthreads();
    const int per = ((n + 31) / 32 + 31) / 32 * 32;
    const int lo = min(n, warp * per), hi = min(n, lo + per);
    int *mine = hist + warp * G;
    constexpr int U = 8;
    // calls f(token, group, lanes of the same group) for the warp's tokens, 32 at a time;
    // requests are runs of tokens, so that a group most often fills the warp
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
                    const bool one = __all_sync(0xffffffffu, g[i] == __shfl_sync(0xffffffffu, g[i], 0));
                    f(b + 32 * i + lane, g[i],
                      one ? 0xffffffffu : __match_any_sync(0xffffffffu, g[i]));
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
        int tok = 0, tile = 0, cost = 0;
        for (int b = 0; b < G; b += 32) {
            const int c = b + lane < G ? first[b + lane] : 0, k = (c + kAdapterTile - 1) / kAdapterTile;
            // as k whole tiles, the tokens of the last one taken back
            const bool none = b + lane == L;
            const int e = k * tile_cost(none, 0) + tile_cost(none, c) - tile_cost(none, 0);
            int sc = c, sk = k, se = e;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int uc = __shfl_up_sync(0xffffffffu, sc, d);
                const int uk = __shfl_up_sync(0xffffffffu, sk, d);
                const int ue = __shfl_up_sync(0xffffffffu, se, d);
                if (lane >= d) {
                    sc += uc;
                    sk += uk;
                    se += ue;
                }
            }
            if (b + lane < G) {
                first[b + lane] = tok + sc - c;
                tile0[b + lane] = tile + sk - k;
                cost0[b + lane] = cost + se - e;
            }
            tok += __shfl_sync(0xffffffffu, sc, 31);
            tile += __shfl_sync(0xffffffffu, sk, 31);
            cost += __shfl_sync(0xffffffffu, se, 31);
        }
        if (lane == 0) {
            first[G] = n;
            tile0[G] = tile;
            p.n_tiles[0] = tile;
            p.n_tiles[1] = cost;
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
        const int k = i - tile0[a], start = first[a] + k * kAdapterTile;
        p.tiles[i] = make_int4(a, start, min(kAdapterTile, first[a + 1] - start),
                               cost0[a] + k * tile_cost(a == L, kAdapterTile));
    }
    walk([&](int t, int g, unsigned same) {
        if (g >= 0)
            p.perm[first[g] + mine[g] + __popc(same & ((1u << lane) - 1))] = t;
        __syncwarp();       // before the leaders count these tokens
        if (g >= 0 && lane == __ffs(same) - 1)
            mine[g] += __popc(same);
    });
}

// ---------------------------------------------------------------- host

// CTAs that share the contraction of a tile: two for each SM in all (above rank 64 the shared
// memory of one fits an SM, and they make two waves), each with two steps at least.  Asks no device, since the workspace depends on it.
int shrink_slices(int n, int L, int K)
{
    const int most = std::max(1, (K + kAdapterStep - 1) / kAdapterStep / 2);
    return std::max(1, std::min({304 / adapter_tiles(n, L), most, kMaxSlices}));
}
// CTAs that share an adapter's tokens, in the same way, each with four steps at least.
int outer_blocks(int K, int N)
{
    return (K + kAdapterCols - 1) / kAdapterCols + (N + kAdapterCols - 1) / kAdapterCols;
}
int outer_splits(int n, int L, int K, int N)
{
    const long long ctas = (long long)outer_blocks(K, N) * L;
    return (int)std::max(1LL, std::min({304 / ctas, (long long)n / (4 * kAdapterStep), 8LL}));
}

AdapterWorkspace adapter_ws(void *base, int n, int L, int r, int K, int N, bool grad)
{
    AdapterWorkspace w{};
    size_t at = 0;
    const auto take = [&](size_t bytes) {
        char *p = static_cast<char *>(base) + at;
        at += (bytes + 255) / 256 * 256;
        return p;
    };
    w.slices = shrink_slices(n, L, grad ? N : K);
    w.splits = grad ? outer_splits(n, L, K, N) : 1;
    const int tiles = w.slices > 1 ? adapter_tiles(n, L) : 0;
    const int outer = w.splits > 1 ? L * outer_blocks(K, N) : 0;
    w.tickets = tiles + outer;
    w.p.n_tiles = reinterpret_cast<int *>(take(8));
    w.p.off = reinterpret_cast<int *>(take(4 * ((size_t)L + 2)));
    w.p.perm = reinterpret_cast<int *>(take(4 * (size_t)n));
    w.p.tiles = reinterpret_cast<int4 *>(take(16 * (size_t)adapter_tiles(n, L)));
    w.p.tickets = reinterpret_cast<unsigned *>(take(4 * (size_t)w.tickets));
    w.outer_tickets = w.p.tickets + tiles;
    w.p.most = reinterpret_cast<unsigned *>(take(4 * (size_t)L));
    w.mid = reinterpret_cast<float *>(take(8 * (size_t)n * rank_pad(r)));
    w.part = reinterpret_cast<float *>(
        take(w.slices > 1 ? 4 * (size_t)w.slices * n * rank_pad(r) : 0));
    w.outer_part = reinterpret_cast<float *>(
        take(4 * (size_t)w.splits * outer * kAdapterCols * rank_pad(r)));
    w.bytes = at;
    return w;
}

cudaError_t launch_plan(const int32_t *ids, int n, int L, const AdapterWorkspace &w, cudaStream_t st)
{
    const size_t smem = sizeof(int) * (32 * ((size_t)L + 1) + 3 * ((size_t)L + 2));
    if (smem > 48 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(
            adapter_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
            (int)(sizeof(int) * (32 * (kAdapterMaxCount + 1) + 3 * (kAdapterMaxCount + 2))));
        if (e != cudaSuccess)
            return e;
    }
    return launch_pdl(adapter_plan_kernel, dim3(1), dim3(1024), smem, st, ids, n, L, w.p, w.tickets);
}

int check_sizes(int dtype, int n, int L, int r, int K, int N)
{
    if (dtype != MOE_FP16 && dtype != MOE_BF16)
        return record_failure(MOE_ERR_UNSUPPORTED, "dtype must be MOE_FP16 or MOE_BF16");
    if (n < 1 || n > kMaxTokens)
        return record_failure(MOE_ERR_INVALID_ARG, "n_tokens must be in 1..1048576");
    if (L < 1 || L > kAdapterMaxCount)
        return record_failure(MOE_ERR_INVALID_ARG, "n_adapters must be in 1..1024");
    if (r < 8 || r > kAdapterMaxRank || r % 8)
        return record_failure(MOE_ERR_INVALID_ARG, "rank must be a multiple of 8 in 8..128");
    if (K < 1 || K > kMaxWidth || N < 1 || N > kMaxWidth)
        return record_failure(MOE_ERR_INVALID_ARG, "cols and rows must be in 1..1048576");
    return MOE_OK;
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
    if (n_tokens < 1 || n_tokens > kMaxTokens || n_adapters < 1 || n_adapters > kAdapterMaxCount ||
        rank < 8 || rank > kAdapterMaxRank || rank % 8 || cols < 1 || cols > kMaxWidth || rows < 1 ||
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
    const AdapterCall c = {x, ldx, A, B, base, ldb, out, ldo, h, scale, n_tokens, n_adapters,
                           rank, cols, rows, sms,
                           adapter_ws(workspace, n_tokens, n_adapters, rank, cols, rows, false)};
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const cudaError_t e = launch_plan(ids, n_tokens, n_adapters, c.w, st);
    return launch_result(e != cudaSuccess    ? e
                         : dtype == MOE_FP16 ? adapter_fp16(c, st)
                                             : adapter_bf16(c, st));
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
    const AdapterGradCall c = {dy, x, lddy, ldx, h, A, B, in, ldb, dx, lddx, dA, dB, scale,
                               n_tokens, n_adapters, rank, cols, rows, sms,
                               adapter_ws(workspace, n_tokens, n_adapters, rank, cols, rows, true)};
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const cudaError_t e = launch_plan(ids, n_tokens, n_adapters, c.w, st);
    return launch_result(e != cudaSuccess    ? e
                         : dtype == MOE_FP16 ? adapter_grad_fp16(c, st)
                                             : adapter_grad_bf16(c, st));
}
