// 4-bit group-quantised products for many tokens, on the tcgen05 tensor cores:
//   y[t][r]  = sum_k x[t][k] W[r][k] (+ bias) (+ residual)      (GRAD = false)
//   dx[t][k] = sum_r dy[t][r] W[r][k]                            (GRAD = true)
//
// The matrix stays packed in its canonical layout; a 128 x 128 block of it (8 KB
// of codes: 128 rows of 64 bytes) is one TMA box, dequantised once per token
// tile, W = (q - z) * s rounded once to the activations' type, into the MMA's A
// operand in tensor memory (M = 128: the outputs' features).  The tokens
// (up to 256 of them) are the MMA's N, their rows the B operand in shared
// memory, read by TMA as they lie.  The contraction index runs along K of the
// MMA in memory order in both directions:
//   forward: a thread owns one weight row (its tensor-memory lane) and
//     unpacks 64 of its K into 32 columns;
//   gradient: the contraction runs over the weight rows, so a thread unpacks
//     four columns of the matrix over pairs of rows (a transposing matrix load
//     puts two rows' nibbles into one word) and stores them in the 16-lane x
//     256-bit tensor memory layout, lane 8 j + g of a quarter holding column
//     4 g + j.
// Why the weights are rounded: an MMA multiplies operands of one 16-bit type, and
// a scale changes with the feature and along the contraction, so it can be
// folded neither into the tokens nor into the finished sums.  The weights in two
// 16-bit parts would take twice the MMAs (4096 tokens 14336 x 4096 fp16 280 us;
// with the contraction twice as long 543 us), scaled sums per group a pass over the
// accumulators every 32 to 128 steps of the contraction.  With the weights as the
// activations' type holds them the output's relative error (2-norm, against 64
// bits) is 0.0023 instead of the 0.0017 of its own rounding in bf16, 0.00028
// instead of 0.00021 in fp16.  A weight beyond fp16's range (a scale above 4366)
// becomes an infinity.
// Roles of a persistent CTA (one per SM): a code producer and a B producer
// (TMA), three groups of four dequant warps taking blocks in turn, one or two
// MMA warps, four epilogue warps.  Tiles of more than 128 tokens need one MMA
// warp; smaller MMAs take less time than one thread needs to issue the next,
// so two warps then run alternate 64-steps into accumulators of their own,
// summed at the end.
// A matrix with too few tiles for the SMs is split along the contraction over a
// cluster of 2 to 8 CTAs, whose partial tiles meet in distributed shared
// memory, in rank order.
// Measured in a replayed graph: 4096 tokens 14336 x 4096 fp16 280 us, 1720
// TFLOP/s, bound by the tensor cores; gradient, 2000 tokens 4096 x 4096 bf16 44.4
// us, 1510 TFLOP/s (288 tiles for 152 SMs: the second wave is not full); 33 tokens
// 6144 x 4096 bf16 15.6 us, bound by the dequantisation.
// Every wait is bounded in time; on expiry the CTA's outputs (its cluster's) are
// NaN and the caller's status word gets MOE_STATUS_TIMEOUT.
#include <algorithm>
#include <cmath>
#include <mutex>
#include <type_traits>

#include "tcgen05.cuh"
#include "w4.cuh"

namespace qe {

namespace {

constexpr int kM = 128;             // output features per tile (MMA M)
constexpr int kBlk = 128;           // contraction elements per code block
constexpr int kBlkBytes = 128 * 64; // codes of a block
constexpr int kGroups = 3;          // dequant groups of four warps
constexpr int kDeq = 4 * kGroups, kEpi = 4;   // warps
constexpr int kEpi0 = kDeq, kProd = kDeq + kEpi, kBProd = kProd + 1, kMma0 = kProd + 2;
constexpr int kGemmThreads = (kMma0 + 2) * 32;

template <int TOK, bool GRAD>
struct LGeo {
    static constexpr int chains = TOK > 128 ? 1 : 2;
    static constexpr int acc_cols = chains * TOK;       // accumulator columns
    static constexpr int a_cols = 32;                   // 64 contraction elements, two per column
    static constexpr int b_stage = TOK * 128;           // TOK rows of 64 elements
    // A and B stages (64 contraction elements each), in lockstep
    static constexpr int as = TOK > 128 ? 5 : TOK > 64 ? 7 : 12;
    // tensor-memory columns behind the A stages: the residual of the tokens from
    // 64 on, two per column
    static constexpr int res0 = acc_cols + as * a_cols, res_cols = (TOK - 64) / 2;
    // code blocks: a multiple of the groups, so that a group always reads the same ones
    static constexpr int cs = TOK > 64 ? 6 : 12;
    static constexpr int b_off = 0, c_off = as * b_stage;
    // gradient: per dequant group two buffers of a block's zero points and
    // scales, as the unpacking's operand words: [4 column quarters][64 row pairs]
    static constexpr int meta_off = c_off + cs * kBlkBytes;
    static constexpr int meta_buf = 4 * 64 * 12;
    static constexpr int bar_off = meta_off + (GRAD ? 2 * kGroups * meta_buf : 0);
    static constexpr int nbars = 2 * cs + 3 * as + 4;
    static constexpr int smem = bar_off + 8 * nbars + 16;
};
template <int TOK, bool GRAD>
constexpr bool lgeo_ok()
{
    using G = LGeo<TOK, GRAD>;
    return G::smem <= 227 * 1024 && G::res0 + G::res_cols <= 512 && G::cs % kGroups == 0 && G::as >= 5 &&
           (TOK > 128 || 128 * TOK * 4 <= G::c_off);    // a partial tile fits in the B stages
}
static_assert(lgeo_ok<256, false>() && lgeo_ok<128, false>() && lgeo_ok<64, false>() &&
                  lgeo_ok<256, true>() && lgeo_ok<128, true>() && lgeo_ok<64, true>(),
              "stages fit shared and tensor memory");

struct GemmCall {
    W4Call c;
    int tok;            // tokens per tile: a multiple of 16, at most TOK
    int mt, nt;         // tiles along the features and the tokens
    int splits;         // CTAs of a cluster along the contraction
    int vec_meta;       // a row's scales and zero points of 128 K allow vector loads
};

// 16 lanes x 32 columns from the warp's registers, 16x256b layout: of every 8
// columns thread (g, t) writes lane g, columns 2 t and 2 t + 1, then lane g + 8.
__device__ __forceinline__ void tmem_st_16x256(uint32_t taddr, const uint32_t (&v)[16])
{
    asm volatile(
        "tcgen05.st.sync.aligned.16x256b.x4.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
        "%11, %12, %13, %14, %15, %16};"
        ::"r"(taddr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]),
          "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]),
          "r"(v[13]), "r"(v[14]), "r"(v[15])
        : "memory");
}

// One answer for the four warps of a dequant group, which also orders their
// shared-memory writes before it against the reads after it.
__device__ __forceinline__ bool group_and(int id, bool v)
{
    uint32_t r;
    asm volatile("{\n .reg .pred p, q;\n setp.ne.b32 p, %1, 0;\n"
                 " barrier.cta.red.and.pred q, %2, 128, p;\n selp.u32 %0, 1, 0, q;\n}"
                 : "=r"(r)
                 : "r"((uint32_t)v), "r"(id)
                 : "memory");
    return r != 0;
}

template <typename S>
struct alignas(2 * sizeof(S)) ScalePair {
    S a, b;
};

// 16 columns to, and 8 from, this warp's 32 tensor-memory lanes.
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&v)[16])
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
        "%11, %12, %13, %14, %15, %16};"
        ::"r"(taddr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]),
          "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]),
          "r"(v[13]), "r"(v[14]), "r"(v[15])
        : "memory");
    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t (&v)[8])
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]),
                   "=r"(v[6]), "=r"(v[7])
                 : "r"(taddr));
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}

template <typename T>
__device__ __forceinline__ void store_out(const W4Call &c, float v, int tok, int f)
{
    using Q = W4<T>;
    if (c.bias)
        v += Q::to_float(static_cast<const T *>(c.bias)[f]);
    if (c.residual)
        v += Q::to_float(static_cast<const T *>(c.residual)[tok * c.ldr + f]);
    static_cast<T *>(c.out)[tok * c.ldo + f] = Q::from_float(v);
}

// Feature of tensor-memory lane m of a tile.
template <bool GRAD>
__device__ __forceinline__ int lane_feature(int m)
{
    return GRAD ? (m & ~31) | ((m & 7) << 2) | ((m >> 3) & 3) : m;
}

template <typename T, bool GRAD, int TOK>
__global__ void __launch_bounds__(kGemmThreads, 1)
    linear_gemm_kernel(const __grid_constant__ CUtensorMap wmap,
                       const __grid_constant__ CUtensorMap bmap, const GemmCall a)
{
    using G = LGeo<TOK, GRAD>;
    using Q = W4<T>;
    constexpr bool kBf16 = sizeof(typename Q::Scale) == 8;
    extern __shared__ __align__(1024) uint8_t smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (saddr(smem) & 1023) {       // the swizzled stages need it; never seen otherwise
        if (threadIdx.x == 0 && a.c.status)
            atomicOr(a.c.status, MOE_STATUS_TIMEOUT);
        return;
    }
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + G::bar_off);
    const uint32_t code_full = saddr(bars), code_empty = code_full + 8 * G::cs;
    const uint32_t a_full = code_empty + 8 * G::cs, b_full = a_full + 8 * G::as;
    const uint32_t stage_empty = b_full + 8 * G::as;    // the MMAs on A and B stage s are done
    const uint32_t acc_full = stage_empty + 8 * G::as, acc_empty = acc_full + 8;
    const uint32_t drain = acc_empty + 8;               // [2]
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + G::nbars);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);

    if (warp == kProd && lane == 0)
        prefetch_map(&wmap);
    if (warp == kBProd && lane == 0)
        prefetch_map(&bmap);
    if (threadIdx.x == 0) {
        for (int s = 0; s < G::cs; s++) {
            bar_init(code_full + 8 * s, 1);
            bar_init(code_empty + 8 * s, 4);
        }
        for (int s = 0; s < G::as; s++) {
            bar_init(a_full + 8 * s, 4);
            bar_init(b_full + 8 * s, 1);
            bar_init(stage_empty + 8 * s, G::chains);
        }
        bar_init(acc_full, G::chains);
        bar_init(acc_empty, kEpi);
        bar_init(drain, 1);
        bar_init(drain + 8, 1);
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == kMma0) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                     ::"r"(saddr(tmem_slot)), "r"(512u)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    pdl_enter();

    const W4Call &c = a.c;
    const int C = GRAD ? c.w.rows : c.w.K;      // contraction length
    const int F = GRAD ? c.w.K : c.w.rows;      // output features
    const int blocks = (C + kBlk - 1) / kBlk;
    const int rank = blockIdx.x % a.splits;
    const int blk0 = (int)((long long)blocks * rank / a.splits);
    const int blk1 = (int)((long long)blocks * (rank + 1) / a.splits);
    // 64-steps of this CTA: two per block, one when the contraction ends in its first half
    const int nsteps = 2 * (blk1 - blk0) - (blk1 == blocks && blk1 > blk0 && C - (blocks - 1) * kBlk <= 64);
    const int tile0 = blockIdx.x / a.splits, tile_step = gridDim.x / a.splits;
    const int tiles = a.mt * a.nt;
    bool ok = true;

    if (warp == kProd) {
        // -------------------------------------------------------- code producer
        if (lane == 0) {
            unsigned cc = 0;
            for (int t = tile0; t < tiles && ok; t += tile_step) {
                const int m0 = t % a.mt * kM;
                for (int b = blk0; b < blk1; b++, cc++) {
                    const uint32_t s = cc % G::cs;
                    if (!bar_wait(code_empty + 8 * s, ((cc / G::cs) & 1) ^ 1, abort_flag)) {
                        ok = false;
                        break;
                    }
                    bar_expect_tx(code_full + 8 * s, kBlkBytes);
                    tma_load_2d(saddr(smem + G::c_off + s * kBlkBytes), &wmap,
                                GRAD ? m0 / 2 : b * (kBlk / 2), GRAD ? b * kBlk : m0,
                                code_full + 8 * s);
                }
            }
            if (!ok) {
                *abort_flag = 1;
                for (unsigned i = cc > (unsigned)G::cs ? cc - G::cs : 0; i < cc; i++) {
                    const unsigned long long t0 = now_ns();
                    while (!bar_try(code_full + 8 * (i % G::cs), (i / G::cs) & 1) &&
                           now_ns() - t0 < kGWaitNs) {
                    }
                }
            }
        }
        __syncwarp();
    } else if (warp == kBProd) {
        // -------------------------------------------------------- B producer
        if (lane == 0) {
            unsigned bc = 0;
            for (int t = tile0; t < tiles && ok; t += tile_step) {
                const int tok0 = t / a.mt * a.tok;
                for (int j = 0; j < nsteps; j++, bc++) {
                    const uint32_t s = bc % G::as;
                    if (!bar_wait(stage_empty + 8 * s, ((bc / G::as) & 1) ^ 1, abort_flag)) {
                        ok = false;
                        break;
                    }
                    bar_expect_tx(b_full + 8 * s, a.tok * 128);
                    tma_load_2d(saddr(smem + G::b_off + s * G::b_stage), &bmap,
                                blk0 * kBlk + j * 64, tok0, b_full + 8 * s);
                }
            }
            if (!ok) {
                *abort_flag = 1;
                for (unsigned i = bc > (unsigned)G::as ? bc - G::as : 0; i < bc; i++) {
                    const unsigned long long t0 = now_ns();
                    while (!bar_try(b_full + 8 * (i % G::as), (i / G::as) & 1) &&
                           now_ns() - t0 < kGWaitNs) {
                    }
                }
            }
        }
        __syncwarp();
    } else if (warp >= kMma0) {
        // -------------------------------------------------------- MMA issuers
        // chain ch takes the steps of its parity into its own accumulator
        // Every lane walks the loop and one elected lane issues, so that the
        // descriptors stay in uniform registers: an issue from a branch of one
        // lane costs several times as much.
        const int ch = __shfl_sync(0xffffffffu, warp - kMma0, 0);
        if (ch < G::chains) {
            const uint32_t idesc = idesc_f16(a.tok, kBf16);
            const uint32_t dacc = tmem + ch * TOK;
            unsigned slot = 0, par = 0, ti = 0;
            bool issued = false;
            for (int t = tile0; t < tiles && ok; t += tile_step, ti++) {
                if (!warp_wait(acc_empty, (ti & 1) ^ 1, abort_flag)) {
                    ok = false;
                    break;
                }
                for (int j = 0; j < nsteps; j++) {
                    // Both chains wait for every step's A and release its stage, so
                    // that stages are released in step order; one of them
                    // multiplies.
                    const bool own = G::chains == 1 || (j & 1) == ch;
                    if (!warp_wait(a_full + 8 * slot, par, abort_flag) ||
                        (own && !warp_wait(b_full + 8 * slot, par, abort_flag))) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t abase = tmem + G::acc_cols + slot * G::a_cols;
                    const uint64_t bdesc = sw128_desc(saddr(smem + G::b_off) + slot * G::b_stage);
                    if (elect_one()) {
                        if (own) {
#pragma unroll
                            for (int kk = 0; kk < 4; kk++)      // 16 each: A 8 columns, B 32 bytes
                                umma_ta(dacc, abase + kk * 8, bdesc + 2 * kk, idesc,
                                        j >= G::chains || kk ? 1u : 0u);
                        }
                        umma_commit(stage_empty + 8 * slot);
                    }
                    __syncwarp();
                    issued = true;
                    if (++slot == (unsigned)G::as) {
                        slot = 0;
                        par ^= 1;
                    }
                }
                if (ok && elect_one())
                    umma_commit(acc_full);
                __syncwarp();
            }
            if (!ok && lane == 0)
                *abort_flag = 1;
            if (issued && elect_one()) {    // every MMA issued has completed before the memory is freed
                umma_commit(drain + 8 * ch);
                const unsigned long long t0 = now_ns();
                while (!bar_try(drain + 8 * ch, 0) && now_ns() - t0 < kGWaitNs) {
                }
            }
        }
        __syncwarp();
    } else if (warp >= kEpi0) {
        // -------------------------------------------------------- epilogue
        const int q = warp & 3;
        unsigned ti = 0;
        for (int t = tile0; t < tiles && ok; t += tile_step, ti++) {
            const int f = t % a.mt * kM + lane_feature<GRAD>(32 * q + lane);
            const int tok0 = t / a.mt * a.tok;
            const uint32_t taddr = tmem + ((uint32_t)(32 * q) << 16);
            const bool two = G::chains == 2 && nsteps > 1;
            const int cols = min(a.tok, c.n - tok0);
            float *part = reinterpret_cast<float *>(smem + G::b_off) +
                          lane_feature<GRAD>(32 * q + lane);    // in feature order
            const bool in = f < F;
            const float bias = c.bias && in ? Q::to_float(static_cast<const T *>(c.bias)[f]) : 0.f;
            T *out = static_cast<T *>(c.out) + tok0 * c.ldo + f;
            // The residual is read while the tile is still multiplied (with the
            // next tile's operands under way a load would take microseconds in the
            // epilogue): 64 tokens into registers, the others, as pairs, into
            // tensor-memory columns of their own.
            const bool add = !GRAD && c.residual && a.splits == 1;
            uint32_t held[2][16];
            if (add) {
                const T *res = static_cast<const T *>(c.residual) + tok0 * c.ldr + f;
                const auto load32 = [&](int c0, uint32_t (&h)[16]) {
                    uint16_t v[32];
#pragma unroll
                    for (int i = 0; i < 32; i++) {
                        v[i] = 0;
                        if (in && c0 + i < cols)
                            v[i] = *reinterpret_cast<const uint16_t *>(res + (c0 + i) * c.ldr);
                    }
#pragma unroll
                    for (int i = 0; i < 16; i++)
                        h[i] = v[2 * i] | (uint32_t)v[2 * i + 1] << 16;
                };
                for (int c0 = 64; c0 < cols; c0 += 32) {
                    load32(c0, held[0]);
                    __syncwarp();
                    tmem_st16(taddr + G::res0 + (c0 - 64) / 2, held[0]);
                }
                load32(0, held[0]);
                load32(32, held[1]);
                __syncwarp();
            }
            if (!warp_wait(acc_full, ti & 1, abort_flag)) {
                ok = false;
                break;
            }
            tc_fence_after();
            // 16 tokens' sums, with 8 words of their residual, to the output
            const auto finish = [&](int c0, auto with, const uint32_t (&h)[8]) {
                float d[16], e[16];
                tmem_ld16(taddr + c0, d);
                if (two) {
                    tmem_ld16(taddr + TOK + c0, e);
#pragma unroll
                    for (int i = 0; i < 16; i++)
                        d[i] += e[i];
                }
                if (a.splits > 1) {     // uniform over the grid
#pragma unroll
                    for (int i = 0; i < 16; i++)
                        part[(c0 + i) * kM] = d[i];
                    return;
                }
                const int left = in ? cols - c0 : 0;
                if (with.value) {
#pragma unroll
                    for (int i = 0; i < 8; i++) {
                        d[2 * i] += Q::low(h[i]);
                        d[2 * i + 1] += Q::high(h[i]);
                    }
                }
                if (left >= 16) {
#pragma unroll
                    for (int i = 0; i < 16; i++, out += c.ldo)
                        *out = Q::from_float(d[i] + bias);
                } else {
#pragma unroll
                    for (int i = 0; i < 16; i++, out += c.ldo)
                        if (i < left)
                            *out = Q::from_float(d[i] + bias);
                }
                __syncwarp();
            };
            if (!add) {
                const uint32_t none[8] = {};
                for (int c0 = 0; c0 < cols; c0 += 16)
                    finish(c0, std::false_type(), none);
            } else {
#pragma unroll
                for (int u = 0; u < 4; u++)
                    if (16 * u < cols) {
                        uint32_t h[8];
#pragma unroll
                        for (int i = 0; i < 8; i++)
                            h[i] = held[u >> 1][8 * (u & 1) + i];
                        finish(16 * u, std::true_type(), h);
                    }
                for (int c0 = 64; c0 < cols; c0 += 16) {
                    uint32_t h[8];
                    tmem_ld8(taddr + G::res0 + (c0 - 64) / 2, h);
                    finish(c0, std::true_type(), h);
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0)
                bar_arrive(acc_empty);
        }
        if (!ok && lane == 0)
            *abort_flag = 1;
        __syncwarp();
    } else {
        // -------------------------------------------------------- dequant
        const int q = warp & 3, wg = warp >> 2, tq = lane & 3;
        const uint32_t tlane = (uint32_t)(32 * q) << 16;
        const int ng = c.w.K / c.w.group, gsh = c.w.group == 128 ? 7 : c.w.group == 64 ? 6 : 5;
        const int per_blk = kBlk / c.w.group;       // groups along 128 K
        const int r = 32 * q + lane;
        // Scales and zero points (0 outside the matrix) of one matrix row over 128
        // K: forward, this thread's row of the tile over the block; gradient,
        // row r of the block over the tile.  They are loaded one block ahead and
        // first touched a block later: a warp stalls on a loaded value where it
        // is used.
        struct Meta {
            uint32_t s[2], z;       // group j's scale in half j, zero point in byte j
            __device__ __forceinline__ uint32_t scale(int j) const
            {
                return j & 1 ? s[j >> 1] >> 16 : s[j >> 1] & 0xffff;
            }
            __device__ __forceinline__ uint32_t zero(int j) const { return z >> (8 * j) & 0xff; }
        };
        const auto load_meta = [&](int m0, int b, Meta &m) {
            const int row = (GRAD ? b * kBlk : m0) + r;
            const int g0 = (GRAD ? m0 : b * kBlk) >> gsh;
            m.s[0] = m.s[1] = m.z = 0;
            if (row >= c.w.rows)
                return;
            const uint16_t *sp = c.w.scales + (long long)row * ng + g0;
            const uint8_t *zp = c.w.zeros + (long long)row * ng + g0;
            if (per_blk == 1) {
                m.s[0] = *sp;       // g0 < ng: a block begins inside the matrix
                m.z = *zp;
            } else if (a.vec_meta) {
                if (per_blk == 2) {
                    m.s[0] = *reinterpret_cast<const uint32_t *>(sp);
                    m.z = *reinterpret_cast<const uint16_t *>(zp);
                } else {
                    const uint2 v = *reinterpret_cast<const uint2 *>(sp);
                    m.s[0] = v.x;
                    m.s[1] = v.y;
                    m.z = *reinterpret_cast<const uint32_t *>(zp);
                }
            } else {
#pragma unroll
                for (int j = 0; j < 4; j++)
                    if (j < per_blk && g0 + j < ng) {
                        m.s[j >> 1] |= (uint32_t)sp[j] << (16 * (j & 1));
                        m.z |= (uint32_t)zp[j] << (8 * j);
                    }
            }
        };
        // this group's place in the CTA's blocks: every kGroups-th one of them
        struct Place {
            int t, m0, b;
            unsigned cc, ac0;       // blocks before this one; 64-steps before this tile
        };
        const int nb = blk1 - blk0;
        const auto settle = [&](Place &p) {
            if (p.b >= blk1) {
                do {
                    p.b -= nb;
                    p.t += tile_step;
                    p.ac0 += nsteps;
                } while (p.b >= blk1);
                p.m0 = p.t % a.mt * kM;
            }
        };
        Place at{tile0, tile0 % a.mt * kM, blk0 + wg, (unsigned)wg, 0u};
        settle(at);
        Meta meta{}, next{};
        if (at.t < tiles)
            load_meta(at.m0, at.b, next);
        for (unsigned buf = 0; at.t < tiles && (GRAD || ok); buf ^= 1) {
            const int b = at.b, steps = b + 1 == blocks && C - b * kBlk <= 64 ? 1 : 2;
            const unsigned cc = at.cc;
            unsigned ac = at.ac0 + 2 * (b - blk0);
            meta = next;
            at.b += kGroups;
            at.cc += kGroups;
            settle(at);
            if (at.t < tiles)       // the next block's arrive while this one is unpacked
                load_meta(at.m0, at.b, next);
            const uint32_t s = cc % G::cs;
            // gradient: this group's words of the block (zero points, then scales)
            uint32_t *zw = reinterpret_cast<uint32_t *>(smem + G::meta_off +
                                                        (2 * wg + buf) * G::meta_buf);
            typename Q::Scale *sw = reinterpret_cast<typename Q::Scale *>(zw + 4 * 64);
            if (GRAD) {
#pragma unroll
                for (int j = 0; j < 4; j++)
                    if (j < per_blk) {      // a row pair's two words, one by each of its lanes
                        const uint32_t s1 = meta.scale(j), z1 = meta.zero(j);
                        const uint32_t s2 = __shfl_xor_sync(0xffffffffu, s1, 1);
                        const uint32_t z2 = __shfl_xor_sync(0xffffffffu, z1, 1);
                        if (lane & 1)
                            sw[64 * j + (r >> 1)] = Q::scale(s2, s1);
                        else
                            zw[64 * j + (r >> 1)] = Q::zero(z1, z2).lo;
                    }
            }
            bool have = ok && warp_wait(code_full + 8 * s, (cc / G::cs) & 1, abort_flag);
            if (GRAD)       // the group's words are written; its warps go on, or leave, together
                have = group_and(1 + wg, have);
            if (!have) {
                ok = false;
                break;
            }
            const uint8_t *blk = smem + G::c_off + s * kBlkBytes;
            uint4 cw[4];
            if (!GRAD) {
                // row r's 16-byte chunk i sits at i ^ (r / 2 % 4) (64-byte swizzle)
#pragma unroll
                for (int i = 0; i < 4; i++)
                    cw[i] = *reinterpret_cast<const uint4 *>(blk + r * 64 +
                                                             ((i ^ ((r >> 1) & 3)) << 4));
                // the codes are in registers before the copy engine writes the block
                // again: without the fence these reads may still be on their way
                fence_async_shared();
                __syncwarp();
                if (lane == 0)
                    bar_arrive(code_empty + 8 * s);
            }
#pragma unroll
            for (int h = 0; h < 2; h++) {
                if (h >= steps)
                    break;
                const uint32_t as = ac % G::as;
                uint32_t col[32];
                if (!GRAD) {
#pragma unroll
                    for (int i = 0; i < 2; i++) {
                        // quarter 2 h + i of the block: its group's
                        const int j = 2 * h + i;
                        const uint32_t zb = per_blk == 1   ? meta.zero(0)
                                            : per_blk == 2 ? meta.zero(j / 2)
                                                           : meta.zero(j);
                        const uint32_t sb = per_blk == 1   ? meta.scale(0)
                                            : per_blk == 2 ? meta.scale(j / 2)
                                                           : meta.scale(j);
                        const typename Q::Zero z = Q::zero(zb, zb);
                        const typename Q::Scale sc = Q::scale(sb, sb);
                        const uint4 v = cw[2 * h + i];
                        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                        for (int u = 0; u < 4; u++) {
                            uint32_t p[4];
                            Q::unpack(w[u], z, p);
#pragma unroll
                            for (int n = 0; n < 4; n++)
                                p[n] = Q::mul(p[n], sc);
                            // fields (i, i + 4) into memory order
                            col[16 * i + 4 * u] = __byte_perm(p[0], p[1], 0x5410);
                            col[16 * i + 4 * u + 1] = __byte_perm(p[2], p[3], 0x5410);
                            col[16 * i + 4 * u + 2] = __byte_perm(p[0], p[1], 0x7632);
                            col[16 * i + 4 * u + 3] = __byte_perm(p[2], p[3], 0x7632);
                        }
                    }
                } else {
                    const int slot = 64 * ((32 * q) >> gsh) + 32 * h + 2 * tq;
                    // Tiles of 8 rows x 16 bytes, transposed, for 16 rows of the
                    // contraction in memory order: the rows 4 tq, + 1 and 4 tq + 2,
                    // + 3 of each 16.  Row r's 16-byte chunk q sits at q ^ (r / 2 %
                    // 4) (64-byte swizzle).
                    uint32_t w[4][2];
#pragma unroll
                    for (int ss = 0; ss < 4; ss += 2) {
                        const int rr = 64 * h + 16 * (ss + (lane >> 4)) + 4 * (lane >> 1 & 3) +
                                       2 * (lane >> 3 & 1) + (lane & 1);
                        uint32_t d[4];
                        ldmatrix4_trans(d, saddr(blk) + rr * 64 + ((q ^ (rr >> 1 & 3)) << 4));
                        w[ss][0] = d[0];
                        w[ss][1] = d[1];
                        w[ss + 1][0] = d[2];
                        w[ss + 1][1] = d[3];
                    }
#pragma unroll
                    for (int ss = 0; ss < 4; ss++) {        // 16 rows: pairs 8 ss + 2 tq, + 1
                        const uint2 zz = *reinterpret_cast<const uint2 *>(zw + slot + 8 * ss);
                        const typename Q::Zero z01 = Q::zero_of(zz.x), z23 = Q::zero_of(zz.y);
                        const ScalePair<typename Q::Scale> sc =
                            *reinterpret_cast<const ScalePair<typename Q::Scale> *>(sw + slot + 8 * ss);
                        uint32_t p[4], p2[4];
                        Q::unpack(w[ss][0], z01, p);
                        Q::unpack(w[ss][1], z23, p2);
                        // columns 0, 1 of the quad to lanes 0..15, 2, 3 to 16..31
#pragma unroll
                        for (int u = 0; u < 4; u++) {
                            const int to = 16 * (u >> 1) + 4 * ss + 2 * (u & 1);
                            col[to] = Q::mul(p[u], sc.a);
                            col[to + 1] = Q::mul(p2[u], sc.b);
                        }
                    }
                    if (h + 1 == steps) {
                        fence_async_shared();       // as above
                        __syncwarp();
                        if (lane == 0)
                            bar_arrive(code_empty + 8 * s);
                    }
                }
                // A parity wait cannot tell a phase from the one two before it.
                // Stages are released in step order, and this group last waited for
                // a step at most 5 before this one, so the use before the one
                // waited for has ended (as >= 5).
                if (!warp_wait(stage_empty + 8 * as, ((ac / G::as) & 1) ^ 1, abort_flag)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t dst = tmem + tlane + G::acc_cols + as * G::a_cols;
                if (!GRAD) {
                    tmem_st32(dst, col);
                } else {
                    uint32_t lo[16], hi[16];
#pragma unroll
                    for (int i = 0; i < 16; i++) {
                        lo[i] = col[i];
                        hi[i] = col[16 + i];
                    }
                    tmem_st_16x256(dst, lo);
                    tmem_st_16x256(dst + (16u << 16), hi);
                    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    bar_arrive(a_full + 8 * as);
                ac++;
            }
        }
        if (!ok && lane == 0)
            *abort_flag = 1;
        __syncwarp();
    }

    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kMma0)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u)
                     : "memory");
    if (*abort_flag) {      // what a wait that gave up left out is no result: NaN
        if (threadIdx.x == 0 && c.status)
            atomicOr(c.status, MOE_STATUS_TIMEOUT);
        float *part = reinterpret_cast<float *>(smem + G::b_off);
        for (int t = tile0; t < tiles; t += tile_step)
            for (int i = threadIdx.x; i < a.tok * kM; i += kGemmThreads) {
                const int tok = t / a.mt * a.tok + i / kM, f = t % a.mt * kM + i % kM;
                if (a.splits > 1)       // the sum over the cluster
                    part[i] = NAN;
                else if (tok < c.n && f < F)
                    static_cast<T *>(c.out)[tok * c.ldo + f] = Q::from_float(NAN);
            }
    }
    if (a.splits > 1) {
        // the one tile of this cluster: rank r adds its share of the tokens
        cluster_arrive();
        cluster_wait();
        const int m0 = tile0 % a.mt * kM, tok0 = tile0 / a.mt * a.tok;
        const int lo = a.tok * rank / a.splits, hi = a.tok * (rank + 1) / a.splits;
        const uint32_t base = saddr(smem + G::b_off);
        for (int i = lo * kM + 4 * threadIdx.x; i < hi * kM; i += 4 * kGemmThreads) {
            const int tok = tok0 + i / kM, f = m0 + i % kM;
            if (tok >= c.n || f >= F)
                continue;
            float4 p[8];
#pragma unroll
            for (int r = 0; r < 8; r++) {
                p[r] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (r < a.splits) {
                    const uint32_t remote = cluster_addr(base + 4 * i, r);
                    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                                 : "=f"(p[r].x), "=f"(p[r].y), "=f"(p[r].z), "=f"(p[r].w)
                                 : "r"(remote));
                }
            }
            float v[4] = {};
#pragma unroll
            for (int r = 0; r < 8; r++) {
                v[0] += p[r].x;
                v[1] += p[r].y;
                v[2] += p[r].z;
                v[3] += p[r].w;
            }
#pragma unroll
            for (int u = 0; u < 4; u++)
                if (f + u < F)
                    store_out<T>(c, v[u], tok, f + u);
        }
        cluster_arrive();
        cluster_wait();     // a CTA's shared memory stays until its peers have read it
    }
}

using EncodeFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                              const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                              const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encoder()
{
    static const EncodeFn fn = [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000,
                                             cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess) {
            cudaGetLastError();
            p = nullptr;
        }
        return reinterpret_cast<EncodeFn>(p);
    }();
    return fn;
}

// Clusters of each size that run at once (they cannot use every SM: a GPC
// holds a whole number of them), looked up once per device.
constexpr int kMaxSplits = 8;
struct Clusters {
    std::once_flag once;
    int n[kMaxSplits + 1] = {};
};

}  // namespace

bool encode_map(CUtensorMap *map, CUtensorMapDataType type, const void *base, uint64_t cols,
            uint64_t rows, uint64_t pitch, uint32_t box_cols, uint32_t box_rows,
            CUtensorMapSwizzle swizzle)
{
    const EncodeFn fn = encoder();
    if (!fn)
        return false;
    const cuuint64_t dims[2] = {cols, rows}, strides[1] = {pitch};
    const cuuint32_t box[2] = {box_cols, box_rows}, estr[2] = {1, 1};
    return fn(map, type, 2, const_cast<void *>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

const int *cluster_table(int dev)
{
    constexpr int kMaxDevices = 64;
    static Clusters table[kMaxDevices];
    static const int none[kMaxSplits + 1] = {};
    if (dev < 0 || dev >= kMaxDevices)
        return none;        // no splits
    Clusters &t = table[dev];
    std::call_once(t.once, [&t] {
        auto kernel = linear_gemm_kernel<__half, false, 128>;
        constexpr int smem = LGeo<128, false>::smem;
        if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) !=
            cudaSuccess) {
            cudaGetLastError();
            return;
        }
        for (int s = 2; s <= kMaxSplits; s++) {
            cudaLaunchConfig_t cfg = {};
            cfg.gridDim = dim3(s);
            cfg.blockDim = dim3(kGemmThreads);
            cfg.dynamicSmemBytes = smem;
            cudaLaunchAttribute attr[1];
            attr[0].id = cudaLaunchAttributeClusterDimension;
            attr[0].val.clusterDim.x = s;
            attr[0].val.clusterDim.y = 1;
            attr[0].val.clusterDim.z = 1;
            cfg.attrs = attr;
            cfg.numAttrs = 1;
            if (cudaOccupancyMaxActiveClusters(&t.n[s], kernel, &cfg) != cudaSuccess) {
                cudaGetLastError();
                t.n[s] = 0;
            }
        }
    });
    return t.n;
}

namespace {

struct Plan {
    int tok, nt, splits;
};

// Tokens per tile and splits along the contraction: the smallest estimated time,
// in SM cycles, of the busiest SM.  Measured: a 64-step of a tile of N tokens
// takes 2 N cycles on the tensor core, and whatever N at least about 480 for its
// dequantisation (560 in the gradient); a tile's epilogue takes about 20 N and
// the exchange of a cluster's partial tiles 2500 + 8 N.
Plan plan(int C, int F, int n, int grad, int num_sms, const int *clusters)
{
    const int mt = (F + kM - 1) / kM, steps = (C + 63) / 64;
    Plan best{};
    double least = 0;
    for (int most = 256; most >= 16; most -= 16) {
        const int nt = (n + most - 1) / most, tok = ((n + nt - 1) / nt + 15) / 16 * 16;
        if (tok == best.tok)
            continue;
        for (int s = 1; s == 1 || (s <= kMaxSplits && tok <= 128 && 4 * s <= steps); s++) {
            const long long ctas = (long long)mt * nt * s;
            if (s > 1 && (long long)mt * nt > clusters[s])
                continue;       // a cluster would wait for another one's SMs
            const double waves = (double)((ctas + num_sms - 1) / num_sms);
            const double step = std::max(2.0 * tok, grad ? 560.0 : 480.0);
            const double cost = waves * ((steps + s - 1) / s * step + 20.0 * tok) +
                                (s > 1 ? 2500 + 8.0 * tok : 0);
            if (!best.tok || cost < least) {
                best = {tok, nt, s};
                least = cost;
            }
        }
    }
    return best;
}

template <typename T, bool GRAD, int TOK>
cudaError_t launch(const GemmCall &a, const CUtensorMap &wmap, const CUtensorMap &bmap, int num_sms,
                   cudaStream_t st)
{
    auto kernel = linear_gemm_kernel<T, GRAD, TOK>;
    const cudaError_t e =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, LGeo<TOK, GRAD>::smem);
    if (e != cudaSuccess)
        return e;
    const long long tiles = (long long)a.mt * a.nt;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(a.splits > 1 ? tiles * a.splits : std::min<long long>(tiles, num_sms)));
    cfg.blockDim = dim3(kGemmThreads);
    cfg.dynamicSmemBytes = LGeo<TOK, GRAD>::smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = a.splits;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kernel, wmap, bmap, a);
}

template <typename T, bool GRAD>
cudaError_t launch_tok(const GemmCall &a, const CUtensorMap &wmap, const CUtensorMap &bmap,
                       int num_sms, cudaStream_t st)
{
    if (a.tok > 128)
        return launch<T, GRAD, 256>(a, wmap, bmap, num_sms, st);
    if (a.tok > 64)
        return launch<T, GRAD, 128>(a, wmap, bmap, num_sms, st);
    return launch<T, GRAD, 64>(a, wmap, bmap, num_sms, st);
}

}  // namespace

// Whether the activations can be read by TMA (rows on 16-byte boundaries).
bool linear_gemm_fits(const W4Call &c)
{
    return reinterpret_cast<uintptr_t>(c.in) % 16 == 0 && c.ldi % 8 == 0;
}

cudaError_t launch_linear_gemm(const W4Call &c, int bf16, int grad, int dev, int num_sms,
                               cudaStream_t st)
{
    const int C = grad ? c.w.rows : c.w.K, F = grad ? c.w.K : c.w.rows;
    const Plan p = plan(C, F, c.n, grad, num_sms, cluster_table(dev));
    const int vec_meta = c.w.K % 128 == 0 && reinterpret_cast<uintptr_t>(c.w.scales) % 8 == 0 &&
                         reinterpret_cast<uintptr_t>(c.w.zeros) % 4 == 0;
    GemmCall a{c, p.tok, (F + kM - 1) / kM, p.nt, p.splits, vec_meta};
    CUtensorMap wmap, bmap;
    if (!encode_map(&wmap, CU_TENSOR_MAP_DATA_TYPE_UINT8, c.w.codes, c.w.K / 2, c.w.rows, c.w.K / 2, 64,
                128, CU_TENSOR_MAP_SWIZZLE_64B) ||
        !encode_map(&bmap, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                c.in, C, c.n, 2 * c.ldi, 64, p.tok, CU_TENSOR_MAP_SWIZZLE_128B))
        return cudaErrorInvalidValue;
    if (bf16)
        return grad ? launch_tok<__nv_bfloat16, true>(a, wmap, bmap, num_sms, st)
                    : launch_tok<__nv_bfloat16, false>(a, wmap, bmap, num_sms, st);
    return grad ? launch_tok<__half, true>(a, wmap, bmap, num_sms, st)
                : launch_tok<__half, false>(a, wmap, bmap, num_sms, st);
}

}  // namespace qe
