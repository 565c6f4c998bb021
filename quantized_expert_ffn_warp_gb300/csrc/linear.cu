// 4-bit group-quantised products for few tokens, on the warp MMA:
//   moe_linear              y[t][r]  = sum_k x[t][k] W[r][k] (+ bias) (+ residual)
//   moe_linear_input_grad   dx[t][k] = sum_r dy[t][r] W[r][k]
// with W = (q - z) * s in the canonical layout ("Strata" article, section 2.2:
// one scale and one zero point per group along K; section 3.4: hand-written
// INT4 GEMV; "Flash-MoE", section 3: dequant matvec).
//
// Both are bound by the stream of packed bytes.  The weights are the MMA's A
// operand (M = 16), the tokens its N = 8 columns.  The MMA's K order is free as
// long as A and B agree, so a lane's MMA elements are the nibbles of whole
// words, and no lane exchanges weights with another.
//
// One CTA per SM.  Each of its (up to 16) warps has its own slice of the matrix
// and its own ring in shared memory, which TMA fills ahead; the warp refills a
// stage itself as soon as it has read it, so that about 128 KB per SM are under
// way whatever the arithmetic does, and no warp waits for another.
//
// Measured in a replayed graph over more inputs than L2 holds: 1 token 2048 x
// 2048 fp16 3.2 us (latency); 8 tokens 4096 x 14336 bf16 14.9 us; 3 tokens 32003
// x 4096 fp16 19.7 us; 8 tokens 256000 x 4096 fp16 114 us, 4.9 TB/s: the issue of
// unpacking and MMA together bounds it (without both 75 us).  Gradient: 2 tokens
// 1027 x 2048 fp16 7.4 us, 8 tokens 14336 x 4096 bf16 15.4 us.
#include <algorithm>
#include <cmath>

#include "w4.cuh"

namespace qe {

namespace {

constexpr int kWarps = 16;              // multiplying warps
constexpr int kRing = 8 * 1024;         // bytes per warp
constexpr int kAdders = 4;              // warps that add: one per scheduler, as they cost issue slots

// ---- y = x W^T -------------------------------------------------------------
// A stage is 16 RT rows x a slice of 256 K, i.e. 128 bytes of each row (128-byte
// swizzle).  The warps of a row tile (16 RT rows) take its slices in turn; up
// to 4096 K a warp has one slice for the whole call, and that slice's
// activations stay in its registers as MMA operands.  Of 128 K, lane (g, t)
// holds word t of each of the four 16-byte pieces v of rows g and g + 8, i.e. K =
// 32 v + 8 t .. + 7, whose fields (i, i + 4) pair with the activations (i, i
// + 4) of the same 8.  So two MMAs cover 32 consecutive K: the products with
// the exact integers q - z are summed over one group and the fp32 sum is
// scaled; no weight is rounded, for any group size.
// A tile's partial sums go to four more warps through shared memory, which add
// them in order and store the results while the others go on.
struct FwdArgs {
    W4Call c;
    int kw_n, rw_n;     // warps along K, and row tiles at a time, of a CTA
    int vec_meta;       // rows of scales and zero points allow vector loads
};

template <int RT>
struct FwdGeo {
    static constexpr int stage = RT * 16 * 128, stages = kRing / stage;
    static constexpr int out = 16 * RT * 8;                // results of a row tile
    static constexpr int red_off = kWarps * kRing;              // [2][kWarps][out] sums
    static constexpr int bar_off = red_off + 2 * 4 * kWarps * out;
    static constexpr int nbars = kWarps * stages + 4;   // full stages; sums full, empty
    static constexpr int smem = bar_off + 8 * nbars + 16;
};
static_assert(FwdGeo<1>::smem <= 227 * 1024 && FwdGeo<2>::smem <= 227 * 1024, "shared memory");

// A row's scales and zero points over 256 K, as loaded.
template <int GS>
struct RowMeta;
template <>
struct RowMeta<128> {
    uint32_t s, z;
    __device__ __forceinline__ void load(const uint16_t *sp, const uint8_t *zp)
    {
        s = *reinterpret_cast<const uint32_t *>(sp);
        z = *reinterpret_cast<const uint16_t *>(zp);
    }
};
template <>
struct RowMeta<64> {
    uint2 s;
    uint32_t z;
    __device__ __forceinline__ void load(const uint16_t *sp, const uint8_t *zp)
    {
        s = *reinterpret_cast<const uint2 *>(sp);
        z = *reinterpret_cast<const uint32_t *>(zp);
    }
};
template <>
struct RowMeta<32> {
    uint4 s;
    uint2 z;
    __device__ __forceinline__ void load(const uint16_t *sp, const uint8_t *zp)
    {
        s = *reinterpret_cast<const uint4 *>(sp);
        z = *reinterpret_cast<const uint2 *>(zp);
    }
};

// The same by single loads; 0 past the row's end (its scale times the padding's
// zeros has to be 0, whatever the last group's scale).
template <int GS>
__device__ __forceinline__ void load_each(RowMeta<GS> &m, const uint16_t *sp, const uint8_t *zp,
                                          int left)
{
    constexpr int N = 256 / GS;
    uint32_t s[(N + 1) / 2] = {}, z[(N + 3) / 4] = {};
#pragma unroll
    for (int i = 0; i < N; i++) {
        if (i < left) {
            s[i / 2] |= (uint32_t)sp[i] << (16 * (i & 1));
            z[i / 4] |= (uint32_t)zp[i] << (8 * (i & 3));
        }
    }
    memcpy(&m.s, s, sizeof(m.s));
    memcpy(&m.z, z, sizeof(m.z));
}

// Group i's zero point and scale out of a row's.
__device__ __forceinline__ uint32_t word_of(uint32_t v, int) { return v; }
__device__ __forceinline__ uint32_t word_of(const uint2 &v, int i) { return i ? v.y : v.x; }
__device__ __forceinline__ uint32_t word_of(const uint4 &v, int i)
{
    return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
}
template <typename Q, typename M>
__device__ __forceinline__ typename Q::Zero group_zero(const M &m, int i)
{
    const uint32_t z = word_of(m.z, i / 4) >> (8 * (i & 3)) & 0xff;
    return Q::zero(z, z);
}
template <typename M>
__device__ __forceinline__ float group_scale(const M &m, int i)
{
    return __half2float(__ushort_as_half((unsigned short)(word_of(m.s, i / 2) >> (16 * (i & 1)))));
}

// After a wait that gave up: the copies still in flight, waited for with a
// limit before the shared memory is given back.
__device__ __forceinline__ void drain(uint32_t full, int stages, unsigned arrived, unsigned issued)
{
    for (; arrived < issued; arrived++) {
        const unsigned long long t0 = now_ns();
        while (!bar_try(full + 8 * (arrived % stages), arrived / stages & 1) &&
               now_ns() - t0 < kGWaitNs) {
        }
    }
}

template <typename T, int GS, int RT>
__global__ void __launch_bounds__(32 * (kWarps + kAdders), 1)
    linear_kernel(const __grid_constant__ CUtensorMap wmap, const FwdArgs a)
{
    using Q = W4<T>;
    using G = FwdGeo<RT>;
    extern __shared__ __align__(1024) uint8_t smem[];
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + G::bar_off);
    const uint32_t red_full = saddr(bars + kWarps * G::stages), red_empty = red_full + 16;
    volatile int *abort_flag = reinterpret_cast<volatile int *>(bars + G::nbars);
    const W4Call &c = a.c;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int warps = a.kw_n * a.rw_n;      // multiplying warps; the next ones add
    const int kw = warp % a.kw_n, rw = warp / a.kw_n;
    const uint32_t full = saddr(bars + warp * G::stages);
    const uint32_t ring = saddr(smem) + warp * kRing;
    if (saddr(smem) & 1023) {       // the swizzled stages need it; never seen otherwise
        if (threadIdx.x == 0 && c.status)
            atomicOr(c.status, MOE_STATUS_TIMEOUT);
        return;
    }
    if (lane == 0) {
        if (warp < warps) {
            prefetch_map(&wmap);
            for (int i = 0; i < G::stages; i++)
                bar_init(full + 8 * i, 1);
        } else if (warp == warps) {
            for (int i = 0; i < 2; i++) {
                bar_init(red_full + 8 * i, warps);
                bar_init(red_empty + 8 * i, kAdders);
            }
            *abort_flag = 0;
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncthreads();
    pdl_enter();

    const int rows = c.w.rows, K = c.w.K, tok0 = blockIdx.y * 8, ng = K / GS;
    const int tiles = (rows + 16 * RT - 1) / (16 * RT), sets = (tiles + a.rw_n - 1) / a.rw_n;
    const int slices = (K + 255) / 256;
    bool ok = true;

    if (warp < warps) {
        // ------------------------------------------------------ multiply
        // a stage's place: set of row tiles, and slice of K
        struct Place {
            int set, slice;
        };
        const auto advance = [&](Place &p) {
            p.slice += a.kw_n;
            if (p.slice >= slices) {
                p.slice = kw;
                p.set += gridDim.x;
            }
        };
        unsigned issued = 0, arrived = 0;       // copies
        const auto fetch = [&](const Place &p, int slot) {
            issued++;
            if (lane == 0) {
                bar_expect_tx(full + 8 * slot, G::stage);
                tma_load_2d(ring + slot * G::stage, &wmap, p.slice * 128,
                            (p.set * a.rw_n + rw) * 16 * RT, full + 8 * slot);
            }
        };
        Place first{(int)blockIdx.x, kw}, filled = first, loaded = first;
        for (int i = 0; i < G::stages; i++)
            if (filled.set < sets) {
                fetch(filled, i);
                advance(filled);
            }

        // Scales and zero points of a stage: lane l those of row l.  They are
        // loaded two stages ahead, about as far as the codes: with that much
        // under way a load takes several microseconds.
        const auto load_meta = [&](const Place &p, RowMeta<GS> &m) {
            // rows past the matrix repeat its last row; their sums are not stored
            const int row = min((p.set * a.rw_n + rw) * 16 * RT + (lane & (16 * RT - 1)), rows - 1);
            const int at = p.slice * (256 / GS);
            const uint16_t *sp = c.w.scales + (long long)row * ng + at;
            const uint8_t *zp = c.w.zeros + (long long)row * ng + at;
            if (a.vec_meta)
                m.load(sp, zp);
            else
                load_each<GS>(m, sp, zp, ng - at);
        };
        RowMeta<GS> ahead[2] = {};
#pragma unroll
        for (int i = 0; i < 2; i++)
            if (loaded.set < sets) {
                load_meta(loaded, ahead[i]);
                advance(loaded);
            }

        // a slice's activations as B operands: fields (i, i + 4) of each 8
        uint32_t xb[2][4][4];
        const auto load_x = [&](int slice) {
#pragma unroll
            for (int j = 0; j < 2; j++)
#pragma unroll
                for (int v = 0; v < 4; v++) {
                    const int tok = tok0 + g, k = slice * 256 + 128 * j + 32 * v + 8 * t;
                    uint4 b = make_uint4(0, 0, 0, 0);
                    if (tok < c.n && k < K)
                        b = *reinterpret_cast<const uint4 *>(static_cast<const T *>(c.in) +
                                                             tok * c.ldi + k);
                    xb[j][v][0] = __byte_perm(b.x, b.z, 0x5410);
                    xb[j][v][1] = __byte_perm(b.x, b.z, 0x7632);
                    xb[j][v][2] = __byte_perm(b.y, b.w, 0x5410);
                    xb[j][v][3] = __byte_perm(b.y, b.w, 0x7632);
                }
        };
        if (slices <= a.kw_n)
            load_x(kw);

        int slot = 0;
        uint32_t parity = 0, buf = 0, red_parity = 1;
        for (int set = blockIdx.x; set < sets; set += gridDim.x) {
            float acc[RT][4];
#pragma unroll
            for (int r = 0; r < RT; r++)
#pragma unroll
                for (int i = 0; i < 4; i++)
                    acc[r][i] = 0.f;
            for (int slice = kw; slice < slices; slice += a.kw_n) {
                if (slices > a.kw_n)
                    load_x(slice);
                const RowMeta<GS> meta = ahead[0];
                ahead[0] = ahead[1];
                if (loaded.set < sets) {
                    load_meta(loaded, ahead[1]);
                    advance(loaded);
                }
                if (ok && !warp_wait(full + 8 * slot, parity, abort_flag)) {
                    ok = false;
                    *abort_flag = 1;
                    __threadfence_block();
                }
                arrived += ok;
                const uint32_t stage = ring + slot * G::stage;
#pragma unroll
                for (int r = 0; r < RT; r++) {
                    // of rows g and g + 8 of this 16-row tile
                    const RowMeta<GS> m0 = shfl_of(meta, 16 * r + g), m1 = shfl_of(meta, 16 * r + g + 8);
#pragma unroll
                    for (int j = 0; j < 2; j++) {
                        uint32_t w0[4], w1[4];
                        // 16-byte piece p of row r sits at p ^ (r % 8)
                        const uint32_t row = stage + (r * 16 + (lane & 7)) * 128 +
                                             (((4 * j + (lane >> 3)) ^ (lane & 7)) << 4);
                        ldmatrix4(w0, row);
                        ldmatrix4(w1, row + 8 * 128);
                        float part[4];
                        typename Q::Zero z0, z1;
                        float f0 = 0.f, f1 = 0.f;
#pragma unroll
                        for (int v = 0; v < 4; v++) {
                            if ((32 * v) % GS == 0) {       // a group begins
                                const int i = (128 * j + 32 * v) / GS;
                                z0 = group_zero<Q>(m0, i);
                                z1 = group_zero<Q>(m1, i);
                                f0 = group_scale(m0, i);
                                f1 = group_scale(m1, i);
                            }
                            uint32_t p[4], q[4];
                            Q::unpack(w0[v], z0, p);
                            Q::unpack(w1[v], z1, q);
                            const uint32_t *b = xb[j][v];
                            if ((32 * v) % GS == 0)
                                mma16816c<T>(part, p[0], q[0], p[1], q[1], b[0], b[1], 0.f, 0.f, 0.f,
                                             0.f);
                            else
                                mma16816<T>(part, p[0], q[0], p[1], q[1], b[0], b[1]);
                            mma16816<T>(part, p[2], q[2], p[3], q[3], b[2], b[3]);
                            if ((32 * v + 32) % GS == 0) {  // and ends
#pragma unroll
                                for (int i = 0; i < 4; i++)
                                    acc[r][i] = fmaf(i < 2 ? f0 : f1, part[i], acc[r][i]);
                            }
                        }
                    }
                }
                // every lane's reads are done before the copy engine writes the stage
                fence_async_shared();
                __syncwarp();
                if (ok && filled.set < sets) {
                    fetch(filled, slot);
                    advance(filled);
                }
                if (++slot == G::stages) {
                    slot = 0;
                    parity ^= 1;
                }
            }
            // this warp's sums, as its lanes hold them
            if (ok && !warp_wait(red_empty + 8 * buf, red_parity, abort_flag)) {
                ok = false;
                *abort_flag = 1;
                __threadfence_block();
            }
            float *red = reinterpret_cast<float *>(smem + G::red_off) + (buf * kWarps + warp) * G::out;
#pragma unroll
            for (int r = 0; r < RT; r++)
#pragma unroll
                for (int i = 0; i < 4; i++)
                    red[(4 * r + i) * 32 + lane] = acc[r][i];
            __syncwarp();
            if (lane == 0)
                bar_arrive(red_full + 8 * buf);
            buf ^= 1;
            if (!buf)
                red_parity ^= 1;
        }
        drain(full, G::stages, arrived, issued);
    } else {
        // ------------------------------------------------------ add and store
        // Two neighbouring lanes' sums per thread: o = 16 (4 r + i) + lane / 2 is row
        // 16 r + 8 (i / 2) + g and the tokens 4 (o % 2) + i % 2 and + 2.
        constexpr int kPairs = G::out / 2;
        static_assert(kPairs <= 32 * kAdders, "a pair per thread");
        const int o = (warp - warps) * 32 + lane, i = o / 16 % 4;
        const int tok = tok0 + 4 * (o & 1) + (i & 1);
        const int in_tile = o / 64 * 16 + 8 * (i >> 1) + o / 2 % 8;
        const float2 *red = reinterpret_cast<const float2 *>(smem + G::red_off) + o;
        uint32_t buf = 0, parity = 0;
        for (int set = blockIdx.x; set < sets; set += gridDim.x) {
            if (ok && !warp_wait(red_full + 8 * buf, parity, abort_flag)) {
                ok = false;
                *abort_flag = 1;
            }
            if (o < kPairs)
                for (int rb = 0; rb < a.rw_n; rb++) {
                    const float2 *p = red + (buf * kWarps + rb * a.kw_n) * kPairs;
                    float v[2] = {};
#pragma unroll 8
                    for (int w = 0; w < a.kw_n; w++) {
                        const float2 q = p[w * kPairs];
                        v[0] += q.x;
                        v[1] += q.y;
                    }
                    // A sum that some warp did not wait for is no result: NaN.  A warp
                    // that gave up set the flag before it arrives, or writes sums, out
                    // of turn.
                    __threadfence_block();
                    const bool spoilt = *abort_flag;
                    const int row = (set * a.rw_n + rb) * 16 * RT + in_tile;
                    if (row >= rows)
                        continue;
                    const float bias = c.bias ? Q::to_float(static_cast<const T *>(c.bias)[row]) : 0.f;
#pragma unroll
                    for (int u = 0; u < 2; u++) {
                        if (tok + 2 * u >= c.n)
                            continue;
                        float s = spoilt ? NAN : v[u] + bias;
                        if (c.residual)
                            s += Q::to_float(static_cast<const T *>(c.residual)[(tok + 2 * u) * c.ldr + row]);
                        static_cast<T *>(c.out)[(tok + 2 * u) * c.ldo + row] = Q::from_float(s);
                    }
                }
            __syncwarp();
            if (lane == 0)
                bar_arrive(red_empty + 8 * buf);
            buf ^= 1;
            if (!buf)
                parity ^= 1;
        }
    }
    if (!ok && lane == 0 && c.status)
        atomicOr(c.status, MOE_STATUS_TIMEOUT);
}

// ---- dx = dy W -------------------------------------------------------------
// A CTA owns 128 columns; a stage is 32 rows x 64 bytes (64-byte swizzle).  The
// rows are the MMA's K and the columns its M.  A transposing matrix load of 8
// rows x 16 bytes gives lane (g, t) the 16-bit piece g (4 columns) of the rows 2 t
// and 2 t + 1 in one word, so that a field holds one column of two rows.  The
// scale differs along the MMA's K:
//   bf16, groups of 128: one scale per row holds for all columns of the CTA, so
//     it multiplies the gradients, dy * s rounded once to bf16 (fp32 range);
//   otherwise it is folded into the weights, (q - z) * s rounded once (in fp16
//     a product of gradient and scale could fall below the normal range; a
//     weight above 65504 becomes an infinity).
// Either way one factor of each term has the activations' type: exact q - z and
// sums scaled per group, as in the forward product, are open only where the
// contraction runs along a group.  Relative error of the output (2-norm, against
// 64 bits) 0.0024 instead of the 0.0017 of its own rounding in bf16, 0.00027
// instead of 0.00021 in fp16.
// The warps of a CTA and the CTAs of a cluster (1 to 8) split the rows; the
// partial sums meet in shared and distributed shared memory, in a fixed order.
constexpr int kThreads = 32 * kWarps;
constexpr int kGradCols = 128, kGradStage = 32 * 64, kGradStages = kRing / kGradStage;
constexpr int kGradSmem = kWarps * kRing + 8 * kWarps * kGradStages + 16;

template <typename T, int GS>
__global__ void __launch_bounds__(kThreads, 1)
    linear_grad_kernel(const __grid_constant__ CUtensorMap wmap, const W4Call c, int vec_in)
{
    using Q = W4<T>;
    constexpr bool kScaleIn = GS == 128 && sizeof(typename Q::Scale) == 8;
    constexpr int kMeta = kGradCols / GS;
    extern __shared__ __align__(1024) uint8_t smem[];
    float *red = reinterpret_cast<float *>(smem);       // [kWarps][8 tokens][128 columns]
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + kWarps * kRing);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(bars + kWarps * kGradStages);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const uint32_t full = saddr(bars + warp * kGradStages);
    const uint32_t ring = saddr(smem) + warp * kRing;
    if (saddr(smem) & 1023) {       // the swizzled stages need it; never seen otherwise
        if (threadIdx.x == 0 && c.status)
            atomicOr(c.status, MOE_STATUS_TIMEOUT);
        return;
    }
    if (lane == 0) {
        prefetch_map(&wmap);
        for (int i = 0; i < kGradStages; i++)
            bar_init(full + 8 * i, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (threadIdx.x == 0)
        *abort_flag = 0;
    __syncthreads();
    pdl_enter();

    const int rows = c.w.rows, K = c.w.K, ng = K / GS;
    const int splits = gridDim.x, rank = blockIdx.x, col0 = blockIdx.y * kGradCols;
    const int tok0 = blockIdx.z * 8;
    const T *dy = static_cast<const T *>(c.in);
    const int first = (rank * kWarps + warp) * 32, r_step = splits * kWarps * 32;

    unsigned issued = 0, arrived = 0;       // copies
    const auto fetch = [&](int r0, int slot) {
        issued++;
        if (lane == 0) {
            bar_expect_tx(full + 8 * slot, kGradStage);
            tma_load_2d(ring + slot * kGradStage, &wmap, col0 / 2, r0, full + 8 * slot);
        }
    };
    for (int i = 0; i < kGradStages; i++)
        if (first + i * r_step < rows)
            fetch(first + i * r_step, i);

    // scales and zero points of a stage: lane l those of row l
    struct Meta {
        uint32_t s[kMeta], z[kMeta];
    };
    const auto load_meta = [&](int r0, Meta &m) {
        // rows past the matrix: scales of 0 (the last row's, infinite, would make
        // NaN of the padding's zeros)
        const bool in = r0 + lane < rows;
        const long long at = (long long)(in ? r0 + lane : 0) * ng;
#pragma unroll
        for (int i = 0; i < kMeta; i++) {
            const int grp = min(col0 / GS + i, ng - 1);
            m.s[i] = in ? c.w.scales[at + grp] : 0;
            m.z[i] = in ? c.w.zeros[at + grp] : 0;
        }
    };

    float acc[8][4];
#pragma unroll
    for (int m = 0; m < 8; m++)
#pragma unroll
        for (int i = 0; i < 4; i++)
            acc[m][i] = 0.f;

    // loaded about as far ahead as the codes: with that much under way a load
    // takes several microseconds
    constexpr int kAhead = GS == 128 ? 4 : 2;
    Meta ahead[kAhead] = {};
#pragma unroll
    for (int i = 0; i < kAhead; i++)
        if (first + i * r_step < rows)
            load_meta(first + i * r_step, ahead[i]);
    bool ok = true;
    unsigned it = 0;
    for (int r0 = first; r0 < rows; r0 += r_step, it++) {
        const Meta meta = ahead[0];
#pragma unroll
        for (int i = 0; i + 1 < kAhead; i++)
            ahead[i] = ahead[i + 1];
        if (r0 + kAhead * r_step < rows)
            load_meta(r0 + kAhead * r_step, ahead[kAhead - 1]);
        uint32_t b[2][2];       // gradients of the rows 2 t, + 1 of each 8
#pragma unroll
        for (int ss = 0; ss < 2; ss++)
#pragma unroll
            for (int h = 0; h < 2; h++) {
                const int tok = tok0 + g, r = r0 + 16 * ss + 8 * h + 2 * t;
                b[ss][h] = 0;
                if (tok < c.n) {
                    const T *p = dy + tok * c.ldi + r;
                    if (vec_in && r + 1 < rows) {
                        b[ss][h] = *reinterpret_cast<const uint32_t *>(p);
                    } else {
                        const uint16_t *u = reinterpret_cast<const uint16_t *>(p);
                        if (r < rows)
                            b[ss][h] = u[0];
                        if (r + 1 < rows)
                            b[ss][h] |= (uint32_t)u[1] << 16;
                    }
                }
            }
        // this lane's row pair (lane & ~1, + 1) as the unpacking's operand words
        typename Q::Zero zp[kMeta];
        typename Q::Scale sp[kMeta];
        uint32_t raw[kMeta];
#pragma unroll
        for (int i = 0; i < kMeta; i++) {
            const uint32_t s2 = __shfl_xor_sync(0xffffffffu, meta.s[i], 1);
            const uint32_t z2 = __shfl_xor_sync(0xffffffffu, meta.z[i], 1);
            const bool odd = lane & 1;
            zp[i] = Q::zero(odd ? z2 : meta.z[i], odd ? meta.z[i] : z2);
            raw[i] = odd ? s2 | meta.s[i] << 16 : meta.s[i] | s2 << 16;
            if (!kScaleIn)
                sp[i] = Q::scale(raw[i] & 0xffff, raw[i] >> 16);
        }
        const int slot = it % kGradStages;
        if (ok && !warp_wait(full + 8 * slot, (it / kGradStages) & 1, abort_flag)) {
            ok = false;
            *abort_flag = 1;
        }
        arrived += ok;
        // w[ss][chunk of 32 columns][half]; row r's chunk p sits at p ^ (r / 2 % 4)
        const uint32_t stage = ring + slot * kGradStage;
        uint32_t w[2][4][2];
#pragma unroll
        for (int ss = 0; ss < 2; ss++)
#pragma unroll
            for (int p = 0; p < 4; p += 2) {
                const int r = 16 * ss + (lane & 15), chunk = p + (lane >> 4);
                uint32_t d[4];
                ldmatrix4_trans(d, stage + r * 64 + ((chunk ^ (r >> 1 & 3)) << 4));
                w[ss][p][0] = d[0];
                w[ss][p][1] = d[1];
                w[ss][p + 1][0] = d[2];
                w[ss][p + 1][1] = d[3];
            }
        // every lane's reads are done before the copy engine writes the stage
        fence_async_shared();
        __syncwarp();
        if (ok && r0 + kGradStages * r_step < rows)
            fetch(r0 + kGradStages * r_step, slot);
#pragma unroll
        for (int ss = 0; ss < 2; ss++) {
            const int from = 16 * ss + 2 * t;
            typename Q::Zero z01, z23;
            typename Q::Scale s01, s23;
            uint32_t b0 = b[ss][0], b1 = b[ss][1];
#pragma unroll
            for (int p = 0; p < 4; p++) {       // 32 columns: 32 p + 4 g + field
                if (32 * p % GS == 0) {         // a group begins
                    const int i = 32 * p / GS;
                    z01 = Q::zero_of(__shfl_sync(0xffffffffu, zp[i].lo, from));
                    z23 = Q::zero_of(__shfl_sync(0xffffffffu, zp[i].lo, from + 8));
                    if (kScaleIn) {
                        const uint32_t sa = __shfl_sync(0xffffffffu, raw[i], from);
                        const uint32_t sb = __shfl_sync(0xffffffffu, raw[i], from + 8);
                        b0 = Q::times(b0, sa & 0xffff, sa >> 16);
                        b1 = Q::times(b1, sb & 0xffff, sb >> 16);
                    } else {
                        s01 = shfl_of(sp[i], from);
                        s23 = shfl_of(sp[i], from + 8);
                    }
                }
                uint32_t f[4], h[4];
                Q::unpack(w[ss][p][0], z01, f);
                Q::unpack(w[ss][p][1], z23, h);
                if (!kScaleIn) {
#pragma unroll
                    for (int i = 0; i < 4; i++) {
                        f[i] = Q::mul(f[i], s01);
                        h[i] = Q::mul(h[i], s23);
                    }
                }
                mma16816<T>(acc[2 * p], f[0], f[1], h[0], h[1], b0, b1);
                mma16816<T>(acc[2 * p + 1], f[2], f[3], h[2], h[3], b0, b1);
            }
        }
    }
    drain(full, kGradStages, arrived, issued);
    __syncthreads();        // the rings become the sums' buffer
    const bool spoilt = *abort_flag;        // what some warp did not wait for is no result

    constexpr int kOut = 8 * kGradCols;
    static_assert(4 * kWarps * kOut <= kWarps * kRing, "the sums fit in the rings");
#pragma unroll
    for (int m = 0; m < 8; m++)
#pragma unroll
        for (int i = 0; i < 4; i++)
            red[warp * kOut + (2 * t + (i & 1)) * kGradCols + 32 * (m >> 1) + 4 * g + 2 * (m & 1) +
                (i >> 1)] = acc[m][i];
    __syncthreads();
    for (int o = threadIdx.x; o < kOut; o += kThreads) {
        float s = red[o];
#pragma unroll
        for (int w = 1; w < kWarps; w++)
            s += red[w * kOut + o];
        red[o] = spoilt ? NAN : s;
    }
    if (splits > 1) {
        cluster_arrive();
        cluster_wait();
    } else {
        __syncthreads();
    }
    T *dx = static_cast<T *>(c.out);
    for (int o = rank * kThreads + threadIdx.x; o < kOut; o += splits * kThreads) {
        const int cc = col0 + o % kGradCols, tok = tok0 + o / kGradCols;
        if (cc >= K || tok >= c.n)
            continue;
        float s = 0.f;
        if (splits > 1) {
            float v[8];
#pragma unroll
            for (int p = 0; p < 8; p++) {
                v[p] = 0.f;
                if (p < splits)
                    asm volatile("ld.shared::cluster.f32 %0, [%1];"
                                 : "=f"(v[p])
                                 : "r"(cluster_addr(saddr(red + o), p)));
            }
#pragma unroll
            for (int p = 0; p < 8; p++)
                s += v[p];
        } else {
            s = red[o];
        }
        dx[tok * c.ldo + cc] = Q::from_float(s);
    }
    if (splits > 1) {   // a CTA's shared memory stays until its peers have read it
        cluster_arrive();
        cluster_wait();
    }
    if (!ok && lane == 0 && c.status)
        atomicOr(c.status, MOE_STATUS_TIMEOUT);
}

// Launch of clusters along x, chained like the library's other kernels.
template <typename... P, typename... A>
cudaError_t launch_cluster(void (*kernel)(P...), dim3 grid, int threads, int smem, int cluster,
                           cudaStream_t st, A... args)
{
    const cudaError_t e =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess)
        return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <typename T, int GS, int RT>
cudaError_t launch_fwd_rt(const W4Call &c, int num_sms, cudaStream_t st)
{
    FwdArgs a{c, 0, 1, 0};
    const int slices = (c.w.K + 255) / 256, tiles = (c.w.rows + 16 * RT - 1) / (16 * RT);
    const int rounds = (slices + kWarps - 1) / kWarps;
    a.kw_n = (slices + rounds - 1) / rounds;
    // several row tiles at a time only when there are enough for every SM
    a.rw_n = std::max(1, std::min(kWarps / a.kw_n, tiles / num_sms));
    a.vec_meta = c.w.K % 256 == 0 && reinterpret_cast<uintptr_t>(c.w.scales) % 16 == 0 &&
                 reinterpret_cast<uintptr_t>(c.w.zeros) % 8 == 0;
    const int sets = (tiles + a.rw_n - 1) / a.rw_n;
    CUtensorMap wmap;
    if (!encode_map(&wmap, CU_TENSOR_MAP_DATA_TYPE_UINT8, c.w.codes, c.w.K / 2, c.w.rows, c.w.K / 2,
                    128, 16 * RT, CU_TENSOR_MAP_SWIZZLE_128B))
        return cudaErrorInvalidValue;
    auto kernel = linear_kernel<T, GS, RT>;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               FwdGeo<RT>::smem);
    if (e != cudaSuccess)
        return e;
    return launch_pdl(kernel, dim3(std::min(sets, num_sms), (c.n + 7) / 8),
                      dim3(32 * (a.kw_n * a.rw_n + kAdders)), FwdGeo<RT>::smem, st, wmap, a);
}

template <typename T, int GS>
cudaError_t launch_fwd(const W4Call &c, int num_sms, cudaStream_t st)
{
    // 32-row tiles join sums, and read activations, half as often; 16-row tiles
    // spread a small matrix over the SMs
    return c.w.rows >= 24 * num_sms ? launch_fwd_rt<T, GS, 2>(c, num_sms, st)
                                    : launch_fwd_rt<T, GS, 1>(c, num_sms, st);
}

template <typename T, int GS>
cudaError_t launch_bwd(const W4Call &c, int dev, int num_sms, cudaStream_t st)
{
    const int strips = (c.w.K + kGradCols - 1) / kGradCols, blocks = (c.n + 7) / 8;
    // every warp of a cluster has a stage, and all clusters run at once
    const int steps = (c.w.rows + 32 * kWarps - 1) / (32 * kWarps);
    const int *clusters = cluster_table(dev);
    int splits = 1;
    for (int s = 2; s <= std::min(8, steps); s++)
        if ((long long)strips * blocks <= clusters[s])
            splits = s;
    const int vec = reinterpret_cast<uintptr_t>(c.in) % 4 == 0 && c.ldi % 2 == 0;
    CUtensorMap wmap;
    if (!encode_map(&wmap, CU_TENSOR_MAP_DATA_TYPE_UINT8, c.w.codes, c.w.K / 2, c.w.rows, c.w.K / 2,
                    64, 32, CU_TENSOR_MAP_SWIZZLE_64B))
        return cudaErrorInvalidValue;
    return launch_cluster(linear_grad_kernel<T, GS>, dim3(splits, strips, blocks), kThreads,
                          kGradSmem, splits, st, wmap, c, vec);
}

template <typename T, int GS>
cudaError_t launch_few(const W4Call &c, int grad, int dev, int num_sms, cudaStream_t st)
{
    return grad ? launch_bwd<T, GS>(c, dev, num_sms, st) : launch_fwd<T, GS>(c, num_sms, st);
}

template <typename T>
cudaError_t launch_group_size(const W4Call &c, int grad, int dev, int num_sms, cudaStream_t st)
{
    switch (c.w.group) {
    case 32: return launch_few<T, 32>(c, grad, dev, num_sms, st);
    case 64: return launch_few<T, 64>(c, grad, dev, num_sms, st);
    default: return launch_few<T, 128>(c, grad, dev, num_sms, st);
    }
}

}  // namespace

// Whether n rows of wa elements, lda apart, share bytes with n rows of wb, ldb
// apart: ranges that meet do, unless equal strides keep the one's rows in the
// gaps of the other's (column slices of one buffer).  Strides are at least the
// rows' lengths.
bool rows_overlap(const void *a, long long lda, int wa, const void *b, long long ldb, int wb, int n,
                  int size)
{
    const char *p = static_cast<const char *>(a), *q = static_cast<const char *>(b);
    if (p >= q + size * ((n - 1) * ldb + wb) || q >= p + size * ((n - 1) * lda + wa))
        return false;
    const long long ld = size * lda, d = ((q - p) % ld + ld) % ld;
    return lda != ldb || d < (long long)size * wa || d + (long long)size * wb > ld;
}

// Whether n rows of w elements of `size` bytes, ld apart, share bytes with the
// range of `bytes` at q: none does when q lies in the gap behind a row.
bool rows_meet(const void *p, long long ld, int w, int n, int size, const void *q, size_t bytes)
{
    const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
    const uintptr_t pitch = size * (uintptr_t)ld, row = size * (uintptr_t)w;
    if (!bytes || b >= a + (n - 1) * pitch + row || b + bytes <= a)
        return false;
    return b < a || (b - a) % pitch < row || (b - a) % pitch + bytes > pitch;
}

// Whether two ranges share bytes.
bool ranges_meet(const void *p, size_t n, const void *q, size_t m)
{
    const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
    return n && m && a < b + m && b < a + n;
}

bool linear_gemm_fits(const W4Call &c);
cudaError_t launch_linear_gemm(const W4Call &c, int bf16, int grad, int dev, int num_sms,
                               cudaStream_t st);
bool device_pointer_here(const void *p, int dev);
int record_failure(int code, const char *msg);
int record_success();

namespace {

constexpr int kFewTokens = 8;
constexpr int kMaxRows = 1 << 20, kMaxCols = 1 << 16;
constexpr int kMaxTokens = 8 * 65535;     // blocks of 8 tokens along a grid dimension

// Rows of 2-byte elements, `ld` apart, to rows `ldo` apart (a multiple of 8
// elements), the gap filled with zeros: a plain coalesced copy, bound by its
// latency at the sizes it serves.
__global__ void __launch_bounds__(256) realign_kernel(const uint16_t *__restrict__ in, long long ld,
                                                      int width, uint16_t *__restrict__ out, int ldo)
{
    pdl_enter();
    const uint16_t *src = in + blockIdx.x * ld;
    uint16_t *dst = out + (long long)blockIdx.x * ldo;
#pragma unroll 8
    for (int i = blockIdx.y * 2048 + threadIdx.x; i < min(ldo, (int)(blockIdx.y + 1) * 2048); i += 256)
        dst[i] = i < width ? src[i] : 0;
}

// Elements per row, and bytes, of an aligned copy of n rows.
int aligned_ld(int width) { return (width + 7) / 8 * 8; }
size_t aligned_bytes(int width, int n) { return 2 * (size_t)aligned_ld(width) * n; }

int run_linear(W4Call c, int dtype, int grad, void *workspace, size_t workspace_bytes, void *stream)
{
    const W4Matrix &w = c.w;
    if (!w.codes || !w.scales || !w.zeros || !c.in || !c.out)
        return record_failure(MOE_ERR_INVALID_ARG, "null pointer argument");
    if (dtype != MOE_FP16 && dtype != MOE_BF16)
        return record_failure(MOE_ERR_UNSUPPORTED, "dtype must be MOE_FP16 or MOE_BF16");
    if (w.group != 32 && w.group != 64 && w.group != 128)
        return record_failure(MOE_ERR_UNSUPPORTED, "group_size must be 32, 64 or 128");
    if (w.rows < 1 || w.rows > kMaxRows)
        return record_failure(MOE_ERR_INVALID_ARG, "rows must be in 1..1048576");
    if (w.K < w.group || w.K > kMaxCols || w.K % w.group)
        return record_failure(MOE_ERR_INVALID_ARG,
                              "cols must be a multiple of group_size in group_size..65536");
    if (c.n < 1 || c.n > kMaxTokens)
        return record_failure(MOE_ERR_INVALID_ARG, "n_tokens must be in 1..524280");
    const int win = grad ? w.rows : w.K, wout = grad ? w.K : w.rows;
    constexpr long long kMaxLd = 1LL << 31;
    if (c.ldi < win || c.ldo < wout || (c.residual && c.ldr < wout) || c.ldi > kMaxLd ||
        c.ldo > kMaxLd || c.ldr > kMaxLd)
        return record_failure(MOE_ERR_INVALID_ARG,
                              "a row stride is below the row's length or above 2^31");
    const auto mis = [](const void *p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) != 0; };
    if (mis(w.codes, 16) || mis(w.scales, 2) || mis(c.in, grad ? 2 : 16) || mis(c.out, 2) ||
        mis(c.bias, 2) || mis(c.residual, 2) || mis(c.status, 4) || (!grad && c.ldi % 8))
        return record_failure(MOE_ERR_INVALID_ARG,
                              grad ? "misaligned pointer (codes need 16 bytes)"
                                   : "misaligned pointer or stride (codes and the rows of x need "
                                     "16 bytes)");
    if (rows_overlap(c.out, c.ldo, wout, c.in, c.ldi, win, c.n, 2))
        return record_failure(MOE_ERR_INVALID_ARG, "the output overlaps the input");
    if (c.residual && !(c.residual == c.out && c.ldr == c.ldo) &&
        rows_overlap(c.out, c.ldo, wout, c.residual, c.ldr, wout, c.n, 2))
        return record_failure(MOE_ERR_INVALID_ARG,
                              "y overlaps residual (it may be residual itself)");
    const bool copy = grad && c.n > kFewTokens && !linear_gemm_fits(c) && workspace &&
                      workspace_bytes >= aligned_bytes(w.rows, c.n);
    if (copy && mis(workspace, 16))
        return record_failure(MOE_ERR_INVALID_ARG, "misaligned workspace (it needs 16 bytes)");
    // what the call writes against what it reads besides
    const size_t n_meta = (size_t)w.rows * (w.K / w.group);
    const struct {
        const void *p;
        size_t bytes;
    } read[] = {{w.codes, (size_t)w.rows * (w.K / 2)}, {w.scales, 2 * n_meta}, {w.zeros, n_meta},
                {c.bias, c.bias ? 2 * (size_t)wout : 0}, {c.status, c.status ? 4u : 0u}};
    const size_t ws_bytes = copy ? aligned_bytes(w.rows, c.n) : 0;
    for (const auto &r : read) {
        if (rows_meet(c.out, c.ldo, wout, c.n, 2, r.p, r.bytes))
            return record_failure(MOE_ERR_INVALID_ARG,
                                  "the output overlaps the matrix, the bias or the status word");
        if (ranges_meet(workspace, ws_bytes, r.p, r.bytes))
            return record_failure(MOE_ERR_INVALID_ARG, "the workspace overlaps another argument");
    }
    if (rows_meet(c.out, c.ldo, wout, c.n, 2, workspace, ws_bytes) ||
        rows_meet(c.in, c.ldi, win, c.n, 2, workspace, ws_bytes))
        return record_failure(MOE_ERR_INVALID_ARG, "the workspace overlaps another argument");
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
        cudaGetLastError();
        return record_failure(MOE_ERR_CUDA, "no usable current CUDA device");
    }
    const void *all[] = {w.codes, w.scales, w.zeros, c.in, c.out, c.bias, c.residual, c.status,
                         copy ? workspace : nullptr};
    for (const void *p : all)
        if (p && !device_pointer_here(p, dev))
            return record_failure(MOE_ERR_INVALID_ARG,
                                  "arguments must be device pointers of the current device");
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaError_t e = cudaSuccess;
    if (copy) {
        const int ldo = aligned_ld(w.rows);
        e = launch_pdl(realign_kernel, dim3(c.n, (ldo + 2047) / 2048), dim3(256), 0, st,
                       static_cast<const uint16_t *>(c.in), c.ldi, w.rows,
                       static_cast<uint16_t *>(workspace), ldo);
        c.in = workspace;
        c.ldi = ldo;
    }
    if (e == cudaSuccess && c.n > kFewTokens && linear_gemm_fits(c))
        e = launch_linear_gemm(c, dtype == MOE_BF16, grad, dev, sms, st);
    else if (e == cudaSuccess)
        e = dtype == MOE_FP16 ? launch_group_size<__half>(c, grad, dev, sms, st)
                              : launch_group_size<__nv_bfloat16>(c, grad, dev, sms, st);
    if (e != cudaSuccess) {
        cudaGetLastError();
        return record_failure(MOE_ERR_CUDA, cudaGetErrorString(e));
    }
    return record_success();
}

}  // namespace

}  // namespace qe

extern "C" int moe_linear(const void *codes, const void *scales, const void *zeros, int rows,
                          int cols, int group_size, const void *x, long long ldx, int n_tokens,
                          int dtype, const void *bias, const void *residual, long long ldr,
                          void *y, long long ldy, int *status, void *stream)
{
    qe::W4Call c{};
    c.w = {static_cast<const uint8_t *>(codes), static_cast<const uint16_t *>(scales),
           static_cast<const uint8_t *>(zeros), rows, cols, group_size};
    c.in = x;
    c.ldi = ldx;
    c.n = n_tokens;
    c.bias = bias;
    c.residual = residual;
    c.ldr = residual ? ldr : 0;
    c.out = y;
    c.ldo = ldy;
    c.status = status;
    return qe::run_linear(c, dtype, 0, nullptr, 0, stream);
}

extern "C" int moe_linear_input_grad(const void *codes, const void *scales, const void *zeros,
                                     int rows, int cols, int group_size, const void *dy,
                                     long long lddy, int n_tokens, int dtype, void *dx,
                                     long long lddx, void *workspace, size_t workspace_bytes,
                                     int *status, void *stream)
{
    qe::W4Call c{};
    c.w = {static_cast<const uint8_t *>(codes), static_cast<const uint16_t *>(scales),
           static_cast<const uint8_t *>(zeros), rows, cols, group_size};
    c.in = dy;
    c.ldi = lddy;
    c.n = n_tokens;
    c.out = dx;
    c.ldo = lddx;
    c.status = status;
    return qe::run_linear(c, dtype, 1, workspace, workspace_bytes, stream);
}

extern "C" size_t moe_linear_input_grad_workspace(int rows, int n_tokens, const void *dy,
                                                  long long lddy)
{
    qe::W4Call c{};
    c.in = dy;
    c.ldi = lddy;
    if (rows < 1 || rows > qe::kMaxRows || n_tokens <= qe::kFewTokens ||
        n_tokens > qe::kMaxTokens || qe::linear_gemm_fits(c))
        return 0;
    return qe::aligned_bytes(rows, n_tokens);
}
