// 4-bit group-quantised products for few tokens, on the warp MMA:
//   moe_linear              y[t][r]  = sum_k x[t][k] W[r][k] (+ bias) (+ residual)
//   moe_linear_input_grad   dx[t][k] = sum_r dy[t][r] W[r][k]
// with W = (q - z) * s in the canonical layout ("Strata" article, section 2.2:
// one scale and one zero point per group along K; section 3.4: hand-written
// INT4 GEMV; "Flash-MoE", section 3: dequant matvec).
//
// Both read every packed byte once per block of tokens and are bound by that
// stream while the tokens are few.  The weights are the MMA's A operand
// (M = 16), the tokens its N = 8 columns.  The MMA's K order is free as long as
// A and B agree, so a lane's MMA elements are the nibbles of words it loads
// contiguously, and no lane exchanges weights with another.
#include <algorithm>

#include "w4.cuh"

namespace qe {

namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;

// ---- y = x W^T -------------------------------------------------------------
// A warp's unit is 16 rows x 512 K: lane (g = lane / 4, t = lane % 4) loads, of
// rows g and g + 8, the 16 bytes at K = 128 j + 32 t for j = 0..3, i.e. the
// warp reads 256 contiguous bytes of each row.  Each 16-byte word is four
// MMA K-steps' worth of half of the lane's A elements: its fields (i, i + 4)
// pair with the activations (i, i + 4) of the same 8 elements.
// Groups of 128: the products with the exact integers q - z are summed per
// group and the fp32 sum is scaled (no rounding of weights).  Smaller groups
// lie inside one MMA: the scale is folded into the weights, one rounding.
template <typename T, int GS, int NT, int RT>
__global__ void __launch_bounds__(kThreads) linear_kernel(W4Call c, int kw_n)
{
    using Q = W4<T>;
    extern __shared__ float red[];      // [kWarps][RT][NT][4][32]
    pdl_enter();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int kw = warp % kw_n, rw = warp / kw_n;
    const int rows = c.w.rows, K = c.w.K, tok0 = blockIdx.y * 8 * NT;
    const int row0 = (blockIdx.x * (kWarps / kw_n) + rw) * 16 * RT;
    const int ng = K / GS;
    const T *x = static_cast<const T *>(c.in);

    float acc[RT][NT][4];
#pragma unroll
    for (int r = 0; r < RT; r++)
#pragma unroll
        for (int m = 0; m < NT; m++)
#pragma unroll
            for (int i = 0; i < 4; i++)
                acc[r][m][i] = 0.f;

    for (int k0 = kw * 512; k0 < K; k0 += kw_n * 512) {
        uint4 wq[RT][4][2];
        uint32_t sz[RT][GS == 128 ? 1 : 4][2];   // scale bits << 16 | zero point
#pragma unroll
        for (int r = 0; r < RT; r++)
#pragma unroll
            for (int h = 0; h < 2; h++) {
                // rows past the matrix repeat its last row; their sums are not stored
                const long long row = min(row0 + r * 16 + g + 8 * h, rows - 1);
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    const int k = k0 + 128 * j + 32 * t;
                    wq[r][j][h] = k < K ? ld_codes16(c.w.codes + row * (K / 2) + k / 2)
                                        : make_uint4(0, 0, 0, 0);
                }
                if (GS == 128) {
                    const long long at = row * ng + min(k0 / 128 + t, ng - 1);
                    sz[r][0][h] = (uint32_t)c.w.scales[at] << 16 | c.w.zeros[at];
                } else {
#pragma unroll
                    for (int j = 0; j < 4; j++) {
                        const long long at = row * ng + min((k0 + 128 * j + 32 * t) / GS, ng - 1);
                        sz[r][j][h] = (uint32_t)c.w.scales[at] << 16 | c.w.zeros[at];
                    }
                }
            }
#pragma unroll
        for (int j = 0; j < 4; j++) {
            const int k = k0 + 128 * j + 32 * t;
            uint4 xv[NT][4];
#pragma unroll
            for (int m = 0; m < NT; m++) {
                const int tok = tok0 + 8 * m + g;
#pragma unroll
                for (int v = 0; v < 4; v++)
                    xv[m][v] = tok < c.n && k < K
                                   ? *reinterpret_cast<const uint4 *>(x + tok * c.ldi + k + 8 * v)
                                   : make_uint4(0, 0, 0, 0);
            }
#pragma unroll
            for (int r = 0; r < RT; r++) {
                uint32_t a0, a1;
                if (GS == 128) {
                    a0 = __shfl_sync(0xffffffffu, sz[r][0][0], (lane & ~3) | j);
                    a1 = __shfl_sync(0xffffffffu, sz[r][0][1], (lane & ~3) | j);
                } else {
                    a0 = sz[r][j][0];
                    a1 = sz[r][j][1];
                }
                const typename Q::Zero z0 = Q::zero(a0 & 0xff, a0 & 0xff);
                const typename Q::Zero z1 = Q::zero(a1 & 0xff, a1 & 0xff);
                const uint32_t w0[4] = {wq[r][j][0].x, wq[r][j][0].y, wq[r][j][0].z, wq[r][j][0].w};
                const uint32_t w1[4] = {wq[r][j][1].x, wq[r][j][1].y, wq[r][j][1].z, wq[r][j][1].w};
                float part[NT][4];
#pragma unroll
                for (int m = 0; m < NT; m++)
#pragma unroll
                    for (int i = 0; i < 4; i++)
                        part[m][i] = GS == 128 ? 0.f : acc[r][m][i];
#pragma unroll
                for (int v = 0; v < 4; v++) {
                    uint32_t p[4], q[4];
                    Q::unpack(w0[v], z0, p);
                    Q::unpack(w1[v], z1, q);
                    if (GS != 128) {
                        const typename Q::Scale s0 = Q::scale(a0 >> 16, a0 >> 16);
                        const typename Q::Scale s1 = Q::scale(a1 >> 16, a1 >> 16);
#pragma unroll
                        for (int i = 0; i < 4; i++) {
                            p[i] = Q::mul(p[i], s0);
                            q[i] = Q::mul(q[i], s1);
                        }
                    }
#pragma unroll
                    for (int m = 0; m < NT; m++) {
                        const uint4 b = xv[m][v];
                        mma16816<T>(part[m], p[0], q[0], p[1], q[1], __byte_perm(b.x, b.z, 0x5410),
                                    __byte_perm(b.x, b.z, 0x7632));
                        mma16816<T>(part[m], p[2], q[2], p[3], q[3], __byte_perm(b.y, b.w, 0x5410),
                                    __byte_perm(b.y, b.w, 0x7632));
                    }
                }
                const float f0 = __half2float(__ushort_as_half((unsigned short)(a0 >> 16)));
                const float f1 = __half2float(__ushort_as_half((unsigned short)(a1 >> 16)));
#pragma unroll
                for (int m = 0; m < NT; m++)
#pragma unroll
                    for (int i = 0; i < 4; i++)
                        acc[r][m][i] = GS == 128 ? fmaf(i < 2 ? f0 : f1, part[m][i], acc[r][m][i])
                                                 : part[m][i];
            }
        }
    }

    // sums of the K slices, in slice order
#pragma unroll
    for (int r = 0; r < RT; r++)
#pragma unroll
        for (int m = 0; m < NT; m++)
#pragma unroll
            for (int i = 0; i < 4; i++)
                red[(((warp * RT + r) * NT + m) * 4 + i) * 32 + lane] = acc[r][m][i];
    __syncthreads();
    constexpr int kOut = 16 * RT * 8 * NT;      // results of one row block
    T *y = static_cast<T *>(c.out);
    const T *bias = static_cast<const T *>(c.bias), *res = static_cast<const T *>(c.residual);
    for (int o = threadIdx.x; o < kOut * (kWarps / kw_n); o += kThreads) {
        const int rr = o % (16 * RT), tt = o / (16 * RT) % (8 * NT), rb = o / kOut;
        const int row = (blockIdx.x * (kWarps / kw_n) + rb) * 16 * RT + rr, tok = tok0 + tt;
        if (row >= rows || tok >= c.n)
            continue;
        const int r = rr / 16, gr = rr % 8, hi = rr % 16 / 8, m = tt / 8, tc = tt % 8;
        const int at = ((r * NT + m) * 4 + 2 * hi + (tc & 1)) * 32 + gr * 4 + tc / 2;
        float s = 0.f;
        for (int w = 0; w < kw_n; w++)
            s += red[(rb * kw_n + w) * RT * NT * 128 + at];
        if (bias)
            s += Q::to_float(bias[row]);
        if (res)
            s += Q::to_float(res[tok * c.ldr + row]);
        y[tok * c.ldo + row] = Q::from_float(s);
    }
}

// ---- dx = dy W -------------------------------------------------------------
// A warp's step is 16 rows x 128 K: lane (g, t) loads, of rows 4 t .. 4 t + 3,
// the 8 bytes at K = 16 g.  The rows are the MMA's K and the columns its M:
// one byte permutation pairs the halves of two rows' words, so that a field
// holds one column of two rows.  The scale differs along the MMA's K, so it is
// folded into the weights (one rounding).  The warps of a CTA and the CTAs of
// a cluster (1 to 8) split the rows; the partial sums meet in shared and
// distributed shared memory, in a fixed order.
template <typename T, int GS, int NT>
__global__ void __launch_bounds__(kThreads) linear_grad_kernel(W4Call c, int vec_in)
{
    using Q = W4<T>;
    extern __shared__ float red[];      // [kWarps][8 * NT tokens][128 columns]
    pdl_enter();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int rows = c.w.rows, K = c.w.K, ng = K / GS;
    const int col0 = blockIdx.x * 128, tok0 = blockIdx.z * 8 * NT;
    const int splits = gridDim.y, rank = blockIdx.y;
    // columns past the matrix read its first columns; their sums are not stored
    const int col = col0 + 16 * g < K ? col0 + 16 * g : 0;
    const T *dy = static_cast<const T *>(c.in);

    float acc[8][NT][4];
#pragma unroll
    for (int m = 0; m < 8; m++)
#pragma unroll
        for (int j = 0; j < NT; j++)
#pragma unroll
            for (int i = 0; i < 4; i++)
                acc[m][j][i] = 0.f;

#pragma unroll 4
    for (int r0 = (rank * kWarps + warp) * 16; r0 < rows; r0 += splits * kWarps * 16) {
        uint2 wq[4];
        uint32_t sc[4], zz[4];
#pragma unroll
        for (int i = 0; i < 4; i++) {
            // rows past the matrix repeat its last row, against gradients of zero
            const long long row = min(r0 + 4 * t + i, rows - 1);
            wq[i] = ld_codes8(c.w.codes + row * (K / 2) + col / 2);
            const long long at = row * ng + col / GS;
            sc[i] = c.w.scales[at];
            zz[i] = c.w.zeros[at];
        }
        uint2 b[NT];
#pragma unroll
        for (int j = 0; j < NT; j++) {
            const int tok = tok0 + 8 * j + g, r = r0 + 4 * t;
            b[j] = make_uint2(0, 0);
            if (tok < c.n) {
                const T *p = dy + tok * c.ldi + r;
                if (vec_in && r + 3 < rows) {
                    b[j] = *reinterpret_cast<const uint2 *>(p);
                } else {
                    const uint16_t *u = reinterpret_cast<const uint16_t *>(p);
                    if (r < rows)
                        b[j].x = u[0];
                    if (r + 1 < rows)
                        b[j].x |= (uint32_t)u[1] << 16;
                    if (r + 2 < rows)
                        b[j].y = u[2];
                    if (r + 3 < rows)
                        b[j].y |= (uint32_t)u[3] << 16;
                }
            }
        }
        const typename Q::Zero z01 = Q::zero(zz[0], zz[1]), z23 = Q::zero(zz[2], zz[3]);
        const typename Q::Scale s01 = Q::scale(sc[0], sc[1]), s23 = Q::scale(sc[2], sc[3]);
#pragma unroll
        for (int q4 = 0; q4 < 4; q4++) {        // four columns: half of one of the two words
            const uint32_t sel = q4 & 1 ? 0x7632 : 0x5410;
            const uint32_t u01 = q4 < 2 ? __byte_perm(wq[0].x, wq[1].x, sel)
                                        : __byte_perm(wq[0].y, wq[1].y, sel);
            const uint32_t u23 = q4 < 2 ? __byte_perm(wq[2].x, wq[3].x, sel)
                                        : __byte_perm(wq[2].y, wq[3].y, sel);
            uint32_t p[4], q[4];
            Q::unpack(u01, z01, p);
            Q::unpack(u23, z23, q);
#pragma unroll
            for (int i = 0; i < 4; i++) {
                p[i] = Q::mul(p[i], s01);
                q[i] = Q::mul(q[i], s23);
            }
#pragma unroll
            for (int j = 0; j < NT; j++) {
                mma16816<T>(acc[2 * q4][j], p[0], p[1], q[0], q[1], b[j].x, b[j].y);
                mma16816<T>(acc[2 * q4 + 1][j], p[2], p[3], q[2], q[3], b[j].x, b[j].y);
            }
        }
    }

    constexpr int kOut = 8 * NT * 128;
#pragma unroll
    for (int m = 0; m < 8; m++)
#pragma unroll
        for (int j = 0; j < NT; j++)
#pragma unroll
            for (int i = 0; i < 4; i++)
                red[warp * kOut + (8 * j + 2 * t + (i & 1)) * 128 + 16 * g + 2 * m + (i >> 1)] =
                    acc[m][j][i];
    __syncthreads();
    for (int o = threadIdx.x; o < kOut; o += kThreads) {
        float s = red[o];
#pragma unroll
        for (int w = 1; w < kWarps; w++)
            s += red[w * kOut + o];
        red[o] = s;
    }
    if (splits > 1) {
        asm volatile("barrier.cluster.arrive.aligned;\n barrier.cluster.wait.aligned;" ::: "memory");
    } else {
        __syncthreads();
    }
    T *dx = static_cast<T *>(c.out);
    const uint32_t base = (uint32_t)__cvta_generic_to_shared(red);
    for (int o = rank * kThreads + threadIdx.x; o < kOut; o += splits * kThreads) {
        const int cc = col0 + o % 128, tok = tok0 + o / 128;
        if (cc >= K || tok >= c.n)
            continue;
        float s = 0.f;
        if (splits > 1) {
            for (int p = 0; p < splits; p++) {
                uint32_t remote;
                float v;
                asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(base + 4 * o), "r"(p));
                asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(remote));
                s += v;
            }
        } else {
            s = red[o];
        }
        dx[tok * c.ldo + cc] = Q::from_float(s);
    }
    if (splits > 1)     // a CTA's shared memory stays until its peers have read it
        asm volatile("barrier.cluster.arrive.aligned;\n barrier.cluster.wait.aligned;" ::: "memory");
}

template <typename T, int GS, int NT>
cudaError_t launch_fwd(const W4Call &c, cudaStream_t st)
{
    constexpr int RT = 1;
    const int units = (c.w.K + 511) / 512;
    const int kw = units >= 8 ? 8 : units >= 4 ? 4 : units >= 2 ? 2 : 1;
    const int rows_cta = 16 * RT * (kWarps / kw);
    const dim3 grid((c.w.rows + rows_cta - 1) / rows_cta, (c.n + 8 * NT - 1) / (8 * NT));
    return launch_pdl(linear_kernel<T, GS, NT, RT>, grid, dim3(kThreads),
                      sizeof(float) * kWarps * RT * NT * 128, st, c, kw);
}

template <typename T, int GS, int NT>
cudaError_t launch_bwd(const W4Call &c, int num_sms, cudaStream_t st)
{
    const size_t smem = sizeof(float) * kWarps * 8 * NT * 128;
    auto kernel = linear_grad_kernel<T, GS, NT>;
    if (smem > 48 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(
            kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess)
            return e;
    }
    const int strips = (c.w.K + 127) / 128, blocks = (c.n + 8 * NT - 1) / (8 * NT);
    const int steps = (c.w.rows + 16 * kWarps - 1) / (16 * kWarps);
    int splits = 1;
    while (splits < 8 && (long long)strips * blocks * splits < 2LL * num_sms && 2 * splits <= steps)
        splits *= 2;
    const int vec = reinterpret_cast<uintptr_t>(c.in) % 8 == 0 && c.ldi % 4 == 0;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(strips, splits, blocks);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 1;
    attr[1].val.clusterDim.y = splits;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kernel, c, vec);
}

template <typename T, int GS>
cudaError_t launch_few(const W4Call &c, int grad, int num_sms, cudaStream_t st)
{
    if (grad)
        return c.n <= 8 ? launch_bwd<T, GS, 1>(c, num_sms, st) : launch_bwd<T, GS, 2>(c, num_sms, st);
    return c.n <= 8 ? launch_fwd<T, GS, 1>(c, st) : launch_fwd<T, GS, 2>(c, st);
}

template <typename T>
cudaError_t launch_group_size(const W4Call &c, int grad, int num_sms, cudaStream_t st)
{
    switch (c.w.group) {
    case 32: return launch_few<T, 32>(c, grad, num_sms, st);
    case 64: return launch_few<T, 64>(c, grad, num_sms, st);
    default: return launch_few<T, 128>(c, grad, num_sms, st);
    }
}

}  // namespace

bool linear_gemm_fits(const W4Call &c);
cudaError_t launch_linear_gemm(const W4Call &c, int bf16, int grad, int dev, int num_sms,
                               cudaStream_t st);
bool device_pointer_here(const void *p, int dev);
int record_failure(int code, const char *msg);
int record_success();

namespace {

constexpr int kFewTokens = 16;
constexpr int kMaxRows = 1 << 20, kMaxCols = 1 << 16, kMaxTokens = 1 << 19;

// The byte range of n rows of `width` 2-byte elements, ld elements apart.
bool overlap(const void *a, long long lda, int wa, const void *b, long long ldb, int wb, int n)
{
    const char *p = static_cast<const char *>(a), *q = static_cast<const char *>(b);
    const long long na = 2 * ((n - 1) * lda + wa), nb = 2 * ((n - 1) * ldb + wb);
    return p < q + nb && q < p + na;
}

int run_linear(const W4Call &c, int dtype, int grad, void *stream)
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
        return record_failure(MOE_ERR_INVALID_ARG, "n_tokens must be in 1..524288");
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
    if (overlap(c.out, c.ldo, wout, c.in, c.ldi, win, c.n))
        return record_failure(MOE_ERR_INVALID_ARG, "the output overlaps the input");
    if (c.residual && !(c.residual == c.out && c.ldr == c.ldo) &&
        overlap(c.out, c.ldo, wout, c.residual, c.ldr, wout, c.n))
        return record_failure(MOE_ERR_INVALID_ARG,
                              "y overlaps residual (it may be residual itself)");
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
        cudaGetLastError();
        return record_failure(MOE_ERR_CUDA, "no usable current CUDA device");
    }
    const void *all[] = {w.codes, w.scales, w.zeros, c.in, c.out, c.bias, c.residual, c.status};
    for (const void *p : all)
        if (p && !device_pointer_here(p, dev))
            return record_failure(MOE_ERR_INVALID_ARG,
                                  "arguments must be device pointers of the current device");
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (c.n > kFewTokens && linear_gemm_fits(c))
        e = launch_linear_gemm(c, dtype == MOE_BF16, grad, dev, sms, st);
    else
        e = dtype == MOE_FP16 ? launch_group_size<__half>(c, grad, sms, st)
                              : launch_group_size<__nv_bfloat16>(c, grad, sms, st);
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
    return qe::run_linear(c, dtype, 0, stream);
}

extern "C" int moe_linear_input_grad(const void *codes, const void *scales, const void *zeros,
                                     int rows, int cols, int group_size, const void *dy,
                                     long long lddy, int n_tokens, int dtype, void *dx,
                                     long long lddx, int *status, void *stream)
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
    return qe::run_linear(c, dtype, 1, stream);
}
