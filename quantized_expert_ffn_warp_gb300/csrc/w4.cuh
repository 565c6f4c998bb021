// Device helpers of the 4-bit products on matrices in the canonical layout
// (codes uint8 [rows][K/2], low nibble = even k; fp16 scales and u8 zero
// points [rows][K/group]): the integer q - z of packed nibbles as exact fp16
// or bf16 pairs, the group scale folded in with one rounding, and the warp MMA.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstring>

#include "internal.cuh"
#include "tcgen05.cuh"

namespace qe {

// A pair type's arithmetic.  Pairs are 32-bit words; fields of a word are the
// nibbles i and i + 4 (its low and high half), i = 0..3.
template <typename T>
struct W4;

// fp16: a nibble or'ed into the mantissa of 1024 reads 1024 + q (or, left in
// the upper nibble of a byte, 1024 + 16 q); subtracting 1024 + z (or, after
// an exact division by 16, 64 + z) leaves q - z without rounding.
template <>
struct W4<__half> {
    struct Zero {
        uint32_t lo, hi;    // 1024 + z; -(64 + z)
    };
    static __device__ __forceinline__ uint32_t u(__half2 h) { return *reinterpret_cast<uint32_t *>(&h); }
    static __device__ __forceinline__ __half2 h(uint32_t v) { return *reinterpret_cast<__half2 *>(&v); }
    // zero points of the word's two halves
    static __device__ __forceinline__ Zero zero(uint32_t z0, uint32_t z1)
    {
        const uint32_t z = z0 | (z1 << 16);
        return zero_of(0x64006400u + z);
    }
    // from its `lo` word: the two words' 16 z differ by a constant
    static __device__ __forceinline__ Zero zero_of(uint32_t lo)
    {
        return {lo, (lo << 4) + (0xD400D400u - (0x64006400u << 4))};
    }
    // the four fields' q - z
    static __device__ __forceinline__ void unpack(uint32_t w, const Zero &z, uint32_t (&p)[4])
    {
        const __half2 sixteenth = __float2half2_rn(0.0625f);
        const uint32_t w8 = w >> 8;
        p[0] = u(__hsub2(h(lop_magic(w, 0x000F000Fu)), h(z.lo)));
        p[1] = u(__hfma2(h(lop_magic(w, 0x00F000F0u)), sixteenth, h(z.hi)));
        p[2] = u(__hsub2(h(lop_magic(w8, 0x000F000Fu)), h(z.lo)));
        p[3] = u(__hfma2(h(lop_magic(w8, 0x00F000F0u)), sixteenth, h(z.hi)));
    }
    struct Scale {
        uint32_t s;
    };
    // fp16 scales (as bits) of the word's two halves
    static __device__ __forceinline__ Scale scale(uint32_t s0, uint32_t s1)
    {
        return {s0 | (s1 << 16)};
    }
    // (q - z) * s, rounded once to fp16
    static __device__ __forceinline__ uint32_t mul(uint32_t p, const Scale &s)
    {
        return u(__hmul2(h(p), h(s.s)));
    }
    static __device__ __forceinline__ uint32_t times(uint32_t v, uint32_t s0, uint32_t s1)
    {
        return u(__hmul2(h(v), h(s0 | (s1 << 16))));
    }
    static __device__ __forceinline__ float low(uint32_t v) { return __low2float(h(v)); }
    static __device__ __forceinline__ float high(uint32_t v) { return __high2float(h(v)); }
    static __device__ __forceinline__ float to_float(__half v) { return __half2float(v); }
    static __device__ __forceinline__ __half from_float(float v) { return __float2half_rn(v); }
};

// bf16: the same with 128 + q (7 mantissa bits hold one nibble).
template <>
struct W4<__nv_bfloat16> {
    struct Zero {
        uint32_t lo;        // 128 + z
    };
    static __device__ __forceinline__ uint32_t u(__nv_bfloat162 h) { return *reinterpret_cast<uint32_t *>(&h); }
    static __device__ __forceinline__ __nv_bfloat162 h(uint32_t v) { return *reinterpret_cast<__nv_bfloat162 *>(&v); }
    static __device__ __forceinline__ Zero zero(uint32_t z0, uint32_t z1)
    {
        return {0x43004300u + (z0 | (z1 << 16))};
    }
    static __device__ __forceinline__ Zero zero_of(uint32_t lo) { return {lo}; }
    static __device__ __forceinline__ void unpack(uint32_t w, const Zero &z, uint32_t (&p)[4])
    {
#pragma unroll
        for (int i = 0; i < 4; i++)
            p[i] = u(__hsub2(h(lop_magic(w >> (4 * i), 0x000F000Fu, 0x43004300u)), h(z.lo)));
    }
    // An fp16 scale has 11 significant bits, bf16 8: the scale travels as the
    // sum of two bf16 values, so that the product below is rounded once.
    struct Scale {
        uint32_t hi, lo;
    };
    static __device__ __forceinline__ Scale scale(uint32_t s0, uint32_t s1)
    {
        const float a = __half2float(__ushort_as_half((unsigned short)s0));
        const float b = __half2float(__ushort_as_half((unsigned short)s1));
        const __nv_bfloat162 hi = __floats2bfloat162_rn(a, b);
        const float2 f = __bfloat1622float2(hi);
        // an infinite or NaN scale has no remainder to add
        const float ra = a - f.x, rb = b - f.y;
        return {u(hi), u(__floats2bfloat162_rn(ra == ra ? ra : 0.f, rb == rb ? rb : 0.f))};
    }
    static __device__ __forceinline__ uint32_t mul(uint32_t p, const Scale &s)
    {
        return u(__hfma2(h(p), h(s.hi), __hmul2(h(p), h(s.lo))));
    }
    // A pair of bf16 values times two fp16 scales (as bits), each rounded once.
    static __device__ __forceinline__ uint32_t times(uint32_t v, uint32_t s0, uint32_t s1)
    {
        const float2 f = __bfloat1622float2(h(v));
        return u(__floats2bfloat162_rn(
            f.x * __half2float(__ushort_as_half((unsigned short)s0)),
            f.y * __half2float(__ushort_as_half((unsigned short)s1))));
    }
    static __device__ __forceinline__ float low(uint32_t v) { return __low2float(h(v)); }
    static __device__ __forceinline__ float high(uint32_t v) { return __high2float(h(v)); }
    static __device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }
    static __device__ __forceinline__ __nv_bfloat16 from_float(float v) { return __float2bfloat16_rn(v); }
};

// D (fp32, 16 x 8) = A (16 x 16) B (16 x 8) + C, one warp.
template <typename T>
__device__ __forceinline__ void mma16816c(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                          uint32_t a3, uint32_t b0, uint32_t b1, float c0, float c1,
                                          float c2, float c3);

template <>
__device__ __forceinline__ void mma16816c<__half>(float (&d)[4], uint32_t a0, uint32_t a1,
                                                  uint32_t a2, uint32_t a3, uint32_t b0,
                                                  uint32_t b1, float c0, float c1, float c2,
                                                  float c3)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%10,%11,%12,%13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
}

template <>
__device__ __forceinline__ void mma16816c<__nv_bfloat16>(float (&d)[4], uint32_t a0, uint32_t a1,
                                                         uint32_t a2, uint32_t a3, uint32_t b0,
                                                         uint32_t b1, float c0, float c1, float c2,
                                                         float c3)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%10,%11,%12,%13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
}

// D += A B.
template <typename T>
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1)
{
    mma16816c<T>(d, a0, a1, a2, a3, b0, b1, d[0], d[1], d[2], d[3]);
}

// Four 8 x 16-byte tiles: lane (g, t) receives word t of row g of each; lane i
// gives the address of row i % 8 of tile i / 8.
__device__ __forceinline__ void ldmatrix4(uint32_t (&d)[4], uint32_t addr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(d[0]), "=r"(d[1]), "=r"(d[2]), "=r"(d[3])
                 : "r"(addr)
                 : "memory");
}

// The same tiles transposed: of each, lane (g, t) receives the 16-bit pieces g of
// rows 2 t (low half) and 2 t + 1 (high half).
__device__ __forceinline__ void ldmatrix4_trans(uint32_t (&d)[4], uint32_t addr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(d[0]), "=r"(d[1]), "=r"(d[2]), "=r"(d[3])
                 : "r"(addr)
                 : "memory");
}

// 2-D TMA map (linear_gemm.cu): boxes of box_rows x box_cols elements of a
// row-major matrix [rows][cols] with rows `pitch` bytes apart.
bool encode_map(CUtensorMap *map, CUtensorMapDataType type, const void *base, uint64_t cols,
                uint64_t rows, uint64_t pitch, uint32_t box_cols, uint32_t box_rows,
                CUtensorMapSwizzle swizzle);
// Clusters of s CTAs (s <= 8), one CTA per SM, that run at once on device
// `dev` (linear_gemm.cu); [0] and [1] are unused.
const int *cluster_table(int dev);

// bar_wait by a whole warp with one answer for all its lanes, so that a wait
// that gives up never splits the warp in front of a collective instruction.
__device__ __forceinline__ bool warp_wait(uint32_t b, uint32_t parity, volatile int *abort_flag)
{
    return __all_sync(0xffffffffu, bar_wait(b, parity, abort_flag));
}

// A lane's word(s) read from lane `src`.
template <typename S>
__device__ __forceinline__ S shfl_of(const S &v, int src)
{
    constexpr int N = sizeof(S) / 4;
    uint32_t u[N];
    memcpy(u, &v, sizeof(S));
#pragma unroll
    for (int i = 0; i < N; i++)
        u[i] = __shfl_sync(0xffffffffu, u[i], src);
    S r;
    memcpy(&r, u, sizeof(S));
    return r;
}

__device__ __forceinline__ void prefetch_map(const CUtensorMap *map)
{
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}

__device__ __forceinline__ void cluster_arrive()
{
    asm volatile("barrier.cluster.arrive.aligned;" ::: "memory");
}

__device__ __forceinline__ void cluster_wait()
{
    asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
}

// This CTA's shared address `addr` in the CTA `rank` of its cluster.
__device__ __forceinline__ uint32_t cluster_addr(uint32_t addr, int rank)
{
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}

// Stores to a shared address of the cluster; counted by barrier `bar` of the same CTA.
__device__ __forceinline__ void st_async(uint32_t addr, float v, uint32_t bar)
{
    asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.f32 [%0], %1, [%2];" ::"r"(
                     addr),
                 "f"(v), "r"(bar)
                 : "memory");
}

// A frozen 4-bit matrix in the canonical layout.
struct W4Matrix {
    const uint8_t *codes;       // [rows][K/2]
    const uint16_t *scales;     // [rows][K/group], fp16
    const uint8_t *zeros;       // [rows][K/group]
    int rows, K, group;
};

// One product: activations in [n][ldi], result out [n][ldo].
struct W4Call {
    W4Matrix w;
    const void *in;
    long long ldi;
    int n;
    const void *bias;           // [rows] or null (forward only)
    const void *residual;       // [n][ldr] or null (forward only)
    long long ldr;
    void *out;
    long long ldo;
    int *status;                // device status word or null
};

}  // namespace qe
