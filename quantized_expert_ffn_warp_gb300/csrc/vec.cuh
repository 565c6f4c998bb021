// 16-byte words of fp32, fp16 or bf16 values, and reductions over a warp.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "internal.cuh"

namespace qe {

template <typename T>
struct Vec {
    static constexpr int N = 16 / sizeof(T);    // values of a word
};

template <typename T>
__device__ __forceinline__ float2 unpack2(uint32_t u);
template <>
__device__ __forceinline__ float2 unpack2<__half>(uint32_t u)
{
    return __half22float2(*reinterpret_cast<const __half2 *>(&u));
}
template <>
__device__ __forceinline__ float2 unpack2<__nv_bfloat16>(uint32_t u)
{
    return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xFFFF0000u));
}
template <typename T>
__device__ __forceinline__ uint32_t pack2(float a, float b);
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float a, float b)
{
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float a, float b)
{
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}

template <typename T>
__device__ __forceinline__ void unpack(const uint4 &q, float (&d)[Vec<T>::N])
{
    const uint32_t u[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; i++) {
        if constexpr (sizeof(T) == 4) {
            d[i] = __uint_as_float(u[i]);
        } else {
            const float2 f = unpack2<T>(u[i]);
            d[2 * i] = f.x;
            d[2 * i + 1] = f.y;
        }
    }
}
template <typename T>
__device__ __forceinline__ uint4 pack(const float (&d)[Vec<T>::N])
{
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; i++) {
        if constexpr (sizeof(T) == 4)
            u[i] = __float_as_uint(d[i]);
        else
            u[i] = pack2<T>(d[2 * i], d[2 * i + 1]);
    }
    return make_uint4(u[0], u[1], u[2], u[3]);
}

template <typename T>
__device__ __forceinline__ float to_float(T v)
{
    if constexpr (sizeof(T) == 4)
        return v;
    else
        return static_cast<float>(v);
}
template <typename T>
__device__ __forceinline__ T from_float(float v);
template <>
__device__ __forceinline__ float from_float<float>(float v) { return v; }
template <>
__device__ __forceinline__ __half from_float<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_float<__nv_bfloat16>(float v)
{
    return __float2bfloat16_rn(v);
}

// Two fp32 values in a register pair, the operand of the paired instructions: one
// issue slot for two additions, products or fused operations, each rounded as its
// scalar form.
struct F2 {
    unsigned long long v;
};
__device__ __forceinline__ F2 f2(float x, float y)
{
    F2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(x), "f"(y));
    return r;
}
__device__ __forceinline__ F2 f2(float x) { return f2(x, x); }
__device__ __forceinline__ float2 split(F2 a)
{
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a.v));
    return r;
}
__device__ __forceinline__ F2 add(F2 a, F2 b)
{
    F2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 mul(F2 a, F2 b)
{
    F2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 fma(F2 a, F2 b, F2 c)
{
    F2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return r;
}
__device__ __forceinline__ float sum(F2 a)
{
    const float2 f = split(a);
    return f.x + f.y;
}

// A 16-byte word's values in pairs, and back with one rounding.
template <typename T>
__device__ __forceinline__ void unpack(const uint4 &q, F2 (&d)[Vec<T>::N / 2])
{
    const uint32_t u[4] = {q.x, q.y, q.z, q.w};
    if constexpr (sizeof(T) == 4) {
        d[0] = f2(__uint_as_float(u[0]), __uint_as_float(u[1]));
        d[1] = f2(__uint_as_float(u[2]), __uint_as_float(u[3]));
    } else {
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const float2 f = unpack2<T>(u[i]);
            d[i] = f2(f.x, f.y);
        }
    }
}
template <typename T>
__device__ __forceinline__ uint4 pack(const F2 (&d)[Vec<T>::N / 2])
{
    uint32_t u[4];
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < 2; i++) {
            const float2 f = split(d[i]);
            u[2 * i] = __float_as_uint(f.x);
            u[2 * i + 1] = __float_as_uint(f.y);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const float2 f = split(d[i]);
            u[i] = pack2<T>(f.x, f.y);
        }
    }
    return make_uint4(u[0], u[1], u[2], u[3]);
}

// The hardware's 2^x: 0 below 2^-126, documented within 2 units in the last place.
__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
constexpr float kLog2E = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kLog2ELow = (float)(1.4426950408889634 - (double)kLog2E);   // what kLog2E lacks

// max(a, b), a NaN if either is one
__device__ __forceinline__ float max_nan(float a, float b)
{
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}

// Largest value of a 16-byte word (a NaN is passed over), and the word with its values
// raised to `low` where they are below (a NaN stays one).
template <typename T>
__device__ __forceinline__ float word_max(const uint4 &q)
{
    const uint32_t u[4] = {q.x, q.y, q.z, q.w};
    if constexpr (sizeof(T) == 4) {
        return fmaxf(fmaxf(__uint_as_float(u[0]), __uint_as_float(u[1])),
                     fmaxf(__uint_as_float(u[2]), __uint_as_float(u[3])));
    } else if constexpr (std::is_same_v<T, __half>) {
        const auto h = [&](int i) { return *reinterpret_cast<const __half2 *>(&u[i]); };
        const __half2 m = __hmax2(__hmax2(h(0), h(1)), __hmax2(h(2), h(3)));
        return fmaxf(__low2float(m), __high2float(m));
    } else {
        const auto h = [&](int i) { return *reinterpret_cast<const __nv_bfloat162 *>(&u[i]); };
        const __nv_bfloat162 m = __hmax2(__hmax2(h(0), h(1)), __hmax2(h(2), h(3)));
        return fmaxf(__low2float(m), __high2float(m));
    }
}
template <typename T>
__device__ __forceinline__ uint4 word_raise(const uint4 &q, float low)
{
    uint32_t u[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; i++) {
        if constexpr (sizeof(T) == 4) {
            u[i] = __float_as_uint(max_nan(__uint_as_float(u[i]), low));
        } else {
            const uint32_t l = pack2<T>(low, low);
            if constexpr (std::is_same_v<T, __half>)
                asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(u[i]) : "r"(u[i]), "r"(l));
            else
                asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(u[i]) : "r"(u[i]), "r"(l));
        }
    }
    return make_uint4(u[0], u[1], u[2], u[3]);
}

__device__ __forceinline__ float max_warp(float v)
{
#pragma unroll
    for (int d = 16; d > 0; d >>= 1)
        v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, d));
    return v;
}
__device__ __forceinline__ float sum_warp(float v)
{
#pragma unroll
    for (int d = 16; d > 0; d >>= 1)
        v += __shfl_xor_sync(0xffffffffu, v, d);
    return v;
}

// Streamed data that is read once.
__device__ __forceinline__ uint4 load_stream(const void *p)
{
    uint4 q;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(q.x), "=r"(q.y), "=r"(q.z), "=r"(q.w)
                 : "l"(p));
    return q;
}

// A row of `len` values at any address as 16-byte words: the first and the last
// may reach past its ends.
template <typename T>
struct RowWords {
    static constexpr int N = Vec<T>::N;
    const T *row;           // first value
    int off, len, count;    // values in front of it in its word; values; words

    __device__ __forceinline__ RowWords(const T *r, int length)
        : row(r), off((int)(((uintptr_t)r & 15) / sizeof(T))), len(length),
          count((off + length + N - 1) / N)
    {
    }
    __device__ __forceinline__ int first(int v) const { return v * N - off; }
    __device__ __forceinline__ bool whole(int v) const
    {
        const int i = first(v);
        return i >= 0 && i + N <= len;
    }
    // whether words v .. v + n - 1 lie inside the row
    __device__ __forceinline__ bool inner(int v, int n) const
    {
        const int i = first(v);
        return i >= 0 && i + n * N <= len;
    }
    // word v into `out`, a row like this one whose words lie alike if `aligned`
    __device__ __forceinline__ void store(T *out, int v, const uint4 &q, bool aligned) const
    {
        if (aligned && whole(v)) {
            *reinterpret_cast<uint4 *>(out + first(v)) = q;
            return;
        }
        float d[N];
        unpack<T>(q, d);
#pragma unroll
        for (int e = 0; e < N; e++) {
            const int i = first(v) + e;
            if (i >= 0 && i < len)
                out[i] = from_float<T>(d[e]);
        }
    }
    // word v; values past the row's ends read `fill`
    __device__ __forceinline__ uint4 load(int v, float fill) const
    {
        if (whole(v))
            return load_stream(row + first(v));
        float d[N];
#pragma unroll
        for (int e = 0; e < N; e++) {
            const int i = first(v) + e;
            d[e] = i >= 0 && i < len ? to_float<T>(row[i]) : fill;
        }
        return pack<T>(d);
    }
};

}  // namespace qe
