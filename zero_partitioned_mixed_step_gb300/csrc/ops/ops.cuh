// Device and host helpers that the operators share: element types, wide
// loads and stores with a scalar way round, warp reductions, the 8-bit casts
// and the checks of arguments.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstddef>
#include <cstdint>
#include <cstring>

#include "zerostep_ops.h"

namespace zo {

constexpr int kBlock = 128;             // elements that share a scale
constexpr float kTinyScale = 0x1p-126f;  // the smallest scale (and the largest 1 / s is 2^126)
constexpr int64_t kMaxDim = INT64_C(0x7FFFFFFF) - 1024;  // a tile's end still fits 32 bits

// ------------------------------------------------------------------ host

inline int cuda_error(cudaError_t e) { return ZERO_ECUDA_BASE - (int)e; }
inline int launch_status()
{
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? ZERO_OK : cuda_error(e);
}
inline bool aligned(const void *p, uintptr_t to)
{
    return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0;
}
inline bool is_half(int t) { return t == ZERO_T_F16 || t == ZERO_T_BF16; }
inline bool is_float(int t) { return is_half(t) || t == ZERO_T_F32; }
inline bool is_fp8(int t) { return t == ZERO_T_E4M3 || t == ZERO_T_E5M2; }
inline int type_bytes(int t) { return t == ZERO_T_F32 ? 4 : is_half(t) ? 2 : 1; }
inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline bool bad_dim(int64_t n) { return n < 0 || n > kMaxDim; }
// A matrix argument: present where it has elements, rows not overlapping, aligned to its element.
inline int check_matrix(const void *p, int64_t rows, int64_t cols, int64_t ld, int bytes)
{
    if (rows > 0 && cols > 0 && (!p || ld < cols || ld > (INT64_C(1) << 40)))
        return ZERO_EINVAL;
    return aligned(p, (uintptr_t)bytes) ? ZERO_OK : ZERO_EALIGN;
}
// Whether every row of a matrix starts on a multiple of `to` bytes.
inline bool rows_aligned(const void *p, int64_t ld, int bytes, uintptr_t to)
{
    return aligned(p, to) && (uint64_t)ld * (uint64_t)bytes % to == 0;
}
// SMs of the current device (a property, kept after the first use).
int device_sms();

// ------------------------------------------------------------------ element types

using f16 = __half;
using bf16 = __nv_bfloat16;

template <class T>
struct Type;
template <>
struct Type<f16> {
    static constexpr int code = ZERO_T_F16;
};
template <>
struct Type<bf16> {
    static constexpr int code = ZERO_T_BF16;
};
template <>
struct Type<float> {
    static constexpr int code = ZERO_T_F32;
};

__device__ __forceinline__ float to_f32(f16 x) { return __half2float(x); }
__device__ __forceinline__ float to_f32(bf16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f32(float x) { return x; }
template <class T>
__device__ __forceinline__ T from_f32(float x);
template <>
__device__ __forceinline__ f16 from_f32<f16>(float x)
{
    return __float2half_rn(x);
}
template <>
__device__ __forceinline__ bf16 from_f32<bf16>(float x)
{
    return __float2bfloat16_rn(x);
}
template <>
__device__ __forceinline__ float from_f32<float>(float x)
{
    return x;
}

// Eight neighbouring elements, kept in 32-bit words (halves two to a word: as
// an array of halves the compiler gives each a register of its own).
template <class T>
struct Raw8 {
    static constexpr int kWords = 2 * (int)sizeof(T);
    uint32_t w[kWords];

    __device__ __forceinline__ float at(int i) const
    {
        if constexpr (sizeof(T) == 4)
            return __uint_as_float(w[i]);
        else if constexpr (Type<T>::code == ZERO_T_BF16)
            return __uint_as_float(i & 1 ? w[i >> 1] & 0xFFFF0000u : w[i >> 1] << 16);
        else
            return __half2float(__ushort_as_half((unsigned short)(w[i >> 1] >> (16 * (i & 1)))));
    }
};

template <class T>
__device__ __forceinline__ uint32_t word_of(float a, float b)  // two halves, rounded
{
    if constexpr (Type<T>::code == ZERO_T_BF16) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&h);
    } else {
        const __half2 h = __floats2half2_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
}

// Eight elements from p, of which the first n exist (the others are zeros).
template <class T>
__device__ __forceinline__ Raw8<T> load_raw(const T *p, int n, bool wide)
{
    Raw8<T> r;
    if (wide && n >= 8) {
        const uint4 *q = reinterpret_cast<const uint4 *>(p);
#pragma unroll
        for (int i = 0; i < Raw8<T>::kWords / 4; ++i) {
            const uint4 x = q[i];
            r.w[4 * i] = x.x;
            r.w[4 * i + 1] = x.y;
            r.w[4 * i + 2] = x.z;
            r.w[4 * i + 3] = x.w;
        }
    } else if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            r.w[i] = i < n ? reinterpret_cast<const uint32_t *>(p)[i] : 0u;
    } else {
        const uint16_t *q = reinterpret_cast<const uint16_t *>(p);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            r.w[i] = (2 * i < n ? (uint32_t)q[2 * i] : 0u) | (2 * i + 1 < n ? (uint32_t)q[2 * i + 1] << 16 : 0u);
    }
    return r;
}

// Eight existing elements from a 16-byte aligned p, used once (LAST) or again soon.
template <bool LAST, class T>
__device__ __forceinline__ Raw8<T> load_full(const T *p)
{
    Raw8<T> r;
    const uint4 *q = reinterpret_cast<const uint4 *>(p);
#pragma unroll
    for (int i = 0; i < Raw8<T>::kWords / 4; ++i) {
        const uint4 x = LAST ? __ldcs(q + i) : __ldg(q + i);
        r.w[4 * i] = x.x;
        r.w[4 * i + 1] = x.y;
        r.w[4 * i + 2] = x.z;
        r.w[4 * i + 3] = x.w;
    }
    return r;
}

template <class T>
__device__ __forceinline__ void store_raw(T *p, int n, bool wide, const Raw8<T> &r)
{
    static_assert(sizeof(T) == 2, "halves");
    if (wide && n >= 8) {
        *reinterpret_cast<uint4 *>(p) = make_uint4(r.w[0], r.w[1], r.w[2], r.w[3]);
    } else {
        uint16_t *q = reinterpret_cast<uint16_t *>(p);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n)
                q[i] = (uint16_t)(r.w[i >> 1] >> (16 * (i & 1)));
    }
}

// The same as fp32 values.  `wide`: p is 16-byte aligned (a rule on the whole matrix).
template <class T>
__device__ __forceinline__ void load8(const T *p, int n, bool wide, float x[8])
{
    const Raw8<T> r = load_raw(p, n, wide);
#pragma unroll
    for (int i = 0; i < 8; ++i)
        x[i] = r.at(i);
}

template <class T>
__device__ __forceinline__ void store8(T *p, int n, bool wide, const float x[8])
{
    if constexpr (sizeof(T) == 4) {
        if (wide && n >= 8) {
            reinterpret_cast<float4 *>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
            reinterpret_cast<float4 *>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i < n)
                    p[i] = x[i];
        }
    } else {
        Raw8<T> r;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            r.w[i] = word_of<T>(x[2 * i], x[2 * i + 1]);
        store_raw(p, n, wide, r);
    }
}

// Eight 8-bit values, packed, to p; `wide`: p is 8-byte aligned.
__device__ __forceinline__ void store8b(uint8_t *p, int n, bool wide, uint2 v)
{
    if (wide && n >= 8) {
        *reinterpret_cast<uint2 *>(p) = v;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n)
                p[i] = (uint8_t)((i < 4 ? v.x : v.y) >> (8 * (i & 3)));
    }
}

// ------------------------------------------------------------------ 8-bit blocks

template <int F8>
struct F8Type;
template <>
struct F8Type<ZERO_T_E4M3> {
    static constexpr float qmax = 448.0f;
    static constexpr __nv_fp8_interpretation_t kind = __NV_E4M3;
};
template <>
struct F8Type<ZERO_T_E5M2> {
    static constexpr float qmax = 57344.0f;
    static constexpr __nv_fp8_interpretation_t kind = __NV_E5M2;
};

// A magnitude's bits order as the magnitude does, with infinity above every
// number and NaN above infinity: an integer maximum over them carries both.
__device__ __forceinline__ uint32_t magnitude(float x) { return __float_as_uint(x) & 0x7FFFFFFFu; }

// Magnitudes of a type's elements as order-preserving bits, two halves at a
// time (the same integer order as fp32's), and their largest as fp32 bits.
template <class T>
struct Amax {  // a half type
    uint32_t two = 0;
    __device__ __forceinline__ void add(uint32_t pair) { two = __vmaxu2(two, pair & 0x7FFF7FFFu); }
    __device__ __forceinline__ uint32_t bits() const
    {
        const uint16_t one = (uint16_t)max(two & 0xFFFFu, two >> 16);
        T x;
        memcpy(&x, &one, 2);
        return magnitude(to_f32(x));
    }
};

// The scale of a block whose largest magnitude is amax (as bits).
template <int F8>
__device__ __forceinline__ float block_scale(uint32_t amax)
{
    const float s = __fdiv_rn(__uint_as_float(amax), F8Type<F8>::qmax);
    return s < kTinyScale ? kTinyScale : s;  // NaN stays
}

template <int F8>
__device__ __forceinline__ uint32_t pack4(float a, float b, float c, float d)
{
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, F8Type<F8>::kind);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, F8Type<F8>::kind);
    return lo | hi << 16;
}

// 1 / s of a block's scale s in two parts, hi rounded down and so lo >= 0.
struct Inverse {
    float hi, lo;
};
__device__ __forceinline__ Inverse inverse(float s)
{
    Inverse r;
    r.hi = __frcp_rd(s);
    r.lo = s == __int_as_float(0x7F800000) ? 0.0f : __fmul_rn(__fmaf_rn(-s, r.hi, 1.0f), r.hi);
    return r;
}

// Two fp32 values at a time.
__device__ __forceinline__ float2 mul2(float2 a, float2 b)
{
    float2 r;
    asm("{ .reg .b64 x, y, z; mov.b64 x, {%2, %3}; mov.b64 y, {%4, %5}; mul.rn.f32x2 z, x, y; mov.b64 {%0, %1}, z; }"
        : "=f"(r.x), "=f"(r.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return r;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c)
{
    float2 r;
    asm("{ .reg .b64 x, y, z, w; mov.b64 x, {%2, %3}; mov.b64 y, {%4, %5}; mov.b64 z, {%6, %7};"
        " fma.rn.f32x2 w, x, y, z; mov.b64 {%0, %1}, w; }"
        : "=f"(r.x), "=f"(r.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return r;
}

// Eight quotients x / s, rounded to fp32 and then to 8 bits.  The fp32 quotient
// is x * hi + round(x * lo), rounded: the correctly rounded one for every pair
// of an fp16 or bf16 x below 2^117 and its block's s, above it and for fp32
// in all but a few of 1e8 pairs (x * round(1 / s) is off by an ulp for a quarter
// of all).  So an element whose quotient is the middle between two 8-bit values,
// which is common where x and the block's largest element have few bits, goes to
// the even one.  As lo is not negative, -0 stays.
template <int F8>
__device__ __forceinline__ uint2 quotients8(const float x[8], Inverse d)
{
    float2 q[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 y = make_float2(x[2 * i], x[2 * i + 1]);
        q[i] = fma2(y, make_float2(d.hi, d.hi), mul2(y, make_float2(d.lo, d.lo)));
    }
    return make_uint2(pack4<F8>(q[0].x, q[0].y, q[1].x, q[1].y), pack4<F8>(q[2].x, q[2].y, q[3].x, q[3].y));
}

// ------------------------------------------------------------------ reductions

template <int N>
__device__ __forceinline__ uint32_t max_over(uint32_t x)  // over N neighbouring lanes
{
#pragma unroll
    for (int o = N / 2; o > 0; o >>= 1)
        x = max(x, __shfl_xor_sync(0xFFFFFFFFu, x, o));
    return x;
}

template <int N>
__device__ __forceinline__ float sum_over(float x)
{
#pragma unroll
    for (int o = N / 2; o > 0; o >>= 1)
        x += __shfl_xor_sync(0xFFFFFFFFu, x, o);
    return x;
}

}  // namespace zo
