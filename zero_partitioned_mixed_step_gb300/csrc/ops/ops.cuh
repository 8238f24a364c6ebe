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

#include "zerostep_ops.h"

namespace zo {

constexpr int kBlock = 128;             // elements that share a scale
constexpr float kTinyScale = 0x1p-126f;  // the smallest scale (and the largest 1 / s is 2^126)
constexpr int64_t kMaxDim = INT64_C(0x7FFFFFFF);

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
// x rounded to T and back
template <class T>
__device__ __forceinline__ float rounded(float x)
{
    return to_f32(from_f32<T>(x));
}

// Eight neighbouring elements as they lie in memory.
template <class T>
struct alignas(sizeof(T) * 8 < 16 ? sizeof(T) * 8 : 16) Pack8 {
    T v[8];
};

// Eight elements from p, of which the first n exist (the others read as 0).
// `wide`: p is 16-byte aligned (a rule on the whole matrix).
template <class T>
__device__ __forceinline__ void load8(const T *p, int n, bool wide, float x[8])
{
    if (wide && n >= 8) {
        const Pack8<T> r = *reinterpret_cast<const Pack8<T> *>(p);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            x[i] = to_f32(r.v[i]);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            x[i] = i < n ? to_f32(p[i]) : 0.0f;
    }
}

template <class T>
__device__ __forceinline__ void store8(T *p, int n, bool wide, const float x[8])
{
    if (wide && n >= 8) {
        Pack8<T> r;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            r.v[i] = from_f32<T>(x[i]);
        *reinterpret_cast<Pack8<T> *>(p) = r;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n)
                p[i] = from_f32<T>(x[i]);
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
