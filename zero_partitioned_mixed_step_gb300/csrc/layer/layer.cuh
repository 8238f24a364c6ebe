// What the kernels of libzerostep_layer.so share: 8-bit forms as kernels write
// and read them, sums over a row's threads, and the checks of their arguments.
#pragma once

#include "../ops/ops.cuh"
#include "zerostep_layer.h"

namespace zo {

// ------------------------------------------------------------------ 8-bit forms

struct Form {  // an output; q NULL = not wanted
    uint8_t *q;
    float *s;
    int64_t ld, lds;
    int32_t wide;  // rows start on 8-byte boundaries
};

inline Form form_of(const zero_fp8_form *f)
{
    Form o{};
    if (f) {
        o.q = static_cast<uint8_t *>(f->q);
        o.s = f->s;
        o.ld = f->ld;
        o.lds = f->lds;
        o.wide = rows_aligned(f->q, f->ld, 1, 8);
    }
    return o;
}

inline int check_form(const zero_fp8_form *f, int64_t rows, int64_t cols)
{
    if (!f)
        return ZERO_OK;
    const int rc = check_matrix(f->q, rows, cols, f->ld, 1);
    return rc ? rc : check_matrix(f->s, ceil_div(cols, kBlock), rows, f->lds, 4);
}

// A kept matrix: 8-bit with scales or of the half type without.
inline int check_kept(const void *x, int64_t ld, const float *s, int64_t lds, int type, int64_t rows, int64_t cols)
{
    const int rc = check_matrix(x, rows, cols, ld, s ? 1 : type_bytes(type));
    return rc || !s ? rc : check_matrix(s, ceil_div(cols, kBlock), rows, lds, 4);
}

// As a float, by a number that the whole launch shares.
__device__ __forceinline__ float scale_of(uint32_t amax, bool e5m2)
{
    const float s = __fdiv_rn(__uint_as_float(amax), e5m2 ? F8Type<ZERO_T_E5M2>::qmax : F8Type<ZERO_T_E4M3>::qmax);
    return s < kTinyScale ? kTinyScale : s;  // NaN stays
}

__device__ __forceinline__ uint2 quotients_of(const float x[8], Inverse d, bool e5m2)
{
    return e5m2 ? quotients8<ZERO_T_E5M2>(x, d) : quotients8<ZERO_T_E4M3>(x, d);
}

__device__ __forceinline__ uint32_t amax8(const float x[8])
{
    uint32_t a = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        a = max(a, magnitude(x[i]));
    return a;
}

// Eight neighbouring elements of a row into a form; the 16 lanes of a 1x128
// block come here together, each with its own amax and zeros where the row has ended.
__device__ __forceinline__ void put_form(const Form &f, int64_t row, int64_t c, int n, const float x[8],
                                         uint32_t amax, bool e5m2)
{
    const float s = scale_of(max_over<16>(amax), e5m2);
    if (n > 0) {
        if ((threadIdx.x & 15) == 0)
            f.s[(c / kBlock) * f.lds + row] = s;
        store8b(f.q + row * f.ld + c, n, f.wide, quotients_of(x, inverse(s), e5m2));
    }
}

// Two 8-bit values as fp32: exact, through the half type, which holds both formats.
template <int F8>
__device__ __forceinline__ float2 two_of(uint32_t pair)
{
    const __half2_raw r = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)pair, F8Type<F8>::kind);
    return __half22float2(__half2(r));
}

// Eight elements as they are kept: 8 bits each, or a half type's.
struct Raw8b {
    uint32_t w[2];

    template <int F8 = ZERO_T_E4M3>
    __device__ __forceinline__ void get(float x[8]) const
    {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 v = two_of<F8>(w[i >> 1] >> (16 * (i & 1)) & 0xFFFFu);
            x[2 * i] = v.x;
            x[2 * i + 1] = v.y;
        }
    }
};

__device__ __forceinline__ Raw8b load_raw8b(const uint8_t *p, int n, bool wide)
{
    Raw8b r;
    if (wide && n >= 8) {
        const uint2 x = *reinterpret_cast<const uint2 *>(p);
        r.w[0] = x.x;
        r.w[1] = x.y;
    } else {
        r.w[0] = r.w[1] = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n)
                r.w[i >> 2] |= (uint32_t)p[i] << (8 * (i & 3));
    }
    return r;
}

// A kept matrix's unit: S8 = 8-bit (times the scale of its block), else halves.
template <class H, bool S8>
struct Kept;
template <class H>
struct Kept<H, true> {
    static constexpr int kBytes = 8;
    Raw8b r;
    __device__ __forceinline__ void load(const void *p, int64_t at, int n, bool wide)
    {
        r = load_raw8b(static_cast<const uint8_t *>(p) + at, n, wide);
    }
    __device__ __forceinline__ void get(float x[8], float s) const
    {
        r.get(x);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            x[i] *= s;
    }
};
template <class H>
struct Kept<H, false> {
    static constexpr int kBytes = 16;
    Raw8<H> r;
    __device__ __forceinline__ void load(const void *p, int64_t at, int n, bool wide)
    {
        r = load_raw(static_cast<const H *>(p) + at, n, wide);
    }
    __device__ __forceinline__ void get(float x[8], float s) const
    {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            x[i] = r.at(i) * s;
    }
};

__device__ __forceinline__ float load_one(const void *p, int type, int64_t at)
{
    if (type == ZERO_T_F16)
        return to_f32(static_cast<const f16 *>(p)[at]);
    if (type == ZERO_T_BF16)
        return to_f32(static_cast<const bf16 *>(p)[at]);
    return static_cast<const float *>(p)[at];
}

// ------------------------------------------------------------------ sums over a row

// N sums over the threads of a row: G = 16 or 32 lanes, or (0) the CTA's
// blockDim.x / 32 warps, at most WARPS (a power of two).  `slot`: WARPS * N floats that
// the CTA does not use between this call's barrier and the next one's.
template <int G, int WARPS, int N>
__device__ __forceinline__ void row_sums(float (&x)[N], float *slot)
{
#pragma unroll
    for (int i = 0; i < N; ++i)
        x[i] = sum_over<G ? G : 32>(x[i]);
    if (G)
        return;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (lane == 0)
#pragma unroll
        for (int i = 0; i < N; ++i)
            slot[i * WARPS + warp] = x[i];
    __syncthreads();
    const int w = lane & (WARPS - 1);
#pragma unroll
    for (int i = 0; i < N; ++i)
        x[i] = sum_over<WARPS>(w < (blockDim.x >> 5) ? slot[i * WARPS + w] : 0.0f);
}

}  // namespace zo
