// What the kernels of libzerostep_layer.so share: 8-bit forms as kernels write
// and read them, sums over a row's threads, and the checks of their arguments.
#pragma once

#include <atomic>

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

// A kernel as a value that a launch's lambda can hand on as a template's argument.
template <auto KERNEL>
struct Kernel {
    static constexpr auto value = KERNEL;
};
// Lets a kernel take that much dynamic shared memory, once for each device: the most that any launch of it
// takes, not the call's own amount, as the limit is the process's, and another thread's may come between
// a call's limit and its launch.
template <auto KERNEL>
inline int allow_smem(int bytes)
{
    static std::atomic<uint64_t> ready{0};  // bits of devices
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess && !(dev < 64 && (ready.load(std::memory_order_acquire) >> dev & 1))) {
        e = cudaFuncSetAttribute(KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e == cudaSuccess && dev < 64)
            ready.fetch_or(UINT64_C(1) << dev, std::memory_order_acq_rel);
    }
    return e == cudaSuccess ? ZERO_OK : cuda_error(e);
}

// A matrix in tiles of 128 columns: CTAs take one row of tiles after the other, so that those
// which run together read whole rows of memory (8192x14336, an activation read back as halves:
// 55.5 us, down the columns 59.6).
struct Tiles {
    int32_t rows, cols;  // tiles down and across
};
struct TileAt {
    int32_t r, c;
};
__device__ __forceinline__ TileAt tile_at(const Tiles &t)
{
    return {(int32_t)(blockIdx.x / (uint32_t)t.cols), (int32_t)(blockIdx.x % (uint32_t)t.cols)};
}
// Whether a 128x128 tile's units of 8, along either side, are whole or absent.
__device__ __forceinline__ bool whole_units(const TileAt &at, int rows, int cols)
{
    return (cols % 8 == 0 || at.c < cols / kBlock) && (rows % 8 == 0 || at.r < rows / kBlock);
}
inline Tiles tiles_of(int64_t rows, int64_t cols, int height)
{
    return {(int32_t)ceil_div(rows, height), (int32_t)ceil_div(cols, kBlock)};
}

// ------------------------------------------------------------------ eight elements

// Eight neighbouring elements of a row are four pairs: Blackwell's fp32 pipes take a
// pair at a time, and these kernels are bound by instructions before they are by memory.
// How rows lie: not where wide accesses want them (16 bytes, 8-bit rows 8); there, with a
// last unit of n < 8, which goes in at most three accesses of 4, 2 and 1 elements (a
// vector's fp32 ones one by one); or there, and 8 divides their length.
enum { kApart = 0, kWide = 1, kWhole = 2 };

__device__ __forceinline__ int left_of(int cols, int c) { return min(8, max(0, cols - c)); }

template <int W, class T>
__device__ __forceinline__ Raw8<T> get_raw(const T *p, int n)
{
    if constexpr (W == kApart) {
        return load_raw(p, n, false);
    } else if constexpr (W == kWhole) {
        Raw8<T> r{};
        if (n > 0)
            r = load_raw(p, 8, true);
        return r;
    } else if constexpr (sizeof(T) == 4) {
        if (n >= 8)
            return load_raw(p, 8, true);
        Raw8<T> r{};
#pragma unroll
        for (int i = 0; i < 7; ++i)
            if (i < n)
                r.w[i] = reinterpret_cast<const uint32_t *>(p)[i];
        return r;
    } else {
        if (n >= 8)
            return load_raw(p, 8, true);
        Raw8<T> r{};
        const uint16_t *q = reinterpret_cast<const uint16_t *>(p);
        uint2 four = make_uint2(0, 0);
        uint32_t two = 0, one = 0;
        if (n & 4)
            four = *reinterpret_cast<const uint2 *>(q);
        if (n & 2)
            two = *reinterpret_cast<const uint32_t *>(q + (n & 4));
        if (n & 1)
            one = q[n & 6];
        r.w[0] = n & 4 ? four.x : n & 2 ? two : one;
        r.w[1] = n & 4 ? four.y : n & 2 ? one : 0u;
        r.w[2] = n & 4 ? n & 2 ? two : one : 0u;
        r.w[3] = (n & 6) == 6 ? one : 0u;
        return r;
    }
}

template <int W, class T>
__device__ __forceinline__ void put_raw(T *p, int n, const Raw8<T> &r)
{
    if (W == kWhole) {
        store_raw(p, 8, true, r);
    } else if (W == kApart || n >= 8) {
        store_raw(p, n, W, r);
    } else {
        uint16_t *q = reinterpret_cast<uint16_t *>(p);
        if (n & 4)
            *reinterpret_cast<uint2 *>(q) = make_uint2(r.w[0], r.w[1]);
        if (n & 2)
            *reinterpret_cast<uint32_t *>(q + (n & 4)) = n & 4 ? r.w[2] : r.w[0];
        if (n & 1)
            q[n & 6] = (uint16_t)((n & 4) ? (n & 2) ? r.w[3] : r.w[2] : (n & 2) ? r.w[1] : r.w[0]);
    }
}

template <class H>
__device__ __forceinline__ float2 pair_of(uint32_t w)
{
    if constexpr (Type<H>::code == ZERO_T_BF16)
        return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
    else {
        __half2 h;
        memcpy(&h, &w, 4);
        return __half22float2(h);
    }
}

template <class H>
__device__ __forceinline__ void pairs_of(const Raw8<H> &r, float2 x[4])
{
#pragma unroll
    for (int i = 0; i < 4; ++i)
        x[i] = pair_of<H>(r.w[i]);
}

// Rounded to H; n > 0.
template <int W, class H>
__device__ __forceinline__ void put_pairs(H *p, int n, const float2 x[4])
{
    if constexpr (sizeof(H) == 4) {
        const float y[8] = {x[0].x, x[0].y, x[1].x, x[1].y, x[2].x, x[2].y, x[3].x, x[3].y};
        store8(p, W == kWhole ? 8 : n, W, y);
    } else {
        Raw8<H> r;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            r.w[i] = word_of<H>(x[i].x, x[i].y);
        put_raw<W>(p, n, r);
    }
}

// Of a vector of any of the types.
template <int W>
__device__ __forceinline__ void get_vector(const void *w, int type, int at, int n, float2 x[4])
{
    if (type == ZERO_T_F16)
        pairs_of(get_raw<W>(static_cast<const f16 *>(w) + at, n), x);
    else if (type == ZERO_T_BF16)
        pairs_of(get_raw<W>(static_cast<const bf16 *>(w) + at, n), x);
    else {
        const Raw8<float> r = get_raw<W>(static_cast<const float *>(w) + at, n);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            x[i] = make_float2(__uint_as_float(r.w[2 * i]), __uint_as_float(r.w[2 * i + 1]));
    }
}

__device__ __forceinline__ float2 both(float a) { return make_float2(a, a); }
__device__ __forceinline__ float2 add2(float2 a, float2 b)
{
    float2 r;
    asm("{ .reg .b64 x, y, z; mov.b64 x, {%2, %3}; mov.b64 y, {%4, %5}; add.rn.f32x2 z, x, y; mov.b64 {%0, %1}, z; }"
        : "=f"(r.x), "=f"(r.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return r;
}

// Behind the n elements of a row's last unit are zeros, which a factor that is not finite makes NaN.  They are
// kept out of the row's sums and its last block's scale: a unit without elements takes 0 as its factor
// (a select, where a branch in the norms takes 2 us of 66 at 8192x4096), a short one has zeros put back.
__device__ __forceinline__ float in_row_only(float factor, int n) { return n > 0 ? factor : 0.0f; }
__device__ __forceinline__ void clear_behind(float2 (&x)[4], int n)
{
#pragma unroll
    for (int i = 0; i < 4; ++i)
        x[i] = make_float2(2 * i < n ? x[i].x : 0.0f, 2 * i + 1 < n ? x[i].y : 0.0f);
}
template <int W>
__device__ __forceinline__ void end_unit(float2 (&x)[4], int n, float factor)
{
    if (W != kWhole && n < 8 && !(fabsf(factor) <= 3.402823466e38f))
        clear_behind(x, n);
}

// ------------------------------------------------------------------ 8-bit blocks

__device__ __forceinline__ float max3(float a, float b, float c)  // of magnitudes; a NaN stays
{
    float r;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
__device__ __forceinline__ uint32_t amax8(const float2 x[4])
{
    float a = max3(x[0].x, x[0].y, x[1].x);
    a = max3(a, x[1].y, x[2].x);
    a = max3(a, x[2].y, x[3].x);
    return __float_as_uint(max3(a, x[3].y, x[3].y));
}
template <class H>
__device__ __forceinline__ uint32_t amax8(const Raw8<H> &r)
{
    Amax<H> a;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        a.add(r.w[i]);
    return a.bits();
}

// The sums of P values (2, 4 or 8) over L lanes (16 or 32), shared out in the same way: value i
// ends with the lanes L / P * i and up.
template <int P, int L>
__device__ __forceinline__ float sum_shared(float (&x)[P])
{
    int bit = L / 2;
#pragma unroll
    for (int half = P / 2; half; half >>= 1, bit >>= 1)
#pragma unroll
        for (int i = 0; i < half; ++i) {
            const bool up = threadIdx.x & bit;
            const float keep = up ? x[i + half] : x[i], give = up ? x[i] : x[i + half];
            x[i] = keep + __shfl_xor_sync(0xFFFFFFFFu, give, bit);
        }
#pragma unroll
    for (; bit; bit >>= 1)
        x[0] += __shfl_xor_sync(0xFFFFFFFFu, x[0], bit);
    return x[0];
}

// The largest of each of N values (1, 2 or 4) over 16 lanes.  The lanes share the
// values out between them as they exchange: value i ends with the lanes
// 16 / N * i and up, which then form its scale once.  log2 N + 4 - log2 N steps, but
// N - 1 + 4 - log2 N shuffles where one value after the other takes 4 N.
template <int N>
__device__ __forceinline__ uint32_t max_shared(uint32_t (&a)[N])
{
    const int lane = threadIdx.x;
    int bit = 8;
#pragma unroll
    for (int half = N / 2; half; half >>= 1, bit >>= 1)
#pragma unroll
        for (int i = 0; i < half; ++i) {
            const bool up = lane & bit;
            const uint32_t keep = up ? a[i + half] : a[i], give = up ? a[i] : a[i + half];
            a[i] = max(keep, __shfl_xor_sync(0xFFFFFFFFu, give, bit));
        }
#pragma unroll
    for (; bit; bit >>= 1)
        a[0] = max(a[0], __shfl_xor_sync(0xFFFFFFFFu, a[0], bit));
    return a[0];
}
template <int N>
__device__ __forceinline__ int shared_index()
{
    return (threadIdx.x & 15) / (16 / N);
}
template <int N>
__device__ __forceinline__ float shared_value(float mine, int i)
{
    return __shfl_sync(0xFFFFFFFFu, mine, 16 / N * i, 16);
}

// amax / qmax, correctly rounded, without a division: with y = 1 / qmax rounded to nearest,
// q = a y and the remainder r = a - qmax q, which is exact, q + r y is the rounded
// quotient (Markstein, IBM J. Res. Dev. 34, 1990).  Infinite and NaN maxima are their
// own scales, and what is below the smallest scale becomes it.
__device__ __forceinline__ float scale_from(uint32_t amax, float qmax, float inv_qmax)
{
    const float a = __uint_as_float(amax), q = a * inv_qmax;
    float s = fmaf(fmaf(-qmax, q, a), inv_qmax, q);
    s = a < __int_as_float(0x7F800000) ? s : a;
    return s < kTinyScale ? kTinyScale : s;
}
template <bool E5M2>
__device__ __forceinline__ float scale_of(uint32_t amax)
{
    return E5M2 ? scale_from(amax, 57344.0f, 1.0f / 57344.0f) : scale_from(amax, 448.0f, 1.0f / 448.0f);
}
// The same for a type that the launch knows: two numbers of it, formed once.
struct Range {
    float qmax, inv;
    __device__ __forceinline__ explicit Range(bool e5m2) : qmax(e5m2 ? 57344.0f : 448.0f), inv(e5m2 ? 1.0f / 57344.0f : 1.0f / 448.0f) {}
    __device__ __forceinline__ float scale(uint32_t amax) const { return scale_from(amax, qmax, inv); }
};

// 1 / s in two parts, the first below it by up to 2^-21 of it: x * hi + x * lo rounds as x / s does, in the
// halves that are kept and in what is computed in fp32 alike.  Quotients are often the middle of two 8-bit
// values, which one product with 1 / s turns over.  As lo is not negative -0 stays.  An infinite block has
// hi = lo = 0: its numbers become 0, its infinities NaN.
__device__ __forceinline__ Inverse inverse_of(float s)
{
    float quick;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(quick) : "f"(s));
    Inverse r;
    r.hi = quick * (1.0f - 0x1p-22f);
    r.lo = s == __int_as_float(0x7F800000) ? 0.0f : fmaf(-s, r.hi, 1.0f) * r.hi;
    return r;
}
template <int N>
__device__ __forceinline__ Inverse shared_value(Inverse mine, int i)
{
    return {shared_value<N>(mine.hi, i), shared_value<N>(mine.lo, i)};
}

// Which type is a template's argument: where it is a number that the launch shares, the
// compiler forms both and selects.
template <bool E5M2>
__device__ __forceinline__ uint2 bytes_of(const float2 q[4])
{
    constexpr int F = E5M2 ? ZERO_T_E5M2 : ZERO_T_E4M3;
    return make_uint2(pack4<F>(q[0].x, q[0].y, q[1].x, q[1].y), pack4<F>(q[2].x, q[2].y, q[3].x, q[3].y));
}
template <bool E5M2>
__device__ __forceinline__ uint2 bytes_of(const float2 x[4], Inverse d)
{
    float2 q[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        q[i] = fma2(x[i], both(d.hi), mul2(x[i], both(d.lo)));
    return bytes_of<E5M2>(q);
}
template <int W>
__device__ __forceinline__ void put_bytes(uint8_t *p, int n, uint2 v)
{
    if (W == kWhole) {
        store8b(p, 8, true, v);
    } else if (W == kApart || n >= 8) {
        store8b(p, n, W, v);
    } else {
        if (n & 4)
            *reinterpret_cast<uint32_t *>(p) = v.x;
        const uint32_t rest = n & 4 ? v.y : v.x;
        if (n & 2)
            *reinterpret_cast<uint16_t *>(p + (n & 4)) = (uint16_t)rest;
        if (n & 1)
            p[n & 6] = (uint8_t)(n & 2 ? rest >> 16 : rest);
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
};
template <int F8 = ZERO_T_E4M3>
__device__ __forceinline__ void pairs_of(const Raw8b &r, float2 x[4])
{
#pragma unroll
    for (int i = 0; i < 4; ++i)
        x[i] = two_of<F8>(i & 1 ? r.w[i >> 1] >> 16 : r.w[i >> 1] & 0xFFFFu);
}

template <int W>
__device__ __forceinline__ Raw8b get_bytes(const uint8_t *p, int n)
{
    Raw8b r{};
    if (W == kWhole ? n > 0 : W == kWide && n >= 8) {
        const uint2 x = *reinterpret_cast<const uint2 *>(p);
        r.w[0] = x.x;
        r.w[1] = x.y;
    } else if (W == kWide) {
        uint32_t four = 0, rest = 0;
        if (n & 4)
            four = *reinterpret_cast<const uint32_t *>(p);
        if (n & 2)
            rest = *reinterpret_cast<const uint16_t *>(p + (n & 4));
        if (n & 1)
            rest |= (uint32_t)p[n & 6] << (n & 2 ? 16 : 0);
        r.w[0] = n & 4 ? four : rest;
        r.w[1] = n & 4 ? rest : 0u;
    } else if (W == kApart) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n)
                r.w[i >> 2] |= (uint32_t)p[i] << (8 * (i & 3));
    }
    return r;
}

// A kept matrix's unit: S8 = 8-bit (its values times the scale of its block), else halves.
template <class H, bool S8>
struct Kept;
template <class H>
struct Kept<H, true> {
    static constexpr int kBytes = 8;
    Raw8b r;
    template <int W>
    __device__ __forceinline__ void load(const void *row, int c, int n)
    {
        r = get_bytes<W>(static_cast<const uint8_t *>(row) + c, n);
    }
    __device__ __forceinline__ void get(float2 x[4]) const { pairs_of(r, x); }
};
template <class H>
struct Kept<H, false> {
    static constexpr int kBytes = 16;
    Raw8<H> r;
    template <int W>
    __device__ __forceinline__ void load(const void *row, int c, int n)
    {
        r = get_raw<W>(static_cast<const H *>(row) + c, n);
    }
    __device__ __forceinline__ void get(float2 x[4]) const { pairs_of(r, x); }
};

// Copies of 8 or 16 bytes into shared memory that run beside the thread; of them
// `bytes` are read and the others become zeros.
template <int BYTES>
__device__ __forceinline__ void copy_async(uint32_t to, const void *from, int bytes)
{
    if constexpr (BYTES == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(bytes) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(to), "l"(from), "r"(bytes) : "memory");
}
__device__ __forceinline__ void commit_copies() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>  // all but the last N groups have arrived
__device__ __forceinline__ void wait_copies()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ float load_one(const void *p, int type, int64_t at)
{
    if (type == ZERO_T_F16)
        return to_f32(static_cast<const f16 *>(p)[at]);
    if (type == ZERO_T_BF16)
        return to_f32(static_cast<const bf16 *>(p)[at]);
    return static_cast<const float *>(p)[at];
}

// ------------------------------------------------------------------ sums over a row

// N sums over a CTA, whose row it is: its blockDim.x / 32 warps, at most WARPS (a power of two).
// `slot`: WARPS * N floats that the CTA does not use between this call's barrier and the next
// one's.
template <int WARPS, int N>
__device__ __forceinline__ void row_sums(float (&x)[N], float *slot)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
    for (int i = 0; i < N; ++i)
        x[i] = sum_over<32>(x[i]);
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
