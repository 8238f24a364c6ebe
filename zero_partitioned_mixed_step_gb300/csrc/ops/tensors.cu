// The global L2 norm over many gradient tensors, and the clipped gradients.
//
//   sumsq = sum_t sum_i (x_ti * inv_scale)^2
//   out   = x * (inv_scale * c),  c = min(1, max_norm / (sqrt(sumsq) + 1e-6))
//
// Both are bound by memory: the norm reads every element once, the clip reads
// and writes it once more (no update can start before the norm is known, and
// a model's gradients are far more than L2 holds).  The tensors' pointers and
// sizes travel as kernel arguments (up to kCapacity of them per launch), so a
// call with new gradients needs no copy to the device and no table there.  A
// tensor is cut into chunks of a size that follows from the list's total
// alone, a CTA takes one, and the hardware hands out the chunks: the sum's
// order depends on the sizes, not on the GPU.
//   1 G halves: norm 285 us, 7.0 TB/s; clip 587 us, 6.8 TB/s (the copy rate)
//   1.88 G bf16 of 8 decoder layers, norm and clip: 1.64 ms, 4.6 TB/s of input
//   and output once each, 6.9 of what has to move
//   124 M halves in 148 tensors, both: 127 us; the CTAs' ends (a chunk's sum over
//   its threads, then the total) show here
#include "ops.cuh"

#include <atomic>
#include <cstring>
#include <type_traits>

namespace zo {

constexpr int kThreads = 256;
constexpr int kUnit = 8;                  // elements of one wide access
constexpr int kBatch = 4;                 // wide accesses of a thread in flight
constexpr int64_t kTargetChunks = 8192;   // of a whole list
constexpr int kCapacity = 1024;           // tensors per launch
constexpr int kEndThreads = 1024;
// From so many chunks on the norm ends in a kernel of its own, launched while the
// chunks are summed: their CTAs need not count themselves then, and 1024
// threads add their sums.  (7565 chunks: 57.6 us for 60.1, with the tensors' own
// sums 66.9 for 79.5.)  A short list saves the launch.
constexpr uint32_t kEndChunks = 512;
constexpr int kHeader = 256;              // bytes of the workspace ahead of the chunk sums

// The workspace's start: zero between calls.
struct Header {
    uint32_t done;  // finished CTAs of the running launch
    uint32_t bad;   // 1: something is not finite
};

int device_sms()
{
    constexpr int kDevices = 64;
    static std::atomic<int> count[kDevices];
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess)
        return 1;
    if (dev >= 0 && dev < kDevices && (sms = count[dev].load(std::memory_order_acquire)) > 0)
        return sms;
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms < 1)
        return 1;
    if (dev >= 0 && dev < kDevices)
        count[dev].store(sms, std::memory_order_release);
    return sms;
}

// A chunk's elements, a multiple of what a CTA of the shortest ones takes: few
// elements want all SMs, more of them chunks that are worth a CTA's start and
// end.  The norm of 1 M halves in chunks of 4096, 8192 and 16384: 6.2, 5.4 and
// 5.7 us; 4 M: 9.8, 8.1, 7.3; 30 M: 37.6 in chunks of 4096, 22.8 of 16384, and
// their clip 29.0 and 20.4.
static int64_t chunk_elems(int64_t total)
{
    const int64_t least = total < 1 << 18 ? 4096 : total < 1 << 22 ? 8192 : 16384;
    const int64_t c = ceil_div(ceil_div(total, kTargetChunks), least) * least;
    return c < least ? least : c;
}

// One launch's tensors.  first[t] is tensor t's first chunk, first[n] the
// number of chunks.  Empty tensors are left out.
template <int CAP, bool OUT>
struct List {
    static constexpr int kCap = CAP;
    const void *x[CAP];
    void *out[OUT ? CAP : 1];
    int64_t numel[CAP];
    uint32_t first[CAP + 1];
    int32_t index[CAP];   // in the caller's list
    uint8_t type[CAP];
    uint8_t out_type[OUT ? CAP : 1];
    int64_t chunk;
    int32_t n;
};

template <int CAP, bool OUT>
__device__ __forceinline__ int find_tensor(const List<CAP, OUT> &l, uint32_t c)
{
    int lo = 0, hi = l.n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (l.first[mid] <= c)
            lo = mid;
        else
            hi = mid - 1;
    }
    return lo;
}

// ------------------------------------------------------------------ norm

// The sum of two pairs (hi, lo) of fp32 values, hi carrying the rounded sum.
__device__ __forceinline__ float2 pair_add(float2 a, float2 b)
{
    const float s = __fadd_rn(a.x, b.x);
    const float bb = __fsub_rn(s, a.x);
    const float err = __fadd_rn(__fsub_rn(a.x, __fsub_rn(s, bb)), __fsub_rn(b.x, bb));
    return make_float2(s, __fadd_rn(__fadd_rn(a.y, b.y), err));
}

// The squares of n elements from p: eight running fp32 sums per thread.
template <class T>
__device__ __forceinline__ float2 sum_chunk(const T *p, int64_t n, float inv)
{
    float acc[kUnit];
#pragma unroll
    for (int i = 0; i < kUnit; ++i)
        acc[i] = 0.0f;
    const bool wide = (reinterpret_cast<uintptr_t>(p) & 15) == 0;
    auto add = [&](const Raw8<T> &x) {
#pragma unroll
        for (int i = 0; i < kUnit; ++i) {
            const float g = __fmul_rn(x.at(i), inv);
            acc[i] = fmaf(g, g, acc[i]);
        }
    };
    int64_t u = threadIdx.x;
    if (wide)  // kBatch loads in flight
        for (; (u + (kBatch - 1) * kThreads + 1) * kUnit <= n; u += kBatch * kThreads) {
            Raw8<T> x[kBatch];
#pragma unroll
            for (int k = 0; k < kBatch; ++k)
                x[k] = load_full<false>(p + (u + k * kThreads) * kUnit);
#pragma unroll
            for (int k = 0; k < kBatch; ++k)
                add(x[k]);
        }
    for (; u * kUnit < n; u += kThreads) {
        const int64_t left = n - u * kUnit;
        add(load_raw(p + u * kUnit, left < kUnit ? (int)left : kUnit, wide));
    }
    float2 s = make_float2(acc[0], 0.0f);
#pragma unroll
    for (int i = 1; i < kUnit; ++i)
        s = pair_add(s, make_float2(acc[i], 0.0f));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        s = pair_add(s, make_float2(__shfl_xor_sync(0xFFFFFFFFu, s.x, o),
                                    __shfl_xor_sync(0xFFFFFFFFu, s.y, o)));
    return s;
}

// The same in binary64, for chunks whose fp32 sum is out of range; *bad is set
// where an element is not finite.  Units of zeros (a chunk of zeros comes here
// too) cost their load alone.
template <class T>
__device__ double sum_chunk_wide(const T *p, int64_t n, float inv, bool *bad)
{
    double s = 0.0;
    const bool wide = (reinterpret_cast<uintptr_t>(p) & 15) == 0;
#pragma unroll 2
    for (int64_t u = threadIdx.x; u * kUnit < n; u += kThreads) {
        const int64_t left = n - u * kUnit;
        float x[kUnit];
        load8(p + u * kUnit, left < kUnit ? (int)left : kUnit, wide, x);
        bool any = false;
#pragma unroll
        for (int i = 0; i < kUnit; ++i)
            any |= x[i] != 0.0f;  // NaN too
        if (any)
            for (int i = 0; i < kUnit; ++i) {
                const float g = __fmul_rn(x[i], inv);
                *bad |= !isfinite(g);
                s += (double)g * g;
            }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
    return s;
}

template <class F>
__device__ __forceinline__ auto by_type(int type, const void *p, int64_t at, F &&f)
{
    if (type == ZERO_T_F16)
        return f(static_cast<const f16 *>(p) + at);
    if (type == ZERO_T_BF16)
        return f(static_cast<const bf16 *>(p) + at);
    return f(static_cast<const float *>(p) + at);
}

// Doubles p[0 .. n) summed by a CTA of T threads in a fixed order; valid in thread 0.
template <int T>
__device__ double cta_sum(const double *p, int64_t n, double *shared)
{
    double s = 0.0;
#pragma unroll 8
    for (int64_t i = threadIdx.x; i < n; i += T)
        s += __ldcg(p + i);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
    __syncthreads();
    if ((threadIdx.x & 31) == 0)
        shared[threadIdx.x >> 5] = s;
    __syncthreads();
    s = 0.0;
    if (threadIdx.x == 0)
        for (int w = 0; w < T / 32; ++w)
            s += shared[w];
    return s;
}

// What follows once every chunk of a launch is summed, by a CTA of T threads:
// the tensors' sums, and the total.
struct NormOut {
    double *tensor_sumsq;
    zero_tensors_stat *stat;
    Header *head;
    double *sums;
    int32_t first_launch, last_launch;
};
template <int T, int CAP>
__device__ __forceinline__ void end_norm(const List<CAP, false> &l, const NormOut &o, double *shared)
{
    auto each = [&](auto lanes) {  // G neighbouring threads to a tensor
        constexpr int G = decltype(lanes)::value;
        const int at = threadIdx.x & (G - 1);
        const uint32_t group = G == 32 ? 0xFFFFFFFFu : ((1u << (G & 31)) - 1) << (threadIdx.x & 31 & ~(G - 1));
        for (int t = threadIdx.x / G; t < l.n; t += T / G) {
            double s = 0.0;
            for (uint32_t i = l.first[t] + at; i < l.first[t + 1]; i += G)
                s += __ldcg(o.sums + i);
#pragma unroll
            for (int k = G / 2; k > 0; k >>= 1)
                s += __shfl_xor_sync(group, s, k);
            if (at == 0)
                o.tensor_sumsq[l.index[t]] = s;
        }
    };
    if (o.tensor_sumsq && l.n > 0) {
        // by what a tensor has on average (300 tensors of one chunk each: 11.6
        // us for 33.8 with a warp to each)
        if (l.first[l.n] > 16 * (uint32_t)l.n)
            each(std::integral_constant<int, 32>{});
        else
            each(std::integral_constant<int, 4>{});
    }
    const double total = cta_sum<T>(o.sums, l.n > 0 ? l.first[l.n] : 0, shared);
    if (threadIdx.x == 0) {
        const double all = o.first_launch ? total : o.stat->sumsq + total;
        o.stat->sumsq = all;
        o.stat->norm = (float)sqrt(all);
        o.head->done = 0;
        if (o.last_launch) {
            o.stat->found_inf = (int32_t)o.head->bad;
            o.head->bad = 0;
        }
    }
}

template <int CAP>
__global__ void __launch_bounds__(kThreads)
    norm_kernel(const __grid_constant__ List<CAP, false> l, float inv, const NormOut out, int ends)
{
    if (!ends)
        asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    __shared__ float2 warp_pair[kThreads / 32];
    __shared__ double warp_sum[kThreads / 32];
    __shared__ int last;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t c = blockIdx.x;
    if (l.n > 0) {
        const int t = find_tensor(l, c);
        const int64_t at = (int64_t)(c - l.first[t]) * l.chunk;
        const int64_t left = l.numel[t] - at;
        const int64_t n = left < l.chunk ? left : l.chunk;
        const float2 s = by_type(l.type[t], l.x[t], at,
                                 [&](auto *p) { return sum_chunk(p, n, inv); });
        if (lane == 0)
            warp_pair[warp] = s;
        __syncthreads();
        // each warp adds the warps' sums, in the same order, and so needs no other's
        float2 a = warp_pair[lane & (kThreads / 32 - 1)];
#pragma unroll
        for (int o = kThreads / 64; o > 0; o >>= 1)
            a = pair_add(a, make_float2(__shfl_xor_sync(0xFFFFFFFFu, a.x, o), __shfl_xor_sync(0xFFFFFFFFu, a.y, o)));
        double sum = (double)a.x + (double)a.y;
        // below 2^-90 some squares of the chunk may have lost bits under
        // fp32's smallest normal number
        if (!(sum >= 0x1p-90 && sum <= 0x1p126)) {
            bool bad = false;
            const double d = by_type(l.type[t], l.x[t], at,
                                     [&](auto *p) { return sum_chunk_wide(p, n, inv, &bad); });
            if (lane == 0)
                warp_sum[warp] = d;
            if (__syncthreads_or(bad) && threadIdx.x == 0)
                atomicOr(&out.head->bad, 1u);
            if (threadIdx.x == 0) {
                sum = warp_sum[0];
                for (int w = 1; w < kThreads / 32; ++w)
                    sum += warp_sum[w];
            }
        }
        if (threadIdx.x == 0)
            out.sums[c] = sum;
    }
    if (!ends)
        return;
    if (threadIdx.x == 0) {
        uint32_t before;  // this CTA's sum goes out ahead of it, the others' are seen after
        asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], 1;" : "=r"(before) : "l"(&out.head->done) : "memory");
        last = before == gridDim.x - 1;
    }
    __syncthreads();
    if (last)
        end_norm<kThreads>(l, out, warp_sum);
}

template <int CAP>
__global__ void __launch_bounds__(kEndThreads)
    norm_end_kernel(const __grid_constant__ List<CAP, false> l, const NormOut out)
{
    __shared__ double warp_sum[kEndThreads / 32];
    asm volatile("griddepcontrol.wait;" ::: "memory");  // the sums are written and seen
    end_norm<kEndThreads>(l, out, warp_sum);
}

// ------------------------------------------------------------------ clip

// What an element is multiplied by: f, then twice g, a power of two that is 1
// wherever f alone has fp32's full precision.
struct Factor {
    float f, g;
    __device__ __forceinline__ float of(float x) const { return __fmul_rn(__fmul_rn(__fmul_rn(x, f), g), g); }
};

// inv * c, c = min(1, max_norm / (sqrt(sumsq) + 1e-6)).  In fp32 where everything
// is well inside its range: GB300's binary64 is slow.  Outside (a norm from
// 2^128 on, say) in binary64, rounded once; of a factor that fp32 would hold with
// few bits or none f keeps the bits and g half the exponent.  (Where x * f * g
// is below fp32's normal numbers, with g <= 2^-49, the end is 0.)
__device__ __forceinline__ Factor clip_factor(double sumsq, float inv, double max_norm)
{
    if (sumsq >= 0x1p-120 && sumsq <= 0x1p120) {
        const float f = __fmul_rn(inv, fminf(1.0f, __fdiv_rn((float)max_norm, __fadd_rn(__fsqrt_rn((float)sumsq), 1e-6f))));
        if (f >= 0x1p-100f)
            return {f, 1.0f};
    }
    if (!(sumsq <= 1.7976931348623157e308))  // no finite sum: as with found_inf
        return {inv, 1.0f};
    const double f = inv * fmin(1.0, max_norm / (sqrt(sumsq) + 1e-6));
    if (f >= 0x1p-100 || f == 0.0)
        return {(float)f, 1.0f};
    // f below 1/2, so that no product overflows; 2^-298 times the largest fp32 is 0
    const int half = min((-ilogb(f) - 2) / 2, 149);
    return {(float)scalbn(f, 2 * half), scalbnf(1.0f, -half)};
}

// Eight scaled elements to a 16-byte aligned p; nothing reads them here again.
template <class U, class T>
__device__ __forceinline__ void put(U *p, const Raw8<T> &x, Factor f)
{
    uint32_t w[Raw8<U>::kWords];
    if constexpr (sizeof(U) == 4)
#pragma unroll
        for (int i = 0; i < 8; ++i)
            w[i] = __float_as_uint(f.of(x.at(i)));
    else
#pragma unroll
        for (int i = 0; i < 4; ++i)
            w[i] = word_of<U>(f.of(x.at(2 * i)), f.of(x.at(2 * i + 1)));
#pragma unroll
    for (int i = 0; i < Raw8<U>::kWords / 4; ++i)
        __stcs(reinterpret_cast<uint4 *>(p) + i, make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]));
}

template <class T, class U>
__device__ __forceinline__ void scale_chunk(const T *p, U *o, int64_t n, Factor f)
{
    const bool wide = (reinterpret_cast<uintptr_t>(p) & 15) == 0;
    const bool wide_out = (reinterpret_cast<uintptr_t>(o) & 15) == 0;
    int64_t u = threadIdx.x;
    if (wide && wide_out)
        for (; (u + (kBatch - 1) * kThreads + 1) * kUnit <= n; u += kBatch * kThreads) {
            Raw8<T> x[kBatch];
#pragma unroll
            for (int k = 0; k < kBatch; ++k)
                x[k] = load_full<true>(p + (u + k * kThreads) * kUnit);
#pragma unroll
            for (int k = 0; k < kBatch; ++k)
                put(o + (u + k * kThreads) * kUnit, x[k], f);
        }
    for (; u * kUnit < n; u += kThreads) {
        const int64_t left = n - u * kUnit;
        const int m = left < kUnit ? (int)left : kUnit;
        float x[kUnit];
        load8(p + u * kUnit, m, wide, x);
#pragma unroll
        for (int i = 0; i < kUnit; ++i)
            x[i] = f.of(x[i]);
        store8(o + u * kUnit, m, wide_out, x);
    }
}

template <int CAP>
__global__ void __launch_bounds__(kThreads)
    clip_kernel(const __grid_constant__ List<CAP, true> l, float inv, double max_norm,
                const zero_tensors_stat *stat)
{
    asm volatile("griddepcontrol.wait;" ::: "memory");  // the norm is there, the tensors are final
    Factor f{inv, 1.0f};
    if (max_norm > 0.0 && stat->found_inf == 0)
        f = clip_factor(stat->sumsq, inv, max_norm);  // (the caller may have added sumsq over ranks)
    // from the list's end backwards: what the norm read last is still in L2
    const uint32_t chunk = gridDim.x - 1 - blockIdx.x;
    const int t = find_tensor(l, chunk);
    if (f.f == 1.0f && f.g == 1.0f && l.out[t] == l.x[t])
        return;  // in place and unchanged
    const int64_t at = (int64_t)(chunk - l.first[t]) * l.chunk;
    const int64_t left = l.numel[t] - at;
    const int64_t n = left < l.chunk ? left : l.chunk;
    by_type(l.type[t], l.x[t], at, [&](auto *p) {
        if (l.out_type[t] == ZERO_T_F16)
            scale_chunk(p, static_cast<f16 *>(l.out[t]) + at, n, f);
        else if (l.out_type[t] == ZERO_T_BF16)
            scale_chunk(p, static_cast<bf16 *>(l.out[t]) + at, n, f);
        else
            scale_chunk(p, static_cast<float *>(l.out[t]) + at, n, f);
    });
}

// ------------------------------------------------------------------ host

// A launch that may begin before the kernel ahead of it ends (and waits for it itself).
template <class... P, class... A>
static int launch_after(void (*kernel)(P...), uint32_t grid, int threads, cudaStream_t stream, const A &...args)
{
    cudaLaunchAttribute early{};
    early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    early.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.stream = stream;
    cfg.attrs = &early;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
    return e == cudaSuccess ? ZERO_OK : cuda_error(e);
}

// Checks a list's sizes; its total.
static int list_total(int n, const int64_t *numel, int64_t *total)
{
    if (n < 0 || (n > 0 && !numel))
        return ZERO_EINVAL;
    int64_t sum = 0;
    for (int t = 0; t < n; ++t) {
        if (numel[t] < 0 || numel[t] > (INT64_C(1) << 45) || sum > (INT64_C(1) << 45))
            return ZERO_EINVAL;
        sum += numel[t];
    }
    *total = sum;
    return ZERO_OK;
}

// Fills a launch's list from the caller's tensor t on; returns the next one.
template <int CAP, bool OUT>
static int fill(List<CAP, OUT> &l, int t, int n, const void *const *x, const int64_t *numel,
                const int32_t *type, void *const *out, const int32_t *out_type, int64_t chunk)
{
    l.chunk = chunk;
    l.n = 0;
    uint32_t c = 0;
    for (; t < n && l.n < CAP; ++t) {
        if (numel[t] == 0)
            continue;
        const int64_t more = ceil_div(numel[t], chunk);
        l.x[l.n] = x[t];
        l.numel[l.n] = numel[t];
        l.first[l.n] = c;
        l.index[l.n] = t;
        l.type[l.n] = (uint8_t)type[t];
        if (OUT) {
            l.out[l.n] = out ? out[t] : const_cast<void *>(x[t]);
            l.out_type[l.n] = (uint8_t)(out ? out_type[t] : type[t]);
        }
        c += (uint32_t)more;
        ++l.n;
    }
    while (t < n && numel[t] == 0)
        ++t;
    l.first[l.n] = c;
    return t;
}

// Runs `launch` on lists of the smallest capacity that holds the tensors.
template <bool OUT, class F>
static int for_each_list(int n, const void *const *x, const int64_t *numel, const int32_t *type,
                         void *const *out, const int32_t *out_type, int64_t total, F &&launch)
{
    const int64_t chunk = chunk_elems(total);
    int full = 0;
    for (int t = 0; t < n; ++t)
        full += numel[t] > 0;
    auto go = [&](auto &l) {
        int t = 0;
        bool first = true;
        do {
            t = fill(l, t, n, x, numel, type, out, out_type, chunk);
            const int rc = launch(l, first, t >= n);
            if (rc)
                return rc;
            first = false;
        } while (t < n);
        return (int)ZERO_OK;
    };
    // the arguments are copied at every launch, so a short list takes a short one
    if (full <= 64) {
        List<64, OUT> l;
        return go(l);
    }
    if (full <= 320) {
        List<320, OUT> l;
        return go(l);
    }
    List<kCapacity - (OUT ? 200 : 0), OUT> l;
    return go(l);
}

static int check_list(int n, const void *const *x, const int64_t *numel, const int32_t *type,
                      int64_t *total)
{
    const int rc = list_total(n, numel, total);
    if (rc)
        return rc;
    if (n > 0 && (!x || !type))
        return ZERO_EINVAL;
    for (int t = 0; t < n; ++t) {
        if (!is_float(type[t]) || (numel[t] > 0 && !x[t]))
            return ZERO_EINVAL;
        if (!aligned(x[t], (uintptr_t)type_bytes(type[t])))
            return ZERO_EALIGN;
    }
    return ZERO_OK;
}

}  // namespace zo

using namespace zo;

extern "C" {

size_t zero_tensors_workspace_bytes(int n, const int64_t *numel)
{
    int64_t total = 0;
    if (list_total(n, numel, &total))
        return 0;
    const int64_t chunk = chunk_elems(total);
    int64_t chunks = 0;
    for (int t = 0; t < n; ++t)
        chunks += ceil_div(numel[t], chunk);
    return (size_t)(kHeader + chunks * (int64_t)sizeof(double));
}

int zero_tensors_norm(int n, const void *const *x, const int64_t *numel, const int32_t *type,
                      float inv_scale, double *tensor_sumsq, zero_tensors_stat *stat, void *ws,
                      size_t ws_bytes, zero_stream_t stream)
{
    int64_t total = 0;
    const int rc = check_list(n, x, numel, type, &total);
    if (rc)
        return rc;
    if (!stat || !ws || !(inv_scale > 0.0f) || !std::isfinite(inv_scale))
        return ZERO_EINVAL;
    if (!aligned(stat, 8) || !aligned(ws, 16) || !aligned(tensor_sumsq, 8))
        return ZERO_EALIGN;
    if (ws_bytes < zero_tensors_workspace_bytes(n, numel))
        return ZERO_ESPACE;
    if (tensor_sumsq)
        for (int t = 0; t < n; ++t)
            if (numel[t] == 0) {  // the kernels see no empty tensor
                const cudaError_t e = cudaMemsetAsync(tensor_sumsq, 0, sizeof(double) * (size_t)n,
                                                      stream);
                if (e != cudaSuccess)
                    return cuda_error(e);
                break;
            }
    Header *head = static_cast<Header *>(ws);
    double *sums = reinterpret_cast<double *>(static_cast<char *>(ws) + kHeader);
    return for_each_list<false>(
        n, x, numel, type, nullptr, nullptr, total, [&](auto &l, bool first, bool last) {
            const uint32_t chunks = l.n ? l.first[l.n] : 1;  // an empty list still ends the norm
            const NormOut o{tensor_sumsq, stat, head, sums, first ? 1 : 0, last ? 1 : 0};
            const bool ends = chunks < kEndChunks;
            norm_kernel<<<chunks, kThreads, 0, stream>>>(l, inv_scale, o, ends ? 1 : 0);
            const int rc = launch_status();
            return rc || ends ? rc : launch_after(norm_end_kernel<l.kCap>, 1, kEndThreads, stream, l, o);
        });
}

int zero_tensors_clip(int n, const void *const *x, const int64_t *numel, const int32_t *type,
                      void *const *out, const int32_t *out_type, float inv_scale, double max_norm,
                      const zero_tensors_stat *stat, zero_stream_t stream)
{
    int64_t total = 0;
    int rc = check_list(n, x, numel, type, &total);
    if (rc)
        return rc;
    if (!stat || !(inv_scale > 0.0f) || !std::isfinite(inv_scale) || !(max_norm >= 0.0) ||
        (out && n > 0 && !out_type))
        return ZERO_EINVAL;
    if (!aligned(stat, 8))
        return ZERO_EALIGN;
    if (out)
        for (int t = 0; t < n; ++t) {
            if (!is_float(out_type[t]) || (numel[t] > 0 && !out[t]) ||
                (numel[t] > 0 && out[t] == x[t] && out_type[t] != type[t]))
                return ZERO_EINVAL;
            if (!aligned(out[t], (uintptr_t)type_bytes(out_type[t])))
                return ZERO_EALIGN;
        }
    if (total == 0)
        return ZERO_OK;
    return for_each_list<true>(n, x, numel, type, out, out_type, total,
                               [&](auto &l, bool, bool) {
                                   return launch_after(clip_kernel<l.kCap>, l.first[l.n], kThreads, stream, l,
                                                       inv_scale, max_norm, stat);
                               });
}

}  // extern "C"
