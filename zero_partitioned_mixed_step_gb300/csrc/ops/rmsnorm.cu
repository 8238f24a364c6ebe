// The residual's addition, the root-mean-square norm and its 8-bit form in
// one pass over the rows, and the gradients.
//
//   h = round(x + r),  rstd = 1 / sqrt(mean(h^2) + eps),  y = h * rstd * w
//   dx = rstd * (g - xhat * mean(g * xhat)) + dr,  g = dy * w, xhat = h * rstd
//   dw = sum over rows of dy * xhat
//
// Both are bound by memory.  A row is held in registers between the sum of
// its squares and its use, so each input is read once and each output written
// once; the row's statistics, the gradients' sums and dw are fp32.  The sizes of
// CTAs are powers of two and a thread takes 8 columns at a time: widths below
// one leave threads idle and fewer bytes in flight (each pass's figures).
#include "ops.cuh"

namespace zo {

// Sum over the T threads of a row (T a power of two; `slot`: T / 32 floats of
// shared memory of that row, unused for T = 32, that nobody else uses).
template <int T>
__device__ __forceinline__ float row_sum(float x, float *slot)
{
    x = sum_over<32>(x);
    if (T == 32)
        return x;
    if ((threadIdx.x & 31) == 0)
        slot[(threadIdx.x % T) >> 5] = x;
    __syncthreads();
    return sum_over<T / 32>(slot[threadIdx.x & (T / 32 - 1)]);
}

// ------------------------------------------------------------------ forward

struct NormParams {
    const void *x, *r, *w;
    void *h, *y;
    uint8_t *q;
    float *s, *rstd;
    int64_t ldx, ldr, ldh, ldy, ldq, lds;
    int64_t rows, cols;
    float eps, inv_cols;
    int32_t wide;    // every matrix and w take 16-byte accesses
    int32_t wide_q;  // q takes 8-byte ones
    int32_t w_type;
};

__device__ __forceinline__ void load_w(const void *w, int type, int64_t at, int n, bool wide,
                                       float x[8])
{
    if (type == ZERO_T_F16)
        load8(static_cast<const f16 *>(w) + at, n, wide, x);
    else if (type == ZERO_T_BF16)
        load8(static_cast<const bf16 *>(w) + at, n, wide, x);
    else
        load8(static_cast<const float *>(w) + at, n, wide, x);
}

__device__ __forceinline__ int in_row(int64_t cols, int64_t c)
{
    const int64_t left = cols - c;
    return left >= 8 ? 8 : left > 0 ? (int)left : 0;
}

// Eight neighbouring elements of a row to y and to the 8-bit form; the 16
// lanes of a 1x128 block come here together.
template <class H, int F8>
__device__ __forceinline__ void put_y(const NormParams &p, int64_t row, int64_t c, int n,
                                      const float h[8], float rstd)
{
    float w[8], y[8];
    load_w(p.w, p.w_type, c, n, p.wide, w);
#pragma unroll
    for (int i = 0; i < 8; ++i)
        y[i] = n > i ? h[i] * rstd * w[i] : 0.0f;
    if (p.y && n > 0)
        store8(static_cast<H *>(p.y) + row * p.ldy + c, n, p.wide, y);
    if (!p.q)
        return;
    uint32_t a = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        a = max(a, magnitude(y[i]));
    a = max_over<16>(a);
    const float s = block_scale<F8>(a);
    if (n > 0) {
        if ((threadIdx.x & 15) == 0)
            p.s[(c / kBlock) * p.lds + row] = s;
        store8b(p.q + row * p.ldq + c, n, p.wide_q, quotients8<F8>(y, inverse(s)));
    }
}

// h's unit: x, or x + r rounded; written where it is wanted.
template <class H>
__device__ __forceinline__ Raw8<H> sum_h(const NormParams &p, int64_t row, int64_t c, int n, Raw8<H> x,
                                         const Raw8<H> &r)
{
    if (p.r)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            x.w[i] = word_of<H>(x.at(2 * i) + r.at(2 * i), x.at(2 * i + 1) + r.at(2 * i + 1));
    if (p.h && n > 0)
        store_raw(static_cast<H *>(p.h) + row * p.ldh + c, n, p.wide, x);
    return x;
}

template <class H>
__device__ __forceinline__ void load_h(const NormParams &p, int64_t row, int64_t c, int n, float h[8])
{
    Raw8<H> r{};
    if (p.r)
        r = load_raw(static_cast<const H *>(p.r) + row * p.ldr + c, n, p.wide);
    const Raw8<H> x = sum_h(p, row, c, n, load_raw(static_cast<const H *>(p.x) + row * p.ldx + c, n, p.wide), r);
#pragma unroll
    for (int i = 0; i < 8; ++i)
        h[i] = x.at(i);
}

// T threads to a row, V units of 8 elements to a thread; CTAs of max(T, 256).
// h, which is of a half type, stays packed between its two uses.
// 8192x4096 with a residual, h, y and 8 bits out: 50.9 us, 5.9 TB/s (0.88 of the
// copy rate); with one unit to each of 512 threads 56.0.  Without y, of the copy
// rate: 32768x1024 0.69, 8192x4096 0.74, 4096x8192 0.65; between, 65536x320 0.21,
// 32768x640 0.41, 8192x2304 0.45, 8192x5120 0.47, 4096x12288 0.48; 262144x64 0.15.
template <class H, int F8, int T, int V>
__global__ void __launch_bounds__(T > 256 ? T : 256, T > 512 ? 1 : T > 256 ? 2 : 5) rmsnorm_kernel(const NormParams p)
{
    constexpr int kCta = T > 256 ? T : 256;
    constexpr int kRows = kCta / T;
    __shared__ float slots[kRows][T / 32];
    const int t = threadIdx.x % T, k = threadIdx.x / T;
    const int64_t row = (int64_t)blockIdx.x * kRows + k;
    const bool live = row < p.rows;
    Raw8<H> h[V], r[V];
    float sq = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int64_t c = (int64_t)(v * T + t) * 8;
        const int n = live ? in_row(p.cols, c) : 0;
        h[v] = load_raw(static_cast<const H *>(p.x) + (live ? row : 0) * p.ldx + c, n, p.wide);
        if (p.r)
            r[v] = load_raw(static_cast<const H *>(p.r) + (live ? row : 0) * p.ldr + c, n, p.wide);
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int64_t c = (int64_t)(v * T + t) * 8;
        h[v] = sum_h(p, live ? row : 0, c, live ? in_row(p.cols, c) : 0, h[v], r[v]);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            sq = fmaf(h[v].at(i), h[v].at(i), sq);
    }
    sq = row_sum<T>(sq, slots[k]);
    const float rstd = __fdiv_rn(1.0f, __fsqrt_rn(sq * p.inv_cols + p.eps));
    if (live && t == 0 && p.rstd)
        p.rstd[row] = rstd;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int64_t c = (int64_t)(v * T + t) * 8;
        float x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            x[i] = h[v].at(i);
        put_y<H, F8>(p, live ? row : 0, c, live ? in_row(p.cols, c) : 0, x, rstd);
    }
}

// Rows too long for the registers: the sum of the squares, then the row again
// (from h where it was written, which this CTA's own threads did).
template <class H, int F8>
__global__ void __launch_bounds__(1024) rmsnorm_long_kernel(const NormParams p)
{
    __shared__ float slot[32];
    const int64_t row = blockIdx.x;
    float sq = 0.0f;
    for (int64_t c = threadIdx.x * 8; c < p.cols; c += 1024 * 8) {
        float h[8];
        load_h<H>(p, row, c, in_row(p.cols, c), h);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            sq = fmaf(h[i], h[i], sq);
    }
    sq = row_sum<1024>(sq, slot);
    const float rstd = __fdiv_rn(1.0f, __fsqrt_rn(sq * p.inv_cols + p.eps));
    if (threadIdx.x == 0 && p.rstd)
        p.rstd[row] = rstd;
    const int64_t end = (p.cols + 1024 * 8 - 1) / (1024 * 8) * (1024 * 8);
    for (int64_t c = threadIdx.x * 8; c < end; c += 1024 * 8) {
        const int n = in_row(p.cols, c);
        float h[8];
        if (p.h) {
            load8(static_cast<const H *>(p.h) + row * p.ldh + c, n, p.wide, h);
        } else {
            load_h<H>(p, row, c, n, h);
        }
        put_y<H, F8>(p, row, c, n, h, rstd);
    }
}

template <class H, int F8>
static int launch_rmsnorm(const NormParams &p, cudaStream_t stream)
{
    auto go = [&](auto kernel, int threads, int rows_per_cta) {
        kernel<<<(unsigned)ceil_div(p.rows, rows_per_cta), threads, 0, stream>>>(p);
        return launch_status();
    };
    if (p.cols <= 256)
        return go(rmsnorm_kernel<H, F8, 32, 1>, 256, 8);
    if (p.cols <= 1024)
        return go(rmsnorm_kernel<H, F8, 128, 1>, 256, 2);
    if (p.cols <= 2048)
        return go(rmsnorm_kernel<H, F8, 256, 1>, 256, 1);
    if (p.cols <= 4096)
        return go(rmsnorm_kernel<H, F8, 256, 2>, 256, 1);
    if (p.cols <= 8192)
        return go(rmsnorm_kernel<H, F8, 512, 2>, 512, 1);
    if (p.cols <= 16384)
        return go(rmsnorm_kernel<H, F8, 1024, 2>, 1024, 1);
    return go(rmsnorm_long_kernel<H, F8>, 1024, 1);
}

// ------------------------------------------------------------------ backward

struct BackParams {
    const void *dy, *h, *w, *dr;
    const float *rstd;
    void *dx;
    // [gridDim.x][cols] sums of dw.  Where 8 divides cols, the columns with c %
    // 8 = 0 first, then those with 1 and so on, so that a warp's stores are side
    // by side; else in order.  Column c is at c / 8 * unit + c % 8 * step.
    float *part;
    int64_t unit, step;
    int64_t lddy, ldh, lddr, lddx;
    int64_t rows, cols;
    float inv_cols;
    int32_t wide;
    int32_t w_type;
};

// A CTA takes every gridDim.x-th row, a thread the same 8 columns of each, so
// dw's sums over the CTA's rows stay in registers.  The next row is on its way
// while this one is reduced, and the halves stay packed, so that 1024 threads
// fit an SM.  A row costs one barrier and two shuffled sums.  The sums of dw go
// out with a warp's 32 threads side by side, and dw's own kernel is launched
// meanwhile.  8192x4096: 44.2 us without dw, 6.1 TB/s, and 47.7 with it, 5.6
// TB/s (in column order and launched after the pass 54.0).  The next row's
// loads took 18 us off; three rows ahead in registers cost 16, in a ring of
// asynchronous copies 1; two rows to a barrier, 512 threads to an SM, 0.6.
// Of the copy rate: 32768x1024 0.83, 4096x8192 0.80; between, 65536x320 0.30,
// 32768x640 0.52, 8192x2304 0.56, 8192x5120 0.67; 262144x64 0.22.
template <class H, int T>
__global__ void __launch_bounds__(T, 1024 / T) rmsnorm_backward_kernel(const BackParams p)
{
    constexpr int kWarps = T / 32;
    __shared__ float slot[2][kWarps];
    const int64_t c = (int64_t)threadIdx.x * 8;
    const int n = in_row(p.cols, c);
    float w[8], dw[8];
    load_w(p.w, p.w_type, c, n, p.wide, w);
#pragma unroll
    for (int i = 0; i < 8; ++i)
        dw[i] = 0.0f;
    Raw8<H> dy_next, h_next, dr_next{};
    float rstd_next;
    auto fetch = [&](int64_t row) {
        const int m = row < p.rows ? n : 0;
        dy_next = load_raw(static_cast<const H *>(p.dy) + row * p.lddy + c, m, p.wide);
        h_next = load_raw(static_cast<const H *>(p.h) + row * p.ldh + c, m, p.wide);
        if (p.dr)
            dr_next = load_raw(static_cast<const H *>(p.dr) + row * p.lddr + c, m, p.wide);
        rstd_next = row < p.rows ? p.rstd[row] : 0.0f;
    };
    fetch(blockIdx.x);
    int turn = 0;
    for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x, turn ^= 1) {
        const Raw8<H> dy = dy_next, h = h_next, dr = dr_next;
        const float rstd = rstd_next;
        fetch(row + gridDim.x);
        float dot = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float xhat = h.at(i) * rstd, d = dy.at(i);
            dw[i] = fmaf(d, xhat, dw[i]);
            dot = fmaf(d * w[i], xhat, dot);
        }
        dot = sum_over<32>(dot);
        if (T > 32) {  // two slots in turn, so one barrier
            if ((threadIdx.x & 31) == 0)
                slot[turn][threadIdx.x >> 5] = dot;
            __syncthreads();
            dot = sum_over<kWarps>(slot[turn][threadIdx.x & (kWarps - 1)]);
        }
        const float m = dot * p.inv_cols;
        if (n > 0) {
            float dx[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                dx[i] = rstd * (dy.at(i) * w[i] - h.at(i) * rstd * m) + (p.dr ? dr.at(i) : 0.0f);
            store8(static_cast<H *>(p.dx) + row * p.lddx + c, n, p.wide, dx);
        }
    }
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // dw's launch may begin
    if (p.part)
        for (int i = 0; i < n; ++i)
            p.part[blockIdx.x * p.cols + threadIdx.x * p.unit + i * p.step] = dw[i];
}

// Rows too long for the registers: dw's sums live in the workspace between
// rows (each thread its own columns), and dy and h are read twice.  4096x12288
// 167 us, 0.35 of the copy rate; 2048x16384 98, 0.40.
template <class H>
__global__ void __launch_bounds__(1024) rmsnorm_backward_long_kernel(const BackParams p)
{
    __shared__ float slot[32];
    float *part = p.part ? p.part + (int64_t)blockIdx.x * p.cols : nullptr;
    if (part)
        for (int64_t c = threadIdx.x * 8; c < p.cols; c += 1024 * 8)
            for (int i = 0; i < in_row(p.cols, c); ++i)
                part[c / 8 * p.unit + i * p.step] = 0.0f;
    for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
        const float rstd = p.rstd[row];
        const H *pdy = static_cast<const H *>(p.dy) + row * p.lddy;
        const H *ph = static_cast<const H *>(p.h) + row * p.ldh;
        float dot = 0.0f;
        for (int64_t c = threadIdx.x * 8; c < p.cols; c += 1024 * 8) {
            const int n = in_row(p.cols, c);
            float dy[8], h[8], w[8];
            load8(pdy + c, n, p.wide, dy);
            load8(ph + c, n, p.wide, h);
            load_w(p.w, p.w_type, c, n, p.wide, w);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float xhat = h[i] * rstd;
                if (part && i < n) {
                    float *sum = part + c / 8 * p.unit + i * p.step;
                    *sum = fmaf(dy[i], xhat, *sum);
                }
                dot = fmaf(dy[i] * w[i], xhat, dot);
            }
        }
        __syncthreads();  // the last row's sums are read
        const float m = row_sum<1024>(dot, slot) * p.inv_cols;
        for (int64_t c = threadIdx.x * 8; c < p.cols; c += 1024 * 8) {
            const int n = in_row(p.cols, c);
            float dy[8], h[8], w[8], dx[8];
            load8(pdy + c, n, p.wide, dy);
            load8(ph + c, n, p.wide, h);
            load_w(p.w, p.w_type, c, n, p.wide, w);
            if (p.dr)
                load8(static_cast<const H *>(p.dr) + row * p.lddr + c, n, p.wide, dx);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                dx[i] = rstd * (dy[i] * w[i] - h[i] * rstd * m) + (p.dr ? dx[i] : 0.0f);
            store8(static_cast<H *>(p.dx) + row * p.lddx + c, n, p.wide, dx);
        }
    }
}

// dw from the CTAs' sums: 8 places to a CTA, whose groups of 8 threads take
// the sums in turn, then the warps in order.  Its launch does not wait for the
// pass over the rows: its CTAs come as that pass's leave, and wait here.
template <int kDwThreads, class W>
__global__ void __launch_bounds__(kDwThreads)
    dw_kernel(const float *part, int64_t parts, int64_t cols, int64_t step, W *dw, int add)
{
    constexpr int kGroups = kDwThreads / 8;
    __shared__ float sh[kGroups][8];
    const int at = threadIdx.x & 7, group = threadIdx.x >> 3;
    const int64_t place = (int64_t)blockIdx.x * 8 + at;
    float s = 0.0f;
    asm volatile("griddepcontrol.wait;" ::: "memory");  // the sums are written and seen
    if (place < cols)
#pragma unroll 8
        for (int64_t k = group; k < parts; k += kGroups)
            s += part[k * cols + place];
    s += __shfl_xor_sync(0xFFFFFFFFu, s, 8);
    s += __shfl_xor_sync(0xFFFFFFFFu, s, 16);
    if ((threadIdx.x & 31) < 8)
        sh[threadIdx.x >> 5][at] = s;
    __syncthreads();
    if (threadIdx.x < 8 && place < cols) {
        const int64_t c = step == 1 ? place : place % step * 8 + place / step;
        s = 0.0f;
#pragma unroll
        for (int w = 0; w < kDwThreads / 32; ++w)
            s += sh[w][at];
        dw[c] = from_f32<W>(add ? to_f32(dw[c]) + s : s);
    }
}

// Many sums of few columns want the threads of a CTA, few sums of many columns
// the CTAs: 1216 sums of 1024 columns 17.7 us with 1024 threads (the whole
// backward), 19.8 with 256; 304 of 4096 50.0 and 47.7; 152 of 8192 52.7 and 49.2.
template <int kDwThreads, class W>
static int launch_dw(const BackParams &p, int64_t sums, W *dw, int add, cudaStream_t stream)
{
    cudaLaunchAttribute early{};
    early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    early.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)ceil_div(p.cols, 8));
    cfg.blockDim = dim3(kDwThreads);
    cfg.stream = stream;
    cfg.attrs = &early;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, dw_kernel<kDwThreads, W>, (const float *)p.part, sums,
                                             p.cols, p.step, dw, add ? 1 : 0);
    return e == cudaSuccess ? ZERO_OK : cuda_error(e);
}

// CTAs of the backward pass (and sums of dw in the workspace): a rule on the
// sizes, not on the GPU, so that dw's bits do not depend on it.
static int64_t backward_parts(int64_t rows, int64_t cols)
{
    const int64_t most = 152 * (cols <= 256 ? 32 : cols <= 1024 ? 8 : cols <= 2048 ? 4 : cols <= 4096 ? 2 : 1);
    return rows < most ? (rows < 1 ? 1 : rows) : most;
}

template <class H>
static int launch_backward(const BackParams &p, int64_t parts, cudaStream_t stream)
{
    auto go = [&](auto kernel, int threads) {
        kernel<<<(unsigned)parts, threads, 0, stream>>>(p);
        return launch_status();
    };
    if (p.cols <= 256)
        return go(rmsnorm_backward_kernel<H, 32>, 32);
    if (p.cols <= 1024)
        return go(rmsnorm_backward_kernel<H, 128>, 128);
    if (p.cols <= 2048)
        return go(rmsnorm_backward_kernel<H, 256>, 256);
    if (p.cols <= 4096)
        return go(rmsnorm_backward_kernel<H, 512>, 512);
    if (p.cols <= 8192)
        return go(rmsnorm_backward_kernel<H, 1024>, 1024);
    return go(rmsnorm_backward_long_kernel<H>, 1024);
}

}  // namespace zo

using namespace zo;

extern "C" {

int zero_rmsnorm_fp8(const void *x, int64_t ldx, const void *residual, int64_t ldr, const void *w,
                     int w_type, int type, int64_t rows, int64_t cols, float eps, void *h,
                     int64_t ldh, void *y, int64_t ldy, int fp8, void *q, int64_t ldq, float *s,
                     int64_t lds, float *rstd, zero_stream_t stream)
{
    if (!is_half(type) || !is_float(w_type) || bad_dim(rows) || bad_dim(cols) || cols < 1 ||
        !(eps >= 0.0f) || !std::isfinite(eps) || !q != !s || (q && !is_fp8(fp8)))
        return ZERO_EINVAL;
    if (rows == 0)
        return ZERO_OK;
    if (!w || (!h && !y && !q && !rstd))
        return ZERO_EINVAL;
    const int b = type_bytes(type);
    int rc = check_matrix(x, rows, cols, ldx, b);
    if (!rc && residual)
        rc = check_matrix(residual, rows, cols, ldr, b);
    if (!rc && h)
        rc = check_matrix(h, rows, cols, ldh, b);
    if (!rc && y)
        rc = check_matrix(y, rows, cols, ldy, b);
    if (!rc && q)
        rc = check_matrix(q, rows, cols, ldq, 1);
    if (!rc && q)
        rc = check_matrix(s, ceil_div(cols, kBlock), rows, lds, 4);
    if (!rc && (!aligned(w, (uintptr_t)type_bytes(w_type)) || !aligned(rstd, 4)))
        rc = ZERO_EALIGN;
    if (rc)
        return rc;
    NormParams p{};
    p.x = x;
    p.r = residual;
    p.w = w;
    p.h = h;
    p.y = y;
    p.q = static_cast<uint8_t *>(q);
    p.s = s;
    p.rstd = rstd;
    p.ldx = ldx;
    p.ldr = ldr;
    p.ldh = ldh;
    p.ldy = ldy;
    p.ldq = ldq;
    p.lds = lds;
    p.rows = rows;
    p.cols = cols;
    p.eps = eps;
    p.inv_cols = 1.0f / (float)cols;
    p.w_type = w_type;
    p.wide = rows_aligned(x, ldx, b, 16) && (!residual || rows_aligned(residual, ldr, b, 16)) &&
             (!h || rows_aligned(h, ldh, b, 16)) && (!y || rows_aligned(y, ldy, b, 16)) &&
             aligned(w, 16);
    p.wide_q = q && rows_aligned(q, ldq, 1, 8);
    const bool e5m2 = q && fp8 == ZERO_T_E5M2;
    if (type == ZERO_T_F16)
        return e5m2 ? launch_rmsnorm<f16, ZERO_T_E5M2>(p, stream)
                    : launch_rmsnorm<f16, ZERO_T_E4M3>(p, stream);
    return e5m2 ? launch_rmsnorm<bf16, ZERO_T_E5M2>(p, stream)
                : launch_rmsnorm<bf16, ZERO_T_E4M3>(p, stream);
}

size_t zero_rmsnorm_workspace_bytes(int64_t rows, int64_t cols)
{
    if (bad_dim(rows) || bad_dim(cols) || cols < 1)
        return 0;
    return (size_t)backward_parts(rows, cols) * (size_t)cols * sizeof(float);
}

int zero_rmsnorm_backward(const void *dy, int64_t lddy, const void *h, int64_t ldh, const void *w,
                          int w_type, const float *rstd, const void *dresidual, int64_t lddr,
                          int type, int64_t rows, int64_t cols, void *dx, int64_t lddx, void *dw,
                          int dw_type, int add_dw, void *ws, size_t ws_bytes, zero_stream_t stream)
{
    if (!is_half(type) || !is_float(w_type) || bad_dim(rows) || bad_dim(cols) || cols < 1 || !w ||
        (rows > 0 && !rstd) || (dw && (!is_float(dw_type) || !ws)))
        return ZERO_EINVAL;
    const int b = type_bytes(type);
    int rc = check_matrix(dy, rows, cols, lddy, b);
    if (!rc)
        rc = check_matrix(h, rows, cols, ldh, b);
    if (!rc)
        rc = check_matrix(dx, rows, cols, lddx, b);
    if (!rc && dresidual)
        rc = check_matrix(dresidual, rows, cols, lddr, b);
    if (!rc && (!aligned(w, (uintptr_t)type_bytes(w_type)) || !aligned(rstd, 4) ||
                (dw && (!aligned(ws, 16) || !aligned(dw, (uintptr_t)type_bytes(dw_type))))))
        rc = ZERO_EALIGN;
    if (!rc && dw && ws_bytes < zero_rmsnorm_workspace_bytes(rows, cols))
        rc = ZERO_ESPACE;
    if (rc)
        return rc;
    const int64_t parts = backward_parts(rows, cols);
    BackParams p{};
    p.dy = dy;
    p.h = h;
    p.w = w;
    p.dr = dresidual;
    p.rstd = rstd;
    p.dx = dx;
    p.part = dw ? static_cast<float *>(ws) : nullptr;
    p.lddy = lddy;
    p.ldh = ldh;
    p.lddr = lddr;
    p.lddx = lddx;
    p.rows = rows;
    p.cols = cols;
    p.unit = cols % 8 == 0 ? 1 : 8;
    p.step = cols % 8 == 0 ? cols / 8 : 1;
    p.inv_cols = 1.0f / (float)cols;
    p.w_type = w_type;
    p.wide = rows_aligned(dy, lddy, b, 16) && rows_aligned(h, ldh, b, 16) &&
             rows_aligned(dx, lddx, b, 16) && (!dresidual || rows_aligned(dresidual, lddr, b, 16)) &&
             aligned(w, 16);
    if (rows > 0) {
        rc = type == ZERO_T_F16 ? launch_backward<f16>(p, parts, stream)
                                : launch_backward<bf16>(p, parts, stream);
        if (rc)
            return rc;
    }
    if (!dw)
        return ZERO_OK;
    const int64_t sums = rows > 0 ? parts : 0;
    auto finish = [&](auto *out) {
        return sums > 512 ? launch_dw<1024>(p, sums, out, add_dw, stream)
                          : launch_dw<256>(p, sums, out, add_dw, stream);
    };
    if (dw_type == ZERO_T_F16)
        return finish(static_cast<f16 *>(dw));
    if (dw_type == ZERO_T_BF16)
        return finish(static_cast<bf16 *>(dw));
    return finish(static_cast<float *>(dw));
}

}  // extern "C"
