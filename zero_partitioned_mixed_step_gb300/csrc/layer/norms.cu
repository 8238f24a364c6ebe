// The norms behind and ahead of a block, its gate and the residual stream in one
// pass over the rows, and the gradients.
//
//   xo = o * ro, ro = 1 / sqrt(mean(o^2) + eps)   (xo = o without a norm behind the block)
//   h = scale * x + gate * w_post * xo
//   y = h * rh * w_pre, rh = 1 / sqrt(mean(h^2) + eps)
//
// Backward, xh = h * rh, g = dy * w_pre, A = gate * w_post:
//   m = mean(g * xh),  dH = rh * (g - xh * m) + dh,  dx = scale * dH
//   d_o = ro * (A * dH - xo * mean(A * xo * dH))
// The second mean needs the first, but as dH is linear in m, three sums that need
// nothing of one another give both, so that a row costs one barrier:
//   D = sum g xh,  P = sum A xo (rh g + dh),  Q = sum A xo xh,  sum A xo dH = P - rh (D / cols) Q
// (|P| and |rh m Q| are sums that dH's own terms bound: nothing is lost that dH keeps).
//
// Both passes are bound by memory: each input is read once and each output
// written once.
#include <initializer_list>
#include <type_traits>

#include "layer.cuh"

namespace zo {

struct Gate {
    const void *p;
    int32_t kind, type;
};

// ------------------------------------------------------------------ forward

struct JoinParams {
    const void *o, *x, *w_post, *w_pre;
    Gate gate;
    void *h, *y;
    Form y8, o8, h8;
    float *rstd_post, *rstd_pre;
    int64_t ldo, ldx, ldh, ldy;
    int64_t rows, cols;
    float scale, eps, inv_cols;
    int32_t w_type, e5m2;
    int32_t wide;    // every matrix takes 16-byte accesses
    int32_t wide_w;  // the vectors do
};

__device__ __forceinline__ float root(float sumsq, float inv_cols, float eps)
{
    return __fdiv_rn(1.0f, __fsqrt_rn(sumsq * inv_cols + eps));
}

// The gate's number where a row has one.
__device__ __forceinline__ float row_gate(const Gate &g, int64_t row)
{
    return g.kind == ZERO_GATE_ONE ? load_one(g.p, g.type, 0) : g.kind == ZERO_GATE_ROWS ? load_one(g.p, g.type, row) : 1.0f;
}

// gate * w_post for 8 columns (`gate`: the row's number).
template <class P>
__device__ __forceinline__ void post_factors(const P &p, int64_t c, int n, float gate, float f[8])
{
#pragma unroll
    for (int i = 0; i < 8; ++i)
        f[i] = gate;
    float w[8];
    if (p.w_post) {
        load_w(p.w_post, p.w_type, c, n, p.wide_w, w);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            f[i] *= w[i];
    }
    if (p.gate.kind == ZERO_GATE_COLS) {
        load_w(p.gate.p, p.gate.type, c, n, p.wide_w, w);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            f[i] *= w[i];
    }
}

// h of 8 columns.
template <class H>
__device__ __forceinline__ void join8(const JoinParams &p, int64_t c, int n, const Raw8<H> &o, const Raw8<H> &x,
                                      float ro, float gate, float h[8])
{
    post_factors(p, c, n, gate, h);
#pragma unroll
    for (int i = 0; i < 8; ++i)
        h[i] = fmaf(p.scale, x.at(i), h[i] * (o.at(i) * ro));
}

// What a row's unit leaves once rh is known.
template <class H>
__device__ __forceinline__ void put_unit(const JoinParams &p, int64_t row, int64_t c, int n, const float h[8], float rh)
{
    if (n > 0)
        store8(static_cast<H *>(p.h) + row * p.ldh + c, n, p.wide, h);
    if (p.h8.q)
        put_form(p.h8, row, c, n, h, amax8(h), false);
    if (!p.y && !p.y8.q)
        return;
    float y[8];
    load_w(p.w_pre, p.w_type, c, n, p.wide_w, y);
#pragma unroll
    for (int i = 0; i < 8; ++i)
        y[i] = h[i] * rh * y[i];
    if (p.y && n > 0)
        store8(static_cast<H *>(p.y) + row * p.ldy + c, n, p.wide, y);
    if (p.y8.q)
        put_form(p.y8, row, c, n, y, amax8(y), p.e5m2);
}

template <class H>
__device__ __forceinline__ uint32_t packed_amax(const Raw8<H> &x)
{
    Amax<H> a;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        a.add(x.w[i]);
    return a.bits();
}

template <class H>
__device__ __forceinline__ void put_o8(const JoinParams &p, int64_t row, int64_t c, int n, const Raw8<H> &o)
{
    float x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
        x[i] = o.at(i);
    put_form(p.o8, row, c, n, x, packed_amax(o), false);
}

// A row to G lanes (16 or 32), or to the CTA (G = 0), V units of 8 to a thread.
template <class H, int V, int G, int MAXT>
__global__ void __launch_bounds__(MAXT) join_kernel(const JoinParams p)
{
    constexpr int kWarps = MAXT / 32;
    __shared__ float slots[2][kWarps];
    const int t = G ? threadIdx.x % (G ? G : 1) : threadIdx.x;
    const int T = G ? G : blockDim.x;
    const int64_t at = G ? (int64_t)blockIdx.x * (MAXT / (G ? G : 1)) + threadIdx.x / (G ? G : 1) : blockIdx.x;
    const bool live = at < p.rows;
    const int64_t row = live ? at : 0;
    const int64_t cols = live ? p.cols : 0;
    Raw8<H> o[V], x[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int64_t c = (int64_t)(v * T + t) * 8;
        const int n = in_row(cols, c);
        o[v] = load_raw(static_cast<const H *>(p.o) + row * p.ldo + c, n, p.wide);
        x[v] = load_raw(static_cast<const H *>(p.x) + row * p.ldx + c, n, p.wide);
    }
    float ro = 1.0f;
    if (p.w_post) {
        float sq[1] = {0.0f};
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
            for (int i = 0; i < 8; ++i)
                sq[0] = fmaf(o[v].at(i), o[v].at(i), sq[0]);
        row_sums<G, kWarps>(sq, slots[0]);
        ro = root(sq[0], p.inv_cols, p.eps);
        if (live && t == 0 && p.rstd_post)
            p.rstd_post[row] = ro;
    }
    const float gate = row_gate(p.gate, row);
    float h[V][8], sq[1] = {0.0f};
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int64_t c = (int64_t)(v * T + t) * 8;
        const int n = in_row(cols, c);
        join8(p, c, n, o[v], x[v], ro, gate, h[v]);
        if (p.o8.q)
            put_o8(p, row, c, n, o[v]);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            sq[0] = fmaf(h[v][i], h[v][i], sq[0]);
    }
    row_sums<G, kWarps>(sq, slots[1]);
    const float rh = root(sq[0], p.inv_cols, p.eps);
    if (live && t == 0 && p.rstd_pre)
        p.rstd_pre[row] = rh;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int64_t c = (int64_t)(v * T + t) * 8;
        put_unit<H>(p, row, c, in_row(cols, c), h[v], rh);
    }
}

// Rows too long for the registers: o for its norm, o and x for h's, and both again
// for what is written (h may be x or o, so nothing is written before that).
template <class H>
__global__ void __launch_bounds__(1024) join_long_kernel(const JoinParams p)
{
    __shared__ float slots[2][32];
    const int64_t row = blockIdx.x;
    const H *po = static_cast<const H *>(p.o) + row * p.ldo;
    const H *px = static_cast<const H *>(p.x) + row * p.ldx;
    float ro = 1.0f;
    if (p.w_post) {
        float sq[1] = {0.0f};
        for (int64_t c = threadIdx.x * 8; c < p.cols; c += 1024 * 8) {
            const Raw8<H> o = load_raw(po + c, in_row(p.cols, c), p.wide);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                sq[0] = fmaf(o.at(i), o.at(i), sq[0]);
        }
        row_sums<0, 32>(sq, slots[0]);
        ro = root(sq[0], p.inv_cols, p.eps);
        if (threadIdx.x == 0 && p.rstd_post)
            p.rstd_post[row] = ro;
    }
    const float gate = row_gate(p.gate, row);
    float h[8], sq[1] = {0.0f};
    for (int64_t c = threadIdx.x * 8; c < p.cols; c += 1024 * 8) {
        const int n = in_row(p.cols, c);
        join8(p, c, n, load_raw(po + c, n, p.wide), load_raw(px + c, n, p.wide), ro, gate, h);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            sq[0] = fmaf(h[i], h[i], sq[0]);
    }
    row_sums<0, 32>(sq, slots[1]);
    const float rh = root(sq[0], p.inv_cols, p.eps);
    if (threadIdx.x == 0 && p.rstd_pre)
        p.rstd_pre[row] = rh;
    const int64_t end = (p.cols + 1024 * 8 - 1) / (1024 * 8) * (1024 * 8);
    for (int64_t c = threadIdx.x * 8; c < end; c += 1024 * 8) {
        const int n = in_row(p.cols, c);
        const Raw8<H> o = load_raw(po + c, n, p.wide);
        join8(p, c, n, o, load_raw(px + c, n, p.wide), ro, gate, h);
        if (p.o8.q)
            put_o8(p, row, c, n, o);
        put_unit<H>(p, row, c, n, h, rh);
    }
}

template <class H>
static int launch_join(const JoinParams &p, cudaStream_t stream)
{
    auto go = [&](auto kernel, int threads, int rows_per_cta) {
        kernel<<<(unsigned)ceil_div(p.rows, rows_per_cta), threads, 0, stream>>>(p);
        return launch_status();
    };
    auto threads = [&](int units) { return (int)(ceil_div(ceil_div(p.cols, 8 * units), 32) * 32); };
    if (p.cols <= 128)
        return go(join_kernel<H, 1, 16, 256>, 256, 16);
    if (p.cols <= 256)
        return go(join_kernel<H, 1, 32, 256>, 256, 8);
    if (p.cols <= 2048)
        return go(join_kernel<H, 1, 0, 256>, threads(1), 1);
    if (p.cols <= 8192)
        return go(join_kernel<H, 2, 0, 512>, threads(2), 1);
    if (p.cols <= 16384)
        return go(join_kernel<H, 2, 0, 1024>, threads(2), 1);
    return go(join_long_kernel<H>, 1024, 1);
}

// ------------------------------------------------------------------ backward

struct SplitParams {
    const void *dy, *dh, *o, *h, *w_post, *w_pre;
    const float *so, *sh, *ro, *rh;
    Gate gate;
    void *d_o, *dx;
    void *dgate_rows;  // a token's gate has its gradient from the row itself
    int32_t dgate_type;
    // Sums of the CTAs: [gridDim.x][cols] of dy * xh, the same of (a token's gate
    // times) dH * xo, and [gridDim.x] of w_post * dH * xo over all columns.
    float *part;
    int32_t want_pre, want_post, want_one;
    int64_t lddy, lddh, ldo, ldh, ldso, ldsh, lddo, lddx;
    int64_t rows, cols;
    float scale, inv_cols;
    int32_t w_type;
    int32_t wide;    // the matrices of `type`, and kept halves, take 16-byte accesses, kept 8-bit ones 8-byte ones
    int32_t wide_w;
};

// A thread's own copies into its own places of shared memory (nobody else reads
// them, so waiting for them is all the order that is needed); bytes behind the row's
// end become zeros.
template <int BYTES>
__device__ __forceinline__ void copy_async(uint32_t to, const void *from, int bytes)
{
    if constexpr (BYTES == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(bytes) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(to), "l"(from), "r"(bytes) : "memory");
}

__device__ __forceinline__ void put_one(void *p, int type, int64_t at, float x)
{
    if (type == ZERO_T_F16)
        static_cast<f16 *>(p)[at] = from_f32<f16>(x);
    else if (type == ZERO_T_BF16)
        static_cast<bf16 *>(p)[at] = from_f32<bf16>(x);
    else
        static_cast<float *>(p)[at] = x;
}

// Eight sums to a CTA's partial row; 32 bytes at once where it can be.
__device__ __forceinline__ void put_part(float *to, int n, bool whole, const float x[8])
{
    if (whole && n == 8) {
        asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to), "f"(x[0]), "f"(x[1]),
                     "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7])
                     : "memory");
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n)
                to[i] = x[i];
    }
}

constexpr int kSmallThreads = 256;  // of CTAs whose rows have 16 or 32 lanes

// A CTA takes a run of neighbouring rows (of a token's scales, whose neighbours share
// sectors, all are then read by one SM), a thread the same V * 8 columns of each, so
// that the sums over rows stay in registers.  RING: STAGES - 1 rows ahead are on
// their way through shared memory, which the registers, full of factors and
// sums, have no room for.
template <class H, bool S8, int V, int G, int MAXT, int STAGES, bool RING>
__global__ void __launch_bounds__(MAXT, 512 / MAXT) split_kernel(const SplitParams p)
{
    using K = Kept<H, S8>;
    constexpr int kWarps = MAXT / 32;
    constexpr int kUnit = 32 + 2 * K::kBytes;  // bytes of a row's unit: dy, dh, o, h
    __shared__ float slots[2][3 * kWarps];
    extern __shared__ __align__(16) unsigned char ring[];
    const int T = G ? G : blockDim.x;
    const int t = G ? threadIdx.x % (G ? G : 1) : threadIdx.x;
    const int groups = G ? MAXT / (G ? G : 1) : 1, group = G ? threadIdx.x / (G ? G : 1) : 0;
    const int64_t all = (int64_t)gridDim.x * groups, me = (int64_t)blockIdx.x * groups + group;
    // rows [first, end): rows / all each, one more for the first rows % all
    const int64_t each = p.rows / all, more = p.rows % all;
    const int64_t first = me * each + min(me, more), end = first + each + (me < more ? 1 : 0);

    int n[V];
    float w[V][8], a[V][8], dw[V][8], da[V][8], one = 0.0f;
    const float fixed = p.gate.kind == ZERO_GATE_ONE ? load_one(p.gate.p, p.gate.type, 0) : 1.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int64_t c = (int64_t)(v * T + t) * 8;
        n[v] = in_row(p.cols, c);
        load_w(p.w_pre, p.w_type, c, n[v], p.wide_w, w[v]);
        post_factors(p, c, n[v], 1.0f, a[v]);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            dw[v][i] = da[v][i] = 0.0f;
    }
    const uint32_t place = RING ? (uint32_t)__cvta_generic_to_shared(ring) : 0u;
    // the unit's four parts lie apart, so that a warp's accesses are side by side
    const uint32_t lanes = blockDim.x;
    auto at = [&](int stage, int v, int part) {
        const uint32_t unit = (uint32_t)(stage * V + v) * lanes * kUnit;
        return unit + (part < 2 ? (uint32_t)(part * lanes + threadIdx.x) * 16
                                : lanes * 32 + (uint32_t)((part - 2) * lanes + threadIdx.x) * K::kBytes);
    };
    auto fetch = [&](int64_t row, int stage) {
        if (row < end) {
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const int64_t c = n[v] > 0 ? (int64_t)(v * T + t) * 8 : 0;  // an address of the row even where nothing is read
                copy_async<16>(place + at(stage, v, 0), static_cast<const H *>(p.dy) + row * p.lddy + c, 2 * n[v]);
                if (p.dh)
                    copy_async<16>(place + at(stage, v, 1), static_cast<const H *>(p.dh) + row * p.lddh + c, 2 * n[v]);
                const unsigned char *o = static_cast<const unsigned char *>(p.o), *h = static_cast<const unsigned char *>(p.h);
                constexpr int b = K::kBytes / 8;
                copy_async<K::kBytes>(place + at(stage, v, 2), o + (row * p.ldo + c) * b, b * n[v]);
                copy_async<K::kBytes>(place + at(stage, v, 3), h + (row * p.ldh + c) * b, b * n[v]);
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    float so_next[V], sh_next[V], ro_next = 1.0f, rh_next = 0.0f, gate_next = fixed;
    auto fetch_scales = [&](int64_t row) {
        if (row >= end)
            return;
        rh_next = p.rh[row];
        if (p.w_post)
            ro_next = p.ro[row];
        if (p.gate.kind == ZERO_GATE_ROWS)
            gate_next = load_one(p.gate.p, p.gate.type, row);
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (S8 && n[v] > 0) {
                const int64_t b = (int64_t)(v * T + t) * 8 / kBlock;
                so_next[v] = p.so[b * p.ldso + row];
                sh_next[v] = p.sh[b * p.ldsh + row];
            }
    };
#pragma unroll
    for (int v = 0; v < V; ++v)
        so_next[v] = sh_next[v] = n[v] > 0 ? 1.0f : 0.0f;
    if (RING)
#pragma unroll
        for (int s = 0; s < STAGES - 1; ++s)
            fetch(first + s, s);
    fetch_scales(first);

    // two groups of 16 lanes share a warp and its shuffles, so both take as many turns
    const int64_t last = G == 16 ? first + each + (more > 0 ? 1 : 0) : end;
    int turn = 0, stage = 0;
    for (int64_t row = first; row < last; ++row, turn ^= 1) {
        const bool live = G != 16 || row < end;
        Raw8<H> dy[V], dh[V];
        K o[V], h[V];
        if (RING) {
            asm volatile("cp.async.wait_group %0;" ::"n"(STAGES - 2) : "memory");
#pragma unroll
            for (int v = 0; v < V; ++v) {
                dy[v] = *reinterpret_cast<const Raw8<H> *>(__builtin_assume_aligned(ring + at(stage, v, 0), 16));
                if (p.dh)
                    dh[v] = *reinterpret_cast<const Raw8<H> *>(__builtin_assume_aligned(ring + at(stage, v, 1), 16));
                o[v] = *reinterpret_cast<const K *>(__builtin_assume_aligned(ring + at(stage, v, 2), K::kBytes));
                h[v] = *reinterpret_cast<const K *>(__builtin_assume_aligned(ring + at(stage, v, 3), K::kBytes));
            }
            // the places of the row before, whose values this thread has used
            fetch(row + STAGES - 1, stage == 0 ? STAGES - 1 : stage - 1);
            stage = stage == STAGES - 1 ? 0 : stage + 1;
        } else {
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const int64_t c = (int64_t)(v * T + t) * 8;
                const int m = live ? n[v] : 0;
                dy[v] = load_raw(static_cast<const H *>(p.dy) + row * p.lddy + c, m, p.wide);
                if (p.dh)
                    dh[v] = load_raw(static_cast<const H *>(p.dh) + row * p.lddh + c, m, p.wide);
                o[v].load(p.o, row * p.ldo + c, m, p.wide);
                h[v].load(p.h, row * p.ldh + c, m, p.wide);
            }
        }
        if (!live) {  // a turn that adds nothing
            dy[0] = Raw8<H>{};
            dh[0] = Raw8<H>{};
            o[0] = K{};
            h[0] = K{};
            so_next[0] = sh_next[0] = rh_next = 0.0f;
            ro_next = 1.0f;
            gate_next = 0.0f;
        }
        const float ro = ro_next, rh = rh_next, gate = gate_next;
        float so[V], sh[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            so[v] = so_next[v] * ro;
            sh[v] = sh_next[v] * rh;
        }
        fetch_scales(row + 1);

        float sum[3] = {0.0f, 0.0f, 0.0f};  // D, P, Q
#pragma unroll
        for (int v = 0; v < V; ++v) {
            float xo[8], xh[8];
            o[v].get(xo, so[v]);
            h[v].get(xh, sh[v]);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float d = dy[v].at(i), g = d * w[v][i], axo = a[v][i] * xo[i];
                dw[v][i] = fmaf(d, xh[i], dw[v][i]);
                sum[0] = fmaf(g, xh[i], sum[0]);
                sum[1] = fmaf(axo, p.dh ? fmaf(rh, g, dh[v].at(i)) : rh * g, sum[1]);
                sum[2] = fmaf(axo, xh[i], sum[2]);
            }
        }
        row_sums<G, kWarps>(sum, slots[turn]);
        const float m = sum[0] * p.inv_cols;
        const float along = fmaf(-rh * m, sum[2], sum[1]);  // sum of w_post (and a channel's gate) * xo * dH
        const float mo = p.w_post ? gate * along * p.inv_cols : 0.0f;
        const float part = p.gate.kind == ZERO_GATE_ROWS ? gate : 1.0f;
        one += along;
        if (t == 0 && live && p.dgate_rows)
            put_one(p.dgate_rows, p.dgate_type, row, along);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            float xo[8], xh[8], dx[8], d_o[8];
            o[v].get(xo, so[v]);
            h[v].get(xh, sh[v]);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float g = dy[v].at(i) * w[v][i];
                float d = rh * fmaf(-xh[i], m, g);
                if (p.dh)
                    d += dh[v].at(i);
                dx[i] = p.scale * d;
                d_o[i] = ro * fmaf(-xo[i], mo, gate * a[v][i] * d);
                da[v][i] = fmaf(part * d, xo[i], da[v][i]);
            }
            const int64_t c = (int64_t)(v * T + t) * 8;
            if (n[v] > 0 && live) {
                store8(static_cast<H *>(p.dx) + row * p.lddx + c, n[v], p.wide, dx);
                store8(static_cast<H *>(p.d_o) + row * p.lddo + c, n[v], p.wide, d_o);
            }
        }
    }
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the columns' launch may begin
    if (!p.part)
        return;
    const int64_t parts = gridDim.x;
    const bool whole = p.cols % 8 == 0;
    if constexpr (G == 0) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int64_t c = (int64_t)(v * T + t) * 8;
            if (p.want_pre)
                put_part(p.part + blockIdx.x * p.cols + c, n[v], whole, dw[v]);
            if (p.want_post)
                put_part(p.part + (parts + blockIdx.x) * p.cols + c, n[v], whole, da[v]);
        }
        if (p.want_one && t == 0)
            p.part[2 * parts * p.cols + blockIdx.x] = one;
    } else {  // the row groups of the CTA, in order
        __shared__ float sums[2][MAXT * 8];
        __shared__ float ones[MAXT / G];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            sums[0][threadIdx.x * 8 + i] = dw[0][i];
            sums[1][threadIdx.x * 8 + i] = da[0][i];
        }
        if (t == 0)
            ones[group] = one;
        __syncthreads();
        for (int c = threadIdx.x; c < p.cols; c += MAXT) {
            float x = 0.0f, y = 0.0f;
            for (int g = 0; g < groups; ++g) {
                x += sums[0][g * G * 8 + c];
                y += sums[1][g * G * 8 + c];
            }
            if (p.want_pre)
                p.part[blockIdx.x * p.cols + c] = x;
            if (p.want_post)
                p.part[(parts + blockIdx.x) * p.cols + c] = y;
        }
        if (p.want_one && threadIdx.x == 0) {
            float x = 0.0f;
            for (int g = 0; g < groups; ++g)
                x += ones[g];
            p.part[2 * parts * p.cols + blockIdx.x] = x;
        }
    }
}

// Rows too long for the registers: the sums over rows live in the workspace between
// rows (each thread its own columns), and the row is read twice.
template <class H, bool S8>
__global__ void __launch_bounds__(1024) split_long_kernel(const SplitParams p)
{
    using K = Kept<H, S8>;
    __shared__ float slots[2][3 * 32];
    const int64_t parts = gridDim.x;
    float *pre = p.part && p.want_pre ? p.part + blockIdx.x * p.cols : nullptr;
    float *post = p.part && p.want_post ? p.part + (parts + blockIdx.x) * p.cols : nullptr;
    const float zero[8] = {}, fixed = p.gate.kind == ZERO_GATE_ONE ? load_one(p.gate.p, p.gate.type, 0) : 1.0f;
    for (int64_t c = threadIdx.x * 8; c < p.cols; c += 1024 * 8) {
        if (pre)
            put_part(pre + c, in_row(p.cols, c), false, zero);
        if (post)
            put_part(post + c, in_row(p.cols, c), false, zero);
    }
    float one = 0.0f;
    int turn = 0;
    for (int64_t row = blockIdx.x; row < p.rows; row += parts, turn ^= 1) {
        const float rh = p.rh[row], ro = p.w_post ? p.ro[row] : 1.0f;
        const float gate = p.gate.kind == ZERO_GATE_ROWS ? load_one(p.gate.p, p.gate.type, row) : fixed;
        const float share = p.gate.kind == ZERO_GATE_ROWS ? gate : 1.0f;
        float w[8], a[8], xo[8], xh[8];
        Raw8<H> dy, dh;
        auto read = [&](int64_t c, int n) {
            load_w(p.w_pre, p.w_type, c, n, p.wide_w, w);
            post_factors(p, c, n, 1.0f, a);
            dy = load_raw(static_cast<const H *>(p.dy) + row * p.lddy + c, n, p.wide);
            if (p.dh)
                dh = load_raw(static_cast<const H *>(p.dh) + row * p.lddh + c, n, p.wide);
            K o, h;
            o.load(p.o, row * p.ldo + c, n, p.wide);
            h.load(p.h, row * p.ldh + c, n, p.wide);
            o.get(xo, S8 ? p.so[c / kBlock * p.ldso + row] * ro : ro);
            h.get(xh, S8 ? p.sh[c / kBlock * p.ldsh + row] * rh : rh);
        };
        float sum[3] = {0.0f, 0.0f, 0.0f};
        for (int64_t c = threadIdx.x * 8; c < p.cols; c += 1024 * 8) {
            const int n = in_row(p.cols, c);
            read(c, n);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float d = dy.at(i), g = d * w[i], axo = a[i] * xo[i];
                if (pre && i < n)
                    pre[c + i] = fmaf(d, xh[i], pre[c + i]);
                sum[0] = fmaf(g, xh[i], sum[0]);
                sum[1] = fmaf(axo, p.dh ? fmaf(rh, g, dh.at(i)) : rh * g, sum[1]);
                sum[2] = fmaf(axo, xh[i], sum[2]);
            }
        }
        row_sums<0, 32>(sum, slots[turn]);
        const float m = sum[0] * p.inv_cols;
        const float along = fmaf(-rh * m, sum[2], sum[1]);
        const float mo = p.w_post ? gate * along * p.inv_cols : 0.0f;
        one += along;
        if (threadIdx.x == 0 && p.dgate_rows)
            put_one(p.dgate_rows, p.dgate_type, row, along);
        for (int64_t c = threadIdx.x * 8; c < p.cols; c += 1024 * 8) {
            const int n = in_row(p.cols, c);
            read(c, n);
            float dx[8], d_o[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                float d = rh * fmaf(-xh[i], m, dy.at(i) * w[i]);
                if (p.dh)
                    d += dh.at(i);
                dx[i] = p.scale * d;
                d_o[i] = ro * fmaf(-xo[i], mo, gate * a[i] * d);
                if (post && i < n)
                    post[c + i] = fmaf(share * d, xo[i], post[c + i]);
            }
            store8(static_cast<H *>(p.dx) + row * p.lddx + c, n, p.wide, dx);
            store8(static_cast<H *>(p.d_o) + row * p.lddo + c, n, p.wide, d_o);
        }
    }
    if (p.part && p.want_one && threadIdx.x == 0)
        p.part[2 * parts * p.cols + blockIdx.x] = one;
}

// The CTAs' sums, in order: 8 columns to a CTA, whose groups of 8 threads take the
// sums in turn, then the warps in order; one CTA more for a gate of one number.
// Its launch does not wait for the pass over the rows: its CTAs come as that
// pass's leave, and wait here.
struct ColumnParams {
    const float *part;
    int64_t parts, cols;
    const void *w_post;
    Gate gate;
    void *dw_pre, *dw_post, *dgate;
    int32_t w_type, out_type, add;
};

__device__ __forceinline__ void add_one(const ColumnParams &p, void *to, int64_t at, float x)
{
    if (to)
        put_one(to, p.out_type, at, p.add ? load_one(to, p.out_type, at) + x : x);
}

template <int THREADS>
__global__ void __launch_bounds__(THREADS) columns_kernel(const ColumnParams p)
{
    __shared__ float sh[2][THREADS / 32][8];
    const int at = threadIdx.x & 7, group = threadIdx.x >> 3;
    const bool last = blockIdx.x == (unsigned)((p.cols + 7) / 8);
    const int64_t c = (int64_t)blockIdx.x * 8 + at;
    float s[2] = {0.0f, 0.0f};
    asm volatile("griddepcontrol.wait;" ::: "memory");  // the sums are written and seen
    if (last) {
        for (int64_t k = threadIdx.x; k < p.parts; k += THREADS)
            s[0] += p.part[2 * p.parts * p.cols + k];
        s[0] += __shfl_xor_sync(0xFFFFFFFFu, s[0], 1);
        s[0] += __shfl_xor_sync(0xFFFFFFFFu, s[0], 2);
        s[0] += __shfl_xor_sync(0xFFFFFFFFu, s[0], 4);
    } else if (c < p.cols) {
        const bool post = p.dw_post || (p.dgate && p.gate.kind == ZERO_GATE_COLS);
#pragma unroll 4
        for (int64_t k = group; k < p.parts; k += THREADS / 8) {
            if (p.dw_pre)
                s[0] += p.part[k * p.cols + c];
            if (post)
                s[1] += p.part[(p.parts + k) * p.cols + c];
        }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        s[i] += __shfl_xor_sync(0xFFFFFFFFu, s[i], 8);
        s[i] += __shfl_xor_sync(0xFFFFFFFFu, s[i], 16);
        if ((threadIdx.x & 31) < 8)
            sh[i][threadIdx.x >> 5][at] = s[i];
    }
    __syncthreads();
    if (threadIdx.x >= 8)
        return;
    s[0] = s[1] = 0.0f;
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) {
        s[0] += sh[0][w][at];
        s[1] += sh[1][w][at];
    }
    if (last) {
        if (threadIdx.x == 0)
            add_one(p, p.dgate, 0, s[0]);
    } else if (c < p.cols) {
        add_one(p, p.dw_pre, c, s[0]);
        const bool cols = p.gate.kind == ZERO_GATE_COLS;
        if (p.dw_post)
            add_one(p, p.dw_post, c, s[1] * (cols ? load_one(p.gate.p, p.gate.type, c) : p.gate.kind == ZERO_GATE_ONE ? load_one(p.gate.p, p.gate.type, 0) : 1.0f));
        if (cols)
            add_one(p, p.dgate, c, p.w_post ? s[1] * load_one(p.w_post, p.w_type, c) : s[1]);
    }
}

// How a backward pass is cut, a rule on the sizes alone, so that the sums' bits do not
// depend on the GPU: threads, rows side by side in a CTA, CTAs.
struct Cut {
    int threads, groups;
    int64_t ctas;
};
static Cut cut_of(int64_t rows, int64_t cols)
{
    Cut c{};
    int64_t most;
    if (cols <= 256) {
        c.threads = kSmallThreads;
        c.groups = kSmallThreads / (cols <= 128 ? 16 : 32);
        most = 152 * 2;
    } else if (cols <= 8192) {
        c.threads = (int)(ceil_div(ceil_div(cols, cols <= 2048 ? 8 : 16), 32) * 32);
        c.groups = 1;
        most = 152 * (512 / c.threads);
    } else {
        c.threads = 1024;
        c.groups = 1;
        most = 152;
    }
    c.ctas = ceil_div(rows, c.groups);
    c.ctas = c.ctas < 1 ? 1 : c.ctas > most ? most : c.ctas;
    return c;
}

template <class H, bool S8>
static int launch_split(const SplitParams &p, const Cut &cut, cudaStream_t stream)
{
    constexpr int kStages = S8 ? 4 : 3;  // two CTAs of 4096 columns fit an SM
    auto go = [&](auto kernel, int units, bool ring) {
        size_t bytes = ring ? (size_t)kStages * units * cut.threads * (S8 ? 48 : 64) : 0;
        if (bytes > 32 * 1024) {
            const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
            if (e != cudaSuccess)
                return cuda_error(e);
        }
        kernel<<<(unsigned)cut.ctas, cut.threads, bytes, stream>>>(p);
        return launch_status();
    };
    auto by_width = [&](auto with_ring) {
        constexpr bool R = decltype(with_ring)::value;
        if (p.cols <= 128)
            return go(split_kernel<H, S8, 1, 16, kSmallThreads, kStages, R>, 1, R);
        if (p.cols <= 256)
            return go(split_kernel<H, S8, 1, 32, kSmallThreads, kStages, R>, 1, R);
        if (p.cols <= 2048)
            return go(split_kernel<H, S8, 1, 0, 256, kStages, R>, 1, R);
        if (p.cols <= 4096)
            return go(split_kernel<H, S8, 2, 0, 256, kStages, R>, 2, R);
        return go(split_kernel<H, S8, 2, 0, 512, kStages, R>, 2, R);
    };
    if (p.cols > 8192) {
        split_long_kernel<H, S8><<<(unsigned)cut.ctas, 1024, 0, stream>>>(p);
        return launch_status();
    }
    return p.wide ? by_width(std::true_type{}) : by_width(std::false_type{});
}

template <int THREADS>
static int launch_columns(const ColumnParams &p, bool one, cudaStream_t stream)
{
    cudaLaunchAttribute early{};
    early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    early.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(ceil_div(p.cols, 8) + (one ? 1 : 0)));
    cfg.blockDim = dim3(THREADS);
    cfg.stream = stream;
    cfg.attrs = &early;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, columns_kernel<THREADS>, p);
    return e == cudaSuccess ? ZERO_OK : cuda_error(e);
}

// A token's gate has no elements, and so may be NULL, where there are no rows.
static bool bad_gate(const void *gate, int kind, int type, int64_t rows)
{
    return kind < ZERO_GATE_NONE || kind > ZERO_GATE_ROWS ||
           (kind != ZERO_GATE_NONE && ((!gate && (kind != ZERO_GATE_ROWS || rows > 0)) || !is_float(type)));
}

static bool gate_aligned(const void *gate, int kind, int type)
{
    return kind == ZERO_GATE_NONE || aligned(gate, (uintptr_t)type_bytes(type));
}

}  // namespace zo

using namespace zo;

extern "C" {

int zero_gated_norms_fp8(const void *o, int64_t ldo, const void *x, int64_t ldx, const void *w_post,
                         const void *w_pre, int w_type, const void *gate, int gate_kind, int gate_type,
                         float scale, int type, int64_t rows, int64_t cols, float eps, void *h, int64_t ldh,
                         void *y, int64_t ldy, int fp8, const zero_fp8_form *y8, const zero_fp8_form *o8,
                         const zero_fp8_form *h8, float *rstd_post, float *rstd_pre, zero_stream_t stream)
{
    if (!is_half(type) || !is_float(w_type) || bad_dim(rows) || bad_dim(cols) || cols < 1 || !(eps >= 0.0f) ||
        !std::isfinite(eps) || !std::isfinite(scale) || bad_gate(gate, gate_kind, gate_type, rows) || (y8 && !is_fp8(fp8)))
        return ZERO_EINVAL;
    if (rows == 0)
        return ZERO_OK;
    if (!w_pre)
        return ZERO_EINVAL;
    const int b = type_bytes(type);
    int rc = check_matrix(o, rows, cols, ldo, b);
    if (!rc)
        rc = check_matrix(x, rows, cols, ldx, b);
    if (!rc)
        rc = check_matrix(h, rows, cols, ldh, b);
    if (!rc && y)
        rc = check_matrix(y, rows, cols, ldy, b);
    for (const zero_fp8_form *f : {y8, o8, h8})
        if (!rc)
            rc = check_form(f, rows, cols);
    const uintptr_t wb = (uintptr_t)type_bytes(w_type);
    if (!rc && (!aligned(w_pre, wb) || !aligned(w_post, wb) || !gate_aligned(gate, gate_kind, gate_type) ||
                !aligned(rstd_post, 4) || !aligned(rstd_pre, 4)))
        rc = ZERO_EALIGN;
    if (rc)
        return rc;
    JoinParams p{};
    p.o = o;
    p.x = x;
    p.w_post = w_post;
    p.w_pre = w_pre;
    p.gate = {gate, gate_kind, gate_type};
    p.h = h;
    p.y = y;
    p.y8 = form_of(y8);
    p.o8 = form_of(o8);
    p.h8 = form_of(h8);
    p.rstd_post = rstd_post;
    p.rstd_pre = rstd_pre;
    p.ldo = ldo;
    p.ldx = ldx;
    p.ldh = ldh;
    p.ldy = ldy;
    p.rows = rows;
    p.cols = cols;
    p.scale = scale;
    p.eps = eps;
    p.inv_cols = 1.0f / (float)cols;
    p.w_type = w_type;
    p.e5m2 = y8 && fp8 == ZERO_T_E5M2;
    p.wide = rows_aligned(o, ldo, b, 16) && rows_aligned(x, ldx, b, 16) && rows_aligned(h, ldh, b, 16) &&
             (!y || rows_aligned(y, ldy, b, 16));
    p.wide_w = aligned(w_pre, 16) && aligned(w_post, 16) && (gate_kind != ZERO_GATE_COLS || aligned(gate, 16));
    return type == ZERO_T_F16 ? launch_join<f16>(p, stream) : launch_join<bf16>(p, stream);
}

size_t zero_gated_norms_workspace_bytes(int64_t rows, int64_t cols)
{
    if (bad_dim(rows) || bad_dim(cols) || cols < 1)
        return 0;
    return (size_t)cut_of(rows, cols).ctas * (size_t)(2 * cols + 1) * sizeof(float);
}

int zero_gated_norms_backward(const void *dy, int64_t lddy, const void *dh, int64_t lddh, const void *o, int64_t ldo,
                              const float *so, int64_t ldso, const void *h, int64_t ldh, const float *sh,
                              int64_t ldsh, const float *rstd_post, const float *rstd_pre, const void *w_post,
                              const void *w_pre, int w_type, const void *gate, int gate_kind, int gate_type,
                              float scale, int type, int64_t rows, int64_t cols, void *d_o, int64_t lddo, void *dx,
                              int64_t lddx, void *dw_post, void *dw_pre, void *dgate, int dw_type, int add, void *ws,
                              size_t ws_bytes, zero_stream_t stream)
{
    const bool any = dw_pre || dw_post || dgate;
    const bool shared = dw_pre || dw_post || (dgate && gate_kind != ZERO_GATE_ROWS);  // sums over rows
    if (!is_half(type) || !is_float(w_type) || bad_dim(rows) || bad_dim(cols) || cols < 1 || !std::isfinite(scale) ||
        !w_pre || bad_gate(gate, gate_kind, gate_type, rows) || !so != !sh || (rows > 0 && !rstd_pre) ||
        (rows > 0 && w_post && !rstd_post) || (dw_post && !w_post) || (dgate && gate_kind == ZERO_GATE_NONE) ||
        (any && !is_float(dw_type)) || (shared && !ws))
        return ZERO_EINVAL;
    const int b = type_bytes(type);
    int rc = check_matrix(dy, rows, cols, lddy, b);
    if (!rc && dh)
        rc = check_matrix(dh, rows, cols, lddh, b);
    if (!rc)
        rc = check_kept(o, ldo, so, ldso, type, rows, cols);
    if (!rc)
        rc = check_kept(h, ldh, sh, ldsh, type, rows, cols);
    if (!rc)
        rc = check_matrix(d_o, rows, cols, lddo, b);
    if (!rc)
        rc = check_matrix(dx, rows, cols, lddx, b);
    const uintptr_t wb = (uintptr_t)type_bytes(w_type), db = any ? (uintptr_t)type_bytes(dw_type) : 1;
    if (!rc && (!aligned(w_pre, wb) || !aligned(w_post, wb) || !gate_aligned(gate, gate_kind, gate_type) ||
                !aligned(rstd_post, 4) || !aligned(rstd_pre, 4) || !aligned(dw_pre, db) || !aligned(dw_post, db) ||
                !aligned(dgate, db) || (shared && !aligned(ws, 32))))
        rc = ZERO_EALIGN;
    if (!rc && shared && ws_bytes < zero_gated_norms_workspace_bytes(rows, cols))
        rc = ZERO_ESPACE;
    if (rc)
        return rc;
    const Cut cut = cut_of(rows, cols);
    const Gate g{gate, gate_kind, gate_type};
    if (rows > 0) {
        SplitParams p{};
        p.dy = dy;
        p.dh = dh;
        p.o = o;
        p.h = h;
        p.w_post = w_post;
        p.w_pre = w_pre;
        p.so = so;
        p.sh = sh;
        p.ro = rstd_post;
        p.rh = rstd_pre;
        p.gate = g;
        p.d_o = d_o;
        p.dx = dx;
        p.dgate_rows = gate_kind == ZERO_GATE_ROWS ? dgate : nullptr;
        p.dgate_type = dw_type;
        p.part = shared ? static_cast<float *>(ws) : nullptr;
        p.want_pre = dw_pre != nullptr;
        p.want_post = dw_post || (dgate && gate_kind == ZERO_GATE_COLS);
        p.want_one = dgate && gate_kind == ZERO_GATE_ONE;
        p.lddy = lddy;
        p.lddh = lddh;
        p.ldo = ldo;
        p.ldh = ldh;
        p.ldso = ldso;
        p.ldsh = ldsh;
        p.lddo = lddo;
        p.lddx = lddx;
        p.rows = rows;
        p.cols = cols;
        p.scale = scale;
        p.inv_cols = 1.0f / (float)cols;
        p.w_type = w_type;
        const int kb = so ? 1 : b, to = so ? 8 : 16;
        p.wide = rows_aligned(dy, lddy, b, 16) && (!dh || rows_aligned(dh, lddh, b, 16)) &&
                 rows_aligned(o, ldo, kb, to) && rows_aligned(h, ldh, kb, to) && rows_aligned(d_o, lddo, b, 16) &&
                 rows_aligned(dx, lddx, b, 16);
        p.wide_w = aligned(w_pre, 16) && aligned(w_post, 16) && (gate_kind != ZERO_GATE_COLS || aligned(gate, 16));
        if (type == ZERO_T_F16)
            rc = so ? launch_split<f16, true>(p, cut, stream) : launch_split<f16, false>(p, cut, stream);
        else
            rc = so ? launch_split<bf16, true>(p, cut, stream) : launch_split<bf16, false>(p, cut, stream);
        if (rc)
            return rc;
    }
    if (!shared)
        return ZERO_OK;
    ColumnParams q{};
    q.part = static_cast<const float *>(ws);
    q.parts = rows > 0 ? cut.ctas : 0;
    q.cols = cols;
    q.w_post = w_post;
    q.gate = g;
    q.dw_pre = dw_pre;
    q.dw_post = dw_post;
    q.dgate = gate_kind == ZERO_GATE_ROWS ? nullptr : dgate;
    q.w_type = w_type;
    q.out_type = dw_type;
    q.add = add != 0;
    const bool one = dgate && gate_kind == ZERO_GATE_ONE;
    return q.parts > 512 ? launch_columns<1024>(q, one, stream) : launch_columns<256>(q, one, stream);
}

}  // extern "C"
