// The norms behind and ahead of a block, its gate and the residual stream in one
// pass over the rows:
//
//   xo = o * ro, ro = 1 / sqrt(mean(o^2) + eps)   (xo = o without a norm behind the block)
//   h = scale * x + gate * w_post * xo
//   y = h * rh * w_pre, rh = 1 / sqrt(mean(h^2) + eps)
//
// Each input is read once and each output written once.  Three 8-bit forms make it a matter of
// instructions too: fp32 values go in pairs, maxima are shared out between lanes and each scale is
// formed once.  8192x4096 bf16, three forms: 66 us, 4.6 TB/s (0.69 of the copy rate), bound by
// waiting: 16 warps to an SM, issue slots 59 % busy, ALU 45, DRAM 49.  The first kernel, with values one
// by one and a division for each scale, took 94.  16384x768 32 us (0.64).  Of the copy rate: 131072x256
// 0.77, 65536x512 0.73, 32768x1024 0.71, 16384x2048 0.70, 14563x2304 0.64, x2309 0.59, 104857x320 0.48,
// and above 4096 columns 6553x5120 0.60, 4096x8192 0.58, 2048x16384 0.46, 1024x32768 0.41.
#include <initializer_list>
#include <type_traits>

#include "norms.cuh"

namespace zo {

struct JoinParams {
    const void *o, *x, *w_post, *w_pre;
    Gate gate;
    void *h, *y;
    Form y8, o8, h8;
    float *rstd_post, *rstd_pre;
    int64_t ldo, ldx, ldh, ldy;
    int64_t rows;
    int32_t cols;
    float scale, eps, inv_cols;
    int32_t w_type, e5m2;
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

template <class H>
__device__ __forceinline__ float square_sum(const Raw8<H> &r)
{
    float2 x[4], s = both(0.0f);
    pairs_of(r, x);
#pragma unroll
    for (int i = 0; i < 4; ++i)
        s = fma2(x[i], x[i], s);
    return s.x + s.y;
}

// Behind a row's end o, x, w_post and w_pre are zeros, and so are h and y.
// h of 8 columns (`by`: the row's gate times ro).
template <int W, class H>
__device__ __forceinline__ void join8(const JoinParams &p, int c, int n, const Raw8<H> &o, const Raw8<H> &x, float by, float2 (&h)[4])
{
    float2 f[4], xo[4], xs[4];
    post_factors<W>(p.w_post, p.w_type, p.gate, c, n, f);
    pairs_of(o, xo);
    pairs_of(x, xs);
#pragma unroll
    for (int i = 0; i < 4; ++i)
        h[i] = fma2(both(p.scale), xs[i], mul2(f[i], mul2(xo[i], both(in_row_only(by, n)))));
    end_unit<W>(h, n, by);
}

// V units of a row, `step` columns apart, into two forms of fp32 values (either may be absent).
template <int W, int V>
__device__ __forceinline__ void put_two(const Form &f, const Form &g, int64_t row, int c, int step, int cols,
                                        const float2 (&x)[V][4], const float2 (&y)[V][4], bool e5m2)
{
    uint32_t a[2 * V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        a[v] = amax8(x[v]);
        a[V + v] = amax8(y[v]);
    }
    const uint32_t most = max_shared(a);
    const int mine = shared_index<2 * V>(), unit = mine % V;
    const bool second = mine >= V;
    const float s = Range(second && e5m2).scale(most);
    const Inverse inv = inverse_of(s);
    const Form &w = second ? g : f;
    const int at = c + unit * step;  // a column of this lane's block; its first decides
    if (threadIdx.x % (16 / (2 * V)) == 0 && w.q && (at & ~(kBlock - 1)) < cols)
        w.s[(at / kBlock) * w.lds + row] = s;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int at_v = c + v * step, n = left_of(cols, at_v);
        const Inverse i0 = shared_value<2 * V>(inv, v), i1 = shared_value<2 * V>(inv, V + v);
        if (f.q && n > 0)
            put_bytes<W>(f.q + row * f.ld + at_v, n, bytes_of<false>(x[v], i0));
        if (g.q && n > 0)
            put_bytes<W>(g.q + row * g.ld + at_v, n, e5m2 ? bytes_of<true>(y[v], i1) : bytes_of<false>(y[v], i1));
    }
}

// V units of halves into the form that zero_fp8_quantize gives them.
template <int W, int V, class H>
__device__ __forceinline__ void put_halves(const Form &f, int64_t row, int c, int step, int cols, const Raw8<H> (&r)[V])
{
    uint32_t a[V];
#pragma unroll
    for (int v = 0; v < V; ++v)
        a[v] = amax8(r[v]);
    const uint32_t most = max_shared(a);
    const float s = scale_of<false>(most);
    const Inverse inv = inverse_of(s);
    const int at = c + shared_index<V>() * step;
    if (threadIdx.x % (16 / V) == 0 && (at & ~(kBlock - 1)) < cols)
        f.s[(at / kBlock) * f.lds + row] = s;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int at_v = c + v * step, n = left_of(cols, at_v);
        const Inverse d = shared_value<V>(inv, v);
        float2 x[4];
        pairs_of(r[v], x);
        if (n > 0)
            put_bytes<W>(f.q + row * f.ld + at_v, n, bytes_of<false>(x, d));
    }
}

// What V units of a row leave once rh is known.
template <int W, int V, class H>
__device__ __forceinline__ void put_units(const JoinParams &p, int64_t row, int c, int step, int cols,
                                          const float2 (&h)[V][4], float rh)
{
    float2 y[V][4];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int at = c + v * step, n = left_of(cols, at);
        if (n > 0)
            put_pairs<W>(static_cast<H *>(p.h) + row * p.ldh + at, n, h[v]);
        get_vector<W>(p.w_pre, p.w_type, at, n, y[v]);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            y[v][i] = mul2(mul2(h[v][i], both(in_row_only(rh, n))), y[v][i]);
        end_unit<W>(y[v], n, rh);
        if (p.y && n > 0)
            put_pairs<W>(static_cast<H *>(p.y) + row * p.ldy + at, n, y[v]);
    }
    if (p.h8.q || p.y8.q)
        put_two<W>(p.h8, p.y8, row, c, step, cols, h, y, p.e5m2);
}

// A CTA takes a run of neighbouring rows, two at a time, a thread the same 8 columns of each:
// its factors stay in registers, and STAGES - 1 turns ahead are on their way through shared
// memory (W other than kApart).  G: a row to 16 or 32 lanes, or (0) to the CTA.
template <class H, int G, int MAXT, int STAGES, int W>
__global__ void __launch_bounds__(MAXT, MAXT == 320 ? 2 : 512 / MAXT) join_kernel(const JoinParams p)
{
    constexpr bool kRing = W != kApart;
    constexpr int kLanes = G ? G : 32;
    __shared__ __align__(16) float slots[2][2][2 * 16];  // of the turn, of the sum
    extern __shared__ __align__(16) unsigned char ring[];
    const int t = G ? threadIdx.x % kLanes : threadIdx.x, c = t * 8;
    const int groups = G ? MAXT / kLanes : 1, group = G ? threadIdx.x / kLanes : 0;
    const int64_t all = (int64_t)gridDim.x * groups, me = (int64_t)blockIdx.x * groups + group;
    const int64_t each = p.rows / all, more = p.rows % all;
    const int64_t first = me * each + min(me, more);
    const int mine = (int)each + (me < more ? 1 : 0), last = G == 16 ? (int)each + (more > 0 ? 1 : 0) : mine;
    const int n = left_of(p.cols, c);
    if (!G) {
        for (int i = threadIdx.x; i < 128; i += blockDim.x)
            (&slots[0][0][0])[i] = 0.0f;
        __syncthreads();
    }
    float2 w[4], a[4];
    get_vector<W>(p.w_pre, p.w_type, c, n, w);
    post_factors<W>(p.w_post, p.w_type, p.gate, c, n, a);
    const float fixed = p.gate.kind == ZERO_GATE_ONE ? load_one(p.gate.p, p.gate.type, 0) : 1.0f;

    const uint32_t lanes = blockDim.x, turn_bytes = lanes * 64;  // o and x of two rows
    const uint32_t place = (kRing ? (uint32_t)__cvta_generic_to_shared(ring) : 0u) + threadIdx.x * 16;
    const H *f_o = static_cast<const H *>(p.o) + first * p.ldo + (n > 0 ? c : 0);
    const H *f_x = static_cast<const H *>(p.x) + first * p.ldx + (n > 0 ? c : 0);
    auto fetch = [&](int k, uint32_t stage) {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int m = k + r < mine ? n : 0;  // where nothing is read the address is still one of the matrix
            copy_async<16>(place + stage + r * lanes * 32, k + r < mine ? f_o : static_cast<const H *>(p.o), 2 * m);
            copy_async<16>(place + stage + (r * 2 + 1) * lanes * 16, k + r < mine ? f_x : static_cast<const H *>(p.x), 2 * m);
            f_o += p.ldo;
            f_x += p.ldx;
        }
        commit_copies();
    };
    if (kRing)
#pragma unroll
        for (int s = 0; s < STAGES - 1; ++s)
            fetch(s * 2, s * turn_bytes);
    H *to_h = static_cast<H *>(p.h) + first * p.ldh + c, *to_y = static_cast<H *>(p.y) + first * p.ldy + c;
    uint8_t *to_o8 = p.o8.q + first * p.o8.ld + c, *to_h8 = p.h8.q + first * p.h8.ld + c, *to_y8 = p.y8.q + first * p.y8.ld + c;
    // the scale that a lane writes: of a row of o8, and of a row of h8 (the lower 8 of 16 lanes) or y8
    const int block = c / kBlock, own2 = shared_index<2>(), own4 = shared_index<4>();
    const bool inside = (c & ~(kBlock - 1)) < p.cols;
    const Form &f4 = own4 < 2 ? p.h8 : p.y8;
    float *to_so = (t & 7) == 0 && inside && p.o8.q ? p.o8.s + block * p.o8.lds + first + own2 : nullptr;
    float *to_s4 = (t & 3) == 0 && inside && f4.q ? f4.s + block * f4.lds + first + (own4 & 1) : nullptr;
    const Range range(own4 >= 2 && p.e5m2);

    uint32_t stage = 0;
    int turn = 0;
    for (int k = 0; k < last; k += 2, turn ^= 1) {
        Raw8<H> o[2], x[2];
        const int m[2] = {k < mine ? n : 0, k + 1 < mine ? n : 0};
        if (kRing) {
            wait_copies<STAGES - 2>();
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                load_shared(o[r].w, place + stage + r * lanes * 32);
                load_shared(x[r].w, place + stage + (r * 2 + 1) * lanes * 16);
            }
            // into the places of the turn before, whose values this thread has used
            fetch(k + (STAGES - 1) * 2, stage == 0 ? (STAGES - 1) * turn_bytes : stage - turn_bytes);
            stage = stage == (STAGES - 1) * turn_bytes ? 0 : stage + turn_bytes;
        } else {
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                o[r] = get_raw<W>(static_cast<const H *>(p.o) + (first + k + r) * p.ldo + c, m[r]);
                x[r] = get_raw<W>(static_cast<const H *>(p.x) + (first + k + r) * p.ldx + c, m[r]);
            }
        }
        float by[2];  // the row's gate times ro
#pragma unroll
        for (int r = 0; r < 2; ++r)
            by[r] = p.gate.kind != ZERO_GATE_ROWS ? fixed : k + r < mine ? load_one(p.gate.p, p.gate.type, first + k + r) : 0.0f;
        if (p.w_post) {
            float sq[2] = {square_sum(o[0]), square_sum(o[1])};
            shared_sums<G>(sq, slots[turn][0]);
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const float ro = root(sq[r], p.inv_cols, p.eps);
                by[r] *= ro;
                if (t == 0 && k + r < mine && p.rstd_post)
                    p.rstd_post[first + k + r] = ro;
            }
        }
        if (p.o8.q) {
            uint32_t most[2] = {amax8(o[0]), amax8(o[1])};
            const float s = scale_of<false>(max_shared(most));
            const Inverse inv = inverse_of(s);
            if (to_so && k + own2 < mine)
                to_so[k] = s;
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const Inverse d = shared_value<2>(inv, r);
                float2 v[4];
                pairs_of(o[r], v);
                if (m[r] > 0)
                    put_bytes<W>(to_o8 + r * p.o8.ld, m[r], bytes_of<false>(v, d));
            }
            to_o8 += 2 * p.o8.ld;
        }
        float2 h[2][4];
        float sq[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            float2 xo[4], xs[4], s2 = both(0.0f);
            pairs_of(o[r], xo);
            pairs_of(x[r], xs);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                h[r][i] = fma2(both(p.scale), xs[i], mul2(a[i], mul2(xo[i], both(in_row_only(by[r], n)))));
            end_unit<W>(h[r], n, by[r]);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                s2 = fma2(h[r][i], h[r][i], s2);
            sq[r] = s2.x + s2.y;
        }
        shared_sums<G>(sq, slots[turn][1]);
        float2 y[2][4];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const float rh = root(sq[r], p.inv_cols, p.eps);
            if (t == 0 && k + r < mine && p.rstd_pre)
                p.rstd_pre[first + k + r] = rh;
            if (m[r] > 0)
                put_pairs<W>(to_h + r * p.ldh, m[r], h[r]);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                y[r][i] = mul2(mul2(h[r][i], both(in_row_only(rh, n))), w[i]);
            end_unit<W>(y[r], n, rh);
            if (p.y && m[r] > 0)
                put_pairs<W>(to_y + r * p.ldy, m[r], y[r]);
        }
        to_h += 2 * p.ldh;
        to_y += 2 * p.ldy;
        if (p.h8.q || p.y8.q) {
            uint32_t most[4] = {amax8(h[0]), amax8(h[1]), amax8(y[0]), amax8(y[1])};
            const float s = range.scale(max_shared(most));
            const Inverse inv = inverse_of(s);
            if (to_s4 && k + (own4 & 1) < mine)
                to_s4[k] = s;
            auto put = [&](auto e5m2) {
                constexpr bool E = decltype(e5m2)::value;
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const Inverse d = shared_value<4>(inv, r), e = shared_value<4>(inv, 2 + r);
                    if (p.h8.q && m[r] > 0)
                        put_bytes<W>(to_h8 + r * p.h8.ld, m[r], bytes_of<false>(h[r], d));
                    if (p.y8.q && m[r] > 0)
                        put_bytes<W>(to_y8 + r * p.y8.ld, m[r], bytes_of<E>(y[r], e));
                }
            };
            if (p.e5m2)
                put(std::true_type{});
            else
                put(std::false_type{});
            to_h8 += 2 * p.h8.ld;
            to_y8 += 2 * p.y8.ld;
        }
    }
    if (kRing)
        wait_copies<0>();  // nothing is on its way when the CTA leaves
}

// Rows of more than 4096 columns: one to a CTA, V units of 8 to a thread.  Clusters of 2 to 4
// CTAs of the kernel above, which exchange their sums, took 117 us for 77 at 4096x8192: the
// cluster's barrier waits for the turn's stores.
template <class H, int V, int MAXT, int W>
__global__ void __launch_bounds__(MAXT) join_wide_kernel(const JoinParams p)
{
    constexpr int kWarps = MAXT / 32;
    __shared__ float slots[2][kWarps];
    const int t = threadIdx.x, step = blockDim.x * 8, c = t * 8, cols = p.cols;
    const int64_t row = blockIdx.x;
    const H *po = static_cast<const H *>(p.o) + row * p.ldo, *px = static_cast<const H *>(p.x) + row * p.ldx;
    Raw8<H> o[V], x[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int n = left_of(cols, c + v * step);
        o[v] = get_raw<W>(po + c + v * step, n);
        x[v] = get_raw<W>(px + c + v * step, n);
    }
    float ro = 1.0f;
    if (p.w_post) {
        float sq[1] = {0.0f};
#pragma unroll
        for (int v = 0; v < V; ++v)
            sq[0] += square_sum(o[v]);
        row_sums<kWarps>(sq, slots[0]);
        ro = root(sq[0], p.inv_cols, p.eps);
        if (t == 0 && p.rstd_post)
            p.rstd_post[row] = ro;
    }
    const float by = row_gate(p.gate, row) * ro;
    float2 h[V][4], s2 = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int n = left_of(cols, c + v * step);
        join8<W>(p, c + v * step, n, o[v], x[v], by, h[v]);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            s2 = fma2(h[v][i], h[v][i], s2);
    }
    if (p.o8.q)
        put_halves<W>(p.o8, row, c, step, cols, o);
    float sq[1] = {s2.x + s2.y};
    row_sums<kWarps>(sq, slots[1]);
    const float rh = root(sq[0], p.inv_cols, p.eps);
    if (t == 0 && p.rstd_pre)
        p.rstd_pre[row] = rh;
    put_units<W, V, H>(p, row, c, step, cols, h, rh);
}

// Rows too long for the registers: o for its norm, o and x for h's, and both again
// for what is written (h may be x or o, so nothing is written before that).
template <class H, int W>
__global__ void __launch_bounds__(1024) join_long_kernel(const JoinParams p)
{
    __shared__ float slots[2][32];
    const int64_t row = blockIdx.x;
    const H *po = static_cast<const H *>(p.o) + row * p.ldo;
    const H *px = static_cast<const H *>(p.x) + row * p.ldx;
    float ro = 1.0f;
    if (p.w_post) {
        float sq[1] = {0.0f};
        for (int64_t c = threadIdx.x * 8; c < p.cols; c += 1024 * 8)
            sq[0] += square_sum(get_raw<W>(po + c, left_of(p.cols, (int)c)));
        row_sums<32>(sq, slots[0]);
        ro = root(sq[0], p.inv_cols, p.eps);
        if (threadIdx.x == 0 && p.rstd_post)
            p.rstd_post[row] = ro;
    }
    const float by = row_gate(p.gate, row) * ro;
    Raw8<H> o[1];
    float2 h[1][4], s2 = make_float2(0.0f, 0.0f);
    auto join = [&](int c) {
        const int n = left_of(p.cols, c);
        o[0] = get_raw<W>(po + c, n);
        join8<W>(p, c, n, o[0], get_raw<W>(px + c, n), by, h[0]);
    };
    for (int64_t c = threadIdx.x * 8; c < p.cols; c += 1024 * 8) {
        join((int)c);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            s2 = fma2(h[0][i], h[0][i], s2);
    }
    float sq[1] = {s2.x + s2.y};
    row_sums<32>(sq, slots[1]);
    const float rh = root(sq[0], p.inv_cols, p.eps);
    if (threadIdx.x == 0 && p.rstd_pre)
        p.rstd_pre[row] = rh;
    const int64_t end = ((int64_t)p.cols + 1024 * 8 - 1) / (1024 * 8) * (1024 * 8);
    for (int64_t c = threadIdx.x * 8; c < end; c += 1024 * 8) {
        join((int)c);
        if (p.o8.q)
            put_halves<W>(p.o8, row, (int)c, 0, p.cols, o);
        put_units<W, 1, H>(p, row, (int)c, 0, p.cols, h, rh);
    }
}

template <class H, int W>
static int launch_join(const JoinParams &p, cudaStream_t stream)
{
    auto threads = [&](int units) { return (int)(ceil_div(ceil_div(p.cols, 8 * units), 32) * 32); };
    auto go = [&](auto kernel, int threads) {
        kernel<<<(unsigned)p.rows, threads, 0, stream>>>(p);
        return launch_status();
    };
    // `most_threads`: of any launch of the kernel
    auto ring = [&](auto kernel, int most_threads, int threads, int groups, int stages) {
        const size_t bytes = W != kApart ? (size_t)stages * threads * 64 : 0;
        if (W != kApart)
            if (const int rc = allow_smem<kernel.value>(stages * most_threads * 64))
                return rc;
        const int64_t most = 152 * ((threads > 256 && threads <= 320 ? 640 : 512) / threads), turns = ceil_div(p.rows, 2 * groups);
        kernel.value<<<(unsigned)(turns < most ? turns : most), threads, bytes, stream>>>(p);
        return launch_status();
    };
    constexpr int kDepth = 4;
    if (p.cols <= 128)
        return ring(Kernel<join_kernel<H, 16, 256, kDepth, W>>{}, 256, 256, 16, kDepth);
    if (p.cols <= 256)
        return ring(Kernel<join_kernel<H, 32, 256, kDepth, W>>{}, 256, 256, 8, kDepth);
    if (p.cols <= 2048)
        return ring(Kernel<join_kernel<H, 0, 256, kDepth, W>>{}, 256, threads(1), 1, kDepth);
    if (p.cols <= 2560)  // two CTAs to an SM where registers are 96 (8192x4096 elements in 14563 rows: 70 us; with one
                       // 87 where this took 66)
        return ring(Kernel<join_kernel<H, 0, 320, kDepth, W>>{}, 320, threads(1), 1, kDepth);
    if (p.cols <= 4096)
        return ring(Kernel<join_kernel<H, 0, 512, kDepth, W>>{}, 512, threads(1), 1, kDepth);
    if (p.cols <= 8192)
        return go(join_wide_kernel<H, 2, 512, W>, threads(2));
    if (p.cols <= 16384)
        return go(join_wide_kernel<H, 2, 1024, W>, threads(2));
    return go(join_long_kernel<H, W>, 1024);
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
    p.cols = (int32_t)cols;
    p.scale = scale;
    p.eps = eps;
    p.inv_cols = 1.0f / (float)cols;
    p.w_type = w_type;
    p.e5m2 = y8 && fp8 == ZERO_T_E5M2;
    bool wide = rows_aligned(o, ldo, b, 16) && rows_aligned(x, ldx, b, 16) && rows_aligned(h, ldh, b, 16) &&
                (!y || rows_aligned(y, ldy, b, 16)) && aligned(w_pre, 16) && aligned(w_post, 16) &&
                (gate_kind != ZERO_GATE_COLS || aligned(gate, 16));
    for (const Form *f : {&p.y8, &p.o8, &p.h8})
        wide = wide && (!f->q || f->wide);
    auto go = [&](auto half) {
        using H = decltype(half);
        return !wide ? launch_join<H, kApart>(p, stream)
                     : cols % 8 ? launch_join<H, kWide>(p, stream) : launch_join<H, kWhole>(p, stream);
    };
    return type == ZERO_T_F16 ? go(f16{}) : go(bf16{});
}

}  // extern "C"
