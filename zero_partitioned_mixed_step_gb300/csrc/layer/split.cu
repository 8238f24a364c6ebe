// The gradients of the norms behind and ahead of a block, its gate and the residual
// stream.  xh = h * rh, g = dy * w_pre, A = gate * w_post:
//
//   m = mean(g * xh),  dH = rh * (g - xh * m) + dh,  dx = scale * dH
//   d_o = ro * (A * dH - xo * mean(A * xo * dH))
//
// The second mean needs the first, but as dH is linear in m, three sums that need
// nothing of one another give both, so that a row costs one barrier:
//   D = sum g xh,  P = sum A xo (rh g + dh),  Q = sum A xo xh,  sum A xo dH = P - rh (D / cols) Q
// (|P| and |rh m Q| are sums that dH's own terms bound: nothing is lost that dH keeps).
//
// Each input is read once and each output written once.  8192x4096 bf16 from 8-bit
// checkpoints: 66 us, 5.1 TB/s (0.76 of the copy rate), the pass over the rows 60 (issue slots 65 %
// busy, FMA 39, DRAM 63), the columns' sums 5; from kept halves 69 (0.85 of a longer floor).  Two
// units of one row to a thread, and so a barrier for each row, took 111, without the ring of
// copies 114.  Of the copy rate, from checkpoints: 262144x128 0.73, 65536x512 0.75, 32768x1024 0.76,
// 16384x2048 0.77, 14563x2304 0.62 (288 of 512 threads; 640 threads with 96 registers took 126 us for
// 80), 14563x2309 0.58; above 4096 columns, where a thread has two units, 6553x5120 0.57, 4096x8192
// 0.60, and above 8192, where a row is read twice, 2730x12288 0.29, 2048x16384 0.32.
#include <type_traits>

#include "norms.cuh"

namespace zo {

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
    int64_t rows;
    int32_t cols;
    float scale, inv_cols;
    int32_t w_type;
};

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
__device__ __forceinline__ void put_part(float *to, int n, bool whole, const float2 x[4])
{
    if (whole && n == 8) {
        asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to), "f"(x[0].x), "f"(x[0].y),
                     "f"(x[1].x), "f"(x[1].y), "f"(x[2].x), "f"(x[2].y), "f"(x[3].x), "f"(x[3].y)
                     : "memory");
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n)
                to[i] = i & 1 ? x[i >> 1].y : x[i >> 1].x;
    }
}

constexpr int kSmallThreads = 256;  // of CTAs whose rows have 16 or 32 lanes

// A CTA takes a run of neighbouring rows (of the blocks' scales, whose neighbours share
// sectors, all are then read by one SM), R at a time, a thread the same V * 8 columns
// of each, so that the sums over rows stay in registers.  W other than kApart: STAGES - 1
// turns ahead are on their way through shared memory, which the registers, full of
// factors and sums, have no room for.  A block's scale and its row's rstd are applied to sums
// and factors, not to the kept values one by one.
template <class H, bool S8, int V, int R, int G, int MAXT, int STAGES, int W>
__global__ void __launch_bounds__(MAXT, MAXT == 320 ? 2 : 512 / MAXT) split_kernel(const SplitParams p)
{
    using K = Kept<H, S8>;
    constexpr bool kRing = W != kApart;
    // The next turn's scales in registers, where a thread has one unit; with two they would spill (4096x8192
    // 105 us, 81 without), and kept halves have none.
    constexpr bool kAhead = S8 && V == 1;
    constexpr int kLanes = G ? G : 32;
    constexpr int kUnit = 32 + 2 * K::kBytes;  // bytes of a row's unit: dy, dh, o, h
    constexpr int kElem = K::kBytes / 8;
    __shared__ __align__(16) float slots[2][kSumPlaces<3 * R> * 16];
    extern __shared__ __align__(16) unsigned char ring[];
    const int T = G ? G : blockDim.x;
    const int t = G ? threadIdx.x % kLanes : threadIdx.x;
    const int groups = G ? MAXT / kLanes : 1, group = G ? threadIdx.x / kLanes : 0;
    const int64_t all = (int64_t)gridDim.x * groups, me = (int64_t)blockIdx.x * groups + group;
    // rows [first, end): rows / all each, one more for the first rows % all
    const int64_t each = p.rows / all, more = p.rows % all;
    const int64_t first = me * each + min(me, more);
    const int mine = (int)each + (me < more ? 1 : 0);
    if (!G) {
        for (int i = threadIdx.x; i < (int)(sizeof(slots) / 4); i += blockDim.x)
            (&slots[0][0])[i] = 0.0f;
        __syncthreads();
    }

    int n[V];
    float2 w[V][4], a[V][4], dw[V][4], da[V][4];
    float one = 0.0f;
    const float fixed = p.gate.kind == ZERO_GATE_ONE ? load_one(p.gate.p, p.gate.type, 0) : 1.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int c = (v * T + t) * 8;
        n[v] = left_of(p.cols, c);
        get_vector<W>(p.w_pre, p.w_type, c, n[v], w[v]);
        post_factors<W>(p.w_post, p.w_type, p.gate, c, n[v], a[v]);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            dw[v][i] = da[v][i] = both(0.0f);
    }
    // a thread's places: the four parts of a unit lie apart, so that a warp's accesses are side by side
    const uint32_t lanes = blockDim.x, unit_bytes = lanes * kUnit, turn_bytes = unit_bytes * V * R;
    const uint32_t base = kRing ? (uint32_t)__cvta_generic_to_shared(ring) : 0u;
    const uint32_t place[4] = {base + threadIdx.x * 16, base + (lanes + threadIdx.x) * 16,
                               base + lanes * 32 + threadIdx.x * K::kBytes,
                               base + lanes * 32 + (lanes + threadIdx.x) * K::kBytes};
    const H *f_dy = static_cast<const H *>(p.dy) + first * p.lddy, *f_dh = static_cast<const H *>(p.dh) + first * p.lddh;
    const unsigned char *f_o = static_cast<const unsigned char *>(p.o) + first * p.ldo * kElem;
    const unsigned char *f_h = static_cast<const unsigned char *>(p.h) + first * p.ldh * kElem;
    // rows k .. k + R - 1 of this group; what is behind the last row, or its end, becomes zeros
    auto fetch = [&](int k, uint32_t stage) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const bool there = k + r < mine;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const int c = there && n[v] > 0 ? (v * T + t) * 8 : 0, m = there ? n[v] : 0;
                const uint32_t to = stage + (r * V + v) * unit_bytes;
                // where nothing is read the address is still one of the matrix
                copy_async<16>(place[0] + to, (there ? f_dy : static_cast<const H *>(p.dy)) + c, 2 * m);
                if (p.dh)
                    copy_async<16>(place[1] + to, (there ? f_dh : static_cast<const H *>(p.dh)) + c, 2 * m);
                copy_async<K::kBytes>(place[2] + to, (there ? f_o : static_cast<const unsigned char *>(p.o)) + c * kElem, kElem * m);
                copy_async<K::kBytes>(place[3] + to, (there ? f_h : static_cast<const unsigned char *>(p.h)) + c * kElem, kElem * m);
            }
            f_dy += p.lddy;
            f_dh += p.lddh;
            f_o += p.ldo * kElem;
            f_h += p.ldh * kElem;
        }
        commit_copies();
    };
    // the next turn's numbers of rows and of their blocks
    float so_next[R][V], sh_next[R][V], ro_next[R], rh_next[R], gate_next[R];
    const float *f_so[V], *f_sh[V];
#pragma unroll
    for (int v = 0; v < V; ++v)
        if (S8) {
            const int64_t b = n[v] > 0 ? (v * T + t) * 8 / kBlock : 0;
            f_so[v] = p.so + b * p.ldso + first;
            f_sh[v] = p.sh + b * p.ldsh + first;
        }
    auto fetch_scales = [&](int k) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const bool there = k + r < mine;
            ro_next[r] = 1.0f;
            rh_next[r] = gate_next[r] = 0.0f;
#pragma unroll
            for (int v = 0; v < V; ++v)
                so_next[r][v] = sh_next[r][v] = !S8 && there ? 1.0f : 0.0f;
            if (!there)
                continue;  // a row that adds nothing
            rh_next[r] = p.rh[first + k + r];
            if (p.w_post)
                ro_next[r] = p.ro[first + k + r];
            gate_next[r] = p.gate.kind == ZERO_GATE_ROWS ? load_one(p.gate.p, p.gate.type, first + k + r) : fixed;
#pragma unroll
            for (int v = 0; v < V; ++v)
                if (S8 && n[v] > 0) {
                    so_next[r][v] = f_so[v][k + r];
                    sh_next[r][v] = f_sh[v][k + r];
                }
        }
    };
    if (kRing)
#pragma unroll
        for (int s = 0; s < STAGES - 1; ++s)
            fetch(s * R, s * turn_bytes);
    if (kAhead)
        fetch_scales(0);

    // two groups of 16 lanes share a warp and its shuffles, so both take as many turns
    const int last = G == 16 ? (int)each + (more > 0 ? 1 : 0) : mine;
    int turn = 0;
    uint32_t stage = 0;
    H *dx_row = static_cast<H *>(p.dx) + first * p.lddx, *do_row = static_cast<H *>(p.d_o) + first * p.lddo;
    for (int k = 0; k < last; k += R, turn ^= 1) {
        Raw8<H> dy[R][V], dh[R][V];
        K o[R][V], h[R][V];
        if (!kAhead)
            fetch_scales(k);
        if (kRing)
            wait_copies<STAGES - 2>();
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int v = 0; v < V; ++v) {
                if (kRing) {
                    const uint32_t from = stage + (r * V + v) * unit_bytes;
                    dh[r][v] = Raw8<H>{};
                    load_shared(dy[r][v].w, place[0] + from);
                    if (p.dh)
                        load_shared(dh[r][v].w, place[1] + from);
                    load_shared(o[r][v].r.w, place[2] + from);
                    load_shared(h[r][v].r.w, place[3] + from);
                } else {
                    const int c = (v * T + t) * 8, m = k + r < mine ? n[v] : 0;
                    const int64_t row = first + k + r;
                    dy[r][v] = get_raw<W>(static_cast<const H *>(p.dy) + row * p.lddy + c, m);
                    dh[r][v] = get_raw<W>(static_cast<const H *>(p.dh) + row * p.lddh + c, p.dh ? m : 0);
                    o[r][v].template load<W>(static_cast<const unsigned char *>(p.o) + row * p.ldo * kElem, c, m);
                    h[r][v].template load<W>(static_cast<const unsigned char *>(p.h) + row * p.ldh * kElem, c, m);
                }
            }
        if (kRing) {
            // into the places of the turn before, whose values this thread has used
            fetch(k + (STAGES - 1) * R, stage == 0 ? (STAGES - 1) * turn_bytes : stage - turn_bytes);
            stage = stage == (STAGES - 1) * turn_bytes ? 0 : stage + turn_bytes;
        }
        float ro[R], rh[R], gate[R], so[R][V], sh[R][V];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            ro[r] = ro_next[r];
            rh[r] = rh_next[r];
            gate[r] = gate_next[r];
#pragma unroll
            for (int v = 0; v < V; ++v) {
                so[r][v] = so_next[r][v] * ro[r];
                sh[r][v] = sh_next[r][v] * rh[r];
            }
        }
        if (kAhead)
            fetch_scales(k + R);

        float sum[3 * R];  // D, P, Q of each row
#pragma unroll
        for (int r = 0; r < R; ++r) {
            sum[3 * r] = sum[3 * r + 1] = sum[3 * r + 2] = 0.0f;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                float2 qo[4], qh[4], d[4], e[4], s0 = both(0.0f), s1 = s0, s2 = s0;
                o[r][v].get(qo);
                h[r][v].get(qh);
                pairs_of(dy[r][v], d);
                pairs_of(dh[r][v], e);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 g = mul2(d[i], w[v][i]), ax = mul2(a[v][i], qo[i]);
                    dw[v][i] = fma2(mul2(d[i], both(sh[r][v])), qh[i], dw[v][i]);
                    s0 = fma2(g, qh[i], s0);
                    s1 = fma2(ax, fma2(both(rh[r]), g, e[i]), s1);
                    s2 = fma2(ax, qh[i], s2);
                }
                sum[3 * r] = fmaf(s0.x + s0.y, sh[r][v], sum[3 * r]);
                sum[3 * r + 1] = fmaf(s1.x + s1.y, so[r][v], sum[3 * r + 1]);
                sum[3 * r + 2] = fmaf((s2.x + s2.y) * sh[r][v], so[r][v], sum[3 * r + 2]);
            }
        }
        shared_sums<G>(sum, slots[turn]);
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int v = 0; v < V; ++v) {
                renew(dy[r][v].w);
                renew(dh[r][v].w);
                renew(o[r][v].r.w);
                renew(h[r][v].r.w);
            }
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const bool live = k + r < mine;
            const float m = sum[3 * r] * p.inv_cols;
            const float along = fmaf(-rh[r] * m, sum[3 * r + 2], sum[3 * r + 1]);  // sum of w_post (and a channel's gate) * xo * dH
            const float mo = p.w_post ? gate[r] * along * p.inv_cols : 0.0f;
            one += along;
            if (t == 0 && live && p.dgate_rows)
                put_one(p.dgate_rows, p.dgate_type, first + k + r, along);
            const float by = ro[r] * gate[r];
            // Without a norm behind the block o, which may not be finite, has no part in d_o.  A select takes 1.3 us of
            // 66 at 8192x4096 and of 83 at 4096x8192, two ways for the row the same and 7.
            const bool post = p.w_post != nullptr;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                float2 qo[4], qh[4], d[4], e[4], x[4], y[4];
                o[r][v].get(qo);
                h[r][v].get(qh);
                pairs_of(dy[r][v], d);
                pairs_of(dh[r][v], e);
                const float km = -rh[r] * m * sh[r][v], ko = -ro[r] * mo * so[r][v];
                const float part = p.gate.kind == ZERO_GATE_ROWS ? gate[r] * so[r][v] : so[r][v];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 g = mul2(d[i], w[v][i]);
                    const float2 dH = fma2(both(km), qh[i], fma2(both(rh[r]), g, e[i]));
                    x[i] = mul2(both(p.scale), dH);
                    const float2 off = mul2(both(ko), qo[i]);
                    y[i] = fma2(a[v][i], mul2(both(by), dH), make_float2(post ? off.x : 0.0f, post ? off.y : 0.0f));
                    da[v][i] = fma2(mul2(both(part), dH), qo[i], da[v][i]);
                }
                const int c = (v * T + t) * 8;
                if (n[v] > 0 && live) {
                    put_pairs<W>(dx_row + c, n[v], x);
                    put_pairs<W>(do_row + c, n[v], y);
                }
            }
            dx_row += p.lddx;
            do_row += p.lddo;
        }
    }
    if (kRing)
        wait_copies<0>();  // nothing is on its way when the CTA leaves
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the columns' launch may begin
    if (!p.part)
        return;
    const int64_t parts = gridDim.x;
    const bool whole = p.cols % 8 == 0;
    if constexpr (G == 0) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int c = (v * T + t) * 8;
            if (p.want_pre)
                put_part(p.part + (int64_t)blockIdx.x * p.cols + c, n[v], whole, dw[v]);
            if (p.want_post)
                put_part(p.part + (parts + blockIdx.x) * p.cols + c, n[v], whole, da[v]);
        }
        if (p.want_one && t == 0)
            p.part[2 * parts * p.cols + blockIdx.x] = one;
    } else {  // the row groups of the CTA, in order
        __shared__ float2 sums[2][MAXT * 4];
        __shared__ float ones[MAXT / G];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            sums[0][threadIdx.x * 4 + i] = dw[0][i];
            sums[1][threadIdx.x * 4 + i] = da[0][i];
        }
        if (t == 0)
            ones[group] = one;
        __syncthreads();
        for (int c = threadIdx.x; c < p.cols; c += MAXT) {
            float x = 0.0f, y = 0.0f;
            for (int g = 0; g < groups; ++g) {
                x += reinterpret_cast<const float *>(sums[0])[g * G * 8 + c];
                y += reinterpret_cast<const float *>(sums[1])[g * G * 8 + c];
            }
            if (p.want_pre)
                p.part[(int64_t)blockIdx.x * p.cols + c] = x;
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
template <class H, bool S8, int W>
__global__ void __launch_bounds__(1024) split_long_kernel(const SplitParams p)
{
    using K = Kept<H, S8>;
    __shared__ float slots[2][3 * 32];
    const int64_t parts = gridDim.x;
    float *pre = p.part && p.want_pre ? p.part + (int64_t)blockIdx.x * p.cols : nullptr;
    float *post = p.part && p.want_post ? p.part + (parts + blockIdx.x) * p.cols : nullptr;
    const float2 zero[4] = {};
    const float fixed = p.gate.kind == ZERO_GATE_ONE ? load_one(p.gate.p, p.gate.type, 0) : 1.0f;
    const bool whole = p.cols % 8 == 0;
    for (int64_t c = threadIdx.x * 8; c < p.cols; c += 1024 * 8) {
        if (pre)
            put_part(pre + c, left_of(p.cols, (int)c), whole, zero);
        if (post)
            put_part(post + c, left_of(p.cols, (int)c), whole, zero);
    }
    // adds x * y to a unit of sums
    auto add = [&](float *to, int64_t c, int n, const float2 x[4], const float2 y[4]) {
        float2 s[4];
        const Raw8<float> r = whole ? get_raw<kWhole>(to + c, n) : get_raw<kApart>(to + c, n);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            s[i] = fma2(x[i], y[i], make_float2(__uint_as_float(r.w[2 * i]), __uint_as_float(r.w[2 * i + 1])));
        put_part(to + c, n, whole, s);
    };
    float one = 0.0f;
    int turn = 0;
    for (int64_t row = blockIdx.x; row < p.rows; row += parts, turn ^= 1) {
        const float rh = p.rh[row], ro = p.w_post ? p.ro[row] : 1.0f;
        const float gate = p.gate.kind == ZERO_GATE_ROWS ? load_one(p.gate.p, p.gate.type, row) : fixed;
        const float share = p.gate.kind == ZERO_GATE_ROWS ? gate : 1.0f;
        float2 w[4], a[4], xo[4], xh[4], d[4], e[4];
        auto read = [&](int c, int n) {
            get_vector<W>(p.w_pre, p.w_type, c, n, w);
            // the short way for whole rows would hold more than 64 registers have room for (12288 columns:
            // 196 us for 173)
            post_factors<W == kWhole ? kWide : W>(p.w_post, p.w_type, p.gate, c, n, a);
            pairs_of(get_raw<W>(static_cast<const H *>(p.dy) + row * p.lddy + c, n), d);
            pairs_of(get_raw<W>(static_cast<const H *>(p.dh) + row * p.lddh + c, p.dh ? n : 0), e);
            K o, h;
            constexpr int kElem = K::kBytes / 8;
            o.template load<W>(static_cast<const unsigned char *>(p.o) + row * p.ldo * kElem, c, n);
            h.template load<W>(static_cast<const unsigned char *>(p.h) + row * p.ldh * kElem, c, n);
            o.get(xo);
            h.get(xh);
            const float so = S8 ? p.so[c / kBlock * p.ldso + row] * ro : ro;
            const float sh = S8 ? p.sh[c / kBlock * p.ldsh + row] * rh : rh;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                xo[i] = mul2(xo[i], both(so));
                xh[i] = mul2(xh[i], both(sh));
            }
        };
        float2 s0 = both(0.0f), s1 = s0, s2 = s0;
        for (int64_t c = threadIdx.x * 8; c < p.cols; c += 1024 * 8) {
            const int n = left_of(p.cols, (int)c);
            read((int)c, n);
            if (pre)
                add(pre, c, n, d, xh);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 g = mul2(d[i], w[i]), ax = mul2(a[i], xo[i]);
                s0 = fma2(g, xh[i], s0);
                s1 = fma2(ax, fma2(both(rh), g, e[i]), s1);
                s2 = fma2(ax, xh[i], s2);
            }
        }
        float sum[3] = {s0.x + s0.y, s1.x + s1.y, s2.x + s2.y};
        row_sums<32>(sum, slots[turn]);
        const float m = sum[0] * p.inv_cols;
        const float along = fmaf(-rh * m, sum[2], sum[1]);
        const float mo = p.w_post ? gate * along * p.inv_cols : 0.0f;
        one += along;
        if (threadIdx.x == 0 && p.dgate_rows)
            put_one(p.dgate_rows, p.dgate_type, row, along);
        for (int64_t c = threadIdx.x * 8; c < p.cols; c += 1024 * 8) {
            const int n = left_of(p.cols, (int)c);
            read((int)c, n);
            float2 x[4], y[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 g = mul2(d[i], w[i]);
                d[i] = fma2(both(-rh * m), xh[i], fma2(both(rh), g, e[i]));
                x[i] = mul2(both(p.scale), d[i]);
                y[i] = mul2(a[i], mul2(both(ro * gate), d[i]));
                if (p.w_post)
                    y[i] = fma2(a[i], mul2(both(ro * gate), d[i]), mul2(both(-ro * mo), xo[i]));
                d[i] = mul2(both(share), d[i]);
            }
            if (post)
                add(post, c, n, d, xo);
            put_pairs<W>(static_cast<H *>(p.dx) + row * p.lddx + c, n, x);
            put_pairs<W>(static_cast<H *>(p.d_o) + row * p.lddo + c, n, y);
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

// How a backward pass is cut, a rule on the sizes and on whether o and h are kept in 8 bits, so that the
// sums' bits do not depend on the GPU: threads, rows side by side in a CTA, CTAs.
struct Cut {
    int threads, groups;
    int64_t ctas;
};
static Cut cut_of(int64_t rows, int64_t cols, bool s8)
{
    Cut c{};
    int64_t most;
    if (cols <= 256) {
        c.threads = kSmallThreads;
        c.groups = kSmallThreads / (cols <= 128 ? 16 : 32);
        most = 152 * 2;
    } else if (cols <= 8192) {
        c.threads = (int)(ceil_div(ceil_div(cols, cols <= 4096 ? 8 : 16), 32) * 32);
        c.groups = 1;
        most = 152 * ((!s8 && cols <= 2560 ? 682 : 512) / c.threads);  // by registers: 96 and 128
    } else {
        c.threads = 1024;
        c.groups = 1;
        most = 152;
    }
    c.ctas = ceil_div(rows, c.groups);
    c.ctas = c.ctas < 1 ? 1 : c.ctas > most ? most : c.ctas;
    return c;
}

template <class H, bool S8, int W>
static int launch_split(const SplitParams &p, const Cut &cut, cudaStream_t stream)
{
    // `most_threads`: of any launch of the kernel
    auto go = [&](auto kernel, int most_threads, int units, int stages) {
        const size_t bytes = W != kApart ? (size_t)stages * units * cut.threads * (S8 ? 48 : 64) : 0;
        if (W != kApart)
            if (const int rc = allow_smem<kernel.value>(stages * units * most_threads * (S8 ? 48 : 64)))
                return rc;
        kernel.value<<<(unsigned)cut.ctas, cut.threads, bytes, stream>>>(p);
        return launch_status();
    };
    if (p.cols <= 128)
        return go(Kernel<split_kernel<H, S8, 1, 1, 16, kSmallThreads, 4, W>>{}, kSmallThreads, 1, 4);
    if (p.cols <= 256)
        return go(Kernel<split_kernel<H, S8, 1, 1, 32, kSmallThreads, 4, W>>{}, kSmallThreads, 1, 4);
    if constexpr (!S8)
        if (p.cols <= 2560)  // 96 registers (32768x1024 fp16 70 us, with 128 77; from checkpoints they spill)
            return go(Kernel<split_kernel<H, S8, 1, 2, 0, 320, 2, W>>{}, 320, 2, 2);
    if (p.cols <= 2048)
        return go(Kernel<split_kernel<H, S8, 1, 2, 0, 256, 3, W>>{}, 256, 2, 3);
    if (p.cols <= 4096)
        return go(Kernel<split_kernel<H, S8, 1, 2, 0, 512, 3, W>>{}, 512, 2, 3);
    if (p.cols <= 8192)
        return go(Kernel<split_kernel<H, S8, 2, 1, 0, 512, 3, W>>{}, 512, 2, 3);
    split_long_kernel<H, S8, W><<<(unsigned)cut.ctas, 1024, 0, stream>>>(p);
    return launch_status();
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

}  // namespace zo

using namespace zo;

extern "C" {

size_t zero_gated_norms_workspace_bytes(int64_t rows, int64_t cols)
{
    if (bad_dim(rows) || bad_dim(cols) || cols < 1)
        return 0;
    // kept halves have the most CTAs
    return (size_t)cut_of(rows, cols, false).ctas * (size_t)(2 * cols + 1) * sizeof(float);
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
    const Cut cut = cut_of(rows, cols, so != nullptr);
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
        p.cols = (int32_t)cols;
        p.scale = scale;
        p.inv_cols = 1.0f / (float)cols;
        p.w_type = w_type;
        const int kb = so ? 1 : b, to = so ? 8 : 16;
        const bool wide = rows_aligned(dy, lddy, b, 16) && (!dh || rows_aligned(dh, lddh, b, 16)) &&
                          rows_aligned(o, ldo, kb, to) && rows_aligned(h, ldh, kb, to) && rows_aligned(d_o, lddo, b, 16) &&
                          rows_aligned(dx, lddx, b, 16) && aligned(w_pre, 16) && aligned(w_post, 16) &&
                          (gate_kind != ZERO_GATE_COLS || aligned(gate, 16));
        auto go = [&](auto half, auto kept) {
            using H = decltype(half);
            constexpr bool S8 = decltype(kept)::value;
            return !wide ? launch_split<H, S8, kApart>(p, cut, stream)
                         : cols % 8 ? launch_split<H, S8, kWide>(p, cut, stream) : launch_split<H, S8, kWhole>(p, cut, stream);
        };
        if (type == ZERO_T_F16)
            rc = so ? go(f16{}, std::true_type{}) : go(f16{}, std::false_type{});
        else
            rc = so ? go(bf16{}, std::true_type{}) : go(bf16{}, std::false_type{});
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
