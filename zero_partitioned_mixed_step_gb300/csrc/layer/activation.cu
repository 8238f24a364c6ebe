// The activation between a feed-forward's products, a = u sig(z(u)) v, in 8 bits,
// and its gradients from 8-bit checkpoints in the forms that the products take.
//
//   silu: z = u;  gelu's tanh form: z = 2 sqrt(2 / pi) (u + 0.044715 u^3)
//   du = da v (sig + u sig (1 - sig) z'),  dv = da u sig
//
// Forward 8192x14336 bf16, gated, three 8-bit forms: 155 us, 5.4 TB/s (0.79 of the copy
// rate; issue slots 73 % busy, ALU 57, DRAM 65).  Backward from checkpoints, du and dv
// in 8 bits along the row and along the tokens, a along the tokens: 301 us, 3.6 TB/s (0.53; issue
// 61 %, ALU 48, DRAM 43), 16 warps to an SM by registers (128).  The transposed forms' values are
// computed twice, once for their scales; conversions and quotients are the larger part of 490
// instructions for 8 elements.  From kept halves 320 us (0.60).
#include <initializer_list>
#include <type_traits>

#include "layer.cuh"

namespace zo {

// sig(z(u)) and z'(u).  exp2 and the reciprocal are approximate to an fp32 unit or two; a
// reciprocal of 2^126 and more is 0.
template <bool GELU>
__device__ __forceinline__ float2 sigmoid_of(float2 u, float2 &dz)
{
    constexpr float kLog2e = 1.4426950408889634f;
    float2 z;
    if (GELU) {
        // beyond 16 the sigmoid is 0 or 1 in fp32; u^3 stays finite (a NaN reaches the result through u)
        const float2 c = make_float2(fminf(fmaxf(u.x, -16.0f), 16.0f), fminf(fmaxf(u.y, -16.0f), 16.0f));
        constexpr float k = 1.5957691216057308f;
        const float2 c2 = mul2(c, c);
        dz = fma2(both(k * 3.0f * 0.044715f), c2, both(k));
        z = mul2(mul2(both(-kLog2e), c), fma2(both(k * 0.044715f), c2, both(k)));
    } else {
        dz = both(1.0f);
        z = mul2(both(-kLog2e), u);
    }
    float2 e, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.x) : "f"(z.x));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.y) : "f"(z.y));
    e = add2(e, both(1.0f));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.x) : "f"(e.x));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.y) : "f"(e.y));
    return r;
}

// ------------------------------------------------------------------ forward

struct ActParams {
    const void *u, *v;
    void *a;
    Form a8, u8, v8;
    int64_t ldu, ldv, lda;
    int32_t rows, cols;
    Tiles tiles;
    int32_t e5m2;
};

constexpr int kActRows = 32;  // rows of a CTA: two to each 16 lanes

// A tile is 128 columns of 32 neighbouring rows, whose scales lie side by side.  CTAs walk the
// tiles with the next one on its way to the registers.
template <class H, bool GELU, int W>
__global__ void __launch_bounds__(256, 3) act_kernel(const ActParams p)
{
    const int lane = threadIdx.x & 15, group = threadIdx.x >> 4;
    const uint32_t across = p.tiles.cols, tiles = p.tiles.rows * across;
    Raw8<H> u_next[2], v_next[2];
    auto fetch = [&](uint32_t tile) {
        const int64_t row = (int64_t)(tile / across) * kActRows + group * 2;
        const int c = (int)(tile % across) * kBlock + lane * 8, nc = tile < tiles ? left_of(p.cols, c) : 0;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int n = row + k < p.rows ? nc : 0;
            u_next[k] = get_raw<W>(static_cast<const H *>(p.u) + (row + k) * p.ldu + c, n);
            if (p.v)
                v_next[k] = get_raw<W>(static_cast<const H *>(p.v) + (row + k) * p.ldv + c, n);
        }
    };
    fetch(blockIdx.x);
    for (uint32_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
        const Raw8<H> u[2] = {u_next[0], u_next[1]}, v[2] = {v_next[0], v_next[1]};
        fetch(tile + gridDim.x);
        const int64_t tc = tile % across, row = (int64_t)(tile / across) * kActRows + group * 2;
        const int c = (int)tc * kBlock + lane * 8, nc = left_of(p.cols, c);
        const int n[2] = {row < p.rows ? nc : 0, row + 1 < p.rows ? nc : 0};
        // the scale that a lane writes of N values, two rows of each form
        auto put_scale = [&](const Form &f, int mine, int every, float s) {
            const int64_t r = row + (mine & 1);
            if (lane % every == 0 && f.q && r < p.rows)
                f.s[tc * f.lds + r] = s;
        };
        auto put_kept = [&](const Form &f, const Raw8<H> &r, int k, Inverse d) {
            float2 x[4];
            pairs_of(r, x);
            if (f.q && n[k] > 0)
                put_bytes<W>(f.q + (row + k) * f.ld + c, n[k], bytes_of<false>(x, d));
        };
        if (p.v && (p.u8.q || p.v8.q)) {
            uint32_t most[4] = {amax8(u[0]), amax8(u[1]), amax8(v[0]), amax8(v[1])};
            const float s = scale_of<false>(max_shared(most));
            const Inverse inv = inverse_of(s);
            const int mine = shared_index<4>();
            put_scale(mine < 2 ? p.u8 : p.v8, mine, 4, s);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const Inverse d = shared_value<4>(inv, k);
                put_kept(k < 2 ? p.u8 : p.v8, k < 2 ? u[k & 1] : v[k & 1], k & 1, d);
            }
        } else if (p.u8.q) {
            uint32_t most[2] = {amax8(u[0]), amax8(u[1])};
            const float s = scale_of<false>(max_shared(most));
            const Inverse inv = inverse_of(s);
            put_scale(p.u8, shared_index<2>(), 8, s);
#pragma unroll
            for (int k = 0; k < 2; ++k)
                put_kept(p.u8, u[k], k, shared_value<2>(inv, k));
        }
        float2 a[2][4];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            float2 x[4], dz;
            pairs_of(u[k], x);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                a[k][i] = mul2(x[i], sigmoid_of<GELU>(x[i], dz));
            if (p.v) {
                pairs_of(v[k], x);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    a[k][i] = mul2(a[k][i], x[i]);
            }
            if (p.a && n[k] > 0)
                put_pairs<W>(static_cast<H *>(p.a) + (row + k) * p.lda + c, n[k], a[k]);
        }
        if (!p.a8.q)
            continue;
        auto put_a8 = [&](auto e5m2) {
            constexpr bool E = decltype(e5m2)::value;
            uint32_t most[2] = {amax8(a[0]), amax8(a[1])};
            const float s = scale_of<E>(max_shared(most));
            const Inverse inv = inverse_of(s);
            put_scale(p.a8, shared_index<2>(), 8, s);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const Inverse d = shared_value<2>(inv, k);
                if (n[k] > 0)
                    put_bytes<W>(p.a8.q + (row + k) * p.a8.ld + c, n[k], bytes_of<E>(a[k], d));
            }
        };
        if (p.e5m2)
            put_a8(std::true_type{});
        else
            put_a8(std::false_type{});
    }
}

// ------------------------------------------------------------------ backward

struct ActBackParams {
    const void *da, *u, *v;
    const float *su, *sv;
    void *du, *dv;
    Form du8, dv8, du8t, dv8t, a8t;
    int64_t ldda, ldu, ldv, ldsu, ldsv, lddu, lddv;
    int32_t rows, cols;
    Tiles tiles;
    int32_t e5m2;
};

constexpr int kBackThreads = 256;  // 16 groups of 16 lanes, 8 rows to a group

// du, dv and a of two elements (dv without v: 0).
struct Slopes {
    float2 du, dv, a;
};
template <bool GATED, bool GELU>
__device__ __forceinline__ Slopes slopes_of(float2 da, float2 u, float2 v)
{
    float2 dz;
    const float2 sig = sigmoid_of<GELU>(u, dz), act = mul2(u, sig);
    const float2 rest = fma2(sig, both(-1.0f), both(1.0f));
    const float2 slope = fma2(act, GELU ? mul2(rest, dz) : rest, sig);
    if (GATED)
        return {mul2(mul2(da, v), slope), mul2(da, act), mul2(act, v)};
    return {mul2(da, slope), both(0.0f), act};
}

// The inputs of a 128x128 tile as they came.  The transposed forms' scales are known only when the whole
// tile is, so its columns are computed again from these, by the same operations and so to the same
// bits: held as values, three forms take 98 KB as bf16, which is a rounding that turns over one in a hundred
// of their bytes, and 197 KB as fp32.  A row's 128 elements are 16 units of 8.  Unit j of a row of
// group g (rows 8g ..) lies at j ^ g, units of halves at j ^ (g % 8).  So 16 lanes that read one
// part of 16 groups' units, lanes from 8 on the other part of halves, and those that write a row's units meet
// different banks.
template <class H, bool S8>
struct Staged {
    using Unit = std::conditional_t<S8, uint2, uint4>;
    uint4 da[kBlock][16];
    Unit u[kBlock][16], v[kBlock][16];  // v: not there without a gate
    static constexpr int bytes(bool gated) { return (int)(sizeof(Staged) - (gated ? 0 : sizeof(Unit) * kBlock * 16)); }
};
__device__ __forceinline__ void stage8(uint4 (&t)[kBlock][16], int group, int i, int j, const uint32_t (&w)[4])
{
    t[group * 8 + i][j ^ (group & 7)] = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void stage8(uint2 (&t)[kBlock][16], int group, int i, int j, const uint32_t (&w)[2])
{
    t[group * 8 + i][j ^ group] = make_uint2(w[0], w[1]);
}
// Columns 8k + 4part .. + 3 of 8 rows: row i's 4 elements.
__device__ __forceinline__ void staged4(const uint4 (&t)[kBlock][16], int lane, int k, int part, uint2 (&w)[8])
{
#pragma unroll
    for (int i = 0; i < 8; ++i)
        w[i] = reinterpret_cast<const uint2 *>(&t[lane * 8 + i][k ^ (lane & 7)])[part];
}
__device__ __forceinline__ void staged4(const uint2 (&t)[kBlock][16], int lane, int k, int part, uint32_t (&w)[8])
{
#pragma unroll
    for (int i = 0; i < 8; ++i)
        w[i] = reinterpret_cast<const uint32_t *>(&t[lane * 8 + i][k ^ lane])[part];
}
// Element m of two rows' 4.
template <class H>
__device__ __forceinline__ float2 down(uint2 a, uint2 b, int m)
{
    return pair_of<H>(__byte_perm(m & 2 ? a.y : a.x, m & 2 ? b.y : b.x, m & 1 ? 0x7632 : 0x5410));
}
template <class H>
__device__ __forceinline__ float2 down(uint32_t a, uint32_t b, int m)
{
    return two_of<ZERO_T_E4M3>(__byte_perm(a, b, m | (m + 4) << 4) & 0xFFFFu);
}

// What a tile's columns need of its rows.
struct TileNumbers {
    uint32_t amax[3][kBlock];  // of the columns of du, a and dv
    Inverse inverse[3][kBlock];
    float2 scale[2][kBlock / 2];  // of u's and v's rows, two at a time
};

// A 128x128 tile: rows first, two at a time with the next two on their way (gradients, their
// 8-bit forms along the row, the columns' largest magnitudes), then, if a transposed form is wanted,
// columns.
template <class H, bool S8, bool GATED, bool GELU, int W>
__device__ __forceinline__ void act_backward_tile(const ActBackParams &p, const TileAt at, Staged<H, S8> &tile, TileNumbers &numbers)
{
    using K = Kept<H, S8>;
    constexpr int kElem = K::kBytes / 8, kForms = GATED ? 3 : 2, kMaxima = GATED ? 4 : 2;
    auto &amax = numbers.amax;
    auto &inverse = numbers.inverse;
    const bool trans = p.du8t.q || p.dv8t.q || p.a8t.q;
    const int j = threadIdx.x & 15, group = threadIdx.x >> 4;
    const int64_t tc = at.c, r0 = (int64_t)at.r * kBlock, c0 = tc * kBlock, first = r0 + group * 8;
    const int c = at.c * kBlock + j * 8, nc = left_of(p.cols, c);
    if (trans) {
        for (int i = threadIdx.x; i < kForms * kBlock; i += kBackThreads)
            (&amax[0][0])[i] = 0;
        __syncthreads();
    }
    Raw8<H> da[2];
    K u[2], v[2];
    float su[2], sv[2];
    // pointers move on by two rows at a time
    const H *f_da = static_cast<const H *>(p.da) + first * p.ldda;
    const unsigned char *f_u = static_cast<const unsigned char *>(p.u) + first * p.ldu * kElem;
    const unsigned char *f_v = static_cast<const unsigned char *>(p.v) + first * p.ldv * kElem;
    const float *f_su = p.su + tc * p.ldsu + first, *f_sv = p.sv + tc * p.ldsv + first;
    const int left = (int)min((int64_t)8, max((int64_t)0, p.rows - first));  // of this group's 8 rows
    auto fetch = [&](int step) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int n = step + i < left ? nc : 0;
            da[i] = get_raw<W>(f_da + c, n);
            u[i].template load<W>(f_u, c, n);
            su[i] = sv[i] = 1.0f;
            if (S8 && n > 0)
                su[i] = f_su[step + i];
            if (GATED) {
                v[i].template load<W>(f_v, c, n);
                if (S8 && n > 0)
                    sv[i] = f_sv[step + i];
            }
            f_da += p.ldda;
            f_u += p.ldu * kElem;
            f_v += p.ldv * kElem;
        }
    };
    H *to_du = static_cast<H *>(p.du) + first * p.lddu + c, *to_dv = static_cast<H *>(p.dv) + first * p.lddv + c;
    uint8_t *to_du8 = p.du8.q + first * p.du8.ld + c, *to_dv8 = p.dv8.q + first * p.dv8.ld + c;
    // a scale that this lane writes, of row (j / (16 / kMaxima)) % 2 of two
    const int mine = shared_index<kMaxima>();
    const bool second = mine >= 2;
    const bool writes = j % (16 / kMaxima) == 0 && (second ? p.dv8.q : p.du8.q);
    float *to_s = (second ? p.dv8.s + tc * p.dv8.lds : p.du8.s + tc * p.du8.lds) + first + (mine & 1);
    fetch(0);
    const Range range(p.e5m2);
    float most[kForms][8] = {};
#pragma unroll 1
    for (int step = 0; step < 8; step += 2) {
        float2 g[2][4], uf[2][4], vf[2][4], du[2][4], dv[2][4], a[2][4];
        const int n[2] = {step < left ? nc : 0, step + 1 < left ? nc : 0};
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            pairs_of(da[i], g[i]);
            u[i].get(uf[i]);
            if (GATED)
                v[i].get(vf[i]);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if (S8)
                    uf[i][k] = mul2(uf[i][k], both(su[i]));
                if (S8 && GATED)
                    vf[i][k] = mul2(vf[i][k], both(sv[i]));
            }
            if (S8) {
                end_unit<W>(uf[i], n[i], su[i]);
                if (GATED)
                    end_unit<W>(vf[i], n[i], sv[i]);
            }
        }
        if (trans)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                stage8(tile.da, group, step + i, j, da[i].w);
                stage8(tile.u, group, step + i, j, u[i].r.w);
                if (GATED)
                    stage8(tile.v, group, step + i, j, v[i].r.w);
                if (S8 && j == 0) {
                    reinterpret_cast<float *>(numbers.scale[0])[group * 8 + step + i] = su[i];
                    reinterpret_cast<float *>(numbers.scale[1])[group * 8 + step + i] = sv[i];
                }
            }
        if (step < 6)
            fetch(step + 2);
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const Slopes d = slopes_of<GATED, GELU>(g[i][k], uf[i][k], vf[i][k]);
                du[i][k] = d.du;
                dv[i][k] = d.dv;
                a[i][k] = d.a;
            }
        if (trans) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                most[0][2 * k] = max3(most[0][2 * k], du[0][k].x, du[1][k].x);
                most[0][2 * k + 1] = max3(most[0][2 * k + 1], du[0][k].y, du[1][k].y);
                most[1][2 * k] = max3(most[1][2 * k], a[0][k].x, a[1][k].x);
                most[1][2 * k + 1] = max3(most[1][2 * k + 1], a[0][k].y, a[1][k].y);
                if (GATED) {
                    most[kForms - 1][2 * k] = max3(most[kForms - 1][2 * k], dv[0][k].x, dv[1][k].x);
                    most[kForms - 1][2 * k + 1] = max3(most[kForms - 1][2 * k + 1], dv[0][k].y, dv[1][k].y);
                }
            }
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            if (p.du && n[i] > 0)
                put_pairs<W>(to_du + i * p.lddu, n[i], du[i]);
            if (GATED && p.dv && n[i] > 0)
                put_pairs<W>(to_dv + i * p.lddv, n[i], dv[i]);
        }
        to_du += 2 * p.lddu;
        to_dv += 2 * p.lddv;
        if (p.du8.q || (GATED && p.dv8.q)) {
            uint32_t m[kMaxima];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                m[i] = amax8(du[i]);
                if (GATED)
                    m[kMaxima - 2 + i] = amax8(dv[i]);
            }
            const float s = range.scale(max_shared(m));
            const Inverse inv = inverse_of(s);
            if (writes && step + (mine & 1) < left)
                to_s[step] = s;
            auto put = [&](auto e5m2) {
                constexpr bool E = decltype(e5m2)::value;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const Inverse d0 = shared_value<kMaxima>(inv, i), d1 = shared_value<kMaxima>(inv, kMaxima - 2 + i);
                    if (p.du8.q && n[i] > 0)
                        put_bytes<W>(to_du8 + i * p.du8.ld, n[i], bytes_of<E>(du[i], d0));
                    if (GATED && p.dv8.q && n[i] > 0)
                        put_bytes<W>(to_dv8 + i * p.dv8.ld, n[i], bytes_of<E>(dv[i], d1));
                }
            };
            if (p.e5m2)
                put(std::true_type{});
            else
                put(std::false_type{});
            to_du8 += 2 * p.du8.ld;
            to_dv8 += 2 * p.dv8.ld;
        }
    }
    if (!trans)
        return;
#pragma unroll
    for (int f = 0; f < kForms; ++f)
#pragma unroll
        for (int k = 0; k < 8; ++k)
            atomicMax(&amax[f][j * 8 + k], __float_as_uint(most[f][k]));  // a maximum: in any order the same
    __syncthreads();
    // A group takes 8 columns from `group * 8` on, 8 rows to a lane; it forms their scales first.
    const int k0 = group * 8, wide_k = p.cols - (int)c0;
    for (int i = j; i < kForms * 8; i += 16) {
        const int f = i >> 3, at_k = k0 + (i & 7);
        const Form &to = f == 0 ? p.du8t : f == 1 ? p.a8t : p.dv8t;
        const float s = (f == 1 ? Range(false) : range).scale(amax[f][at_k]);
        inverse[f][at_k] = inverse_of(s);
        if (to.q && at_k < wide_k)
            to.s[r0 / kBlock * to.lds + c0 + at_k] = s;
    }
    __syncwarp();
    const int64_t row = r0 + j * 8;
    const int nr = row < p.rows ? left_of(p.rows, (int)row) : 0;
    float2 fu[4], fv[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (S8) {
            fu[i] = numbers.scale[0][j * 4 + i];
            fv[i] = numbers.scale[1][j * 4 + i];
        }
    auto columns = [&](auto e5m2) {
        constexpr bool E = decltype(e5m2)::value;
        using Part = std::conditional_t<S8, uint32_t, uint2>;
#pragma unroll 1
        for (int half = 0; half < 2; ++half) {
            const int part = half ^ (j >> 3), first_k = k0 + part * 4;
            uint8_t *to_du = p.du8t.q + (c0 + first_k) * p.du8t.ld + row, *to_a = p.a8t.q + (c0 + first_k) * p.a8t.ld + row;
            uint8_t *to_dv = p.dv8t.q + (c0 + first_k) * p.dv8t.ld + row;
            uint2 wd[8];
            Part wu[8], wv[8];
            staged4(tile.da, j, group, part, wd);
            staged4(tile.u, j, group, part, wu);
            if (GATED)
                staged4(tile.v, j, group, part, wv);
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                float2 du[4], dv[4], a[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float2 x = down<H>(wu[2 * i], wu[2 * i + 1], m), y = both(0.0f);
                    if (GATED)
                        y = down<H>(wv[2 * i], wv[2 * i + 1], m);
                    if (S8) {
                        x = mul2(x, fu[i]);
                        if (GATED)
                            y = mul2(y, fv[i]);
                    }
                    const Slopes d = slopes_of<GATED, GELU>(down<H>(wd[2 * i], wd[2 * i + 1], m), x, y);
                    du[i] = d.du;
                    dv[i] = d.dv;
                    a[i] = d.a;
                }
                const int at_k = first_k + m;
                if (nr > 0 && at_k < wide_k) {
                    if (p.du8t.q)
                        put_bytes<W>(to_du, nr, bytes_of<E>(du, inverse[0][at_k]));
                    if (p.a8t.q)
                        put_bytes<W>(to_a, nr, bytes_of<false>(a, inverse[1][at_k]));
                    if (GATED && p.dv8t.q)
                        put_bytes<W>(to_dv, nr, bytes_of<E>(dv, inverse[kForms - 1][at_k]));
                }
                to_du += p.du8t.ld;
                to_a += p.a8t.ld;
                to_dv += p.dv8t.ld;
            }
        }
    };
    if (p.e5m2)
        columns(std::true_type{});
    else
        columns(std::false_type{});
}

// Where 8 does not divide the rows or the columns, each tile is asked whether it has a short unit to reckon
// with, as only those at the ends do: 8191x14336 takes about what 8192x14336 does, and a third more where
// the call decides.
template <class H, bool S8, bool GATED, bool GELU, int W>
__global__ void __launch_bounds__(kBackThreads, 2) act_backward_kernel(const ActBackParams p)
{
    extern __shared__ __align__(16) unsigned char dynamic[];
    Staged<H, S8> &tile = *reinterpret_cast<Staged<H, S8> *>(dynamic);
    __shared__ TileNumbers numbers;
    const TileAt at = tile_at(p.tiles);
    if (W == kWide && whole_units(at, p.rows, p.cols))
        act_backward_tile<H, S8, GATED, GELU, kWhole>(p, at, tile, numbers);
    else
        act_backward_tile<H, S8, GATED, GELU, W>(p, at, tile, numbers);
}

template <class H, bool S8, bool GATED, bool GELU, int W>
static int launch_act_backward(const ActBackParams &p, int64_t grid, cudaStream_t stream)
{
    const bool trans = p.du8t.q || p.dv8t.q || p.a8t.q;
    const int bytes = trans ? Staged<H, S8>::bytes(GATED) : 0;
    constexpr auto kernel = act_backward_kernel<H, S8, GATED, GELU, W>;
    if (const int rc = allow_smem<kernel>(Staged<H, S8>::bytes(GATED)))
        return rc;
    kernel<<<(unsigned)grid, kBackThreads, bytes, stream>>>(p);
    return launch_status();
}

template <class H, bool S8, int W>
static int choose_act_backward(const ActBackParams &p, bool gelu, int64_t grid, cudaStream_t stream)
{
    if (p.v)
        return gelu ? launch_act_backward<H, S8, true, true, W>(p, grid, stream)
                    : launch_act_backward<H, S8, true, false, W>(p, grid, stream);
    return gelu ? launch_act_backward<H, S8, false, true, W>(p, grid, stream)
                : launch_act_backward<H, S8, false, false, W>(p, grid, stream);
}

}  // namespace zo

using namespace zo;

extern "C" {

int zero_activation_fp8(const void *u, int64_t ldu, const void *v, int64_t ldv, int act, int type, int64_t rows,
                        int64_t cols, void *a, int64_t lda, int fp8, const zero_fp8_form *a8,
                        const zero_fp8_form *u8, const zero_fp8_form *v8, zero_stream_t stream)
{
    if (!is_half(type) || bad_dim(rows) || bad_dim(cols) || (act != ZERO_ACT_SILU && act != ZERO_ACT_GELU) ||
        (a8 && !is_fp8(fp8)) || (v8 && !v))
        return ZERO_EINVAL;
    if (rows == 0 || cols == 0)
        return ZERO_OK;
    if (!a && !a8 && !u8 && !v8)
        return ZERO_EINVAL;
    const int b = type_bytes(type);
    int rc = check_matrix(u, rows, cols, ldu, b);
    if (!rc && v)
        rc = check_matrix(v, rows, cols, ldv, b);
    if (!rc && a)
        rc = check_matrix(a, rows, cols, lda, b);
    for (const zero_fp8_form *f : {a8, u8, v8})
        if (!rc)
            rc = check_form(f, rows, cols);
    if (rc)
        return rc;
    ActParams p{};
    p.u = u;
    p.v = v;
    p.a = a;
    p.a8 = form_of(a8);
    p.u8 = form_of(u8);
    p.v8 = form_of(v8);
    p.ldu = ldu;
    p.ldv = ldv;
    p.lda = lda;
    p.rows = (int32_t)rows;
    p.cols = (int32_t)cols;
    p.tiles = tiles_of(rows, cols, kActRows);
    bool wide = rows_aligned(u, ldu, b, 16) && (!v || rows_aligned(v, ldv, b, 16)) && (!a || rows_aligned(a, lda, b, 16));
    for (const Form *f : {&p.a8, &p.u8, &p.v8})
        wide = wide && (!f->q || f->wide);
    p.e5m2 = a8 && fp8 == ZERO_T_E5M2;
    const int64_t tiles = (int64_t)p.tiles.rows * p.tiles.cols, most = 152 * 3;  // three CTAs to an SM
    if (tiles > kMaxDim)
        return ZERO_EINVAL;
    auto go = [&](auto kernel) {
        kernel<<<(unsigned)(tiles < most ? tiles : most), 256, 0, stream>>>(p);
        return launch_status();
    };
    auto by_type = [&](auto half) {
        using H = decltype(half);
        auto by_act = [&](auto gelu) {
            constexpr bool G = decltype(gelu)::value;
            return !wide ? go(act_kernel<H, G, kApart>)
                         : cols % 8 ? go(act_kernel<H, G, kWide>) : go(act_kernel<H, G, kWhole>);
        };
        return act == ZERO_ACT_GELU ? by_act(std::true_type{}) : by_act(std::false_type{});
    };
    return type == ZERO_T_F16 ? by_type(f16{}) : by_type(bf16{});
}

int zero_activation_backward_fp8(const void *da, int64_t ldda, const void *u, int64_t ldu, const float *su,
                                 int64_t ldsu, const void *v, int64_t ldv, const float *sv, int64_t ldsv, int act,
                                 int type, int64_t rows, int64_t cols, void *du, int64_t lddu, void *dv,
                                 int64_t lddv, int fp8, const zero_fp8_form *du8, const zero_fp8_form *dv8,
                                 const zero_fp8_form *du8t, const zero_fp8_form *dv8t, const zero_fp8_form *a8t,
                                 zero_stream_t stream)
{
    if (!is_half(type) || bad_dim(rows) || bad_dim(cols) || (act != ZERO_ACT_SILU && act != ZERO_ACT_GELU) ||
        (!v && (dv || dv8 || dv8t || sv)) || (v && !su != !sv) || ((du8 || dv8 || du8t || dv8t) && !is_fp8(fp8)))
        return ZERO_EINVAL;
    if (rows == 0 || cols == 0)
        return ZERO_OK;
    if (!du && !dv && !du8 && !dv8 && !du8t && !dv8t && !a8t)
        return ZERO_EINVAL;
    const int b = type_bytes(type);
    int rc = check_matrix(da, rows, cols, ldda, b);
    if (!rc)
        rc = check_kept(u, ldu, su, ldsu, type, rows, cols);
    if (!rc && v)
        rc = check_kept(v, ldv, sv, ldsv, type, rows, cols);
    if (!rc && du)
        rc = check_matrix(du, rows, cols, lddu, b);
    if (!rc && dv)
        rc = check_matrix(dv, rows, cols, lddv, b);
    for (const zero_fp8_form *f : {du8, dv8})
        if (!rc)
            rc = check_form(f, rows, cols);
    for (const zero_fp8_form *f : {du8t, dv8t, a8t})
        if (!rc)
            rc = check_form(f, cols, rows);
    if (rc)
        return rc;
    ActBackParams p{};
    p.da = da;
    p.u = u;
    p.v = v;
    p.su = su;
    p.sv = sv;
    p.du = du;
    p.dv = dv;
    p.du8 = form_of(du8);
    p.dv8 = form_of(dv8);
    p.du8t = form_of(du8t);
    p.dv8t = form_of(dv8t);
    p.a8t = form_of(a8t);
    p.ldda = ldda;
    p.ldu = ldu;
    p.ldv = ldv;
    p.ldsu = ldsu;
    p.ldsv = ldsv;
    p.lddu = lddu;
    p.lddv = lddv;
    p.rows = (int32_t)rows;
    p.cols = (int32_t)cols;
    p.tiles = tiles_of(rows, cols, kBlock);
    const int kb = su ? 1 : b, to = su ? 8 : 16;
    bool wide = rows_aligned(da, ldda, b, 16) && (!du || rows_aligned(du, lddu, b, 16)) &&
                (!dv || rows_aligned(dv, lddv, b, 16)) && rows_aligned(u, ldu, kb, to) &&
                (!v || rows_aligned(v, ldv, kb, to));
    for (const Form *f : {&p.du8, &p.dv8, &p.du8t, &p.dv8t, &p.a8t})
        wide = wide && (!f->q || f->wide);
    p.e5m2 = fp8 == ZERO_T_E5M2;
    const int64_t grid = (int64_t)p.tiles.rows * p.tiles.cols;
    if (grid > kMaxDim)
        return ZERO_EINVAL;
    const bool gelu = act == ZERO_ACT_GELU;
    auto go = [&](auto half, auto kept) {
        using H = decltype(half);
        constexpr bool S8 = decltype(kept)::value;
        return !wide ? choose_act_backward<H, S8, kApart>(p, gelu, grid, stream)
                     : cols % 8 || rows % 8 ? choose_act_backward<H, S8, kWide>(p, gelu, grid, stream)
                                            : choose_act_backward<H, S8, kWhole>(p, gelu, grid, stream);
    };
    if (type == ZERO_T_F16)
        return su ? go(f16{}, std::true_type{}) : go(f16{}, std::false_type{});
    return su ? go(bf16{}, std::true_type{}) : go(bf16{}, std::false_type{});
}

}  // extern "C"
