// The activation between a feed-forward's products, a = u sig(z(u)) v, in 8 bits,
// and its gradients from 8-bit checkpoints in the forms that the products take.
//
//   silu: z = u;  gelu's tanh form: z = 2 sqrt(2 / pi) (u + 0.044715 u^3)
//   du = da v (sig + u sig (1 - sig) z'),  dv = da u sig
#include <initializer_list>

#include "layer.cuh"

namespace zo {

// sig(z(u)) and z'(u).  exp and the quotient are approximate to a few fp32 units; a
// quotient by 2^126 and more is 0.
template <bool GELU>
__device__ __forceinline__ float sigmoid_of(float u, float &dz)
{
    float z = u;
    dz = 1.0f;
    if (GELU) {
        // beyond 16 the sigmoid is 0 or 1 in fp32; u^3 stays finite (a NaN reaches the result through u)
        const float c = fminf(fmaxf(u, -16.0f), 16.0f), k = 1.5957691216057308f, c2 = c * c;
        z = k * c * fmaf(0.044715f, c2, 1.0f);
        dz = k * fmaf(3.0f * 0.044715f, c2, 1.0f);
    }
    return __fdividef(1.0f, 1.0f + __expf(-z));
}

// ------------------------------------------------------------------ forward

struct ActParams {
    const void *u, *v;
    void *a;
    Form a8, u8, v8;
    int64_t ldu, ldv, lda, rows, cols;
    int64_t row_tiles;
    int32_t wide, e5m2;
};

template <class H>
__device__ __forceinline__ void put_kept(const Form &f, int64_t row, int64_t c, int n, const Raw8<H> &r)
{
    Amax<H> a;
    float x[8];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        a.add(r.w[i]);
#pragma unroll
    for (int i = 0; i < 8; ++i)
        x[i] = r.at(i);
    put_form(f, row, c, n, x, a.bits(), false);
}

constexpr int kActRows = 32;  // rows of a CTA: two to each 16 lanes

// A CTA takes 128 columns of 32 neighbouring rows, whose scales lie side by side.
template <class H, bool GELU>
__global__ void __launch_bounds__(256) act_kernel(const ActParams p)
{
    const int64_t c = blockIdx.x / p.row_tiles * kBlock + (threadIdx.x & 15) * 8;
    const int64_t r0 = blockIdx.x % p.row_tiles * kActRows + (threadIdx.x >> 4);
    const int nc = in_row(p.cols, c);
    Raw8<H> u[2], v[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const int64_t row = r0 + 16 * k;
        const int n = row < p.rows ? nc : 0;
        u[k] = load_raw(static_cast<const H *>(p.u) + row * p.ldu + c, n, p.wide);
        if (p.v)
            v[k] = load_raw(static_cast<const H *>(p.v) + row * p.ldv + c, n, p.wide);
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const int64_t row = r0 + 16 * k;
        const int n = row < p.rows ? nc : 0;
        float a[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float dz;
            a[i] = u[k].at(i) * sigmoid_of<GELU>(u[k].at(i), dz);
            if (p.v)
                a[i] *= v[k].at(i);
        }
        if (p.a && n > 0)
            store8(static_cast<H *>(p.a) + row * p.lda + c, n, p.wide, a);
        if (p.a8.q)
            put_form(p.a8, row, c, n, a, amax8(a), p.e5m2);
        if (p.u8.q)
            put_kept(p.u8, row, c, n, u[k]);
        if (p.v8.q)
            put_kept(p.v8, row, c, n, v[k]);
    }
}

// ------------------------------------------------------------------ backward

struct ActBackParams {
    const void *da, *u, *v;
    const float *su, *sv;
    void *du, *dv;
    Form du8, dv8, du8t, dv8t, a8t;
    int64_t ldda, ldu, ldv, ldsu, ldsv, lddu, lddv, rows, cols;
    int64_t row_tiles;
    int32_t wide, wide_kept, e5m2;
};

constexpr int kBackThreads = 512;  // 32 groups of 16 lanes, 4 rows to a group

// bf16 values of the 128x128 tile on their way to the transposed forms: a row's 128
// values are 16 units of 8; unit j of row r lies at j ^ (r / 16), its halves
// exchanged where r / 8 is odd.  So 4 neighbouring columns c = 4k .. of row r are the
// 8 bytes at place k ^ (r / 8): the 16 lanes of a column (8 rows each) read
// different banks, and so do the 16 lanes of a row as they write.
struct Staged {
    uint2 row[kBlock][32];
};
__device__ __forceinline__ void stage8(Staged &t, int r, int j, const float x[8])
{
    const uint2 lo = make_uint2(word_of<bf16>(x[0], x[1]), word_of<bf16>(x[2], x[3]));
    const uint2 hi = make_uint2(word_of<bf16>(x[4], x[5]), word_of<bf16>(x[6], x[7]));
    const bool turned = r >> 3 & 1;
    const uint2 a = turned ? hi : lo, b = turned ? lo : hi;
    *reinterpret_cast<uint4 *>(&t.row[r][2 * (j ^ r >> 4)]) = make_uint4(a.x, a.y, b.x, b.y);
}

// Four columns (from 4k on) of a tile, 8 rows to each of 16 lanes, into a transposed
// form.  amax: of the tile's columns, of the fp32 values.
__device__ __forceinline__ void put_columns(const Form &f, const Staged &t, const uint32_t *amax, int k, int64_t c0,
                                            int64_t cols, int64_t r0, int64_t rows, bool e5m2)
{
    const int lane = threadIdx.x & 15;
    uint2 w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
        w[i] = t.row[lane * 8 + i][k ^ lane];
    // each lane forms one of the four scales
    const float s = scale_of(amax[4 * k + (lane & 3)], e5m2);
    const Inverse mine = inverse(s);
    const int64_t c = c0 + 4 * k;
    if (lane < 4 && c + lane < cols)
        f.s[r0 / kBlock * f.lds + c + lane] = s;
    const int64_t row = r0 + lane * 8;
    const int n = in_row(rows, row);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const Inverse d = {__shfl_sync(0xFFFFFFFFu, mine.hi, j, 16), __shfl_sync(0xFFFFFFFFu, mine.lo, j, 16)};
        float x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t two = j < 2 ? w[i].x : w[i].y;
            x[i] = __uint_as_float(j & 1 ? two & 0xFFFF0000u : two << 16);
        }
        const uint2 q = quotients_of(x, d, e5m2);
        if (n > 0 && c + j < cols)
            store8b(f.q + (c + j) * f.ld + row, n, f.wide, q);
    }
}

// A CTA takes a 128x128 tile: rows first (gradients, their 8-bit forms along the row,
// the columns' largest magnitudes), then, if a transposed form is wanted, columns.
template <class H, bool S8, bool GATED, bool GELU>
__global__ void __launch_bounds__(kBackThreads, 1) act_backward_kernel(const ActBackParams p)
{
    using K = Kept<H, S8>;
    constexpr int kRows = kBlock * 16 / kBackThreads;
    extern __shared__ __align__(16) unsigned char dynamic[];
    Staged *tile = reinterpret_cast<Staged *>(dynamic);  // du, a and dv
    __shared__ uint32_t amax[3][kBlock];
    const bool trans = p.du8t.q || p.dv8t.q || p.a8t.q;
    const int j = threadIdx.x & 15, group = threadIdx.x >> 4;
    const int64_t tr = blockIdx.x % p.row_tiles, tc = blockIdx.x / p.row_tiles;
    const int64_t r0 = tr * kBlock, c0 = tc * kBlock, c = c0 + j * 8;
    const int nc = in_row(p.cols, c);
    if (trans) {
        for (int i = threadIdx.x; i < 3 * kBlock; i += kBackThreads)
            (&amax[0][0])[i] = 0;
        __syncthreads();
    }
    Raw8<H> da[kRows];
    K u[kRows], v[kRows];
    float su[kRows], sv[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        const int64_t row = r0 + group * kRows + i;
        const int n = row < p.rows ? nc : 0;
        da[i] = load_raw(static_cast<const H *>(p.da) + row * p.ldda + c, n, p.wide);
        u[i].load(p.u, row * p.ldu + c, n, p.wide_kept);
        su[i] = S8 && n > 0 ? p.su[tc * p.ldsu + row] : 1.0f;
        if (GATED) {
            v[i].load(p.v, row * p.ldv + c, n, p.wide_kept);
            sv[i] = S8 && n > 0 ? p.sv[tc * p.ldsv + row] : 1.0f;
        }
    }
    uint32_t most[GATED ? 3 : 2][8] = {};
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        const int r = group * kRows + i;
        const int64_t row = r0 + r;
        const int n = row < p.rows ? nc : 0;
        float uf[8], vf[8], du[8], dv[8], a[8];
        u[i].get(uf, su[i]);
        if (GATED)
            v[i].get(vf, sv[i]);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            float dz;
            const float sig = sigmoid_of<GELU>(uf[k], dz), act = uf[k] * sig, g = da[i].at(k);
            const float slope = fmaf(act * (1.0f - sig), dz, sig);
            if (GATED) {
                du[k] = g * vf[k] * slope;
                dv[k] = g * act;
                a[k] = act * vf[k];
            } else {
                du[k] = g * slope;
                a[k] = act;
            }
        }
        if (p.du && n > 0)
            store8(static_cast<H *>(p.du) + row * p.lddu + c, n, p.wide, du);
        if (p.du8.q)
            put_form(p.du8, row, c, n, du, amax8(du), p.e5m2);
        if (GATED && p.dv && n > 0)
            store8(static_cast<H *>(p.dv) + row * p.lddv + c, n, p.wide, dv);
        if (GATED && p.dv8.q)
            put_form(p.dv8, row, c, n, dv, amax8(dv), p.e5m2);
        if (trans) {
            stage8(tile[0], r, j, du);
            stage8(tile[1], r, j, a);
            if (GATED)
                stage8(tile[2], r, j, dv);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                most[0][k] = max(most[0][k], magnitude(du[k]));
                most[1][k] = max(most[1][k], magnitude(a[k]));
                if (GATED)
                    most[GATED ? 2 : 0][k] = max(most[GATED ? 2 : 0][k], magnitude(dv[k]));
            }
        }
    }
    if (!trans)
        return;
#pragma unroll
    for (int f = 0; f < (GATED ? 3 : 2); ++f)
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const uint32_t m = max(most[f][k], __shfl_xor_sync(0xFFFFFFFFu, most[f][k], 16));
            if ((threadIdx.x & 16) == 0)
                atomicMax(&amax[f][j * 8 + k], m);  // a maximum: in any order the same
        }
    __syncthreads();
    if (p.du8t.q)
        put_columns(p.du8t, tile[0], amax[0], group, c0, p.cols, r0, p.rows, p.e5m2);
    if (p.a8t.q)
        put_columns(p.a8t, tile[1], amax[1], group, c0, p.cols, r0, p.rows, false);
    if (GATED && p.dv8t.q)
        put_columns(p.dv8t, tile[2], amax[2], group, c0, p.cols, r0, p.rows, p.e5m2);
}

template <class H, bool S8, bool GATED, bool GELU>
static int launch_act_backward(const ActBackParams &p, int64_t grid, cudaStream_t stream)
{
    const bool trans = p.du8t.q || p.dv8t.q || p.a8t.q;
    const int bytes = trans ? (GATED ? 3 : 2) * (int)sizeof(Staged) : 0;
    auto kernel = act_backward_kernel<H, S8, GATED, GELU>;
    if (bytes) {
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e != cudaSuccess)
            return cuda_error(e);
    }
    kernel<<<(unsigned)grid, kBackThreads, bytes, stream>>>(p);
    return launch_status();
}

template <class H, bool S8>
static int choose_act_backward(const ActBackParams &p, bool gelu, int64_t grid, cudaStream_t stream)
{
    if (p.v)
        return gelu ? launch_act_backward<H, S8, true, true>(p, grid, stream)
                    : launch_act_backward<H, S8, true, false>(p, grid, stream);
    return gelu ? launch_act_backward<H, S8, false, true>(p, grid, stream)
                : launch_act_backward<H, S8, false, false>(p, grid, stream);
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
    p.rows = rows;
    p.cols = cols;
    p.row_tiles = ceil_div(rows, kActRows);
    p.wide = rows_aligned(u, ldu, b, 16) && (!v || rows_aligned(v, ldv, b, 16)) && (!a || rows_aligned(a, lda, b, 16));
    p.e5m2 = a8 && fp8 == ZERO_T_E5M2;
    const int64_t grid = p.row_tiles * ceil_div(cols, kBlock);
    if (grid > kMaxDim)
        return ZERO_EINVAL;
    auto go = [&](auto kernel) {
        kernel<<<(unsigned)grid, 256, 0, stream>>>(p);
        return launch_status();
    };
    if (type == ZERO_T_F16)
        return act == ZERO_ACT_GELU ? go(act_kernel<f16, true>) : go(act_kernel<f16, false>);
    return act == ZERO_ACT_GELU ? go(act_kernel<bf16, true>) : go(act_kernel<bf16, false>);
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
    p.rows = rows;
    p.cols = cols;
    p.row_tiles = ceil_div(rows, kBlock);
    p.wide = rows_aligned(da, ldda, b, 16) && (!du || rows_aligned(du, lddu, b, 16)) &&
             (!dv || rows_aligned(dv, lddv, b, 16));
    const int kb = su ? 1 : b, to = su ? 8 : 16;
    p.wide_kept = rows_aligned(u, ldu, kb, to) && (!v || rows_aligned(v, ldv, kb, to));
    p.e5m2 = fp8 == ZERO_T_E5M2;
    const int64_t grid = p.row_tiles * ceil_div(cols, kBlock);
    if (grid > kMaxDim)
        return ZERO_EINVAL;
    const bool gelu = act == ZERO_ACT_GELU;
    if (type == ZERO_T_F16)
        return su ? choose_act_backward<f16, true>(p, gelu, grid, stream)
                  : choose_act_backward<f16, false>(p, gelu, grid, stream);
    return su ? choose_act_backward<bf16, true>(p, gelu, grid, stream)
              : choose_act_backward<bf16, false>(p, gelu, grid, stream);
}

}  // extern "C"
