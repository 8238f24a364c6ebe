// The product of two 8-bit matrices with a scale for each block of 128.
//
//   out[i, j] (+)= sum_b sa[b, i] sb[b, j] (sum over k in block b of a[i, k] b[j, k])
#include "ops.cuh"

namespace zo {

struct MatmulParams {
    const uint8_t *a, *b;
    const float *sa, *sb;
    void *out;
    int64_t lda, ldb, ldsa, ldsb, ldo;
    int64_t m, n, k;
    int32_t a_type, b_type, b_tile, out_type, add;
};

__device__ __forceinline__ float fp8_value(uint8_t x, int type)
{
    const __half_raw r = __nv_cvt_fp8_to_halfraw(x, type == ZERO_T_E4M3 ? __NV_E4M3 : __NV_E5M2);
    return __half2float(__half(r));
}

__global__ void __launch_bounds__(256) matmul_kernel(const MatmulParams p)
{
    __shared__ float as[16][17], bs[16][17];
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const int64_t i0 = (int64_t)blockIdx.y * 16, j0 = (int64_t)blockIdx.x * 16;
    const int64_t i = i0 + ty, j = j0 + tx;
    float acc = 0.0f;
    for (int64_t k0 = 0; k0 < p.k; k0 += kBlock) {
        float part = 0.0f;
        for (int64_t kk = k0; kk < k0 + kBlock && kk < p.k; kk += 16) {
            const int64_t c = kk + tx;
            __syncthreads();
            as[ty][tx] = i0 + ty < p.m && c < p.k ? fp8_value(p.a[(i0 + ty) * p.lda + c], p.a_type) : 0.0f;
            bs[ty][tx] = j0 + ty < p.n && c < p.k ? fp8_value(p.b[(j0 + ty) * p.ldb + c], p.b_type) : 0.0f;
            __syncthreads();
#pragma unroll
            for (int e = 0; e < 16; ++e)
                part = fmaf(as[ty][e], bs[tx][e], part);
        }
        if (i < p.m && j < p.n) {
            const int64_t kb = k0 / kBlock;
            acc = fmaf(part, p.sa[kb * p.ldsa + i] * p.sb[kb * p.ldsb + (p.b_tile ? j / kBlock : j)], acc);
        }
    }
    if (i >= p.m || j >= p.n)
        return;
    const int64_t at = i * p.ldo + j;
    if (p.out_type == ZERO_T_F16) {
        f16 *o = static_cast<f16 *>(p.out) + at;
        *o = from_f32<f16>(p.add ? to_f32(*o) + acc : acc);
    } else if (p.out_type == ZERO_T_BF16) {
        bf16 *o = static_cast<bf16 *>(p.out) + at;
        *o = from_f32<bf16>(p.add ? to_f32(*o) + acc : acc);
    } else {
        float *o = static_cast<float *>(p.out) + at;
        *o = p.add ? *o + acc : acc;
    }
}

}  // namespace zo

using namespace zo;

extern "C" {

size_t zero_fp8_matmul_workspace_bytes(int64_t m, int64_t n, int64_t k)
{
    if (bad_dim(m) || bad_dim(n) || bad_dim(k))
        return 0;
    return 256;
}

int zero_fp8_matmul(const void *a, int a_type, int64_t lda, const float *sa, int64_t ldsa,
                    const void *b, int b_type, int64_t ldb, const float *sb, int64_t ldsb,
                    int b_tile, void *out, int out_type, int64_t ldo, int64_t m, int64_t n,
                    int64_t k, int add, void *ws, size_t ws_bytes, zero_stream_t stream)
{
    if (!is_fp8(a_type) || !is_fp8(b_type) || !is_float(out_type) || bad_dim(m) || bad_dim(n) ||
        bad_dim(k) || (b_tile != 0 && b_tile != 1) || !ws)
        return ZERO_EINVAL;
    if (m == 0 || n == 0)
        return ZERO_OK;
    int rc = check_matrix(out, m, n, ldo, type_bytes(out_type));
    if (!rc)
        rc = check_matrix(a, m, k, lda, 1);
    if (!rc)
        rc = check_matrix(b, n, k, ldb, 1);
    if (!rc)
        rc = check_matrix(sa, ceil_div(k, kBlock), m, ldsa, 4);
    if (!rc)
        rc = check_matrix(sb, ceil_div(k, kBlock), b_tile ? ceil_div(n, kBlock) : n, ldsb, 4);
    if (!rc && (!aligned(ws, 16) || (k > 0 && (!rows_aligned(a, lda, 1, 16) || !rows_aligned(b, ldb, 1, 16)))))
        rc = ZERO_EALIGN;
    if (!rc && ws_bytes < zero_fp8_matmul_workspace_bytes(m, n, k))
        rc = ZERO_ESPACE;
    if (rc)
        return rc;
    MatmulParams p{};
    p.a = static_cast<const uint8_t *>(a);
    p.b = static_cast<const uint8_t *>(b);
    p.sa = sa;
    p.sb = sb;
    p.out = out;
    p.lda = lda;
    p.ldb = ldb;
    p.ldsa = ldsa;
    p.ldsb = ldsb;
    p.ldo = ldo;
    p.m = m;
    p.n = n;
    p.k = k;
    p.a_type = a_type;
    p.b_type = b_type;
    p.b_tile = b_tile;
    p.out_type = out_type;
    p.add = add ? 1 : 0;
    const dim3 grid((unsigned)ceil_div(n, 16), (unsigned)ceil_div(m, 16));
    matmul_kernel<<<grid, 256, 0, stream>>>(p);
    return launch_status();
}

}  // extern "C"
