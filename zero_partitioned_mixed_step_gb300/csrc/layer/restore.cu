// An 8-bit matrix read back, x = q * s * row * col, and its transpose in 8 bits: the
// operand of a weight's gradient made from a checkpoint, without the tensor in a half
// type in between.
//
// Bound by memory.  A CTA takes a 128x128 tile, 8 rows to 16 lanes of 8 columns.
// The bytes go through shared memory as they are: within a tile a row has one scale
// and one factor, so a transposed value is a byte times a row's and a column's number.
#include "layer.cuh"

namespace zo {

struct RestoreParams {
    const uint8_t *q;
    const float *s, *row;
    const void *col;
    void *x;
    Form t8;
    int64_t ldq, lds, ldx, rows, cols;
    int64_t row_tiles;
    int32_t col_type, wide_q, wide_x, wide_col;
};

constexpr int kRestoreThreads = 256;

template <int F8, class X>
__global__ void __launch_bounds__(kRestoreThreads) restore_kernel(const RestoreParams p)
{
    // row r's 8 bytes of columns 8j .. lie at j ^ (r / 8), so that the 16 lanes of a column,
    // 8 rows each, read different banks
    __shared__ uint2 tile[kBlock][16];
    __shared__ float factor[kBlock];
    const int j = threadIdx.x & 15, group = threadIdx.x >> 4;
    const int64_t tr = blockIdx.x % p.row_tiles, tc = blockIdx.x / p.row_tiles;
    const int64_t r0 = tr * kBlock, c0 = tc * kBlock, c = c0 + j * 8;
    const int nc = in_row(p.cols, c);
    Raw8b q[8];
    const uint8_t *from = p.q + (r0 + group * 8) * p.ldq + c;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        q[i] = load_raw8b(from + i * p.ldq, r0 + group * 8 + i < p.rows ? nc : 0, p.wide_q);
    if (threadIdx.x < kBlock) {
        const int64_t row = r0 + threadIdx.x;
        float f = 0.0f;
        if (row < p.rows) {
            f = p.s[tc * p.lds + row];
            if (p.row)
                f *= p.row[row];
        }
        factor[threadIdx.x] = f;
    }
    if (p.t8.q)
#pragma unroll
        for (int i = 0; i < 8; ++i)
            tile[group * 8 + i][j ^ group] = make_uint2(q[i].w[0], q[i].w[1]);
    __syncthreads();
    if (p.x && nc > 0) {
        float col[8];
        if (p.col)
            load_w(p.col, p.col_type, c, nc, p.wide_col, col);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int64_t row = r0 + group * 8 + i;
            if (row >= p.rows)
                break;
            const float f = factor[group * 8 + i];
            float x[8];
            q[i].get<F8>(x);
#pragma unroll
            for (int k = 0; k < 8; ++k)
                x[k] = p.col ? x[k] * f * col[k] : x[k] * f;
            store8(static_cast<X *>(p.x) + row * p.ldx + c, nc, p.wide_x, x);
        }
    }
    if (!p.t8.q)
        return;
    const int lane = j;
    float f[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
        f[i] = factor[lane * 8 + i];
    const int64_t row = r0 + lane * 8;
    const int n = in_row(p.rows, row);
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        const int k = group + 16 * half;  // columns 4k ..
        float x[4][8];
        uint32_t a[4] = {};
        const int64_t at = c0 + 4 * k;
        float col[4];
#pragma unroll
        for (int m = 0; m < 4; ++m)
            col[m] = p.col && at + m < p.cols ? load_one(p.col, p.col_type, at + m) : 1.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint2 two = tile[lane * 8 + i][k >> 1 ^ lane];
            const uint32_t w = k & 1 ? two.y : two.x;
            const float2 lo = two_of<F8>(w & 0xFFFFu), hi = two_of<F8>(w >> 16);
            x[0][i] = lo.x * f[i];
            x[1][i] = lo.y * f[i];
            x[2][i] = hi.x * f[i];
            x[3][i] = hi.y * f[i];
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                if (p.col)
                    x[m][i] *= col[m];
                a[m] = max(a[m], magnitude(x[m][i]));
            }
        }
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            const float s = block_scale<F8>(max_over<16>(a[m]));
            if (at + m >= p.cols)
                continue;
            if (lane == 0)
                p.t8.s[tr * p.t8.lds + at + m] = s;
            if (n > 0)
                store8b(p.t8.q + (at + m) * p.t8.ld + row, n, p.t8.wide, quotients8<F8>(x[m], inverse(s)));
        }
    }
}

template <class X>
static int launch_restore(const RestoreParams &p, int fp8, int64_t grid, cudaStream_t stream)
{
    if (fp8 == ZERO_T_E5M2)
        restore_kernel<ZERO_T_E5M2, X><<<(unsigned)grid, kRestoreThreads, 0, stream>>>(p);
    else
        restore_kernel<ZERO_T_E4M3, X><<<(unsigned)grid, kRestoreThreads, 0, stream>>>(p);
    return launch_status();
}

}  // namespace zo

using namespace zo;

extern "C" int zero_fp8_restore(const void *q, int fp8, int64_t ldq, const float *s, int64_t lds, const float *row,
                                const void *col, int col_type, int64_t rows, int64_t cols, void *x, int x_type,
                                int64_t ldx, const zero_fp8_form *t8, zero_stream_t stream)
{
    if (!is_fp8(fp8) || bad_dim(rows) || bad_dim(cols) || (col && !is_float(col_type)) || (x && !is_float(x_type)))
        return ZERO_EINVAL;
    if (rows == 0 || cols == 0)
        return ZERO_OK;
    if (!x && !t8)
        return ZERO_EINVAL;
    int rc = check_matrix(q, rows, cols, ldq, 1);
    if (!rc)
        rc = check_matrix(s, ceil_div(cols, kBlock), rows, lds, 4);
    if (!rc && x)
        rc = check_matrix(x, rows, cols, ldx, type_bytes(x_type));
    if (!rc)
        rc = check_form(t8, cols, rows);
    if (!rc && (!aligned(row, 4) || (col && !aligned(col, (uintptr_t)type_bytes(col_type)))))
        rc = ZERO_EALIGN;
    if (rc)
        return rc;
    RestoreParams p{};
    p.q = static_cast<const uint8_t *>(q);
    p.s = s;
    p.row = row;
    p.col = col;
    p.x = x;
    p.t8 = form_of(t8);
    p.ldq = ldq;
    p.lds = lds;
    p.ldx = ldx;
    p.rows = rows;
    p.cols = cols;
    p.row_tiles = ceil_div(rows, kBlock);
    p.col_type = col_type;
    p.wide_q = rows_aligned(q, ldq, 1, 8);
    p.wide_x = x && rows_aligned(x, ldx, type_bytes(x_type), 16);
    p.wide_col = aligned(col, 16);
    const int64_t grid = p.row_tiles * ceil_div(cols, kBlock);
    if (grid > kMaxDim)
        return ZERO_EINVAL;
    if (x && x_type == ZERO_T_F16)
        return launch_restore<f16>(p, fp8, grid, stream);
    if (x && x_type == ZERO_T_F32)
        return launch_restore<float>(p, fp8, grid, stream);
    return launch_restore<bf16>(p, fp8, grid, stream);
}
