// An 8-bit matrix read back, x = q * s * row * col, and its transpose in 8 bits: the
// operand of a weight's gradient made from a checkpoint, without the tensor in a half
// type in between.
//
// A CTA takes a 128x128 tile, 8 rows to 16 lanes of 8 columns.  The bytes go through
// shared memory as they are: within a tile a row has one scale and one factor, so a
// transposed value is a byte times a row's and a column's number.
//
// 8192x14336 as bf16: 55 us, 6.4 TB/s (0.95 of the copy rate).  8192x4096 transposed with both
// factors: 21 us, 3.3 TB/s (0.49; issue slots 66 % busy, ALU 59): taking bytes apart and together
// again is what it does, and four CTAs to an SM take 2048 tiles in 3.4 waves.  CTAs that walk the tiles with two more on their way took 23, and the
// first case 63.
#include "layer.cuh"

namespace zo {

struct RestoreParams {
    const uint8_t *q;
    const float *s, *row;
    const void *col;
    void *x;
    Form t8;
    int64_t ldq, lds, ldx;
    int32_t rows, cols;
    Tiles tiles;
    int32_t col_type;
};

constexpr int kRestoreThreads = 256;

template <int F8, class X, int W>
__device__ __forceinline__ void restore_tile(const RestoreParams &p, const TileAt tile_of, uint2 (&tile)[kBlock][16], float (&factor)[kBlock])
{
    const int lane = threadIdx.x & 15, group = threadIdx.x >> 4;
    const int64_t tr = tile_of.r, tc = tile_of.c, r0 = tr * kBlock, c0 = tc * kBlock;
    const int c = tile_of.c * kBlock + lane * 8, nc = left_of(p.cols, c);
    const int nr = r0 + group * 8 < p.rows ? left_of(p.rows, (int)(r0 + group * 8)) : 0;
    Raw8b q[8];
    const uint8_t *from = p.q + (r0 + group * 8) * p.ldq + c;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        q[i] = get_bytes<W>(from + i * p.ldq, i < nr ? nc : 0);
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
            tile[group * 8 + i][lane ^ group] = make_uint2(q[i].w[0], q[i].w[1]);
    __syncthreads();
    if (p.x && nc > 0) {
        float2 col[4];
        if (p.col)
            get_vector<W>(p.col, p.col_type, c, nc, col);
        X *to = static_cast<X *>(p.x) + (r0 + group * 8) * p.ldx + c;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < nr) {
                const float f = factor[group * 8 + i];
                float2 x[4];
                pairs_of<F8>(q[i], x);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    x[k] = mul2(x[k], both(f));
                    if (p.col)
                        x[k] = mul2(x[k], col[k]);
                }
                put_pairs<W>(to + i * p.ldx, nc, x);
            }
    }
    if (!p.t8.q)
        return;
    float2 f[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        f[i] = *reinterpret_cast<const float2 *>(&factor[lane * 8 + 2 * i]);
    const int64_t row = r0 + lane * 8;
    const int n = row < p.rows ? left_of(p.rows, (int)row) : 0;
    const uint32_t *words = reinterpret_cast<const uint32_t *>(&tile[lane * 8][group ^ lane]);
    uint8_t *to = p.t8.q + (c0 + group * 8) * p.t8.ld + row;
#pragma unroll 1
    for (int half = 0; half < 2; ++half) {
        const int64_t at = c0 + group * 8 + half * 4;  // four columns
        float2 x[4][4];  // of a column, rows 2i and 2i + 1
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t a = words[2 * i * 32 + half], b = words[(2 * i + 1) * 32 + half];
#pragma unroll
            for (int m = 0; m < 4; ++m)
                x[m][i] = mul2(two_of<F8>(__byte_perm(a, b, m | (m + 4) << 4) & 0xFFFFu), f[i]);
        }
        if (p.col)
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                const float col = at + m < p.cols ? load_one(p.col, p.col_type, at + m) : 1.0f;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    x[m][i] = mul2(x[m][i], both(col));
            }
        if (W != kWhole && n < 8)  // rows behind the last: 0 times a column's factor may be NaN
#pragma unroll
            for (int m = 0; m < 4; ++m)
                clear_behind(x[m], n);
        uint32_t a[4];
#pragma unroll
        for (int m = 0; m < 4; ++m)
            a[m] = W != kWhole || n > 0 ? amax8(x[m]) : 0u;
        const float s = scale_of<F8 == ZERO_T_E5M2>(max_shared(a));
        const Inverse inv = inverse_of(s);
        const int mine = shared_index<4>();
        if (lane % 4 == 0 && at + mine < p.cols)
            p.t8.s[tr * p.t8.lds + at + mine] = s;
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            const Inverse d = shared_value<4>(inv, m);
            if (n > 0 && at + m < p.cols)
                put_bytes<W>(to, n, bytes_of<F8 == ZERO_T_E5M2>(x[m], d));
            to += p.t8.ld;
        }
    }
}

// As for the activation's gradients, only the last tiles of rows or columns that 8 does not divide have short units
// to reckon with (8191x4096 23 us, 24 where all do).
template <int F8, class X, int W>
__global__ void __launch_bounds__(kRestoreThreads) restore_kernel(const RestoreParams p)
{
    // row r's 8 bytes of columns 8j .. lie at j ^ (r / 8), so that the 16 lanes of a column,
    // 8 rows each, read different banks
    __shared__ uint2 tile[kBlock][16];
    __shared__ __align__(16) float factor[kBlock];
    const TileAt at = tile_at(p.tiles);
    if (W == kWide && whole_units(at, p.rows, p.cols))
        restore_tile<F8, X, kWhole>(p, at, tile, factor);
    else
        restore_tile<F8, X, W>(p, at, tile, factor);
}

template <class X, int W>
static int launch_restore(const RestoreParams &p, int fp8, int64_t grid, cudaStream_t stream)
{
    if (fp8 == ZERO_T_E5M2)
        restore_kernel<ZERO_T_E5M2, X, W><<<(unsigned)grid, kRestoreThreads, 0, stream>>>(p);
    else
        restore_kernel<ZERO_T_E4M3, X, W><<<(unsigned)grid, kRestoreThreads, 0, stream>>>(p);
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
    p.rows = (int32_t)rows;
    p.cols = (int32_t)cols;
    p.tiles = tiles_of(rows, cols, kBlock);
    p.col_type = col_type;
    const bool wide = rows_aligned(q, ldq, 1, 8) && (!x || rows_aligned(x, ldx, type_bytes(x_type), 16)) &&
                      aligned(col, 16) && (!t8 || p.t8.wide);
    const int64_t grid = (int64_t)p.tiles.rows * p.tiles.cols;
    if (grid > kMaxDim)
        return ZERO_EINVAL;
    auto go = [&](auto out) {
        using X = decltype(out);
        return !wide ? launch_restore<X, kApart>(p, fp8, grid, stream)
                     : cols % 8 || rows % 8 ? launch_restore<X, kWide>(p, fp8, grid, stream)
                                            : launch_restore<X, kWhole>(p, fp8, grid, stream);
    };
    if (x && x_type == ZERO_T_F16)
        return go(f16{});
    if (x && x_type == ZERO_T_F32)
        return go(0.0f);
    return go(bf16{});
}
