// A matrix in 8-bit floating point with a scale for each 1x128 block or
// 128x128 tile, and its transpose:
//
//   s = max(amax / qmax, 2^-126),  q = round(x / s)
//
// Bound by memory: x is read once and both forms are written from the same
// registers.  A CTA takes a 128x128 tile; each thread holds an 8x8 patch (8
// neighbouring rows, 8 neighbouring columns), so that a row's 16 bytes load at
// once, a row's amax is a reduction over 16 lanes, a column's over 8 registers
// and the 16 row groups, and 8 rows of a column pack into the 8 bytes that the
// transposed form has side by side.  What keeps it from the copy rate is the
// latency of a tile's way through loads, maxima and barriers, which only the
// other three CTAs of the SM cover; no unit is the limit (8192x4096, both forms:
// issue slots 55 % busy, ALU 48, DRAM 40).
//   8192x4096 bf16, both forms:  29.2 us, 4.7 TB/s (0.69 of the copy rate)
//   14336x4096 bf16, 128x128 tiles, both forms:  41.2 us, 5.7 TB/s (0.84)
// The quotients' second product costs the first 1.5 us and the tiles nothing.
//   8192x4096, 1x128 blocks, one form alone: bf16 20.6 us (0.72 of the copy rate), its
//   transpose 25.4 (0.59); fp32 32.9 (0.75), 37.0 (0.67), both 44.7 (0.66)
#include "ops.cuh"

namespace zo {

constexpr int kQThreads = 256;  // 16 row groups x 16 column groups of 8x8

struct QuantParams {
    const void *x;
    int64_t rows, cols, ldx;
    uint8_t *q, *qt;
    int64_t ldq, ldqt;
    float *s, *st;
    int64_t lds, ldst;
    int32_t wide_x, wide_q, wide_qt;
    int32_t row_tiles;
};

// A thread's 8x8 patch as it lies in memory.  Halves stay packed: half the
// registers, so that four CTAs fit an SM (28.9 us for three's 31.2 at 8192x4096,
// both forms, with one product to a quotient), and their magnitudes are compared
// two at a time.
template <class T>
struct Patch {
    Raw8<T> row[8];

    __device__ __forceinline__ float at(int i, int j) const { return row[i].at(j); }
    __device__ __forceinline__ uint32_t row_amax(int i) const
    {
        if constexpr (sizeof(T) == 2) {
            Amax<T> a;
#pragma unroll
            for (int k = 0; k < 4; ++k)
                a.add(row[i].w[k]);
            return a.bits();
        } else {
            uint32_t a = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j)
                a = max(a, magnitude(at(i, j)));
            return a;
        }
    }
    // columns 2k and 2k + 1
    __device__ __forceinline__ uint2 column_amax(int k) const
    {
        if constexpr (sizeof(T) == 2) {
            Amax<T> a;
#pragma unroll
            for (int i = 0; i < 8; ++i)
                a.add(row[i].w[k]);
            Amax<T> lo, hi;
            lo.two = a.two & 0xFFFFu;
            hi.two = a.two >> 16;
            return make_uint2(lo.bits(), hi.bits());
        } else {
            uint2 a = make_uint2(0, 0);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                a.x = max(a.x, magnitude(at(i, 2 * k)));
                a.y = max(a.y, magnitude(at(i, 2 * k + 1)));
            }
            return a;
        }
    }
};

// TILE: one scale per tile.  TRANS: the transposed form is wanted (q may be
// too: p.q says so).
template <class T, int F8, bool TILE, bool TRANS>
__global__ void __launch_bounds__(kQThreads, sizeof(T) == 2 ? 4 : 2) quantize_kernel(const QuantParams p)
{
    __shared__ uint32_t amax_sh[16][kBlock];  // a row group's amax of each column
    __shared__ Inverse inv_sh[kBlock];
    __shared__ uint2 t_sh[TRANS ? kBlock : 1][16];
    const int cg = threadIdx.x & 15, rg = threadIdx.x >> 4;
    const int64_t tr = blockIdx.x % p.row_tiles, tc = blockIdx.x / p.row_tiles;
    const int64_t r0 = tr * kBlock + rg * 8, c0 = tc * kBlock + cg * 8;
    const int nc = (int)min((int64_t)8, p.cols - c0);   // may be <= 0
    const int nr = (int)min((int64_t)8, p.rows - r0);
    const T *x = static_cast<const T *>(p.x) + r0 * p.ldx + c0;

    Patch<T> v;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        v.row[i] = load_raw(x + i * p.ldx, i < nr ? nc : 0, p.wide_x);

    Inverse inv_tile{};
    if (TILE) {
        uint32_t a = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            a = max(a, v.row_amax(i));
        a = max_over<32>(a);
        if ((threadIdx.x & 31) == 0)
            amax_sh[0][threadIdx.x >> 5] = a;
        __syncthreads();
        a = 0;
#pragma unroll
        for (int w = 0; w < kQThreads / 32; ++w)
            a = max(a, amax_sh[0][w]);
        const float s = block_scale<F8>(a);
        inv_tile = inverse(s);
        if (threadIdx.x == 0) {
            if (p.q)
                p.s[tc * p.lds + tr] = s;
            if (TRANS)
                p.st[tr * p.ldst + tc] = s;
        }
    }
    if (p.q) {
        // a row's amax is over the 16 lanes of its row group: the lanes halve
        // the rows between them as they exchange, so that lane i ends with
        // rows i % 8's and its scale is formed once (8 shuffles, not 32)
        uint32_t mine = 0;
        if (!TILE) {
            uint32_t a[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                a[i] = v.row_amax(i);
#pragma unroll
            for (int half = 4; half; half >>= 1)
#pragma unroll
                for (int i = 0; i < half; ++i) {
                    const bool up = cg & half;
                    const uint32_t keep = up ? a[i + half] : a[i], give = up ? a[i] : a[i + half];
                    a[i] = max(keep, __shfl_xor_sync(0xFFFFFFFFu, give, half));
                }
            mine = max(a[0], __shfl_xor_sync(0xFFFFFFFFu, a[0], 8));
        }
        Inverse inv_mine{};
        if (!TILE) {
            const float s = block_scale<F8>(mine);
            inv_mine = inverse(s);
            if (cg < 8 && cg < nr)
                p.s[tc * p.lds + r0 + cg] = s;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            Inverse d = inv_tile;
            if (!TILE)
                d = {__shfl_sync(0xFFFFFFFFu, inv_mine.hi, i, 16), __shfl_sync(0xFFFFFFFFu, inv_mine.lo, i, 16)};
            float x[8];
#pragma unroll
            for (int j = 0; j < 8; ++j)
                x[j] = v.at(i, j);
            const uint2 o = quotients8<F8>(x, d);
            if (i < nr)
                store8b(p.q + (r0 + i) * p.ldq + c0, nc, p.wide_q, o);
        }
    }
    if (!TRANS)
        return;

    if (!TILE) {
        // the columns' amax over the tile's 128 rows
#pragma unroll
        for (int k = 0; k < 4; ++k)
            *reinterpret_cast<uint2 *>(&amax_sh[rg][cg * 8 + 2 * k]) = v.column_amax(k);
        __syncthreads();
        if (threadIdx.x < kBlock) {
            uint32_t a = 0;
#pragma unroll
            for (int g = 0; g < 16; ++g)
                a = max(a, amax_sh[g][threadIdx.x]);
            const float s = block_scale<F8>(a);
            inv_sh[threadIdx.x] = inverse(s);
            const int64_t c = tc * kBlock + threadIdx.x;
            if (c < p.cols)
                p.st[tr * p.ldst + c] = s;
        }
        __syncthreads();
    }
    // The transposed tile through shared memory: column c's 128 bytes lie as 16
    // units of 8 rows, unit g at place g ^ (c / 8), so that the 16 column
    // groups of a half-warp, whose columns are 1024 bytes apart, write to
    // different banks.
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        float x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            x[i] = v.at(i, j);
        t_sh[cg * 8 + j][rg ^ cg] = quotients8<F8>(x, TILE ? inv_tile : inv_sh[cg * 8 + j]);
    }
    __syncthreads();
    // 16 threads write a column's 128 rows
    const int64_t row = tr * kBlock + cg * 8;
    const int n = (int)min((int64_t)8, p.rows - row);
    if (n > 0)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int c = i * 16 + rg;
            const int64_t col = tc * kBlock + c;
            if (col < p.cols)
                store8b(p.qt + col * p.ldqt + row, n, p.wide_qt, t_sh[c][cg ^ (c >> 3)]);
        }
}

template <class T, int F8>
static int launch_quantize(const QuantParams &p, bool tile, cudaStream_t stream)
{
    const int64_t grid = p.row_tiles * ceil_div(p.cols, kBlock);
    if (grid > kMaxDim)
        return ZERO_EINVAL;
    auto go = [&](auto kernel) {
        kernel<<<(unsigned)grid, kQThreads, 0, stream>>>(p);
        return launch_status();
    };
    if (p.qt)
        return tile ? go(quantize_kernel<T, F8, true, true>) : go(quantize_kernel<T, F8, false, true>);
    return tile ? go(quantize_kernel<T, F8, true, false>) : go(quantize_kernel<T, F8, false, false>);
}

}  // namespace zo

using namespace zo;

extern "C" int zero_fp8_quantize(const void *x, int type, int64_t rows, int64_t cols, int64_t ldx,
                                 int fp8, int tile, void *q, int64_t ldq, float *s, int64_t lds,
                                 void *qt, int64_t ldqt, float *st, int64_t ldst,
                                 zero_stream_t stream)
{
    if (!is_float(type) || !is_fp8(fp8) || bad_dim(rows) || bad_dim(cols) || (tile != 0 && tile != 1))
        return ZERO_EINVAL;
    if (rows == 0 || cols == 0)
        return ZERO_OK;
    if ((!q && !qt) || !q != !s || !qt != !st)
        return ZERO_EINVAL;
    int rc = check_matrix(x, rows, cols, ldx, type_bytes(type));
    if (!rc && q)
        rc = check_matrix(q, rows, cols, ldq, 1);
    if (!rc && q)
        rc = check_matrix(s, ceil_div(cols, kBlock), tile ? ceil_div(rows, kBlock) : rows, lds, 4);
    if (!rc && qt)
        rc = check_matrix(qt, cols, rows, ldqt, 1);
    if (!rc && qt)
        rc = check_matrix(st, ceil_div(rows, kBlock), tile ? ceil_div(cols, kBlock) : cols, ldst, 4);
    if (rc)
        return rc;
    QuantParams p{};
    p.x = x;
    p.rows = rows;
    p.cols = cols;
    p.ldx = ldx;
    p.q = static_cast<uint8_t *>(q);
    p.ldq = ldq;
    p.s = s;
    p.lds = lds;
    p.qt = static_cast<uint8_t *>(qt);
    p.ldqt = ldqt;
    p.st = st;
    p.ldst = ldst;
    p.wide_x = rows_aligned(x, ldx, type_bytes(type), 16);
    p.wide_q = q && rows_aligned(q, ldq, 1, 8);
    p.wide_qt = qt && rows_aligned(qt, ldqt, 1, 8);
    p.row_tiles = (int32_t)ceil_div(rows, kBlock);
    auto by_fp8 = [&](auto x_type) {
        using T = decltype(x_type);
        return fp8 == ZERO_T_E4M3 ? launch_quantize<T, ZERO_T_E4M3>(p, tile != 0, stream)
                                  : launch_quantize<T, ZERO_T_E5M2>(p, tile != 0, stream);
    };
    if (type == ZERO_T_F16)
        return by_fp8(f16{});
    if (type == ZERO_T_BF16)
        return by_fp8(bf16{});
    return by_fp8(0.0f);
}
