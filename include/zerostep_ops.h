/*
 * zerostep_ops.h — C ABI of libzerostep_ops.so: the operators that a program
 * runs around the partitioned step on one GB300 GPU (sm_103a) when its
 * products are in 8-bit floating point.
 *
 *   zero_rmsnorm_fp8        residual addition, root-mean-square norm, the
 *                           result in 8 bits with a scale for each block of 128
 *   zero_rmsnorm_backward   its gradients
 *   zero_fp8_quantize       a matrix in 8 bits with a scale for each block of
 *                           128, and its transpose
 *   zero_fp8_matmul         the product of two such matrices
 *   zero_tensors_norm       the global L2 norm over many gradient tensors
 *   zero_tensors_clip       the clipped gradients, in place or into the flat
 *                           half buffer that zero_step_fused reads
 *
 * Conventions: as zerostep.h (the caller owns every buffer, device work is
 * enqueued on `stream` and nothing synchronises the host, arguments are
 * validated before anything is enqueued, the same return codes).  All data
 * pointers are device pointers of the current device; arrays of pointers and
 * sizes are host arrays read during the call.  Matrices are row-major with a
 * row stride ld (in elements, at least the row's length); elements between a
 * row's end and the next row are neither read nor written.  An input may not
 * overlap an output unless its description allows it.  A pointer must be
 * aligned to its element; rows that start on 16-byte boundaries run with wide
 * accesses (zero_fp8_matmul requires them).  Sizes are 0 .. 2^31 - 1025
 * per dimension and offsets are formed in 64 bits.  All calls can be captured in
 * a CUDA graph.  Results do not depend on the launch shape or on other work
 * on the GPU: no floating-point atomics, sums in a fixed order.
 *
 * Blocks of 128.  The 8-bit form of a matrix X[rows, cols] is q[rows, cols]
 * (ZERO_T_E4M3 or ZERO_T_E5M2) and fp32 scales s, block columns first:
 *   one for each 1x128 block:   s[(c / 128) * lds + r],       lds >= rows
 *   one for each 128x128 tile:  s[(c / 128) * lds + r / 128], lds >= ceil(rows / 128)
 * with X[r, c] ~ q[r, c] * s.  The last block of a row and the last tile may
 * be short.  s = max(amax / qmax, 2^-126), amax the largest magnitude of the
 * block and qmax the type's largest value (448 and 57344); q is X / s rounded
 * to fp32 and then to the type, to nearest even (of fp32 elements, and where amax
 * is 2^117 or more, a few in 1e8 meet the fp32 quotient's neighbour).  A block of
 * zeros has q = 0.
 * A block that holds a NaN or an infinity has s = NaN or infinity, and q * s is
 * NaN throughout it, so that what is computed from it is not finite and the
 * step skips.
 */
#ifndef ZEROSTEP_OPS_H
#define ZEROSTEP_OPS_H

#include "zerostep.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types.  The half types have zero_dtype's values. */
typedef enum {
    ZERO_T_F16 = 0,
    ZERO_T_BF16 = 1,
    ZERO_T_F32 = 4,
    ZERO_T_E4M3 = 8, /* 4 exponent bits, 3 of fraction, no infinities, largest value 448 */
    ZERO_T_E5M2 = 9  /* 5 exponent bits, 2 of fraction, largest value 57344 */
} zero_type;

/* What zero_tensors_norm leaves for zero_tensors_clip: DEVICE-resident, 16
 * bytes, 8-byte aligned, owned by the caller.  Ranks that hold different
 * tensors add their sumsq and OR their found_inf before the clip. */
typedef struct {
    double sumsq;      /* sum of the squares of all elements, times inv_scale^2 */
    float norm;        /* its square root (infinite from 2^128 on; the clip goes by sumsq) */
    int32_t found_inf; /* 1 if an element times inv_scale is NaN or infinite */
} zero_tensors_stat;

/* Bytes of workspace that zero_tensors_norm needs for these tensors (0 for
 * invalid sizes).  ZERO-FILL IT ONCE before its first use: it holds two
 * counters, which every call that runs to completion returns to zero.  One
 * workspace may serve lists of different sizes, one call after the other. */
ZERO_API size_t zero_tensors_workspace_bytes(int n, const int64_t *numel);

/*
 * The global norm over n tensors: stat->sumsq = sum over tensors t and their
 * elements of (x * inv_scale)^2, stat->norm, stat->found_inf.
 *  x[n], numel[n], type[n]: the tensors (contiguous; F16, BF16 or F32, mixed
 *    as they come); x[t] may be NULL where numel[t] = 0.  n = 0 and empty
 *    tensors give a norm of +0.
 *  tensor_sumsq: NULL, or n doubles (device) that receive each tensor's sum.
 * The squares are summed in fp32 over runs of a chunk (at least 4096
 * elements, one CTA each), the runs in pairs of fp32 values and the chunks in
 * binary64, in an order that depends on the sizes alone; a chunk whose fp32
 * sum leaves the type's normal range is summed again in binary64, so squares
 * that overflow or vanish in fp32 are not lost.
 */
ZERO_API int zero_tensors_norm(int n, const void *const *x, const int64_t *numel,
                               const int32_t *type, float inv_scale, double *tensor_sumsq,
                               zero_tensors_stat *stat, void *ws, size_t ws_bytes,
                               zero_stream_t stream);

/*
 * out = x * (inv_scale * c), formed in fp32 and rounded to out's type, with
 * c = min(1, max_norm / (sqrt(stat->sumsq) + 1e-6)) as the step's own clip;
 * c = 1 when stat->found_inf, so that what is not finite stays so and reaches
 * the step, which skips, and c = 1 when max_norm is 0 (no clipping) or sumsq is not
 * finite.
 *  out: NULL = in place (out_type is not read), or n pointers with the types
 *    out_type[n]; out[t] may equal x[t] when the types are the same.
 *    Pointers into the flat half buffer at the layout's tensor offsets make it
 *    the gradient that the step reads.
 *  inv_scale: under a loss scale S, 1 / S in zero_tensors_norm (max_norm is about
 *    the unscaled gradients) and, into the step's buffer, 1 here: the step
 *    divides what it reads by S itself, and the half type holds the small
 *    gradients only while they are scaled.  1 / S here gives unscaled
 *    gradients, for a reader that expects those.
 * In place with a factor of exactly 1 nothing is written.
 */
ZERO_API int zero_tensors_clip(int n, const void *const *x, const int64_t *numel,
                               const int32_t *type, void *const *out, const int32_t *out_type,
                               float inv_scale, double max_norm, const zero_tensors_stat *stat,
                               zero_stream_t stream);

/*
 * x[rows, cols] (F16, BF16 or F32) in 8 bits (fp8: ZERO_T_E4M3 or _E5M2).
 *  tile: 0 = a scale for each 1x128 block; 1 = for each 128x128 tile.
 *  q, s: x's 8-bit form, or both NULL.
 *  qt, st: the transpose's 8-bit form, [cols, rows] with blocks along x's
 *    rows: st[(r / 128) * ldst + c] (or c / 128 with tile), or both NULL.
 *  With tile = 1 both forms hold the same values.
 */
ZERO_API int zero_fp8_quantize(const void *x, int type, int64_t rows, int64_t cols, int64_t ldx,
                               int fp8, int tile, void *q, int64_t ldq, float *s, int64_t lds,
                               void *qt, int64_t ldqt, float *st, int64_t ldst,
                               zero_stream_t stream);

/* Bytes of workspace that zero_fp8_matmul needs for these sizes (0 for invalid
 * ones).  ZERO-FILL IT ONCE before its first use; a call leaves it ready for
 * the next one of any sizes that it is large enough for.  Its first 4 bytes
 * are an error word: nonzero if a kernel gave up waiting for its own copies
 * or products (never expected; that call's output is then undefined, and the
 * word stays until the caller clears it). */
ZERO_API size_t zero_fp8_matmul_workspace_bytes(int64_t m, int64_t n, int64_t k);

/*
 * out[i, j] = (add ? out[i, j] : 0) + sum over k-blocks b of
 *   sa[b, i] * sb[b, j] * (sum over k in b of a[i, k] * b[j, k])
 * a[m, k] has a scale for each 1x128 block, b[n, k] one for each 128x128 tile
 * (b_tile = 1) or 1x128 block (b_tile = 0), both as zero_fp8_quantize lays
 * them out.  Either may be E4M3 or E5M2.  The products of a block are summed
 * in fp32 by the tensor cores, the blocks in fp32 in ascending order (in
 * groups, the groups in ascending order, where few outputs make the kernel
 * split k: a rule on the sizes alone); out (F16, BF16 or F32) is rounded once.
 * sa * sb is formed first, in fp32: a product of scales below 2^-126 loses bits
 * (below 2^-150 its block counts as zero), one of 2^128 or more is infinite.
 *   forward:              a = activations [tokens, in],   b = weights [out, in] in tiles
 *   input's gradient:     a = gradients [tokens, out],    b = transposed weights [in, out] in tiles
 *   weights' gradient:    a = transposed gradients [out, tokens],
 *                         b = transposed activations [in, tokens], both in 1x128 blocks
 *  a, b: 16-byte aligned, lda and ldb multiples of 16 (ZERO_EALIGN).
 *  k = 0 gives out = 0 (or leaves it, with add).  A sum added to an fp32 out
 *    whose rows start on 16-byte boundaries is flushed to zero where it is below
 *    fp32's smallest normal number.
 */
ZERO_API int zero_fp8_matmul(const void *a, int a_type, int64_t lda, const float *sa, int64_t ldsa,
                             const void *b, int b_type, int64_t ldb, const float *sb, int64_t ldsb,
                             int b_tile, void *out, int out_type, int64_t ldo, int64_t m,
                             int64_t n, int64_t k, int add, void *ws, size_t ws_bytes,
                             zero_stream_t stream);

/*
 * For each row: h = x + residual, rounded to `type` (h = x without one);
 * rstd = 1 / sqrt(mean(h^2) + eps); y = h * rstd * w.
 *  x, residual (or NULL), h (or NULL), y (or NULL): [rows, cols] of `type`
 *    (F16 or BF16).  h may be x or residual itself.
 *  w: [cols] of w_type (F16, BF16 or F32).
 *  q, s: y (before its rounding to `type`) in 8 bits with a scale for each
 *    1x128 block, or both NULL.
 *  rstd: [rows] fp32, for the backward pass, or NULL.
 *  cols >= 1; eps >= 0.  The squares are summed in fp32: a row whose squares
 *    overflow it has rstd = 0.
 */
ZERO_API int zero_rmsnorm_fp8(const void *x, int64_t ldx, const void *residual, int64_t ldr,
                              const void *w, int w_type, int type, int64_t rows, int64_t cols,
                              float eps, void *h, int64_t ldh, void *y, int64_t ldy, int fp8,
                              void *q, int64_t ldq, float *s, int64_t lds, float *rstd,
                              zero_stream_t stream);

/* Bytes of workspace that zero_rmsnorm_backward needs (0 for invalid sizes;
 * contents undefined before and after). */
ZERO_API size_t zero_rmsnorm_workspace_bytes(int64_t rows, int64_t cols);

/*
 * Gradients of y = h * rstd * w (the rounding to 8 bits passes them on):
 *   xhat = h * rstd, g = dy * w
 *   dx = rstd * (g - xhat * mean(g * xhat)) + dresidual
 *   dw = (add_dw ? dw : 0) + sum over rows of dy * xhat
 * dx is the gradient of h and so of x and of the residual alike.
 *  dy, h, dresidual (or NULL), dx: [rows, cols] of `type`.  dx may be dy or
 *    dresidual itself.  dw: [cols] of dw_type (F16, BF16 or F32), or NULL.
 *  rows = 0: dw = 0 (or as it is, with add_dw).
 */
ZERO_API int zero_rmsnorm_backward(const void *dy, int64_t lddy, const void *h, int64_t ldh,
                                   const void *w, int w_type, const float *rstd,
                                   const void *dresidual, int64_t lddr, int type, int64_t rows,
                                   int64_t cols, void *dx, int64_t lddx, void *dw, int dw_type,
                                   int add_dw, void *ws, size_t ws_bytes, zero_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* ZEROSTEP_OPS_H */
