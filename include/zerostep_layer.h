/*
 * zerostep_layer.h — C ABI of libzerostep_layer.so: what lies between the 8-bit
 * products of a layer (zerostep_ops.h) on one GB300 GPU (sm_103a): the norms
 * behind and ahead of a block, the activation, and the tensors that the backward
 * pass needs, kept in 8 bits.
 *
 *   zero_gated_norms_fp8          norm of a block's output, its gate, the residual
 *                                 stream, the norm ahead of the next block, in 8 bits
 *   zero_gated_norms_backward     its gradients
 *   zero_activation_fp8           silu or gelu, gated or not, in 8 bits
 *   zero_activation_backward_fp8  its gradients in the 8-bit forms that the products
 *                                 of the inputs' and the weights' gradients take
 *   zero_fp8_restore              an 8-bit matrix read back, and transposed in 8 bits
 *
 * Conventions: as zerostep_ops.h (buffers of the caller, device pointers of the
 * current device, row-major matrices with a row stride in elements, elements
 * between a row's end and the next row neither read nor written, sizes 0 ..
 * 2^31 - 1025, work enqueued on `stream`, arguments validated before anything is
 * enqueued, the same return codes; calls can be captured in a CUDA graph; no
 * floating-point atomics, sums in an order that the sizes fix, and in
 * zero_gated_norms_backward whether o and h are kept in 8 bits).  An input may not
 * overlap an output, nor an output another, unless the description allows it.
 * Rows that start on 16-byte boundaries (8-bit ones: 8) run with wide accesses.
 *
 * Checkpoints.  What the backward pass reads of the forward pass is an 8-bit form
 * as zero_fp8_quantize makes it, E4M3 with an fp32 scale for each 1x128 block
 * (8.25 bits an element for 16), or the tensor itself in its half type.  The
 * gradients are those of the formulas below with the values that were kept.  Every
 * 8-bit output is the form that zero_fp8_quantize gives of the fp32 values.
 */
#ifndef ZEROSTEP_LAYER_H
#define ZEROSTEP_LAYER_H

#include "zerostep_ops.h"

#ifdef __cplusplus
extern "C" {
#endif

/* An 8-bit matrix with a scale for each 1x128 block: element (r, c) is
 * q[r * ld + c] * s[(c / 128) * lds + r].  Where a call takes a pointer to one,
 * NULL = not wanted. */
typedef struct {
    void *q;
    int64_t ld;
    float *s;
    int64_t lds;
} zero_fp8_form;

/* What a block's output is multiplied by on its way into the stream. */
typedef enum {
    ZERO_GATE_NONE = 0, /* nothing */
    ZERO_GATE_ONE = 1,  /* one number */
    ZERO_GATE_COLS = 2, /* [cols], one for each channel */
    ZERO_GATE_ROWS = 3  /* [rows], one for each token */
} zero_gate;

typedef enum {
    ZERO_ACT_SILU = 0, /* u sigmoid(u) */
    ZERO_ACT_GELU = 1  /* gelu's tanh form: u sigmoid(2 sqrt(2 / pi) (u + 0.044715 u^3)) */
} zero_act;

/*
 * For each row of the block's output o and the stream x:
 *   rstd_post = 1 / sqrt(mean(o^2) + eps),  n = o * rstd_post * w_post
 *     (without w_post there is no norm behind the block: n = o)
 *   h = scale * x + gate * n
 *   rstd_pre = 1 / sqrt(mean(h^2) + eps),   y = h * rstd_pre * w_pre
 *  o, x, h, y (or NULL): [rows, cols] of `type` (F16 or BF16).  h is rounded for
 *    storing; the norm and the 8-bit forms are of its fp32 value.  h may be x or o
 *    itself.
 *  w_post (or NULL), w_pre: [cols] of w_type; gate: as gate_kind says, of
 *    gate_type (both F16, BF16 or F32).
 *  y8: y in 8 bits (fp8: E4M3 or E5M2).  o8, h8: checkpoints of o and h (E4M3).
 *  rstd_post, rstd_pre: [rows] fp32, for the backward pass, or NULL.  rstd_post is
 *    not written without w_post.
 *  cols >= 1; eps >= 0.  The squares are summed in fp32: a row whose squares
 *    overflow it has rstd = 0.
 */
ZERO_API int zero_gated_norms_fp8(const void *o, int64_t ldo, const void *x, int64_t ldx,
                                  const void *w_post, const void *w_pre, int w_type,
                                  const void *gate, int gate_kind, int gate_type, float scale,
                                  int type, int64_t rows, int64_t cols, float eps, void *h,
                                  int64_t ldh, void *y, int64_t ldy, int fp8,
                                  const zero_fp8_form *y8, const zero_fp8_form *o8,
                                  const zero_fp8_form *h8, float *rstd_post, float *rstd_pre,
                                  zero_stream_t stream);

/* Bytes of workspace that zero_gated_norms_backward needs (0 for invalid sizes;
 * contents undefined before and after, 32-byte aligned).  One workspace may serve
 * one call after the other, of sizes that it is large enough for, not two at once. */
ZERO_API size_t zero_gated_norms_workspace_bytes(int64_t rows, int64_t cols);

/*
 * Gradients of zero_gated_norms_fp8.  xh = h * rstd_pre, xo = o * rstd_post (xo = o
 * and w_post = 1 without w_post):
 *   g = dy * w_pre,  dH = rstd_pre * (g - xh * mean(g * xh)) + dh
 *   dx = scale * dH
 *   G = gate * w_post * dH,  d_o = rstd_post * (G - xo * mean(G * xo))
 *     (d_o = gate * dH without w_post)
 *   dw_pre = sum over rows of dy * xh,  dw_post = sum over rows of gate * dH * xo
 *   dgate = w_post * dH * xo summed over what a gate's number is shared by
 *  dy, dh (the gradient that reaches h along the stream, or NULL), d_o, dx:
 *    [rows, cols] of `type`.  d_o may be dy and dx may be dh, or each the other.
 *  o, h: what was kept, both of `type` with so = sh = NULL, or both E4M3 with the
 *    scales so and sh of their 1x128 blocks.
 *  dw_pre, dw_post (without w_post: NULL), dgate: of dw_type (F16, BF16 or F32),
 *    dgate of the gate's shape; each or NULL.  add: dw_pre, dw_post and the dgate of
 *    one number or of channels are added to what is there; a token's dgate
 *    is written.
 *  ws: needed for dw_pre, dw_post and a dgate of one number or of channels.
 *  rows = 0: the sums are 0 (or as they are, with add).
 */
ZERO_API int zero_gated_norms_backward(const void *dy, int64_t lddy, const void *dh, int64_t lddh,
                                       const void *o, int64_t ldo, const float *so, int64_t ldso,
                                       const void *h, int64_t ldh, const float *sh, int64_t ldsh,
                                       const float *rstd_post, const float *rstd_pre,
                                       const void *w_post, const void *w_pre, int w_type,
                                       const void *gate, int gate_kind, int gate_type, float scale,
                                       int type, int64_t rows, int64_t cols, void *d_o,
                                       int64_t lddo, void *dx, int64_t lddx, void *dw_post,
                                       void *dw_pre, void *dgate, int dw_type, int add, void *ws,
                                       size_t ws_bytes, zero_stream_t stream);

/*
 * a = act(u) * v (a = act(u) without v).
 *  u, v (or NULL), a (or NULL): [rows, cols] of `type` (F16 or BF16).  a may be u
 *    or v itself.
 *  a8: a (before its rounding to `type`) in 8 bits (fp8: E4M3 or E5M2).
 *  u8, v8: checkpoints of u and v (E4M3).
 * The sigmoid counts as 0 where it is below 2^-126.
 */
ZERO_API int zero_activation_fp8(const void *u, int64_t ldu, const void *v, int64_t ldv, int act,
                                 int type, int64_t rows, int64_t cols, void *a, int64_t lda,
                                 int fp8, const zero_fp8_form *a8, const zero_fp8_form *u8,
                                 const zero_fp8_form *v8, zero_stream_t stream);

/*
 * Gradients of zero_activation_fp8 for the gradient da of a, and a again:
 *   du = da * v * act'(u),  dv = da * act(u)
 *  da: [rows, cols] of `type`.  u, v (or NULL): what was kept, of `type` with su = sv =
 *    NULL, or E4M3 with the scales of their 1x128 blocks.
 *  du, dv: [rows, cols] of `type`, or NULL.  Either may be da itself.
 *  du8, dv8: in 8 bits (fp8: E4M3 or E5M2).
 *  du8t, dv8t (fp8), a8t (E4M3): the transposes' 8-bit forms, [cols, rows] with
 *    blocks along the rows of u: the operands of the weights' gradients.
 *  Without v: dv, dv8 and dv8t are NULL.
 * Every form is that of the fp32 values, which are rounded once.
 */
ZERO_API int zero_activation_backward_fp8(const void *da, int64_t ldda, const void *u, int64_t ldu,
                                          const float *su, int64_t ldsu, const void *v, int64_t ldv,
                                          const float *sv, int64_t ldsv, int act, int type,
                                          int64_t rows, int64_t cols, void *du, int64_t lddu,
                                          void *dv, int64_t lddv, int fp8, const zero_fp8_form *du8,
                                          const zero_fp8_form *dv8, const zero_fp8_form *du8t,
                                          const zero_fp8_form *dv8t, const zero_fp8_form *a8t,
                                          zero_stream_t stream);

/*
 * x = q * s * row * col, formed in fp32: an 8-bit matrix q[rows, cols] (fp8: E4M3 or
 * E5M2) with scales s for 1x128 blocks read back, with a factor for each row and each
 * column (the norm of a checkpoint h is h * rstd * w).
 *  row: [rows] fp32 or NULL; col: [cols] of col_type (F16, BF16 or F32) or NULL.
 *  x: [rows, cols] of x_type (F16, BF16 or F32), or NULL.
 *  t8: the transpose's 8-bit form, [cols, rows] of q's type with blocks along q's
 *    rows.
 */
ZERO_API int zero_fp8_restore(const void *q, int fp8, int64_t ldq, const float *s, int64_t lds,
                              const float *row, const void *col, int col_type, int64_t rows,
                              int64_t cols, void *x, int x_type, int64_t ldx,
                              const zero_fp8_form *t8, zero_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* ZEROSTEP_LAYER_H */
