/*
 * gclip_block.h -- the memory-bound operators of a block of the kind that
 * most language models have now, next to those of gclip_layer.h: RMS norm
 * with the residual's addition, the (gated) activation, and what both can
 * leave in 8 bits: the norm's output, for a product of 8-bit operands, and
 * checkpoints of what a backward pass starts from, at half the bytes of a
 * 16-bit matrix.
 *
 *   Backprop lesson (unhomeschool.com, vi), section "Forward pass": a block
 *   is x += attn(norm(x)); x += mlp(norm(x)).  Section "One gradient tensor
 *   per weight tensor": the norm's weight has a gradient, which the
 *   microbatches add up with += (section "Accumulation across microbatches")
 *   -- the `accumulate` flag below -- before the clip.
 *
 * Everything works on the rows of matrices of `size` columns:
 *
 *   norm        rstd = 1 / sqrt(sum(x^2) / size + eps),  y = x * rstd * weight
 *   gradient    n = x * rstd,  g = dy * weight,
 *               dx = rstd * (g - n * sum(g * n) / size),
 *               dweight = sum over the rows of dy * n
 *   residual    h = residual + dropout(x), rounded to the storage format,
 *               then y = norm(h) of the rounded h; its gradient
 *               dresidual = dh + (the norm's dx at h),  dx = dropout(dresidual)
 *   activation  y = act(gate) * up, or act(gate) without up; its gradient
 *               dgate = dy * up * act'(gate),  dup = dy * act(gate)
 *   8 bits      scale = max(a / 448, 2^-112) with a the largest finite
 *               magnitude of the columns that share it; the value is
 *               v / scale rounded to e4m3 (OCP 8-bit float, largest 448), and
 *               stands for value * scale.  (In binary32: a times the rounded
 *               1/448, v times the rounded 1/scale.)  What is not finite
 *               becomes a NaN, which the clip's non-finite check finds later on.
 *
 * Conventions: those of gclip_layer.h (matrices, in place, overlaps, arithmetic
 * in binary32 with one rounding to the storage format, bit-identical results
 * from run to run, capture, rows of 0).  Besides:
 *   - The squares of a row of 8 to 16384 columns are summed in binary32, and
 *     again of the row scaled by 2^-96 where that overflows; those of others in
 *     binary64.  The gradients' sums are binary32, but for a row's of more than
 *     16384 columns: binary64, of binary32 sums of eight.
 *   - What an 8-bit matrix is given for is computed from the stored 8-bit
 *     values: the norm's gradient takes n = (value * scale) * rstd with the
 *     rstd of the forward pass.
 */
#ifndef GCLIP_BLOCK_H
#define GCLIP_BLOCK_H

#include <stdint.h>

#include "gclip.h"
#include "gclip_layer.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Columns that share a scale, counted from a row's first. */
#define GCLIP_SCALE_BLOCK 128

/* Which columns of a row share a scale. */
typedef enum gclip_scales {
  GCLIP_SCALES_BLOCK = 0, /* GCLIP_SCALE_BLOCK each: (size + 127) / 128 scales a row */
  GCLIP_SCALES_ROW = 1    /* all: one scale a row */
} gclip_scales;

/* A matrix in 8 bits.  values has an address and an ld that are multiples of
 * 8, and ld >= size: rows are read and written in groups of 8 bytes, so the
 * bytes from size to the next multiple of 8 are the row's too (what is
 * written there is unspecified, what is read there ignored). */
typedef struct gclip_packed8 {
  void* values; /* e4m3; NULL: there is none */
  int64_t ld;   /* distance of the rows in bytes */
  float* scales; /* [rows][scales a row], adjacent */
  int32_t mode; /* gclip_scales */
  int32_t reserved; /* 0 */
} gclip_packed8;

/* One forward call of the norm. */
typedef struct gclip_rms_forward {
  int64_t rows, size;
  int32_t dtype;        /* gclip_dtype of the matrices */
  int32_t weight_dtype; /* of weight: GCLIP_F32 or dtype */
  double eps;           /* finite, at least 2^-126 */
  const void* x;
  int64_t ldx;
  const void* residual; /* gclip_residual_rms_forward only */
  int64_t ldresidual;
  const void* weight; /* size elements, or NULL: 1 */
  void* h;            /* gclip_residual_rms_forward only */
  int64_t ldh;
  void* y; /* y or y8: one of them */
  int64_t ldy;
  gclip_packed8 y8;
  gclip_packed8 kept; /* of x, or of the residual step's h; GCLIP_SCALES_BLOCK */
  float* rstd;        /* rows elements, for the backward pass; NULL: not kept */
} gclip_rms_forward;

/* One backward call of the norm. */
typedef struct gclip_rms_backward {
  int64_t rows, size;
  int32_t dtype;        /* gclip_dtype of the matrices */
  int32_t weight_dtype; /* of weight: GCLIP_F32 or dtype */
  int32_t grad_dtype;   /* of dweight: GCLIP_F32 or dtype */
  int32_t accumulate;   /* nonzero: dweight is added to, with one rounding */
  const void* dy;       /* gradient of y */
  int64_t lddy;
  const void* dh; /* gradient of h from its other uses; gclip_residual_rms_backward only; NULL: none */
  int64_t lddh;
  const void* x; /* what was normed, x or the residual step's h; x or x8: one of them */
  int64_t ldx;
  gclip_packed8 x8;
  const float* rstd; /* as the forward call left it */
  const void* weight; /* NULL: 1 */
  void* dresidual;    /* gclip_residual_rms_backward only */
  int64_t lddresidual;
  void* dx; /* NULL in gclip_residual_rms_backward without a drop, where it would equal dresidual */
  int64_t lddx;
  void* dweight;   /* size elements, or NULL: not wanted */
  void* workspace; /* 16-byte aligned device memory, for this call alone until it has run */
  int64_t workspace_bytes; /* at least gclip_rms_workspace(rows, size) */
} gclip_rms_backward;

/* y = norm(x). */
gclip_status gclip_rmsnorm_forward(const gclip_rms_forward* a, void* stream);

/* dx and dweight of gclip_rmsnorm_forward. */
gclip_status gclip_rmsnorm_backward(const gclip_rms_backward* a, void* stream);

/* h = residual + dropout(x), y = norm(h).  drop may be NULL: none. */
gclip_status gclip_residual_rms_forward(const gclip_rms_forward* a, const gclip_dropout* drop, void* stream);

/* dresidual, dx and dweight of gclip_residual_rms_forward, with the same drop. */
gclip_status gclip_residual_rms_backward(const gclip_rms_backward* a, const gclip_dropout* drop, void* stream);

/* Bytes of workspace that a backward call of this shape needs; 0 without
 * rows, and for arguments that such a call would refuse.  Host only. */
int64_t gclip_rms_workspace(int64_t rows, int64_t size);

/* act(x); of a NaN a NaN. */
typedef enum gclip_activation {
  GCLIP_ACT_SILU = 0,      /* x / (1 + exp(-x)) */
  GCLIP_ACT_GELU = 1,      /* x (1 + erf(x / sqrt(2))) / 2 */
  GCLIP_ACT_GELU_TANH = 2, /* x (1 + tanh(sqrt(2 / pi) (x + 0.044715 x^3))) / 2 */
  GCLIP_ACT_RELU = 3       /* x above 0, else 0; its derivative at 0 is 0 */
} gclip_activation;

/* One forward or backward call of the activation. */
typedef struct gclip_activate {
  int64_t rows, size;
  int32_t dtype; /* gclip_dtype of the matrices */
  int32_t kind;  /* gclip_activation */
  const void* gate; /* backward: gate or gate8, one of them */
  int64_t ldgate;
  const void* up; /* NULL, up8 too: not gated */
  int64_t ldup;
  gclip_packed8 gate8; /* forward: written where given; backward: read; GCLIP_SCALES_BLOCK */
  gclip_packed8 up8;   /* as gate8, with up: both or neither */
  void* y;             /* backward: computed again where wanted; NULL: not wanted */
  int64_t ldy;
  const void* dy; /* the rest: gclip_activation_backward only */
  int64_t lddy;
  void* dgate;
  int64_t lddgate;
  void* dup; /* with up */
  int64_t lddup;
} gclip_activate;

/* y = act(gate) * up, and the checkpoints. */
gclip_status gclip_activation_forward(const gclip_activate* a, void* stream);

/* dgate and dup (and y) from dy, and gate and up or their checkpoints. */
gclip_status gclip_activation_backward(const gclip_activate* a, void* stream);

/* A matrix into 8 bits, and out of them. */
gclip_status gclip_pack(const void* x, int64_t ldx, const gclip_packed8* out, int64_t rows, int64_t size,
                         int32_t dtype, void* stream);
gclip_status gclip_unpack(const gclip_packed8* x, void* out, int64_t ldout, int64_t rows, int64_t size,
                           int32_t dtype, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* GCLIP_BLOCK_H */
