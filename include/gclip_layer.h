/*
 * gclip_layer.h -- the memory-bound layers of a pre-norm training step, next
 * to the gradient list that clips what they produce: layer norm, dropout
 * whose mask is never stored, and the residual step that runs both in one
 * pass, each with its gradient.
 *
 *   Backprop lesson (unhomeschool.com, vi), section "Forward pass": a block
 *   is x += attn(LN(x)); x += mlp(LN(x)).  Section "One gradient tensor per
 *   weight tensor": the norms' weight and bias each have a gradient, which
 *   the microbatches add up with += (section "Accumulation across
 *   microbatches") -- the `accumulate` flag below -- before the clip.
 *
 * Everything works on the rows of matrices of `size` columns:
 *
 *   norm      mean = sum(x) / size,  var = sum((x - mean)^2) / size,
 *             rstd = 1 / sqrt(var + eps),  y = (x - mean) * rstd * weight + bias
 *   gradient  n = (x - mean) * rstd,  g = dy * weight,
 *             dx = rstd * (g - sum(g) / size - n * sum(g * n) / size),
 *             dweight = sum over the rows of dy * n,  dbias = sum over the rows of dy
 *   dropout   y = x * s where kept, else 0 (a gclip_dropout below); its
 *             gradient is the same map
 *   residual  h = residual + dropout(x), rounded to the storage format, then
 *             y = norm(h) of the rounded h; its gradient
 *             dresidual = dh + (the norm's dx at h),  dx = dropout(dresidual)
 *
 * Conventions: those of gclip.h (device pointers, stream, statuses; argument
 * errors are detected on the host before anything is enqueued).  Besides:
 *   - Every call only enqueues kernels and keeps nothing between calls, so
 *     calls on different streams may overlap (with a workspace each) and any
 *     call may be captured into a HIP graph.
 *   - A matrix is an address and a leading dimension `ld...`: the distance of
 *     its rows in elements.  Columns are adjacent.  Any alignment to the
 *     element size and any ld will do: ld >= size for what is written, ld >= 0
 *     for what is read (0: one row for all).  16-byte alignment is faster.
 *   - What is written may be exactly a matrix that is read (same address and
 *     ld: in place), and otherwise overlaps nothing.  Two matrices that lie
 *     in one buffer as different columns of the same ld do not overlap.
 *   - Arithmetic is binary32, with one rounding to the storage format.  The
 *     statistics of rows of 8 to 16384 columns are binary32 sums, taken again
 *     of the row scaled by 2^-96 where they overflow; those of shorter and
 *     longer rows are binary64 sums.  So a finite row's y is finite unless it
 *     leaves the format itself, and so are its gradients while its sums of
 *     dy * weight, and of that times n, stay in binary32.
 *   - Results are bit-identical from run to run.  They may differ in the last
 *     bits between calls of other shapes: few rows take kernels that sum a row
 *     in another order (up to 512 rows forward; up to 2048 rows of up to 2048
 *     columns in a 16-bit format backward), so a token's y can depend on how
 *     many rows are with it.  h and the masks never do.
 *   - A NaN or infinity stays in its row (dweight and dbias apart), and
 *     where dropout drops an element it is 0 whatever it held.
 *   - rows may be 0: nothing is written but dweight and dbias, whose sums
 *     are then empty.  size is at least 1 for the norms.
 */
#ifndef GCLIP_LAYER_H
#define GCLIP_LAYER_H

#include <stdint.h>

#include "gclip.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Which elements a dropout keeps.  Element (r, c) takes the 16-bit half
 * number c mod 8 (the low half of a word first) of Philox4x32-10 (Salmon,
 * Moraes, Dror and Shaw, "Parallel random numbers: as easy as 1, 2, 3", SC
 * 2011) on the counter (c div 8, r, site, step + *d_step) under the key (low,
 * high word of seed), and is kept when that is at least
 * t = floor(65536 p + 1/2).  A kept element is multiplied by
 * 65536 / (65536 - t), rounded to binary32, so the mean is kept exactly for
 * the probability t / 65536 that is used (p to 16 bits: half as many
 * generator calls as with 32, and 2^-17 is far below what matters of a p).
 * The same values give the same mask, for the backward pass. */
typedef struct gclip_dropout {
  double p;               /* probability of dropping, 0 <= p <= 1 */
  uint64_t seed;
  uint32_t step;          /* another mask every step ... */
  uint32_t site;          /* ... and for every place of a step that drops */
  const uint32_t* d_step; /* device word, added to step modulo 2^32: a captured graph
                             gets a new mask each replay from it; NULL for none */
} gclip_dropout;

/* Largest extent of a matrix, in rows and in columns. */
#define GCLIP_LAYER_MAX_EXTENT 0x7ffffff0

/* One forward call. */
typedef struct gclip_layer_forward {
  int64_t rows, size;
  int32_t dtype;        /* gclip_dtype of the matrices */
  int32_t weight_dtype; /* of weight and bias: GCLIP_F32 or dtype */
  double eps;           /* finite, at least 2^-126 */
  const void* x;
  int64_t ldx;
  const void* residual; /* gclip_residual_forward only */
  int64_t ldresidual;
  const void* weight; /* size elements, or NULL: 1 */
  const void* bias;   /* size elements, or NULL: 0 */
  void* h;            /* gclip_residual_forward only */
  int64_t ldh;
  void* y;
  int64_t ldy;
  float* mean; /* rows elements each, for the backward pass; both NULL: not kept */
  float* rstd;
} gclip_layer_forward;

/* One backward call. */
typedef struct gclip_layer_backward {
  int64_t rows, size;
  int32_t dtype;        /* gclip_dtype of the matrices */
  int32_t weight_dtype; /* of weight: GCLIP_F32 or dtype */
  int32_t grad_dtype;   /* of dweight and dbias: GCLIP_F32 or dtype */
  int32_t accumulate;   /* nonzero: dweight and dbias are added to, with one rounding */
  const void* dy;       /* gradient of y */
  int64_t lddy;
  const void* dh; /* gradient of h from its other uses; gclip_residual_backward only; NULL: none */
  int64_t lddh;
  const void* x; /* the matrix that was normed: x, or the residual step's h */
  int64_t ldx;
  const float* mean; /* as the forward call left them */
  const float* rstd;
  const void* weight; /* NULL: 1 */
  void* dresidual;    /* gclip_residual_backward only */
  int64_t lddresidual;
  void* dx; /* NULL in gclip_residual_backward without a drop, where it would equal dresidual */
  int64_t lddx;
  void* dweight; /* size elements, or NULL: not wanted */
  void* dbias;   /* size elements, or NULL: not wanted */
  void* workspace; /* 16-byte aligned device memory, for this call alone until it has run */
  int64_t workspace_bytes; /* at least gclip_layer_workspace(rows, size) */
} gclip_layer_backward;

/* y = norm(x). */
gclip_status gclip_layernorm_forward(const gclip_layer_forward* a, void* stream);

/* dx, dweight and dbias of gclip_layernorm_forward. */
gclip_status gclip_layernorm_backward(const gclip_layer_backward* a, void* stream);

/* h = residual + dropout(x), y = norm(h).  drop may be NULL: none. */
gclip_status gclip_residual_forward(const gclip_layer_forward* a, const gclip_dropout* drop, void* stream);

/* dresidual, dx, dweight and dbias of gclip_residual_forward, with the same drop. */
gclip_status gclip_residual_backward(const gclip_layer_backward* a, const gclip_dropout* drop, void* stream);

/* y = dropout(x): forward, and with the gradient in x backward.  y may be x. */
gclip_status gclip_dropout_apply(const void* x, int64_t ldx, void* y, int64_t ldy, int64_t rows, int64_t size,
                                 int32_t dtype, const gclip_dropout* drop, void* stream);

/* Bytes of workspace that a backward call of this shape needs; 0 without
 * rows, and for arguments that such a call would refuse.  Host only. */
int64_t gclip_layer_workspace(int64_t rows, int64_t size);

#ifdef __cplusplus
}
#endif

#endif /* GCLIP_LAYER_H */
