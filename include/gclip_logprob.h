/*
 * gclip_logprob.h -- log probabilities of given tokens, with the entropy and
 * the likeliest alternatives, and their gradient: the loss that the backward
 * pass starts from whose gradients the list clips.
 *
 *   Backprop lesson (unhomeschool.com, vi), section "Forward pass": the
 *   logits of every position against the next token, a softmax cross entropy.
 *
 * Of each row x of `size` logits, with its target t:
 *
 *   m = max(x),  s = log(sum(exp(x - m))),  log p = x - m - s,
 *   logp = log p[t],  entropy = -sum(p * log p)
 *   top: the `top` largest log probabilities, largest first, and their
 *   columns; of equal ones the lowest column first
 *   gradient  dx = dlogp * (1[t] - p) - dentropy * p * (log p + entropy),
 *   from m and s, the row's stats: their sum alone, the logarithm of the sum
 *   of exponentials, loses s beside an m of large magnitude, as in a row of
 *   which a mask of the lowest finite number has left nothing
 *
 * Conventions: those of gclip_layer.h (matrices, in place, statuses, streams,
 * capture, bit-identical results).  Besides:
 *   - A logit of -infinity is a token that cannot come: p = 0, which adds
 *     nothing to the entropy and has no gradient but the target's own dlogp.
 *     In a row of nothing else m, s and logp are -infinity, the entropy is 0
 *     and so is the gradient.
 *     A row with a NaN or +infinity has NaN for its s, logp, entropy and
 *     gradient; its top counts a NaN above everything.
 *   - A row whose target is `ignore` counts for nothing, whatever it holds: its
 *     logp, entropy and gradient are 0 (its stats too), its top has columns -1
 *     with log probabilities of -infinity.  The forward call does not read such
 *     rows of more than 1024 logits; shorter ones, and all of them in the
 *     backward call, are read to no effect.  Any other target that is no column
 *     gives NaN for logp, and a gradient of NaN.
 *   - Sums are binary32, of at most 32 terms in a lane and then of those,
 *     relative to the largest logit so far; a row's results are taken from
 *     them in binary64 and rounded once, those of rows of up to 2048 logits in
 *     binary32.
 */
#ifndef GCLIP_LOGPROB_H
#define GCLIP_LOGPROB_H

#include <stdint.h>

#include "gclip.h"
#include "gclip_layer.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Most alternatives of a call. */
#define GCLIP_LOGPROB_MAX_TOP 32

typedef struct gclip_logprobs {
  int64_t rows, size;
  int32_t dtype; /* gclip_dtype of the logits */
  int32_t top;   /* 0 to GCLIP_LOGPROB_MAX_TOP, at most size; forward only */
  const void* logits;
  int64_t ld;
  const int64_t* targets; /* rows elements; NULL (forward only): no logp */
  int64_t ignore;         /* the target of rows that count for nothing */
  float* stats;           /* [rows][2]: m, s; forward: written, NULL: not wanted; backward: read */
  float* logp;            /* rows elements; forward only */
  float* entropy;         /* rows elements; backward: with dentropy */
  float* top_logp;        /* [rows][top] */
  int64_t* top_ids;       /* [rows][top] */
  const float* dlogp;     /* the rest: backward only.  Rows elements */
  const float* dentropy;  /* rows elements; NULL: none */
  void* dlogits;          /* may be logits */
  int64_t lddlogits;
  void* workspace; /* forward only: 16-byte aligned device memory, for this call alone until it has run */
  int64_t workspace_bytes; /* at least gclip_logprob_workspace(rows, size, top) */
} gclip_logprobs;

/* stats, logp, entropy and top, those whose pointers are given. */
gclip_status gclip_logprob_forward(const gclip_logprobs* a, void* stream);

/* dlogits of logp and entropy, from the forward call's stats and entropy. */
gclip_status gclip_logprob_backward(const gclip_logprobs* a, void* stream);

/* Bytes of workspace that a forward call of this shape needs; 0 for arguments
 * that such a call would refuse.  Host only. */
int64_t gclip_logprob_workspace(int64_t rows, int64_t size, int32_t top);

#ifdef __cplusplus
}
#endif

#endif /* GCLIP_LOGPROB_H */
