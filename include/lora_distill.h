/*
 * lora_distill.h — distillation from a teacher's top logits, loss and
 * gradient, for NVIDIA B200 (sm_100a): C ABI.
 *
 * The operation.  Per row z of the student's bf16 logits [N, V], with the
 * teacher's K highest logits a_i at the vocabulary entries c_i:
 *
 *   t = s * z                       logit scaling (s = logit_scale)
 *   t = cap * tanh(t / cap)         if cap > 0 (softcap)
 *   q = softmax(t / T) over all V entries       (T = temperature)
 *   p = softmax(a / T) over the K entries
 *   loss = T^2 * sum_i p_i (log p_i - log q_{c_i})      (0 where p_i = 0)
 *
 *   backward, for an upstream gradient dloss of each row:
 *   dz_j = dloss * T * (q_j - sum of p_i with c_i = j) * dt_j/dz_j,
 *   dt/dz = s, or s * (1 - (t/cap)^2) with softcapping
 *
 * An entry whose id is -1 is absent (rows may have fewer than K entries).  A
 * row with no entry, or whose entries are all -inf, has loss 0 and gradient 0,
 * and so has a row whose label equals ignore_index (labels may be NULL: every
 * row takes part); labels are used for nothing else.  An id may stand twice in
 * a row: its terms add up.
 *
 * Layout and types.  logits and dlogits are bf16 with row stride ld elements
 * (ld >= V, a multiple of 8), 16-byte aligned; the teacher's values [N, K] are
 * bf16 or fp32 and its ids [N, K] int32 or int64, densely packed, aligned to
 * their own size; labels int64 [N]; loss and dloss fp32 [N].  N, V, K >= 1,
 * V <= 327680, K <= 1024.  A row of logits is read once and stays in the
 * shared memory of a thread-block cluster, so loss and gradient together move
 * 4 bytes a logit; dlogits may be the logits buffer itself.  The same call
 * gives the same bits; a row's last bits may depend on the rows beside it.
 * Other conventions: lora_step.h.
 *
 * The quotients 1 / T and s / T (with softcapping cap / T and s / cap) must stay
 * below 10^37.
 *
 * Logarithms of probabilities are fp32's: off by some 10^-5 and 2^-21 of their
 * distance from the row's largest, whatever the level of the logits.  With
 * softcapping 2^-22 cap / T is added up to cap = 128 T; above, t is formed to
 * fp32's precision first (2^-20 of the row's largest |t| / T), which takes about
 * 1.8 times as long.  A row's loss is T^2 times a difference of such logarithms,
 * and off by T^2 times as much.  Probabilities and gradients below 2^-126 may be 0.
 *
 * A teacher id below -1 or not below V is a device-side finding: the entry
 * counts as absent, the row's loss is NaN, and lora_step_device_status reports
 * LORA_MLP_ERR_INVALID_ARG.  LORA_MLP_ERR_DEVICE_TIMEOUT there means that a
 * wait between blocks ran out (about 2 s) and the results are not complete.
 */
#ifndef LORA_DISTILL_H
#define LORA_DISTILL_H

#include "lora_step.h"

#ifdef __cplusplus
extern "C" {
#endif

#define LORA_DISTILL_VALUES_BF16 0
#define LORA_DISTILL_VALUES_FP32 1
#define LORA_DISTILL_IDS_INT32 0
#define LORA_DISTILL_IDS_INT64 1

typedef struct lora_distill_shape {
    int64_t N;             /* rows (tokens)                                  */
    int64_t V;             /* logits per row                                 */
    int64_t ld;            /* row stride of logits and dlogits in elements   */
    int64_t K;             /* teacher entries per row                        */
    float temperature;     /* T, finite and > 0                              */
    float logit_scale;     /* s, finite and non-zero (1 = no scaling)        */
    float softcap;         /* cap: 0 = no softcapping, else finite and > 0   */
    int32_t values_type;   /* LORA_DISTILL_VALUES_*                          */
    int32_t ids_type;      /* LORA_DISTILL_IDS_*                             */
    int64_t ignore_index;  /* label of rows that take no part                */
} lora_distill_shape;

/* loss [N].  One launch. */
int lora_distill_forward(const lora_distill_shape* shape, const void* logits, const void* values, const void* ids,
                         const int64_t* labels, float* loss, void* stream);

/* dlogits [N, ld] (columns >= V untouched) for dloss [N].  One launch. */
int lora_distill_backward(const lora_distill_shape* shape, const void* logits, const void* values, const void* ids,
                          const int64_t* labels, const float* dloss, void* dlogits, void* stream);

/* dlogits for the upstream gradient dout[0] of the loss that
 * lora_distill_loss reduced: a row that takes part gets dloss = dout[0] *
 * fwd_out[1], fwd_out being that call's out.  One launch. */
int lora_distill_backward_reduced(const lora_distill_shape* shape, const void* logits, const void* values,
                                  const void* ids, const int64_t* labels, const float* dout, const float* fwd_out,
                                  void* dlogits, void* stream);

/* Reductions of the rows' losses into one. */
#define LORA_DISTILL_REDUCTION_SUM 1
#define LORA_DISTILL_REDUCTION_MEAN 2 /* over the rows whose label is not ignore_index (over 1 if there is none) */

/* Workspace bytes of lora_distill_loss (the rows' losses and a counter).  Host only. */
int lora_distill_sizes(const lora_distill_shape* shape, size_t* workspace_bytes);

/* The reduced loss and, where dlogits is not NULL, its gradient in the same
 * pass over the logits.  out is fp32 [2], 8-byte aligned: out[0] the loss
 * (summed in fp64 in a fixed order), out[1] its derivative with respect to the
 * loss of a row that takes part.  dlogits is the gradient of out[0].  Two
 * launches. */
int lora_distill_loss(const lora_distill_shape* shape, const void* logits, const void* values, const void* ids,
                      const int64_t* labels, int reduction, float* out, void* dlogits, void* workspace,
                      size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* LORA_DISTILL_H */
