/*
 * lora_qk_rope.h — norms of queries and keys for each head with the position
 * rotation in the same pass, forward and backward, for NVIDIA B200 (sm_100a):
 * C ABI.
 *
 * The operation, for each head x [D] of a query or key at position p, with
 * the gain [D] of the queries or of the keys:
 *
 *   n = x * rstd * gain,   rstd = 1 / sqrt(mean(x^2) + eps)
 *   y = R(p) n:  each pair (a, b) of the first `rot` elements turns by its angle,
 *       a' = a cos - b sin,   b' = b cos + a sin;   the elements behind stay.
 *
 * Pairs are (i, i + rot/2), or (2i, 2i + 1) with `interleaved`; pair i of
 * position p turns by the angle whose cosine and sine are cos[p, i] and
 * sin[p, i].  Without gains (q_gain = k_gain = NULL) there is no norm: n = x.
 *
 * Backward, for the gradient dy of y, with dn = R(p)^T dy:
 *
 *   dgain = sum over tokens and heads of dn * x * rstd
 *   dx    = rstd * (dn*gain - xh * mean(dn*gain*xh)),   xh = x * rstd
 *
 * (dx = dn without gains).  rstd is formed again from x: nothing is saved.
 * Arithmetic is fp32, each result rounded once.
 *
 * Layout and types.  Queries [B, S, Hq, D], keys [B, S, Hk, D], their results
 * and gradients are bf16 views: 16-byte aligned, strides of batch, position
 * and head in elements, multiples of 8, the D elements of a head next to each
 * other.  So parts of one projection's output and heads-first tensors need no
 * copy.  A view that is written does not overlap itself: in ascending order,
 * each of its strides is at least what the axes before it span.  It may be
 * exactly the view of the same heads that is read (q_out = q; dq = dq_out, or dq =
 * q), and overlaps no other.  cos and sin are fp32 [P, rot/2], 16-byte aligned; gains bf16 [D],
 * 16-byte aligned; their gradients fp32 [D], 4-byte aligned.  positions are
 * int64, 8-byte aligned: entry b * position_stride + s, in [0, P); NULL means
 * position s.  B, S, Hq, Hk >= 1; D and rot multiples of 16,
 * 16 <= rot <= D <= 512; B S (ceil(Hq / 2) + ceil(Hk / 2)) below 2^31.  Other
 * conventions: lora_step.h.
 *
 * A position outside [0, P) is a device-side finding: the heads of its token
 * get NaN (and add nothing to dgain), and lora_step_device_status reports
 * LORA_MLP_ERR_INVALID_ARG.
 */
#ifndef LORA_QK_ROPE_H
#define LORA_QK_ROPE_H

#include "lora_step.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct lora_qk_shape {
    int64_t B, S;            /* sequences, positions of each    */
    int64_t Hq, Hk;          /* heads of queries and of keys    */
    int64_t D;               /* elements of a head              */
    int64_t rot;             /* of which the first rot turn     */
    int64_t P;               /* rows of cos and sin             */
    int64_t position_stride; /* of positions between sequences (0: shared by all) */
    float eps;
    int32_t interleaved;     /* 0: pairs (i, i + rot/2), 1: (2i, 2i + 1) */
} lora_qk_shape;

/* A [B, S, heads, D] view; strides in elements. */
typedef struct lora_qk_view {
    void* data;
    int64_t stride_b, stride_s, stride_h;
} lora_qk_view;

/* q_out, k_out from q, k.  One launch. */
int lora_qk_rope_forward(const lora_qk_shape* shape, const lora_qk_view* q, const lora_qk_view* k,
                         const void* q_gain, const void* k_gain, const float* cos, const float* sin,
                         const int64_t* positions, const lora_qk_view* q_out, const lora_qk_view* k_out,
                         void* stream);

/* Workspace bytes of lora_qk_rope_backward for the gains' gradients; a call
 * without them needs none (workspace may be NULL).  Host only. */
int lora_qk_rope_sizes(const lora_qk_shape* shape, size_t* workspace_bytes);

/* dq, dk (views) and, where dq_gain and dk_gain are not NULL, the gains'
 * gradients, from the forward's q, k and the gradients dq_out, dk_out of its
 * results.  Without gains q and k are not read (they may be NULL), and
 * dq_gain, dk_gain must be NULL; the workspace is used for dq_gain and dk_gain
 * alone.  One launch, two with the gains' gradients. */
int lora_qk_rope_backward(const lora_qk_shape* shape, const lora_qk_view* q, const lora_qk_view* k,
                          const void* q_gain, const void* k_gain, const float* cos, const float* sin,
                          const int64_t* positions, const lora_qk_view* dq_out, const lora_qk_view* dk_out,
                          const lora_qk_view* dq, const lora_qk_view* dk, float* dq_gain, float* dk_gain,
                          void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* LORA_QK_ROPE_H */
