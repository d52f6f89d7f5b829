/*
 * lora_embedding.h — token embedding lookup with scaling, and its gradient by
 * sorted tokens, for NVIDIA B200 (sm_100a): C ABI.
 *
 * The operation.  With a bf16 table E [V, d] and token ids [N]:
 *
 *   out[t] = bf16(scale * E[id_t])
 *   dE[v]  = scale * sum over t with id_t = v of dOut[t],   0 where no token has id v
 *
 * Tokens whose id is padding_idx add nothing to dE (their lookup is the
 * ordinary one).  Sums run in fp32 over the tokens of an id in a fixed order
 * that depends on the ids alone, and are rounded once.
 *
 * Layout and types.  E, out and dOut are bf16, row-major, densely packed,
 * 16-byte aligned; ids are int64, 8-byte aligned; dE is bf16 or fp32 [V, d],
 * every row written.  N, V and d are at least 1, N and d at most 2^30 and V at
 * most 2^31 - 2; d is a multiple of 8.  The gradient's sort reads 2 KB for each
 * pair of tiles of 4096 tokens in each pass: nothing beside dOut at a step's
 * usual size, as long as the rest at some 10^7 tokens, and far longer at the
 * limit.  Other conventions: lora_step.h.
 *
 * An id outside [0, V) is a device-side finding: its row of out is NaN, it
 * adds nothing to dE, and lora_step_device_status reports
 * LORA_MLP_ERR_INVALID_ARG.  (padding_idx is no such id, whatever its value.)
 */
#ifndef LORA_EMBEDDING_H
#define LORA_EMBEDDING_H

#include "lora_step.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Type of dE. */
#define LORA_EMBEDDING_GRAD_BF16 0
#define LORA_EMBEDDING_GRAD_FP32 1

/* out [N, d] from ids [N] and E [V, d].  One launch. */
int lora_embedding_forward(int64_t N, int64_t V, int64_t d, float scale, const int64_t* ids, const void* E,
                           void* out, void* stream);

/* Workspace bytes of lora_embedding_backward (sorted ids and the partial sums
 * of ids that many tokens share).  Host only. */
int lora_embedding_sizes(int64_t N, int64_t V, int64_t d, size_t* workspace_bytes);

/* dE [V, d] from dOut [N, d] and ids [N].  padding_idx < 0: none.  Three
 * launches for N <= 8192; above, three and one for each 9 bits of V. */
int lora_embedding_backward(int64_t N, int64_t V, int64_t d, float scale, int64_t padding_idx, int grad_type,
                            const int64_t* ids, const void* dOut, void* dE, void* workspace,
                            size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* LORA_EMBEDDING_H */
