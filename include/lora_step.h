/*
 * lora_step.h — what the operators around a fine-tuning step's dense layers
 * share (lora_embedding.h, lora_qk_rope.h, lora_distill.h): the device-side
 * status word, kernel timing and the launch count.
 *
 * Conventions are those of lora_mlp.h: 0 or a negative LORA_MLP_ERR_* code;
 * every pointer is caller-owned device memory of the current device; all work
 * is enqueued on `stream` (a cudaStream_t, NULL = legacy default stream);
 * nothing is allocated or synchronised; argument errors are found on the host
 * before anything is enqueued; results are bitwise deterministic.  A workspace
 * belongs to one call at a time: calls (or captured graphs) that may run at
 * once on several streams need one each.
 */
#ifndef LORA_STEP_H
#define LORA_STEP_H

#include <stddef.h>
#include <stdint.h>

#include "lora_mlp.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Reads and clears the device-side status of these operators on the current
 * device: LORA_MLP_OK, or LORA_MLP_ERR_INVALID_ARG after a token id, position
 * or teacher id outside its range (each header says what such an entry's
 * result is), or LORA_MLP_ERR_DEVICE_TIMEOUT after a bounded wait between
 * blocks ran out (lora_distill.h); after both, the latter.  Synchronises
 * `stream`. */
int lora_step_device_status(void* stream, int* status);

/* Kernel timing of these operators, as lora_mlp_timing_enable and
 * lora_mlp_timing_collect are for the others. */
int lora_step_timing_enable(int enable);
int lora_step_timing_collect(lora_mlp_kernel_time* out, int max, int* count);

/* Kernels of these operators launched in this process (all devices). */
int64_t lora_step_launch_count(void);

/* Test hook for the failure path, as lora_mlp_debug_force_timeout is for the
 * others: while enabled, no wait of the distillation's kernels is ever over, and
 * each gives up after `wait_cycles` SM cycles.  The kernels then return, with
 * LORA_MLP_ERR_DEVICE_TIMEOUT for lora_step_device_status and outputs that are
 * not complete.  enable = 0 restores normal operation.  Process-wide; not for
 * production. */
int lora_step_debug_force_timeout(int enable, int64_t wait_cycles);

#ifdef __cplusplus
}
#endif

#endif /* LORA_STEP_H */
