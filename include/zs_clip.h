/*
 * zs_clip.h -- global-norm clipping of the multi-tensor step (zs.h): the norm of
 * the gradient over every bound piece of a PER_TENSOR plan, and AdamW from the
 * clipped gradient, with the non-finite skip. What zs_grad_stats and
 * zs_adamw_shard_step_accum are to one flat fp32 accumulator, these are to many
 * bf16 grad pieces:
 *
 *   zs_reduce_shard_multi            grad pieces (zs.h)
 *   zs_grad_stats_multi              this rank's squared norm and flag
 *   (all-gather of both over ranks)
 *   zs_clip_scale                    factor and skip (zs.h)
 *   zs_adamw_shard_step_multi_clip   the step
 *
 * Conventions are those of zs.h. Factor and skip stay on the device, and every
 * call may be captured into a HIP graph. A replay follows the gradient, the
 * factor and the skip; the step's hyperparameters are passed by value, so that it
 * repeats the step count and the learning rate of the call that was captured: a
 * training loop captures the norm and the factor and makes the step's call anew
 * (scalars in device memory are taken by the _dc calls of zs.h alone).
 * Replays read the table that `workspace` then holds: bound again to the same plan
 * and number of contributions, they follow the new pieces; unbound, the sum and
 * the flag are 0 and nothing is stepped. Bound to anything else, the graph has to
 * be captured again.
 */
#ifndef ZS_CLIP_H
#define ZS_CLIP_H

#include "zs.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Device bytes of zs_grad_stats_multi's stats_workspace; -1 for a NULL or FLAT
 * plan. */
int64_t zs_grad_stats_multi_workspace_bytes(const zs_plan* plan);

/* Over the grad pieces bound to `workspace`: *sumsq_out = the sum of the
 * elements' squares in double (a fixed-order reduction, so repeated calls give
 * identical bits) and *nonfinite_out = 1 if any element is NaN or infinite, else
 * 0; both are always written. A replicated tensor, which every rank holds whole,
 * counts in the sum of rank 0 alone, so that the ranks' sums add up to the
 * squared norm of the whole gradient; its elements are looked at for the flag on
 * every rank. grad has to be bound (a plan without elements gives 0 and 0).
 * sumsq_out is 8-byte, nonfinite_out 4-byte
 * aligned; stats_workspace 16-byte, owned by the call while it is in flight, and
 * holding nothing between calls. The three overlap neither each other nor
 * `workspace`. */
zs_status zs_grad_stats_multi(const zs_plan* plan, const void* workspace, double* sumsq_out, int32_t* nonfinite_out,
                              void* stats_workspace, int64_t stats_workspace_bytes, void* stream);

/* zs_adamw_shard_step_multi_groups with element gradient f32(grad) * *scale
 * (one fp32 product; scale NULL: 1), writing param and full where they are
 * bound. If skip is non-NULL and *skip != 0 nothing is written. scale and skip
 * are device pointers. grad, master, m and v have to be bound, unless the plan
 * has no elements. */
zs_status zs_adamw_shard_step_multi_clip(const zs_plan* plan, const zs_adamw_hparams* hps, int32_t n_groups,
                                         const float* scale, const int32_t* skip, const void* workspace,
                                         void* stream);

#ifdef __cplusplus
}
#endif

#endif /* ZS_CLIP_H */
