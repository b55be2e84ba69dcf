// Host side of the clipping of the multi-tensor step: argument validation. As
// in zs_api.cpp every argument is checked before anything is enqueued.
#include <cstdint>

#include "zs_checks.h"
#include "zs_clip_internal.h"

using namespace zs;

extern "C" {

int64_t zs_grad_stats_multi_workspace_bytes(const zs_plan* plan) {
    if (!plan || plan->layout != ZS_LAYOUT_PER_TENSOR) return -1;
    return norm_bytes((int64_t)plan->chunk_piece.size());
}

zs_status zs_grad_stats_multi(const zs_plan* plan, const void* workspace, double* sumsq_out, int32_t* nonfinite_out,
                              void* stats_workspace, int64_t stats_workspace_bytes, void* stream) {
    if (!plan) return report(ZS_EINVAL, "plan is NULL");
    BoundTables t;
    if (zs_status st = bound_tables(plan, workspace, kHasGrad, &t)) return st;
    if (zs_status st = check_array(sumsq_out, 8, "sumsq_out")) return st;
    if (zs_status st = check_array(nonfinite_out, 4, "nonfinite_out")) return st;
    if (zs_status st = check_array(stats_workspace, 16, "stats_workspace")) return st;
    const int64_t need = zs_grad_stats_multi_workspace_bytes(plan);
    if (stats_workspace_bytes < need)
        return report(ZS_ENOMEM, "stats_workspace holds %lld bytes, the call needs %lld",
                      (long long)stats_workspace_bytes, (long long)need);
    const Span out[3] = {span(sumsq_out, 8), span(nonfinite_out, 4), span(stats_workspace, need)};
    const char* name[3] = {"sumsq_out", "nonfinite_out", "stats_workspace"};
    const Span table = span(workspace, t.bytes);
    for (int i = 0; i < 3; ++i) {
        if (zs_status st = check_apart(out[i], table, name[i], "workspace")) return st;
        for (int j = i + 1; j < 3; ++j)
            if (zs_status st = check_apart(out[i], out[j], name[i], name[j])) return st;
    }
    trace_call("zs_grad_stats_multi", plan, 0, 0, plan->S, stream);
    return report_hip(launch_multi_norm(workspace, t, (int64_t)plan->chunk_piece.size(), sumsq_out, nonfinite_out,
                                        stats_workspace, stream),
                      "multi norm launch");
}

zs_status zs_adamw_shard_step_multi_clip(const zs_plan* plan, const zs_adamw_hparams* hps, int32_t n_groups,
                                         const float* scale, const int32_t* skip, const void* workspace,
                                         void* stream) {
    if (!plan) return report(ZS_EINVAL, "plan is NULL");
    BoundTables t;
    if (zs_status st = bound_tables(plan, workspace, kHasGrad | kHasState, &t)) return st;
    CoefTable ct;
    if (zs_status st = group_coefs(plan, hps, n_groups, &ct)) return st;
    if (zs_status st = check_opt_array(scale, 4, "scale")) return st;
    if (zs_status st = check_opt_array(skip, 4, "skip")) return st;
    trace_call("zs_adamw_shard_step_multi_clip", plan, 0, 0, plan->S, stream);
    return report_hip(launch_multi_clip(ct, workspace, t, (int64_t)plan->chunk_piece.size(), scale, skip, stream),
                      "multi clipped step launch");
}

}  // extern "C"
