// Host side of the verification of drafted tokens: argument validation. As in
// zs_api.cpp every argument is checked before anything is enqueued.
#include <cstdint>

#include "zs_checks.h"
#include "zs_drafts_internal.h"

namespace {

using namespace zs;

zs_status check_sizes(int64_t requests, int32_t drafts, int64_t vocab) {
    if (drafts < 0 || drafts > ZS_VERIFY_MAX_DRAFTS)
        return report(ZS_EINVAL, "drafts = %d outside [0, %d]", drafts, ZS_VERIFY_MAX_DRAFTS);
    if (requests < 0 || requests > kMaxRows / (drafts + 1))
        return report(ZS_EINVAL, "requests = %lld outside [0, %lld] for %d drafted tokens", (long long)requests,
                      (long long)(kMaxRows / (drafts + 1)), drafts);
    if (vocab < 1 || vocab > kMaxVocab)
        return report(ZS_EINVAL, "vocab = %lld outside [1, 2^30]", (long long)vocab);
    return ZS_OK;
}

}  // namespace

extern "C" {

int64_t zs_verify_drafts_workspace_bytes(int64_t requests, int32_t drafts, int64_t vocab) {
    if (check_sizes(requests, drafts, vocab)) return -1;
    return verify_layout(requests, drafts, vocab).bytes;
}

zs_status zs_verify_drafts(const void* target_logits, int32_t dtype, int64_t requests, int32_t drafts, int64_t vocab,
                           int64_t target_stride, const void* draft_logits, int64_t draft_stride,
                           const int32_t* draft_tokens, const int32_t* draft_lens, const float* uniforms,
                           double temperature, int32_t* accepted, int32_t* tokens, float* logprobs, void* workspace,
                           int64_t workspace_bytes, void* stream) {
    if (zs_status st = check_dtype(dtype, "dtype")) return st;
    if (zs_status st = check_sizes(requests, drafts, vocab)) return st;
    if (zs_status st = check_stride(target_stride, vocab, "target_stride")) return st;
    if (draft_logits)
        if (zs_status st = check_stride(draft_stride, vocab, "draft_stride")) return st;
    if (zs_status st = check_temperature(temperature)) return st;
    if (requests == 0) return ZS_OK;
    const int64_t esz = elem_bytes(dtype), places = requests * (drafts + 1);
    if (zs_status st = check_array(target_logits, (uintptr_t)esz, "target_logits")) return st;
    if (zs_status st = check_opt_array(draft_logits, (uintptr_t)esz, "draft_logits")) return st;
    if (drafts > 0)
        if (zs_status st = check_array(draft_tokens, 4, "draft_tokens")) return st;
    if (zs_status st = check_opt_array(draft_lens, 4, "draft_lens")) return st;
    if (zs_status st = check_array(uniforms, 4, "uniforms")) return st;
    if (zs_status st = check_array(accepted, 4, "accepted")) return st;
    if (zs_status st = check_array(tokens, 4, "tokens")) return st;
    if (zs_status st = check_opt_array(logprobs, 4, "logprobs")) return st;
    if (zs_status st = check_array(workspace, 16, "workspace")) return st;
    const VerifyLayout layout = verify_layout(requests, drafts, vocab);
    if (workspace_bytes < layout.bytes)
        return report(ZS_ENOMEM, "workspace holds %lld bytes, the call needs %lld", (long long)workspace_bytes,
                      (long long)layout.bytes);
    const void* tokens_in = drafts > 0 ? draft_tokens : nullptr;
    const void* draft_in = drafts > 0 ? draft_logits : nullptr;
    const Span in[5] = {matrix_span(target_logits, places, vocab, target_stride, esz),
                        draft_in ? matrix_span(draft_in, requests * drafts, vocab, draft_stride, esz) : span(nullptr, 0),
                        span(tokens_in, 4 * requests * drafts), span(draft_lens, 4 * requests),
                        span(uniforms, 4 * places)};
    const char* in_name[5] = {"target_logits", "draft_logits", "draft_tokens", "draft_lens", "uniforms"};
    const Span out[4] = {span(accepted, 4 * requests), span(tokens, 4 * places), span(logprobs, 4 * places),
                         span(workspace, layout.bytes)};
    const char* out_name[4] = {"accepted", "tokens", "logprobs", "workspace"};
    for (int i = 0; i < 4; ++i) {
        for (int j = 0; j < 5; ++j)
            if (zs_status st = check_apart(out[i], in[j], out_name[i], in_name[j])) return st;
        for (int j = i + 1; j < 4; ++j)
            if (zs_status st = check_apart(out[i], out[j], out_name[i], out_name[j])) return st;
    }
    const VerifyArgs a{Rows{target_logits, target_stride}, Rows{draft_in, draft_stride}, requests, vocab, drafts,
                       static_cast<const int32_t*>(tokens_in), draft_lens, uniforms, accepted, tokens, logprobs};
    trace_call("zs_verify_drafts", nullptr, 0, 0, places * vocab, stream);
    return report_hip(launch_verify(a, dtype, temperature, workspace, stream), "verification launch");
}

}  // extern "C"
