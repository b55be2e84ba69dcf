// Host side of the language-model operators: argument validation. As in
// zs_api.cpp every argument is checked before anything is enqueued.
#include <cstdint>

#include "zs_checks.h"
#include "zs_lm_internal.h"

namespace {

using namespace zs;

// Largest weight matrix: a wave (64 work-items) a row in one launch, columns
// counted in int32.
constexpr int64_t kMaxOut = int64_t(1) << 25;
constexpr int64_t kMaxIn = int64_t(1) << 29;

// What the calls over logits share.
zs_status check_logits(const void* logits, int32_t dtype, int64_t rows, int64_t vocab, int64_t row_stride,
                       float temperature) {
    if (zs_status st = check_dtype(dtype, "dtype")) return st;
    if (rows < 0 || rows > kMaxRows)
        return report(ZS_EINVAL, "rows = %lld outside [0, %lld]", (long long)rows, (long long)kMaxRows);
    if (vocab < 1 || vocab > kMaxVocab)
        return report(ZS_EINVAL, "vocab = %lld outside [1, 2^30]", (long long)vocab);
    if (zs_status st = check_stride(row_stride, vocab, "row_stride")) return st;
    if (zs_status st = check_temperature(temperature)) return st;
    if (rows == 0) return ZS_OK;
    return check_array(logits, (uintptr_t)elem_bytes(dtype), "logits");
}

// grad_logits is logits itself or lies apart from it.
zs_status check_grad(const void* logits, int32_t dtype, int64_t rows, int64_t vocab, int64_t row_stride,
                     const void* grad, int64_t grad_stride) {
    const int64_t esz = elem_bytes(dtype);
    if (zs_status st = check_array(grad, (uintptr_t)esz, "grad_logits")) return st;
    if (zs_status st = check_stride(grad_stride, vocab, "grad_stride")) return st;
    if (grad == logits && (grad_stride == row_stride || rows == 1)) return ZS_OK;
    return check_apart(matrix_span(grad, rows, vocab, grad_stride, esz),
                       matrix_span(logits, rows, vocab, row_stride, esz), "grad_logits", "logits");
}

}  // namespace

extern "C" {

zs_status zs_quant_matvec(const zs_plan* plan, int32_t tensor, int64_t out_features, int64_t in_features,
                          int32_t bits, int32_t block, const void* codes_all, const float* scales_all,
                          const void* x_bf16, int64_t x_stride, int32_t rows, void* y, int32_t y_dtype,
                          int64_t y_stride, void* stream) {
    if (!plan) return report(ZS_EINVAL, "plan is NULL");
    if (plan->layout != ZS_LAYOUT_FLAT) return report(ZS_EINVAL, "the quantized gather needs a FLAT plan");
    const int64_t n_scales = zs_quant_num_scales(plan, block);
    if (n_scales < 0 || zs_quant_code_bytes(plan, bits) < 0)
        return report(ZS_EINVAL, "bits = %d must be 4 or 8 and block = %d a power of two in [%d, %d]", bits, block,
                      zs::kQuantMinBlock, zs::kQuantMaxBlock);
    if (tensor < 0 || tensor >= (int32_t)plan->tensors.size())
        return report(ZS_EINVAL, "tensor %d is not one of the plan's %d", tensor, (int)plan->tensors.size());
    const zs::TensorEntry& t = plan->tensors[(size_t)tensor];
    if (out_features < 0 || in_features < 0 || out_features > kMaxOut || in_features > kMaxIn ||
        out_features * in_features != t.numel)
        return report(ZS_EINVAL, "tensor %d has %lld elements, not %lld x %lld (at most 2^25 x 2^29)", tensor,
                      (long long)t.numel, (long long)out_features, (long long)in_features);
    if (rows < 0 || rows > ZS_QUANT_MATVEC_MAX_ROWS)
        return report(ZS_EINVAL, "rows = %d outside [0, %d]", rows, ZS_QUANT_MATVEC_MAX_ROWS);
    if (zs_status st = check_dtype(y_dtype, "y_dtype")) return st;
    if (zs_status st = check_stride(x_stride, in_features, "x_stride")) return st;
    if (zs_status st = check_stride(y_stride, out_features, "y_stride")) return st;
    if (rows == 0 || out_features == 0) return ZS_OK;
    const int64_t y_esz = elem_bytes(y_dtype);
    if (zs_status st = check_array(y, (uintptr_t)y_esz, "y")) return st;
    if (in_features > 0) {
        if (zs_status st = check_array(codes_all, 16, "codes_all")) return st;
        if (zs_status st = check_array(scales_all, 16, "scales_all")) return st;
        if (zs_status st = check_array(x_bf16, 2, "x_bf16")) return st;
        const Span ys = matrix_span(y, rows, out_features, y_stride, y_esz);
        if (zs_status st = check_apart(ys, matrix_span(x_bf16, rows, in_features, x_stride, 2), "y", "x_bf16"))
            return st;
        if (zs_status st = check_apart(ys, span(codes_all, plan->T / 8 * bits), "y", "codes_all")) return st;
        if (zs_status st = check_apart(ys, span(scales_all, 4 * n_scales * plan->world), "y", "scales_all")) return st;
    }
    zs::QuantWeight w{codes_all, scales_all, t.flat_off,  out_features, in_features,
                      plan->S,   n_scales,   plan->world, bits,         0};
    while ((1 << w.block_shift) < block) ++w.block_shift;
    zs::trace_call("zs_quant_matvec", plan, 0, t.flat_off, t.numel, stream);
    return zs::report_hip(zs::launch_quant_matvec(w, zs::Rows{x_bf16, x_stride}, rows, y, y_dtype, y_stride, stream),
                          "quantized product launch");
}

zs_status zs_token_logprobs(const void* logits, int32_t dtype, int64_t rows, int64_t vocab, int64_t row_stride,
                            const int32_t* tokens, float temperature, float* logprob, float* entropy, float* stats,
                            int32_t top, int32_t* top_ids, float* top_logprobs, void* stream) {
    if (zs_status st = check_logits(logits, dtype, rows, vocab, row_stride, temperature)) return st;
    if (top < 0 || top > ZS_LOGPROBS_MAX_TOP || top > vocab)
        return report(ZS_EINVAL, "top = %d outside [0, min(vocab, %d)]", top, ZS_LOGPROBS_MAX_TOP);
    if (rows == 0) return ZS_OK;
    if (zs_status st = check_array(tokens, 4, "tokens")) return st;
    if (zs_status st = check_opt_array(logprob, 4, "logprob")) return st;
    if (zs_status st = check_opt_array(entropy, 4, "entropy")) return st;
    if (zs_status st = check_opt_array(stats, 4, "stats")) return st;
    if (top > 0) {
        if (zs_status st = check_array(top_ids, 4, "top_ids")) return st;
        if (zs_status st = check_array(top_logprobs, 4, "top_logprobs")) return st;
    } else if (top_ids || top_logprobs) {
        return report(ZS_EINVAL, "top_ids and top_logprobs need top > 0");
    }
    if (!logprob && !entropy && !stats && top == 0) return report(ZS_EINVAL, "no output is given");
    const Span in[2] = {matrix_span(logits, rows, vocab, row_stride, elem_bytes(dtype)), span(tokens, 4 * rows)};
    const char* in_name[2] = {"logits", "tokens"};
    const Span out[5] = {span(logprob, 4 * rows), span(entropy, 4 * rows), span(stats, 8 * rows),
                         span(top_ids, 4 * rows * top), span(top_logprobs, 4 * rows * top)};
    const char* out_name[5] = {"logprob", "entropy", "stats", "top_ids", "top_logprobs"};
    for (int i = 0; i < 5; ++i) {
        for (int j = 0; j < 2; ++j)
            if (zs_status st = check_apart(out[i], in[j], out_name[i], in_name[j])) return st;
        for (int j = i + 1; j < 5; ++j)
            if (zs_status st = check_apart(out[i], out[j], out_name[i], out_name[j])) return st;
    }
    const zs::LogprobsOut o{logprob, entropy, stats, top_ids, top_logprobs, top};
    zs::trace_call("zs_token_logprobs", nullptr, 0, 0, rows * vocab, stream);
    return zs::report_hip(zs::launch_logprobs(zs::Rows{logits, row_stride}, dtype, rows, vocab, tokens, temperature, o,
                                              stream),
                          "log-probability launch");
}

zs_status zs_token_logprobs_backward(const void* logits, int32_t dtype, int64_t rows, int64_t vocab,
                                     int64_t row_stride, const int32_t* tokens, float temperature,
                                     const float* stats, const float* entropy, const float* grad_logprob,
                                     const float* grad_entropy, void* grad_logits, int64_t grad_stride, void* stream) {
    if (zs_status st = check_logits(logits, dtype, rows, vocab, row_stride, temperature)) return st;
    if (rows == 0) return ZS_OK;
    if (zs_status st = check_array(tokens, 4, "tokens")) return st;
    if (zs_status st = check_array(stats, 4, "stats")) return st;
    if (zs_status st = check_array(grad_logprob, 4, "grad_logprob")) return st;
    if (zs_status st = check_opt_array(grad_entropy, 4, "grad_entropy")) return st;
    if (grad_entropy)
        if (zs_status st = check_array(entropy, 4, "entropy (needed by grad_entropy)")) return st;
    if (zs_status st = check_grad(logits, dtype, rows, vocab, row_stride, grad_logits, grad_stride)) return st;
    const Span g = matrix_span(grad_logits, rows, vocab, grad_stride, elem_bytes(dtype));
    const Span in[5] = {span(tokens, 4 * rows), span(stats, 8 * rows), span(grad_entropy ? entropy : nullptr, 4 * rows),
                        span(grad_logprob, 4 * rows), span(grad_entropy, 4 * rows)};
    const char* in_name[5] = {"tokens", "stats", "entropy", "grad_logprob", "grad_entropy"};
    for (int i = 0; i < 5; ++i)
        if (zs_status st = check_apart(g, in[i], "grad_logits", in_name[i])) return st;
    const zs::LogprobsGradIn gi{tokens, stats, entropy, grad_logprob, grad_entropy};
    zs::trace_call("zs_token_logprobs_backward", nullptr, 0, 0, rows * vocab, stream);
    return zs::report_hip(zs::launch_logprobs_grad(zs::Rows{logits, row_stride}, dtype, rows, vocab, temperature, gi,
                                                   grad_logits, grad_stride, stream),
                          "log-probability gradient launch");
}

zs_status zs_distill_topk(const void* logits, int32_t dtype, int64_t rows, int64_t vocab, int64_t row_stride,
                          const int32_t* teacher_ids, const float* teacher_logits, int32_t k, float temperature,
                          const float* row_weight, float* loss, void* grad_logits, int64_t grad_stride, void* stream) {
    if (zs_status st = check_logits(logits, dtype, rows, vocab, row_stride, temperature)) return st;
    if (k < 1 || k > ZS_DISTILL_MAX_K) return report(ZS_EINVAL, "k = %d outside [1, %d]", k, ZS_DISTILL_MAX_K);
    if (rows == 0) return ZS_OK;
    if (zs_status st = check_array(teacher_ids, 4, "teacher_ids")) return st;
    if (zs_status st = check_array(teacher_logits, 4, "teacher_logits")) return st;
    if (zs_status st = check_opt_array(row_weight, 4, "row_weight")) return st;
    if (zs_status st = check_array(loss, 4, "loss")) return st;
    if (grad_logits)
        if (zs_status st = check_grad(logits, dtype, rows, vocab, row_stride, grad_logits, grad_stride)) return st;
    const int64_t esz = elem_bytes(dtype);
    const Span l = span(loss, 4 * rows);
    const Span g = grad_logits ? matrix_span(grad_logits, rows, vocab, grad_stride, esz) : span(nullptr, 0);
    const Span in[3] = {span(teacher_ids, 4 * rows * k), span(teacher_logits, 4 * rows * k),
                        span(row_weight, 4 * rows)};
    const char* in_name[3] = {"teacher_ids", "teacher_logits", "row_weight"};
    for (int i = 0; i < 3; ++i) {
        if (zs_status st = check_apart(l, in[i], "loss", in_name[i])) return st;
        if (zs_status st = check_apart(g, in[i], "grad_logits", in_name[i])) return st;
    }
    if (zs_status st = check_apart(l, matrix_span(logits, rows, vocab, row_stride, esz), "loss", "logits")) return st;
    if (zs_status st = check_apart(l, g, "loss", "grad_logits")) return st;
    const zs::Teacher t{teacher_ids, teacher_logits, k, row_weight};
    zs::trace_call("zs_distill_topk", nullptr, 0, 0, rows * vocab, stream);
    return zs::report_hip(zs::launch_distill(zs::Rows{logits, row_stride}, dtype, rows, vocab, t, temperature, loss,
                                             grad_logits, grad_stride, stream),
                          "distillation launch");
}

}  // extern "C"
