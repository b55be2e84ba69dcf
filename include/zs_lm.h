/*
 * zs_lm.h -- language-model operators beside the shard-local step (zs.h):
 * what a training loop runs right before the step, where a loss turns logits
 * into the first gradient, and right after it, where the gathered low-bit
 * parameters are multiplied with.
 *
 *   zs_quant_matvec             products of a few rows with a weight matrix
 *                               read straight from the quantized gather's
 *                               payload (zs_quantize_shard's codes and scales)
 *   zs_token_logprobs           log-probabilities of given tokens, entropy
 *   zs_token_logprobs_backward  and the best alternatives, with the gradient
 *   zs_distill_topk             distillation from a teacher's top logits: loss
 *                               and gradient of the logits in one call
 *
 * Conventions are those of zs.h: caller-owned device memory, no allocation,
 * arguments validated on the host before anything is enqueued on `stream`, no
 * synchronization, zs_last_error(), one ZS_LOG trace line a call. None of the
 * calls needs a workspace, keeps anything from one call for the next or uses
 * an atomic on device memory: equal inputs give equal bits, and every call may
 * be captured into a HIP graph and run beside others on other streams. Kernels
 * run on the stream's device, which has to be current for a NULL stream and
 * has to hold every buffer of the call.
 *
 * Logits, gradients of logits, x and y are row-major matrices whose rows start
 * `stride` elements apart (the row's length <= stride <= 2^38) and need only be
 * aligned to their elements; elements between a row's end and the next row's
 * start are neither read nor written. Calls over logits take up to 2^22 - 1
 * rows. fp32 and int32 arrays are contiguous and
 * 4-byte aligned, codes_all and scales_all 16-byte aligned. Buffers that may
 * not overlap may still lie between each other's rows, as columns of one matrix
 * do; two matrices whose rows start different numbers of bytes apart have to
 * lie in address ranges apart.
 *
 * Sums, maxima and softmax statistics are held in fp32 or wider; a result is
 * rounded once, when it is stored.
 */
#ifndef ZS_LM_H
#define ZS_LM_H

#include "zs.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum zs_dtype { ZS_DTYPE_BF16 = 0, ZS_DTYPE_F32 = 1 } zs_dtype;

/* Rows of x one zs_quant_matvec call takes. */
#define ZS_QUANT_MATVEC_MAX_ROWS 64
/* Alternatives zs_token_logprobs lists. */
#define ZS_LOGPROBS_MAX_TOP 32
/* Teacher entries a row of zs_distill_topk holds. */
#define ZS_DISTILL_MAX_K 1024

/* ------------------------------------------------------------------ products with the quantized gather
 * y[r, o] = sum over i of W[o, i] * x[r, i], o < out_features, r < rows, with W
 * tensor `tensor` of the plan (out_features x in_features, row-major) as the
 * quantized gather delivers it: W[o, i] = f32(code) * scale, the value that
 * zs_dequant_gather rounds to bf16, here not rounded. codes_all and scales_all
 * are the N ranks' payloads end to end, exactly as zs_dequant_gather takes
 * them; nothing else of the payload is read. Any tensor offset, width, shard
 * length and block (a power of two in [8, 256]) is accepted. Products of 1 to 4
 * rows run near the memory's speed where tensor offset, in_features and shard
 * length are multiples of block and block >= 32; more rows take longer (28672 x
 * 8192 in 4 bits: 27 us with 1 row, 33 with 4, 45 with 16, 102 with 64), so do
 * blocks out of line with the rows, and smaller blocks longest. A block whose
 * scale is NaN (an infinity or NaN among its parameters) gives NaN in the rows
 * of W that have elements in it, and an infinity or NaN in x gives infinities
 * or NaN in its row of y. Codes are multiplied with x and summed over up to 128
 * columns before the scale: |x| up to 2^122 (4 bits) or 2^114 (8 bits) cannot
 * overflow there, larger values may give infinities or NaN in their row of y.
 *
 * FLAT plans. bits 4 or 8. out_features <= 2^25, in_features <= 2^29. x is bf16, y bf16 or fp32 (y_dtype).
 * 0 <= rows <= ZS_QUANT_MATVEC_MAX_ROWS (more rows: dequantize once and use a
 * matrix product); rows == 0 or out_features == 0 does nothing, in_features
 * == 0 gives zeros. y may not overlap any input. */
zs_status zs_quant_matvec(const zs_plan* plan, int32_t tensor, int64_t out_features, int64_t in_features,
                          int32_t bits, int32_t block, const void* codes_all, const float* scales_all,
                          const void* x_bf16, int64_t x_stride, int32_t rows, void* y, int32_t y_dtype,
                          int64_t y_stride, void* stream);

/* ------------------------------------------------------------------ log-probabilities of given tokens
 * Per row r of logits (vocab elements of dtype), with d_j = (logits[r, j] -
 * max) / temperature and s = sum of exp(d_j):
 *   stats[r]        = { max, log s }                 (two fp32; optional)
 *   logprob[r]      = d_t - log s, t = tokens[r]     (optional)
 *   entropy[r]      = log s - (sum of exp(d_j) d_j) / s  (optional)
 *   top_ids[r, i]   = the token with the i-th largest logit, i < top, the
 *                     lower token first among equal logits
 *   top_logprobs[r, i] = its log-probability
 * A logit of -infinity is a masked token: probability 0, log-probability
 * -infinity, nothing added to the entropy.
 *   tokens[r] < 0       the row is skipped: its logits do not matter, every
 *                       fp32 output of it is 0 and its top_ids are -1.
 *   tokens[r] >= vocab  logprob[r] is NaN, the other outputs as usual.
 *   every logit -infinity   logprob -infinity, entropy 0, stats { -infinity,
 *                       0 }, top_ids 0, 1, ... with -infinity.
 *   a NaN or +infinity in the row   logprob, entropy, log s and top_logprobs
 *                       are NaN and top_ids -1.
 * temperature in [1e-6, 1e6]. 0 <= top <= min(vocab, ZS_LOGPROBS_MAX_TOP);
 * top_ids and top_logprobs [rows, top] are given together, for top > 0 only.
 * vocab in [1, 2^30]. rows == 0 does nothing. Outputs may not overlap logits
 * or tokens. */
zs_status zs_token_logprobs(const void* logits, int32_t dtype, int64_t rows, int64_t vocab, int64_t row_stride,
                            const int32_t* tokens, float temperature, float* logprob, float* entropy, float* stats,
                            int32_t top, int32_t* top_ids, float* top_logprobs, void* stream);

/* The gradient of any loss over logprob and entropy: with p_j = exp(d_j -
 * log s) and l_j = log p_j from the forward call's stats,
 *   grad_logits[r, j] = ( grad_logprob[r] * ([j == t] - p_j)
 *                         - grad_entropy[r] * p_j * (l_j + entropy[r]) ) / temperature
 * of the logits' dtype. grad_entropy is optional; entropy (the forward call's)
 * is given with it. Skipped rows (token < 0) and rows whose every logit is
 * -infinity get zeros, other rows whose token is >= vocab or whose log s is NaN
 * get NaN. grad_logits may be logits itself (same address and stride); otherwise
 * the two may not overlap. */
zs_status zs_token_logprobs_backward(const void* logits, int32_t dtype, int64_t rows, int64_t vocab,
                                     int64_t row_stride, const int32_t* tokens, float temperature,
                                     const float* stats, const float* entropy, const float* grad_logprob,
                                     const float* grad_entropy, void* grad_logits, int64_t grad_stride, void* stream);

/* ------------------------------------------------------------------ distillation
 * The teacher gives k entries a row: token ids and fp32 logits (or
 * log-probabilities) [rows, k], in any order, a negative id marking an unused
 * entry. With T = temperature, q = softmax over the row's used entries of
 * teacher_logits / T and log p = log-softmax over the vocabulary of logits / T:
 *   loss[r]           = w T^2 * sum over entries of q (log q - log p[id])
 *   grad_logits[r, j] = w T * (p_j - sum over entries with id == j of q)
 * w = row_weight[r] (NULL: 1). grad_logits (optional) is of the logits' dtype
 * and is the gradient of the sum of the losses. An id that occurs twice counts
 * twice. An entry of teacher logit -infinity has q = 0 and adds nothing; a
 * token masked in the student (-infinity) that has q > 0 makes the loss
 * infinite, its gradient staying finite.
 *   row_weight[r] == 0, or no used entry with q > 0   loss 0, gradient 0; the
 *                       row's logits do not matter.
 *   every student logit -infinity   p = 0.
 *   an id >= vocab, a NaN or +infinity among the row's logits or used teacher
 *   logits              loss and the row's whole gradient are NaN.
 * 1 <= k <= ZS_DISTILL_MAX_K; temperature, vocab and the overlap rule as
 * above. */
zs_status zs_distill_topk(const void* logits, int32_t dtype, int64_t rows, int64_t vocab, int64_t row_stride,
                          const int32_t* teacher_ids, const float* teacher_logits, int32_t k, float temperature,
                          const float* row_weight, float* loss, void* grad_logits, int64_t grad_stride, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* ZS_LM_H */
