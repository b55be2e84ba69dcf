/*
 * zs_drafts.h -- verification of drafted tokens beside the log-probabilities of
 * zs_lm.h: a small model drafts some tokens of each request, the large one
 * computes the logits of all of them in one pass, and this call says how many
 * stand and draws the token behind them, so that what comes out is distributed
 * as the large model's own tokens.
 *
 * Conventions are those of zs_lm.h, with a caller-allocated device workspace:
 * a call in flight owns its workspace, which holds nothing between calls; two
 * calls (or two captured graphs) may use the same one only if one follows the
 * other on the device.
 */
#ifndef ZS_DRAFTS_H
#define ZS_DRAFTS_H

#include "zs_lm.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Drafted tokens a request may have. */
#define ZS_VERIFY_MAX_DRAFTS 64

/* Device workspace bytes of zs_verify_drafts; -1 on a bad argument. They serve
 * every call of no more requests, drafts and vocabulary. */
int64_t zs_verify_drafts_workspace_bytes(int64_t requests, int32_t drafts, int64_t vocab);

/* Request b has n_b = draft_lens[b] drafted tokens (draft_lens NULL: all have
 * `drafts`; a larger value counts as `drafts`): draft_tokens[b, i], i < n_b.
 * Row b * (drafts + 1) + i of target_logits is the target model's answer to the
 * request and its first i drafted tokens; row b * drafts + i of draft_logits is
 * what drafted token i was drawn from. Rows behind a request's are not read.
 * With p_i and q_i the softmax of those rows over temperature (draft_logits
 * NULL: q_i is 1 at the drafted token), x_i the drafted tokens and u the
 * request's row of uniforms [requests, drafts + 1], each in [0, 1):
 *   token i stands while u_i * q_i(x_i) < p_i(x_i);
 *   accepted[b] = a, the number that stand before the first that does not;
 *   tokens[b, 0 .. a-1] are those, and tokens[b, a] is drawn with u_drafts: from
 *     max(p_a - q_a, 0) if token a fell (from p_a if that is 0 everywhere),
 *     from p_n if all n_b stand: the lowest token whose running sum exceeds
 *     u_drafts times the sum of all; tokens[b, a+1 ..] = -1;
 *   logprobs[b, i] = log p_i(tokens[b, i]) for i <= a, 0 behind (optional).
 * Softmax, borders and running sums are computed in 64 bits, in which a token
 * less than 2^-1000 times as likely as the likeliest has probability 0. A logit
 * of -infinity is a masked token, never drawn; a drafted token outside [0,
 * vocab) falls, and without draft_logits takes nothing from p. u_drafts at or
 * above 1 draws the last token that has a share, a negative or NaN one the
 * first; a NaN u_i lets a token fall.
 *   draft_lens[b] < 0   the request is skipped: accepted 0, tokens -1,
 *                       logprobs 0; its rows do not matter.
 *   a NaN or +infinity in a row that is needed, or a needed target row of
 *   -infinity alone     the request ends there: accepted is that row's number,
 *                       the token -1 and its log-probability NaN.
 *   a draft row of -infinity alone   q = 0.
 * Logits are of one dtype; rows and strides as in zs_lm.h, with requests *
 * (drafts + 1) < 2^22; vocab in [1, 2^30], temperature in [1e-6, 1e6],
 * 0 <= drafts <= ZS_VERIFY_MAX_DRAFTS (0: one token is drawn from each row).
 * requests == 0 does nothing. draft_tokens and draft_logits may be NULL for
 * drafts == 0. workspace is 16-byte aligned. Outputs and workspace overlap
 * nothing else. */
zs_status zs_verify_drafts(const void* target_logits, int32_t dtype, int64_t requests, int32_t drafts, int64_t vocab,
                           int64_t target_stride, const void* draft_logits, int64_t draft_stride,
                           const int32_t* draft_tokens, const int32_t* draft_lens, const float* uniforms,
                           double temperature, int32_t* accepted, int32_t* tokens, float* logprobs, void* workspace,
                           int64_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* ZS_DRAFTS_H */
