/*
 * specverify_rows.h - operators of libspecverify on the logits rows around the
 * verify step (include/specverify.h): what a server does to the rows before
 * it, and what a trainer of the draft does with them after it.
 *
 *   sv_adjust_logits      penalties for repeated tokens, biases and grammar
 *                         masks, applied to target and draft rows alike before
 *                         verification ("11.1 核心原理: Draft + Verify 与
 *                         Rejection Sampling", section 11.1.2: the transforms
 *                         of p are applied to q too)
 *   sv_top_logits         a teacher row's k best log-probabilities and the log
 *                         of the mass outside them
 *   sv_distill_forward,   the loss of a draft (student) row against such a
 *   sv_distill_backward,  record, its gradient, and both from one pass
 *   sv_distill_loss_grad  ("投机解码 Speculative Decoding", section 4.2: the
 *                         draft is distilled toward the target to raise the
 *                         acceptance rate)
 *
 * Memory, execution and error conventions are those of specverify.h: device
 * memory owned by the caller, contiguous row-major, asynchronous on `stream`
 * of the current device, arguments validated on the host before any launch,
 * data problems never fault.  logits, out, student and grad are 16-byte
 * aligned.  R = 0 or B = 0 is a valid empty call.
 */
#ifndef SPECVERIFY_ROWS_H
#define SPECVERIFY_ROWS_H

#include "specverify.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Limits checked by the entry points. */
#define SV_MAX_HISTORY (1 << 23)   /* tokens of one sequence's history */
#define SV_MAX_BIAS 1024           /* bias entries of one sequence */
#define SV_MAX_MASKS (1 << 24)     /* rows of the mask table */
#define SV_MAX_ROWS (1 << 24)      /* rows of one call */

/*
 * Penalties for repeated tokens, biases and masks.  Row i of sequence b
 * (i <= gamma, or gamma_b[b] in a ragged round) predicts the token after the
 * sequence's history and its drafts d_0 .. d_{i-1}.  For every token v, in
 * float32 and in this order, rounded once to the logits' type:
 *
 *   c    = occurrences of v among the generated tokens: history positions
 *          prompt_len .. history_len - 1 and the drafts before row i
 *   seen = c > 0 or v stands in the prompt (history positions < prompt_len)
 *   x    = logit;  if seen:  x = x > 0 ? x / repetition : x * repetition
 *   x   -= frequency * c + (c > 0 ? presence : 0)
 *   x   += the bias of v, where the sequence lists one
 *   x    = -inf where the row's mask does not allow v
 *
 *   B, gamma, V     sizes as in sv_verify_sample
 *   logits, out     [B][gamma+1][V] of `dtype`; out may be logits itself (in
 *                   place), otherwise the two must not overlap.  Rows behind a
 *                   ragged sequence's last are neither read nor written.
 *   draft_tokens    [B][gamma] int32, or NULL: no drafted token counts
 *   gamma_b         [B] int32 (clamped to [0, gamma]), or NULL: gamma
 *   history         [B][H] int32 tokens behind each sequence, H in
 *                   0..SV_MAX_HISTORY, with history_len [B] int32 (clamped to
 *                   [0, H]) and prompt_len [B] int32 (clamped to [0,
 *                   history_len]; NULL: 0).  NULL history: none.
 *   repetition      [B] float32 > 0, or NULL: 1
 *   frequency, presence  [B] float32, or NULL: 0
 *   bias_tokens, bias_values  [B][NB] int32 and float32, NB in
 *                   0..SV_MAX_BIAS.  Of a token listed twice the last entry
 *                   counts.
 *   mask            [M][ceil(V / 32)] 32-bit words, bit v % 32 of word v / 32
 *                   set where v is allowed, or NULL: everything is
 *   mask_index      [B][gamma+1] int32: the mask row of each logits row; a
 *                   negative index allows everything, one >= M nothing (the
 *                   row becomes -inf throughout, which the verify step reports
 *                   as SV_SEQ_BAD_ROW).  NULL: row i of sequence b uses mask
 *                   row b * (gamma+1) + i, and M must be B * (gamma+1).
 * Token ids outside [0, V) in drafts, history and biases count for nothing.
 * Needs no workspace.
 */
sv_status sv_adjust_logits(int B, int gamma, int V, const void* logits, sv_dtype dtype, void* out,
                           const int32_t* draft_tokens, const int32_t* gamma_b,
                           const int32_t* history, int H, const int32_t* history_len, const int32_t* prompt_len,
                           const float* repetition, const float* frequency, const float* presence,
                           const int32_t* bias_tokens, const float* bias_values, int NB,
                           const uint32_t* mask, int M, const int32_t* mask_index,
                           sv_stream_t stream);

/*
 * The record of teacher rows that distillation reads.  For each of R rows,
 * with K the first k of its tokens by (logit descending, index ascending):
 *
 *   indices    [R][k] int32     the tokens of K in that order; -1 where the
 *                               row has fewer than k logits above -inf
 *   logprobs   [R][k] float32   logit / temperature - lse, lse = ln sum_v
 *                               exp(logit_v / temperature); -inf where the
 *                               index is -1
 *   tail       [R] float32      ln sum_{v not in K} exp(logit_v / temperature)
 *                               - lse; -inf if nothing is left outside
 *
 * A row holding NaN or +inf, or only -inf, gives indices -1 and NaN values.
 * k in 1..SV_MAX_TOP_K; logits [R][V] of `dtype`, R in 0..SV_MAX_ROWS.  The
 * workspace follows the contract of specverify.h (zero-filled before its
 * first use, left zero-filled, one per concurrent call);
 * sv_top_logits_workspace_bytes returns 0 for invalid sizes (it asks the
 * current device for its number of SMs: with at least as many rows a call
 * needs no more than the minimum, so fewer rows can need more than many).
 */
size_t sv_top_logits_workspace_bytes(int R, int V, int k);
sv_status sv_top_logits(int R, int V, const void* logits, sv_dtype dtype, int k, float temperature,
                        int32_t* indices, float* logprobs, float* tail,
                        void* workspace, size_t workspace_bytes, sv_stream_t stream);

/*
 * Distillation from a teacher's top logits.  For each of R rows, with the
 * student's q = softmax(student / temperature) over V tokens and the teacher's
 * p = softmax over the row's listed log-probabilities (and the tail's, if
 * given: then p has one more outcome, "any token not listed", whose student
 * probability is q_t = sum of q over the tokens not listed):
 *
 *   loss = weight * ( sum_j p_j (ln p_j - ln q[indices_j])
 *                     + p_t (ln p_t - ln q_t) )
 *   dloss/dstudent_v = weight / temperature *
 *        ( q_v - sum_{j: indices_j = v} p_j     v listed
 *          q_v (1 - p_t / q_t)                  otherwise )
 *
 * (p_t = 0 without a tail; terms with p = 0 are 0, and so are those of a p
 * that lies below float32's range, 2^-125 of the largest.)  The softmax over the
 * listed values makes them logits as much as log-probabilities: a constant
 * added to a row's values (tail included) changes nothing.  The loss is not
 * scaled by temperature^2.
 *
 *   student     [R][V] of `dtype`
 *   indices, logprobs  [R][k] int32 and float32, k in 1..SV_MAX_TOP_K; entries
 *               whose index is outside [0, V) are ignored; a token listed
 *               twice counts with both values, and once in q
 *   tail        [R] float32, or NULL: no such outcome
 *   weight      [R] float32, or NULL: 1.  A row whose weight is 0 costs no pass
 *               over its logits and may hold anything: loss 0, gradient 0.
 *   loss        [R] float32
 *   stats       [R][SV_DISTILL_STAT_WORDS] float32 written by the forward
 *               pass for the backward pass of the same inputs
 *   grad_loss   [R] float32, the gradient with respect to each row's loss
 *               (grad_loss_stride 1), or one value for all rows
 *               (grad_loss_stride 0, what a sum of the losses hands back)
 *   grad        [R][V] of `dtype`; sv_distill_loss_grad forms the gradient of
 *               the sum of the losses.  grad may be student itself (in
 *               place), otherwise the two must not overlap.
 *
 * A row with no usable entry and no tail has loss 0 and gradient 0.  A student
 * row that holds NaN or +inf, or only -inf, or a teacher row that holds NaN or
 * +inf, gives NaN.  Warps that wait for one another do so for a second or so at most,
 * where a row takes microseconds; if a wait runs out nevertheless, losses,
 * statistics and gradients of all rows that it may concern are NaN throughout.
 * No workspace.
 *
 * The calls that form the loss are fastest for k <= 256 and rows of at most
 * 131072 float32 or 262144 16-bit values; beyond, another kernel takes two to
 * three times as long (512 float32 rows, k = 64: 66 us at V = 131072, 212 at
 * V = 152064).
 */
#define SV_DISTILL_STAT_WORDS 8
sv_status sv_distill_forward(int R, int V, const void* student, sv_dtype dtype, const int32_t* indices,
                             const float* logprobs, const float* tail, int k, float temperature, const float* weight,
                             float* loss, float* stats, sv_stream_t stream);
sv_status sv_distill_backward(int R, int V, const void* student, sv_dtype dtype, const int32_t* indices,
                              const float* logprobs, int k, float temperature, const float* weight,
                              const float* stats, const float* grad_loss, int grad_loss_stride, void* grad,
                              sv_stream_t stream);
sv_status sv_distill_loss_grad(int R, int V, const void* student, sv_dtype dtype, const int32_t* indices,
                               const float* logprobs, const float* tail, int k, float temperature, const float* weight,
                               float* loss, void* grad, sv_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* SPECVERIFY_ROWS_H */
