/*
 * peagle_sample.h -- C ABI of sampling on one GB300 (sm_103a): a token for
 * each row of logits, and the verification of drafts, whose results are the
 * num_accepted and sampled_ids of the next pe_expand_batch ([blog] "P-EAGLE:
 * Faster LLM Inference with Parallel Speculative Decoding in vLLM": the
 * target verifies the K drafts; accepted ones and one token more go into the
 * next step).  Beside pe_lmhead_argmax, which takes the largest logit.
 *
 * The distribution of a row of logits x_0 .. x_{V-1}.  NaN counts as -inf and
 * +inf as the largest finite fp32 number; m is the largest logit.
 *   e_i = exp((x_i - m) * inv) in fp32, inv = 1 / temperature in fp32
 *   W_i = e_i * 2^31, rounded to a whole number (ties to even; 0 for -inf)
 * Tokens in the order of falling logits (equal ones: the lower id first) are
 * kept while all of these hold:
 *   W_i > 0
 *   top-k   fewer than top_k tokens come before it (top_k <= 0: all pass)
 *   min-p   e_i >= min_p, that is a probability of at least min_p times the
 *           largest (min_p <= 0 or NaN: all pass; above 1: as 1)
 *   top-p   the W of the tokens before it sum to less than top_p times the W
 *           of all that pass the other two (top_p >= 1 or NaN: all pass);
 *           the first token always passes
 * A kept token has the probability W_i / total, total = sum of the kept W.
 * A temperature that is not above 0 (NaN too), or whose reciprocal is not
 * finite, keeps the first token alone: greedy.  All sums are of whole
 * numbers, so they are exact and no order of additions changes a token.
 * A token is drawn from a number u of [0, 1): the first one, in the order of
 * the ids, at which the kept W so far exceed floor(u * total) (both as fp64;
 * u outside [0, 1) is taken as the nearest inside, NaN as 0).  u has the numbers
 * that fp32 has, or those that its maker gives it (mostly 2^-24 apart): a token
 * into whose share of [0, 1) none of them falls is never drawn, so the tail is
 * drawn from as finely as u is, not as finely as W.
 *
 * Conventions are those of peagle.h: caller-owned device memory, asynchronous
 * on `stream`, host-checkable errors returned before anything is launched, no
 * C++ exception across the ABI, every tensor on the current device.
 * Data-dependent violations never trap: the kernel skips what it cannot do and
 * records the first code (PE_DEV_*, peagle.h) in *err, a caller-owned device
 * word that starts at 0 and is only ever changed from 0 (err may be NULL:
 * nothing is recorded).  No handle and no workspace: calls may overlap as
 * long as no buffer that one writes is used by the other.
 */
#ifndef PEAGLE_SAMPLE_H_
#define PEAGLE_SAMPLE_H_

#include <stdint.h>

#include "peagle.h"

#ifdef __cplusplus
extern "C" {
#endif

/* A row's distribution: token i is kept where W_i > 0 and its logit is above
 * `cut`, or equal to it with i <= cut_token.  32 bytes, 16-byte aligned. */
typedef struct {
  float max;         /* m; -inf: no token (every logit -inf or NaN) */
  float inv;         /* 1 / temperature; 0 for a greedy row */
  float cut;         /* logit and id of the last kept token; -inf and V - 1 */
  int32_t cut_token; /* where every token of W > 0 is kept */
  int64_t total;     /* sum of the kept W; 0: no token */
  int32_t token;     /* the token drawn; -1: none */
  int32_t reserved;  /* 0 */
} pe_dist;

/* Draw a token for each of `rows` rows of logits.
 *
 * logits [rows, vocab] of `dtype` (pe_dtype), rows `stride` elements apart.
 * temperature, top_k, top_p, min_p: [rows], or NULL (temperature 1; the
 * others: no such filter).  u [rows].  tokens [rows] (-1: the row has no
 * token); logprobs: NULL, or [rows], ln of the drawn token's probability
 * (-inf without a token); dist: NULL, or [rows], what pe_verify takes of a
 * drafter's rows.
 * PE_ERR_INVALID_ARGUMENT: rows or vocab < 1, another dtype, a stride
 * shorter than a row, a null pointer, logits or a vector not aligned to their
 * elements, dist not 16-byte aligned.  PE_ERR_UNSUPPORTED: vocab past 393216, rows past
 * 2^27. */
pe_status pe_sample(int32_t rows, int32_t vocab, int32_t dtype, const void* logits,
                    int64_t stride, const float* temperature, const int32_t* top_k,
                    const float* top_p, const float* min_p, const float* u, int32_t* tokens,
                    float* logprobs, pe_dist* dist, void* stream);

/* Verify the drafts of B requests by rejection sampling.
 *
 * The verify windows lie back to back, as in pe_expand_batch: request r has
 * rows cu_in[r] .. cu_in[r + 1] - 1, at least one; ids[t] is the token of row
 * t (a window's first token is known to be right, the others are its drafts)
 * and row t of the logits is the target's distribution after it, so row t
 * judges the draft ids[t + 1] and a window's last row judges none.  The
 * filters [B] are those of pe_sample, for all rows of a request.  With P the
 * probability in row t and Q that in the drafter's row:
 *   greedy drafts (draft_logits NULL): the draft d is accepted where accept_u
 *     < P(d).  The first rejected draft is replaced by a token drawn from P
 *     without d.
 *   sampled drafts: accepted where accept_u * Q(d) < P(d); replaced by a
 *     token drawn from max(P - Q, 0).
 * (As u * total < W(d) and u * Wq(d) * total < W(d) * totalq in fp64; a draft
 * with P(d) = 0 is never accepted, a greedy one with P(d) = 1 always; accept_u
 * is taken as it is, and one that is NaN accepts no other draft.  For
 * max(P - Q, 0): with p = W * a, q = Wq * aq in fp32, a = 2^31 / total
 * rounded to fp32, the weights are p - q in fp32, rounded to whole numbers;
 * where they sum to 0, p rounded to whole numbers.)
 * Where every draft is accepted, the token is drawn from the last row's P.
 * That token is drawn with u[r].
 *
 * logits [T, vocab] of `dtype`, rows `stride` apart; ids, accept_u [T];
 * cu_in [B + 1]; u [B].  draft_logits: NULL, or [T - B, vocab] of the same
 * dtype, rows draft_stride apart, the drafter's logits of all drafts in the
 * order of ids (row t's draft has row t - r of them); draft_dist [T - B], what
 * pe_sample wrote for them (T = B: both may be anything).
 * num_accepted [B]: drafts before the first rejected one; sampled_ids [B]:
 * the token after them (-1: the row has no token; pe_expand_batch takes both
 * as they are).  logprobs: NULL, or [T]: ln of the probability P of the token
 * that follows row t, for the accepted drafts and the drawn token (-inf: 0),
 * and 0 for the rows after it.  dist [T]: the rows' distributions (token: for
 * greedy drafts the one that a rejection in row t would give; for sampled
 * drafts -1, but for a window's last row).  Rows of no window are left as
 * they were.
 * Device errors: PE_DEV_BAD_ROW (a window that is empty, not within [0, T), or
 * out of order: an entry of cu_in before it lies behind its start, or one after
 * it before its end, so that windows that overlap are bad, each of them; or, of
 * sampled drafts, one whose drafts have no rows t - r within [0, T - B), as may
 * be beside empty windows: num_accepted 0 and sampled_ids -1, its rows are left
 * as they were, and the other windows are judged),
 * PE_DEV_BAD_TOKEN (a draft outside [0, vocab), behind a rejected one too:
 * rejected as one with P = 0, Q = 0).
 * PE_ERR_INVALID_ARGUMENT: B < 1, T < B, vocab < 1, another dtype, a stride
 * shorter than a row, a null or misaligned pointer, draft_logits without
 * draft_dist.  PE_ERR_UNSUPPORTED: vocab past 393216, T past 2^27. */
pe_status pe_verify(int32_t B, int32_t T, int32_t vocab, int32_t dtype, const void* logits,
                    int64_t stride, const int32_t* ids, const int32_t* cu_in,
                    const float* temperature, const int32_t* top_k, const float* top_p,
                    const float* min_p, const float* accept_u, const float* u,
                    const void* draft_logits, int64_t draft_stride, const pe_dist* draft_dist,
                    int32_t* num_accepted, int32_t* sampled_ids, float* logprobs, pe_dist* dist,
                    int32_t* err, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* PEAGLE_SAMPLE_H_ */
