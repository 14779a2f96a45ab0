/*
 * peagle_cache.h -- C ABI of the paged KV cache operators on one GB300
 * (sm_103a): writing new tokens into a cache, attending to it one token at a
 * time, and trimming it by accumulated attention weight.
 *
 * They work on the pools that pe_draft_forward reads ([blog] "P-EAGLE:
 * Faster LLM Inference with Parallel Speculative Decoding in vLLM",
 * engineering section: paged KV cache, block tables), one layer at a time
 * (pe_kv_evict: several layers), without a handle.
 *
 * Position p of a request lives in page block_table[r][p / 16], offset
 * p % 16, and its key is rotated to angle p * theta^(-2 i / head_dim)
 * (rotate-half pairs (i, i + head_dim / 2)), as in pe_draft_forward.
 *
 * Conventions are those of peagle.h: caller-owned device memory unless a
 * parameter says "host", asynchronous on `stream`, host-checkable errors
 * returned before anything is launched, no C++ exception across the ABI.
 * Every tensor lives on the current device.  Data-dependent violations never
 * trap: the kernel skips what it cannot do and records the first code
 * (PE_DEV_*, peagle.h) in *err, a caller-owned device word that starts at 0
 * and is only ever changed from 0 (err may be NULL: nothing is recorded).
 * No call waits on another CTA's progress except at a cluster barrier.
 * Overlapping calls are safe as long as no buffer that one writes (pools,
 * outputs, workspace) is used by the other.
 */
#ifndef PEAGLE_CACHE_H_
#define PEAGLE_CACHE_H_

#include <stdint.h>

#include "peagle.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  PE_KV_BF16 = 0,
  PE_KV_F32 = 1,
  PE_KV_E4M3 = 2 /* OCP FP8 E4M3 codes, one byte an element (pe_set_kv_cache_fp8) */
} pe_kv_dtype;

/* One layer's pools.  k, v: [num_blocks, n_kv_heads, 16, head_dim] of dtype;
 * e4m3 pools stand for code * k_scale (v_scale), the scales are not used
 * otherwise.  scores: NULL, or [num_blocks, n_kv_heads, 16] fp32, the weight
 * that each cached position has received so far.  All 16-byte aligned;
 * head_dim 64 or 128.  q and the new k and v rows are fp32 beside PE_KV_F32
 * pools and bf16 beside the others ("activation type" below). */
typedef struct {
  void* k;
  void* v;
  float* scores;
  int32_t num_blocks;
  int32_t n_kv_heads;
  int32_t head_dim;
  int32_t dtype; /* pe_kv_dtype */
  float k_scale;
  float v_scale;
} pe_kv_pool;

/* Rotate T new rows of q and k to their positions and write k and v into the
 * cache.
 *
 * Row t belongs to request req[t] (req NULL: request t, and T = B) and sits
 * at position pos[t].  q_out[t] = rotated q[t]; the page slot of pos[t] gets
 * the rotated k[t] and v[t], and its score (where the pool has scores) 0.
 * rope_theta 0 rotates nothing.  Angles are right to 2^-26 of a turn and, for
 * rope_theta >= 1, pos * 2^-51 of one; results are rounded once to their type (e4m3: x / scale, nearest even,
 * saturated at +-448).  A row with pos[t] < 0 is padding: nothing of it is
 * written.
 *
 * q [T, n_heads, head_dim] (NULL: no q, then q_out is NULL too), k, v [T,
 * n_kv_heads, head_dim], q_out like q: rows `*_stride` elements apart, heads
 * contiguous, rows 16-byte aligned.  q_out may be q itself.  block_table [B,
 * bt_stride].  No two rows may name the same slot.
 * Device errors: PE_DEV_BAD_ROW (req outside [0, B)), PE_DEV_BAD_POSITION
 * (pos past the table), PE_DEV_BAD_BLOCK: the row's k and v are not written
 * (q_out is).
 * PE_ERR_INVALID_ARGUMENT: T or B < 1, req NULL with T != B, n_heads not a
 * positive multiple of n_kv_heads, a stride shorter than a row, a null or
 * misaligned pointer, rope_theta negative or not finite.
 * PE_ERR_UNSUPPORTED: head_dim other than 64 and 128. */
pe_status pe_kv_append(const pe_kv_pool* pool, int32_t T, int32_t B, int32_t n_heads,
                       float rope_theta, const void* q, int64_t q_stride, const void* k,
                       int64_t k_stride, const void* v, int64_t v_stride, const int32_t* pos,
                       const int32_t* req, const int32_t* block_table, int32_t bt_stride,
                       void* q_out, int64_t q_out_stride, int32_t* err, void* stream);

/* Bytes of workspace of a pe_attn_decode call of B requests on the current
 * device; 0 on a bad argument.  bt_stride 0: what every call needs (the
 * lengths do not matter).  bt_stride > 0: with room for the logits of a table
 * of that width, at most 1 GiB of them, which a call with accumulate keeps
 * there instead of working them out twice.  It keeps those of up to 16 query
 * heads a kv head (fp32 pools: 8 of head_dim 64, 4 of 128); with more heads
 * none, and bt_stride changes nothing past 16 (fp32: give 0). */
int64_t pe_attn_decode_workspace(int32_t B, int32_t n_heads, int32_t n_kv_heads,
                                 int32_t head_dim, int32_t bt_stride);

/* Attention of one new token per request over its cached positions.
 *
 * Query head h of request b attends kv head h / (n_heads / n_kv_heads) at
 * positions max(0, seq_lens[b] - window) .. seq_lens[b] - 1 (window 0: all):
 * out[b, h] = sum_j softmax_j(scale q.k_j) v_j, lse[b, h] = ln sum_j
 * exp(scale q.k_j).  The new token's own k and v are cached already
 * (pe_kv_append).  A row that attends nothing (seq_lens[b] <= 0, or every
 * logit -inf) gives 0 and -inf.  Nothing past seq_lens[b] and no page that
 * holds none of the attended positions is read; what lies in an attended
 * page past the end may be anything, NaN too.
 * accumulate 1: pool->scores of each attended position grows by the sum over
 * its kv head's query heads of their softmax weights.  Each position's sum
 * has a fixed order; where several requests of the call share a page, the
 * order of the requests' additions is not fixed.
 *
 * q [B, n_heads, head_dim] and out like q (not q itself, nor overlapping it),
 * of the activation type: rows `*_stride` elements apart, heads contiguous,
 * rows 16-byte aligned.  lse:
 * NULL, or fp32 [B, n_heads].  block_table [B, bt_stride], seq_lens [B].
 * Logits, maxima, sums and lse are held in fp32, and so are the weights of
 * fp32 pools and those added to scores.  The weights that multiply v beside
 * other pools are pairs of 16-bit numbers: right to 2^-17 of themselves, with
 * e4m3 pools to 2^-21 of themselves or 2^-37 of the largest.  Beside e4m3
 * pools an element of q is right to 2^-25 of its row's largest.  Exponentials
 * are the hardware's, right to 2^-21.  workspace: 16-byte aligned,
 * workspace_bytes at least pe_attn_decode_workspace(.., 0); contents need not
 * be set and do not carry over; calls that may overlap need one each.
 * Device errors: PE_DEV_BAD_POSITION (seq_lens[b] < 0 or past the table:
 * read as 0 or the table's end), PE_DEV_BAD_BLOCK (the page's positions are
 * left out).
 * PE_ERR_INVALID_ARGUMENT: B < 1, window < 0, scale (times the K scale) not
 * finite or too large for its sums to be, out == q, n_heads not
 * a positive multiple of n_kv_heads, accumulate without pool->scores, a
 * stride shorter than a row, a null or misaligned pointer, a short
 * workspace.  PE_ERR_UNSUPPORTED: head_dim other than 64 and 128, or B *
 * bt_stride * n_heads past 2^31 - 1.  An attended v of +-inf gives +-inf or
 * NaN. */
pe_status pe_attn_decode(const pe_kv_pool* pool, int32_t B, int32_t n_heads, float scale,
                         const void* q, int64_t q_stride, const int32_t* block_table,
                         int32_t bt_stride, const int32_t* seq_lens, int32_t window, void* out,
                         int64_t out_stride, float* lse, int32_t accumulate, void* workspace,
                         int64_t workspace_bytes, int32_t* err, void* stream);

/* Trim requests' caches to at most `budget` positions by accumulated weight.
 *
 * A request with seq_lens[b] = L <= budget keeps everything.  Otherwise each
 * layer and kv head keeps positions < sinks, positions >= L - recent, and of
 * the rest the budget - sinks - recent with the largest scores (equal
 * scores: the lowest position; a NaN score counts as -inf), in order:
 * kept[layer, b, h, j] is the old position of new position j (-1 for j >=
 * new_lens[b] = min(L, budget)).  k, v and score of kept[j] move to j; the
 * key is rotated by (j - kept[j]) theta^(-2 i / head_dim), which makes it
 * the key of position j (rope_theta 0: keys are moved as they are; a key
 * that stays at its position is copied bit for bit; e4m3: the codes'
 * rotation, rounded and saturated; each trim of a request rounds its moved
 * keys once, after a rotation that with 16- and 8-bit pools is right to 2^-20
 * of a pair's length).  Scores of positions new_lens[b] .. the end of its page are
 * set to 0.  A drafter or decoder then goes on at position new_lens[b].
 *
 * dst_table [B, dst_stride]: the pages that receive the result, none of
 * which may be a page of block_table that the call reads (pages shared with
 * other requests can be trimmed this way).  dst_table NULL or block_table: in
 * place, in the request's first pages; its pages may then not be shared, and scores up to
 * L are set to 0.  In place needs whole requests to be trimmed by one call
 * for each layer; the layers of one call are independent.
 *
 * pools: HOST array of n_layers pools (all with scores, of the same shape and
 * dtype, each in memory of its own; num_blocks may differ), copied.  block_table [B,
 * bt_stride], seq_lens [B], kept [n_layers, B, n_kv_heads, budget], new_lens
 * [B] (not seq_lens itself).
 * Device errors: PE_DEV_BAD_POSITION (seq_lens[b] < 0 or past the table:
 * read as 0 or the table's end; a new position past dst_table: not written),
 * PE_DEV_BAD_BLOCK (a bad source page scores -inf and moves nothing; a bad
 * destination page is not written).
 * PE_ERR_INVALID_ARGUMENT: n_layers outside [1, 64], B < 1, budget < 1,
 * sinks or recent < 0 or together above budget, rope_theta negative or not
 * finite, pools that differ, share memory or have no scores, a null or
 * misaligned pointer, new_lens == seq_lens, dst_table == block_table with
 * another stride.  PE_ERR_UNSUPPORTED: head_dim other than 64 and 128, more
 * than 2^31 - 1 entries of kept, budget past 2^30 or bt_stride past 2^26. */
pe_status pe_kv_evict(int32_t n_layers, const pe_kv_pool* pools, int32_t B,
                      const int32_t* block_table, int32_t bt_stride, const int32_t* seq_lens,
                      int32_t budget, int32_t sinks, int32_t recent, float rope_theta,
                      const int32_t* dst_table, int32_t dst_stride, int32_t* kept,
                      int32_t* new_lens, int32_t* err, void* stream);

/* Collect scores in the drafting step.  After this call every layer l of
 * pe_draft_forward adds, besides what it does anyway, the attention weights
 * of each request's next-token row (the first of its K sampled rows; query
 * heads of a kv head summed) over positions 0 .. the row's own to scores[l]
 * [num_blocks, Hkv, 16] fp32, 16-byte aligned, of the pools that the step is
 * given.  No other result changes.  The step's attention computes rows in
 * tiles and keeps no weights, so they come from a pass of their own over each
 * layer's K (three launches a layer): collect on the steps where they
 * are worth it.  The step does not clear scores: a request that takes over
 * pages finds theirs (pe_kv_append and pe_kv_evict clear what they free or
 * fill).
 * scores: HOST array of n_layers device pointers, copied; NULL turns the
 * collecting off.  The first call allocates the pass's workspace on the
 * handle: make it outside a graph capture.  A step with a larger batch or
 * table than before allocates room for its logits: at least twice the room
 * before and at most 1 GiB, all of which stays with the handle (2 GiB in the
 * end).  Logits that find no room, because the step is being captured or
 * there is no memory, are worked out twice; room that could not be had is
 * asked for again after the next pe_set_kv_scores.  Calls on one handle must
 * not overlap.  PE_ERR_INVALID_ARGUMENT: a null or misaligned entry;
 * PE_ERR_OUT_OF_MEMORY. */
pe_status pe_set_kv_scores(pe_handle* h, float* const* scores);

#ifdef __cplusplus
}
#endif

#endif /* PEAGLE_CACHE_H_ */
