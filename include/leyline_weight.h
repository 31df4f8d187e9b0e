/*
 * leyline_weight.h - eviction by attention weight on a paged KV cache (MI355X,
 * gfx950): how much attention each cached row gets, and the keep mask that drops
 * the rows that get the least.  Also the serving step's attention with capped
 * scores, which the weights then follow.
 *
 *   begin -> for each layer: append, attend (lse), weigh -> keep_heaviest ->
 *   kv_evict_compact with its mask
 *
 * Weights are a caller-owned float32 buffer, one row per page-table row of the
 * pool (sequence s at weights + s * weight_stride), one value per cached row in
 * row order.  It starts as zeros; ll_step_weigh adds to it and ll_keep_heaviest
 * moves it together as the eviction by its mask moves the cached rows.  Whoever
 * splices or re-indexes a sequence, or frees it and uses its number again, sets its
 * row anew.
 *
 * Ownership, errors and streams are those of leyline.h and leyline_step.h.
 */
#ifndef LEYLINE_WEIGHT_H
#define LEYLINE_WEIGHT_H

#include "leyline_step.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ll_step_attend with scores that a cap bounds:
 *   s_j = cap * tanh(scale * q . k_j / cap),  out = sum_j softmax(s)_j v_j,
 * lse = log sum exp s_j.  cap = 0: ll_step_attend itself.  Otherwise everything that
 * leyline_step.h says of ll_step_attend holds; a score of -inf counts -cap.
 * Errors: as ll_step_attend, and LL_EINVAL for a cap outside {0, [2^-40, 2^40]} or a
 * scale that is neither 0 nor, in magnitude, in [cap * 2^-64, cap * 2^64]. */
ll_status ll_step_attend_capped(ll_step* step, const ll_attend_desc* desc, float cap, void* stream);

typedef struct {
  int64_t tokens;             /* tokens that q, q_pe and lse have room for, as in ll_append_desc */
  int32_t layer;
  int32_t causal;             /* this and the next four: as the attention that made lse */
  int64_t window;
  float scale;
  float cap;                  /* 0: none */
  const void* q;              /* MLA: [T][num_heads][512]; GQA: [T][num_heads][head_dim] */
  int64_t q_token_stride, q_head_stride;
  const void* q_pe;           /* MLA: [T][num_heads][64]; GQA: NULL */
  int64_t q_pe_token_stride, q_pe_head_stride;
  const float* lse;           /* of the attention: float32 [T][num_heads] dense, 4-byte aligned */
  float* weights;             /* float32 [max_seqs of the pool][weight_stride], 4-byte aligned */
  int64_t weight_stride;      /* values from one sequence to the next: the rows of each sequence of the step or
                                 more (under capture: of a whole page-table row) */
  float decay;                /* of what a row's weight was, in [0, 1]; 0: whatever it was, NaN too, counts nothing */
} ll_weigh_desc;

/* The attention that each cached row of the step's sequences gets from the step's
 * tokens in one layer, over all query heads:
 *   weights[s][j] = decay * weights[s][j] + sum_t sum_h exp(s_thj - lse[t][h])
 * over the tokens t of sequence s that see row j.  (A step that goes through several
 * layers decays in the first one, if at all.)  The sum over a token's rows is the
 * number of heads (a score and its lse are float32: their roundings, 2^-24 of each, are
 * the weights' relative errors).  A token and head whose lse is -inf sees nothing and
 * adds nothing.
 * Rows past a sequence's last one, and other sequences', are left as they were; a
 * sequence without tokens in the step decays too.  Scores and sums are float32, in a
 * fixed order: the same call on the same plan gives the same bits.  May be captured as
 * append and attend may (leyline_step.h).
 * Errors: LL_EINVAL (as ll_step_attend_capped; weights or lse NULL or not 4-byte aligned, a
 * weight_stride that is too short, decay outside [0, 1]), LL_EDEVICE. */
ll_status ll_step_weigh(ll_step* step, const ll_weigh_desc* desc, void* stream);

/* Keep masks for kv_evict_compact by weight.  Of the n rows that sequence
 * seq_ids[i] holds, min(budgets[i], n) are kept: the first `sinks` and the last
 * `recent` rows, and of the others those of largest weight, of equal ones the earlier
 * rows.  (A NaN counts as more than infinity; -0 and 0 are equal.)  The mask goes to
 * keep_dev + keep_offsets[i], n bytes of 0 or 1, as kv_evict_compact takes it.
 * kept_weights (NULL: none; weights itself, or a buffer that does not overlap it), of
 * the same stride, gets the kept rows' weights in order, then zeros up to the old
 * length, the rest of its row left as it was.
 * weights: see above; seq_ids, budgets and keep_offsets are host arrays, read before
 * the call returns.  Each sequence at most once; masks may not overlap.  n == 0 is a
 * no-op.
 * Errors: LL_EINVAL (unknown or repeated sequence, budget below 0 or below sinks + recent, negative sinks,
 * recent or offset, overlapping masks, NULL or misaligned buffers, a weight_stride shorter than a sequence),
 * LL_EUNSUPPORTED (the stream is capturing, or a sequence of 2^31 rows or more), LL_EDEVICE. */
ll_status ll_keep_heaviest(ll_pool* pool, const int32_t* seq_ids, int32_t n, const int64_t* budgets,
                           int64_t sinks, int64_t recent, const float* weights, float* kept_weights,
                           int64_t weight_stride, uint8_t* keep_dev, const int64_t* keep_offsets, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* LEYLINE_WEIGHT_H */
