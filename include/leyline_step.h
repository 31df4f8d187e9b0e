/*
 * leyline_step.h - the serving step of a paged KV cache (MI355X, gfx950): the
 * new tokens' rows go into the cache, and their queries read it.
 *
 * A step belongs to a pool of leyline.h (MLA or GQA / MHA) and to a number of
 * query heads.  ll_step_begin says which sequences take part and how many
 * tokens each brings; it grows them and makes, once, what every layer of the
 * model then uses: the tokens' cache rows, the cos / sin of their positions
 * and the split of the attention over the chip.  ll_step_append and
 * ll_step_attend then run once per layer.  "Token t" below is the t-th token of
 * the step: the tokens of the first sequence in order, then the second's, ...
 *
 *   begin(seqs, counts, grow)   ->  for each layer: append, attend
 *
 * Values are bf16; sums, norms, softmax statistics and the rotation are float32,
 * and each result is rounded to bf16 once (attend: the softmax weights are
 * rounded to bf16 as well, for the matrix instructions).
 *
 * Ownership, errors and streams are those of leyline.h: buffers belong to the
 * caller until the stream work that uses them has finished, checks run before
 * anything changes, a call follows the pool's previous one on the device also
 * across streams, and only begin may wait on the host (for room in the staging
 * ring, or for a device-planned eviction to settle).  A step is as little
 * thread-safe as its pool.
 *
 * Lifetime.  A step fits the sequences as begin left them.  Once a splice,
 * eviction, reindex, ll_seq_set_pages, ll_seq_free or another step's growing
 * begin has changed one of them, append and attend return LL_EINVAL until the
 * next begin.  Steps of a destroyed pool refuse every call; ll_step_destroy
 * may come before or after ll_pool_destroy.
 *
 * Graphs.  append and attend may be captured (begin may not: LL_EUNSUPPORTED).
 * They then cover the whole capacity of the step and read its current plan from
 * device memory: begin the next tokens, on the stream the graph runs on, and
 * replay.  Eager calls between are planned for their own tokens.  A graph's
 * attention keeps the tiles (query rows that a workgroup takes) of the begin before
 * the step's first capture, whatever later begins bring: capture behind a begin
 * like those that the graph will replay, and keep a step of fitting max_tokens for
 * each kind (single tokens, prompts).  Nothing orders a replay but its stream: the
 * replays of a step, its begins and the pool's other calls have to follow one
 * another on one stream or be ordered by the caller, since one step has one
 * workspace.  A graph is not replayed once its step or its pool has ended, nor on
 * sequences that something else has changed since the step's begin (a replay cannot
 * refuse them; it stays inside the pool, but may write rows of other sequences).
 *
 * One begin, one tile: the attention of all its sequences runs in tiles that fit the
 * one with the most tokens.  Single tokens beside a long chunk are faster in a begin
 * and calls of their own, by a second step.
 *
 * A stream that a call ran on has to exist until a call on another stream, or the
 * end of the pool, has followed.
 */
#ifndef LEYLINE_STEP_H
#define LEYLINE_STEP_H

#include "leyline.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct ll_step ll_step;

typedef struct {
  int32_t num_heads;   /* query heads: any number (MLA), a multiple of num_kv_heads (GQA) */
  int32_t max_seqs;    /* sequences of one begin, at most: 1 .. the pool's max_seqs */
  int32_t max_tokens;  /* tokens of one begin, at most: 1 .. 2^22, and max_tokens * num_heads <= 2^25 */
} ll_step_desc;

/* Types of the norm weights. */
enum { LL_TYPE_BF16 = 0, LL_TYPE_F32 = 1 };

/* Create a step on a pool: device buffers for its plan and for the parts of
 * split attention, all sized here.  The pool's head_dim may be at most 256.
 * Errors: LL_EINVAL, LL_EUNSUPPORTED (head_dim above 256, page-table rows of
 * 2^31 - 1024 cached rows or more, or more sequences times KV heads than one
 * dispatch holds: about 2^23), LL_ENOMEM,
 * LL_EDEVICE, LL_EPOISONED. */
ll_status ll_step_create(ll_pool* pool, const ll_step_desc* desc, ll_step** out);

/* Wait for the pool's device work and free the step.  NULL is ignored. */
void ll_step_destroy(ll_step* step);

/* The next step: counts[i] >= 0 tokens of sequence seq_ids[i], i < n, each
 * sequence at most once.
 * grow = 1: every sequence gets counts[i] more rows (fresh pages are the lowest
 * free ones, in batch order), its new tokens have the positions next_position,
 * next_position + 1, ..., and its next position moves on by counts[i].
 * grow = 0: the tokens are the last counts[i] rows that the sequence holds
 * (append rewrites them, attend asks from them), at the positions before its
 * next position.
 * Errors: LL_EINVAL (unknown or repeated sequence, counts[i] < 0, more than
 * max_seqs sequences or max_tokens tokens, grow = 0 with more tokens than rows),
 * LL_ERANGE (a page-table row is too short), LL_ENOMEM (too few free pages),
 * LL_EUNSUPPORTED (the stream is capturing), LL_EDEVICE. */
ll_status ll_step_begin(ll_step* step, const int32_t* seq_ids, const int32_t* counts, int32_t n,
                        int32_t grow, void* stream);

/* One layer's new rows and queries.  Strides are in values; pointers are 16-byte
 * aligned and strides multiples of 8; a value axis is dense.  Inputs may be
 * views of one projection's output. */
typedef struct {
  int64_t tokens;             /* tokens that a, b, q and q_out have room for: the step's or more (the first
                                 ones are used), its max_tokens or more under capture */
  int32_t layer;
  int32_t norm_type;          /* LL_TYPE_BF16 or LL_TYPE_F32, of norm and q_norm */
  const void* a;              /* MLA: c_kv [T][512] (a_head_stride unused); GQA: K [T][num_kv_heads][head_dim] */
  int64_t a_token_stride, a_head_stride;
  const void* b;              /* MLA: k_pe [T][64], not yet rotated; GQA: V, shaped as K */
  int64_t b_token_stride, b_head_stride;
  const void* norm;           /* RMS-norm weight of c_kv (512) or of each K head (head_dim); NULL: no norm */
  const void* q;              /* MLA: the rotated part of the queries [T][num_heads][64]; GQA: [T][num_heads][head_dim] */
  int64_t q_token_stride, q_head_stride;
  void* q_out;                /* the queries' results, shaped as q; q itself (same strides) is allowed */
  int64_t q_out_token_stride, q_out_head_stride;
  const void* q_norm;         /* RMS-norm weight of each query head (GQA only); NULL: no norm */
  float eps;                  /* of the norms: x * rsqrt(mean(x^2) + eps) * weight */
} ll_append_desc;

/* Write the tokens' rows of one layer into the cache and prepare their queries:
 *   MLA: row = norm(c_kv), R(position) k_pe;     q_out = R(position) q
 *   GQA: K head = R(position) norm(k), V head = v;  q_out = R(position) norm(q)
 * where R turns the pool's RoPE band (GQA: the first rotary_dim values of a head)
 * with the pool's pairing and base, from the float64 angle's cos and sin rounded
 * to float32.  a = b = NULL leaves the cache alone, q = NULL the queries.  q_out
 * may be q, and may not overlap the inputs otherwise.
 * Errors: LL_EINVAL (layer, too few tokens, NULL or misaligned pointer or stride, overlapping
 * q_out rows, q_out = q with other strides, negative eps, a changed sequence, no begin yet), LL_EDEVICE. */
ll_status ll_step_append(ll_step* step, const ll_append_desc* desc, void* stream);

typedef struct {
  int64_t tokens;             /* tokens that q, q_pe, out and lse have room for, as in ll_append_desc */
  int32_t layer;
  int32_t causal;             /* 1: a token sees the rows up to its own; 0: every row of its sequence */
  int64_t window;             /* > 0 (with causal): only the last `window` of those; 0: all */
  float scale;                /* of the scores; finite, and so is scale * log2 e */
  const void* q;              /* MLA: [T][num_heads][512], in the latent space; GQA: [T][num_heads][head_dim] */
  int64_t q_token_stride, q_head_stride;
  const void* q_pe;           /* MLA: the rotated part [T][num_heads][64]; GQA: NULL */
  int64_t q_pe_token_stride, q_pe_head_stride;
  void* out;                  /* MLA: [T][num_heads][512] (latent); GQA: [T][num_heads][head_dim] */
  int64_t out_token_stride, out_head_stride;
  float* lse;                 /* NULL, or log sum exp of the scores, float32 [T][num_heads] dense, 4-byte aligned */
} ll_attend_desc;

/* Attention of the step's tokens over one layer of the cache:
 *   out[t][h] = sum_j p_j v_j,  p = softmax_j(scale * q[t][h] . k_j)
 * over the rows j of the token's sequence that it sees, in row order (an evicted
 * row is no row; positions play no part).  MLA: k_j is the whole row, v_j its
 * first 512 values, shared by all heads; GQA: head h reads KV head
 * h / (num_heads / num_kv_heads).  Rows that a token does not see never reach its
 * result, whatever they hold; a token that sees none gets zeros and lse = -inf, and
 * so does one whose scores are all -inf.  (A seen row with a score of -inf next to
 * others with finite ones has weight 0; whether 0 times an infinity in its value
 * makes the result NaN depends on the plan.)  out may not overlap q or q_pe.
 * Results do not depend on the other sequences' contents, and the same call on the
 * same plan gives the same bits.
 * Errors: LL_EINVAL (layer, too few tokens, NULL or misaligned pointer or stride, overlapping out
 * rows, a scale that is not finite, window < 0 or without causal, a changed
 * sequence, no begin yet), LL_EDEVICE. */
ll_status ll_step_attend(ll_step* step, const ll_attend_desc* desc, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* LEYLINE_STEP_H */
