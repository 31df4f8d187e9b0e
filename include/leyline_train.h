/*
 * leyline_train.h - the trainer's attention under an engine's evictions (MI355X,
 * gfx950): one pass over whole rollouts in which every token sees exactly the keys
 * that the cache held when it was generated, forward and backward.
 *
 * The mask is the death times of kvs_death_times (leyline.h): query q of a rollout
 * sees key k iff k <= q < death[k], for any int32 values (at or below k: nobody sees
 * the key; n_pad or more: everyone from k on).  A key of a document that ends before
 * token e dies at e, so that documents packed into one rollout are death times too.
 *
 * Values are bf16; sums, softmax statistics and gradients' sums are float32, and each
 * result is rounded to bf16 once.  For the matrix instructions the softmax weights and
 * the scores' gradients are rounded to bf16 as well (2^-9 of each on average, of the
 * order of the results' own rounding; in dq a score gradient's rounding counts with the
 * key's distance from the query's weighted mean key, so that what the keys have in
 * common adds nothing to it).
 *
 * What a query does not see never reaches its result or the gradients of others,
 * whatever it holds.  The same call gives the same bits.
 *
 * Buffers are the caller's device memory; the calls enqueue kernels on `stream`, keep
 * nothing and may be captured.  A context may be used from several streams at once by
 * these calls, each with a workspace of its own.
 */
#ifndef LEYLINE_TRAIN_H
#define LEYLINE_TRAIN_H

#include "leyline.h"

#ifdef __cplusplus
extern "C" {
#endif

/* A bf16 tensor [n][n_pad][heads][width] with a dense last axis: strides in values,
 * multiples of 8, data 16-byte aligned. */
typedef struct {
  void* data;
  int64_t rollout_stride, token_stride, head_stride;
} kvs_heads;

typedef struct {
  int32_t n;                  /* rollouts */
  int32_t heads;              /* query heads: a multiple of kv_heads; head h reads KV head h / (heads / kv_heads) */
  int64_t n_pad;              /* tokens of each, 1 .. 2^31 - 2 */
  int32_t kv_heads;
  int32_t key_dim;            /* width of a query and a key head: a multiple of 8 up to 256 */
  int32_t value_dim;          /* width of a value and an output head: a multiple of 8 up to 256 */
  float scale;                /* of the scores; with the cap as in leyline_weight.h */
  float cap;                  /* scores are cap * tanh(scale q . k / cap); 0: scale q . k */
  const int32_t* death;       /* [n][n_pad] dense */
  kvs_heads q;                /* [n][n_pad][heads][key_dim] */
  kvs_heads k;                /* [n][n_pad][kv_heads][key_dim] */
  kvs_heads v;                /* [n][n_pad][kv_heads][value_dim] */
  kvs_heads out;              /* [n][n_pad][heads][value_dim]: written by kvs_attend, read by kvs_attend_backward */
  float* lse;                 /* float32 [n][n_pad][heads] dense, 4-byte aligned: as out */
  void* workspace;            /* 16-byte aligned device memory that nothing else uses until the work is done */
  int64_t workspace_bytes;    /* at least what kvs_attend_workspace says */
} kvs_attend_desc;

/* Bytes of workspace that kvs_attend (backward = 0) or kvs_attend_backward (1) needs
 * for this n, n_pad, heads, kv_heads, key_dim and value_dim (the rest of desc is not
 * read): for a longer n_pad never less.  Errors: LL_EINVAL, LL_EUNSUPPORTED (as
 * kvs_attend). */
ll_status kvs_attend_workspace(const kvs_attend_desc* desc, int32_t backward, int64_t* bytes);

/* out[q][h] = sum_k p_k v_k and lse[q][h] = log sum_k exp s_k over the keys that
 * query q sees, p = softmax(s).  A query that sees none gets zeros and lse = -inf, and
 * so does one whose scores are all -inf.  out may not overlap the inputs.
 * Errors: LL_EINVAL (sizes outside the ranges above, a scale or cap outside theirs,
 * NULL or misaligned pointers or strides, overlapping rows of out, a workspace that is
 * too small), LL_EUNSUPPORTED (more work than one launch holds: n * heads *
 * ceil(n_pad / 64) of 2^23 or more), LL_EDEVICE. */
ll_status kvs_attend(kvs_ctx* ctx, const kvs_attend_desc* desc, void* stream);

/* The gradients of kvs_attend: with dout the gradient of out (lse has none),
 *   delta = sum_d dout out,  ds = p (dout . v - delta) scale (1 - tanh^2),
 *   dv = sum_q p dout,  dk = sum_q ds q,  dq = sum_k ds k,
 * dk and dv summed over the heads that share a KV head.  delta is what sum_k p dout . v
 * gives (the same but for the rounding of out, which only a first guess is taken from).  out and lse are those that
 * kvs_attend gave for the same inputs.  dq, dk and dv are written whole (zeros where
 * nothing is seen) and may not overlap anything else.  Errors: as kvs_attend. */
typedef struct {
  kvs_attend_desc f;
  kvs_heads dout;             /* shaped as out */
  kvs_heads dq, dk, dv;       /* shaped as q, k, v */
} kvs_attend_backward_desc;
ll_status kvs_attend_backward(kvs_ctx* ctx, const kvs_attend_backward_desc* desc, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* LEYLINE_TRAIN_H */
