// The serving step's host types and the checks that its calls share (step.cpp,
// weight.cpp).  Not part of the C ABI.
#pragma once

#include <vector>

#include "../../include/leyline_step.h"
#include "host_common.h"
#include "pool_internal.h"
#include "step_internal.h"

namespace ll {

// A plan of the attention: the current begin's, in tiles of `tile` query rows.
struct Plan {
  int32_t tile = 16;
  int64_t items = 0;
  int64_t shares = 0;            // of them shares of split tiles, which a second kernel joins
  StepCounts* d_counts = nullptr;
  AttendItem* d_items = nullptr;
};

}  // namespace ll

struct ll_step {
  ll_pool* pool = nullptr;       // cleared when the pool ends
  int32_t device = 0;
  int32_t heads = 0, kv_heads = 1, group = 1;
  int32_t max_seqs = 0, max_tokens = 0;
  int32_t value_dim = 0;         // width of an output head
  int64_t max_items = 0;         // of a plan
  bool captured = false;         // a graph holds plans[0]: its tile stays
  // What graphs read, and eager calls too unless a graph holds another tile than
  // they would take: they have a plan of their own then.  One at a time uses the
  // partial results.
  ll::Plan plans[2];
  int eager = 0;
  // device: [counts, items, twice | sequences | rows | tab | theta | parts]
  char* d_buf = nullptr;
  ll::StepSeq* d_seqs = nullptr;
  int32_t* d_rows = nullptr;
  float* d_tab = nullptr;
  double* d_theta = nullptr;
  float* d_part_o = nullptr;
  float* d_part_ml = nullptr;
  int64_t part_values = 0;       // room in d_part_o
  // the step begun last
  bool begun = false;
  std::vector<int32_t> seqs;
  std::vector<uint64_t> gens;
  std::vector<int64_t> lens;     // rows of each sequence
  int64_t most = 0;              // tokens of the one that brings the most
  int64_t tokens = 0;
};

namespace ll {

constexpr int64_t kMaxStride = int64_t{1} << 32;

inline ll_status check_step(const ll_step* s) {
  if (!s) return fail(LL_EINVAL, "step is NULL");
  if (!s->pool) return fail(LL_EINVAL, "the step's pool has been destroyed");
  return pool_check(s->pool);
}

// The step still fits its sequences.
inline ll_status check_current(const ll_step* s) {
  if (!s->begun) return fail(LL_EINVAL, "the step has not begun");
  for (size_t i = 0; i < s->seqs.size(); ++i)
    if (s->pool->seqs[s->seqs[i]].gen != s->gens[i])
      return fail(LL_EINVAL, "sequence %d has changed since the step began", s->seqs[i]);
  return LL_OK;
}

inline ll_status is_capturing(hipStream_t st, bool* out) {
  hipStreamCaptureStatus c = hipStreamCaptureStatusNone;
  hipError_t e = hipStreamIsCapturing(st, &c);
  if (e != hipSuccess) {
    (void)hipGetLastError();
    return fail(LL_EUNSUPPORTED, "the stream's capture state: %s", hipGetErrorString(e));
  }
  *out = c != hipStreamCaptureStatusNone;
  return LL_OK;
}

// A stride that no second token or head uses says nothing.
inline int64_t used(int64_t stride, int64_t n) { return n > 1 ? stride : 0; }

inline ll_status check_plane(const void* p, int64_t ts, int64_t hs, const char* name) {
  if (!p) return fail(LL_EINVAL, "%s is NULL", name);
  if (reinterpret_cast<uintptr_t>(p) & 15) return fail(LL_EINVAL, "%s is not 16-byte aligned", name);
  if ((ts & 7) || (hs & 7) || ts < 0 || hs < 0 || ts > kMaxStride || hs > kMaxStride)
    return fail(LL_EINVAL, "%s: strides must be multiples of 8 values in [0, 2^32]", name);
  return LL_OK;
}

// What an attention over a layer says of its scores.
inline ll_status check_scores(const ll_pool* p, int32_t layer, int32_t causal, int64_t window, float scale, float cap) {
  if (layer < 0 || layer >= p->desc.num_layers) return fail(LL_EINVAL, "layer %d out of range", layer);
  if (causal != 0 && causal != 1) return fail(LL_EINVAL, "causal must be 0 or 1");
  if (window < 0 || (window > 0 && !causal)) return fail(LL_EINVAL, "window must be >= 0, and needs causal");
  return check_scale(scale, cap);
}

// The caller's buffers hold every token that the call may touch: the step's, or
// under capture (later begins are replayed) as many as the step can have.
inline ll_status check_room(const ll_step* s, int64_t tokens, bool capturing) {
  const int64_t need = capturing ? s->max_tokens : s->tokens;
  if (tokens < need) return fail(LL_EINVAL, "buffers for %lld tokens, but the call may touch %lld", (long long)tokens, (long long)need);
  return LL_OK;
}

// Eager calls follow the pool's earlier work; a captured one is the caller's to
// order.
inline ll_status start(ll_step* s, hipStream_t st, bool capturing) {
  return capturing ? LL_OK : pool_begin_call(s->pool, st);
}

inline void finish(ll_step* s, hipStream_t st, bool capturing) {
  if (capturing) return;
  s->pool->last_stream = st;
  s->pool->unevented = true;
}

}  // namespace ll
