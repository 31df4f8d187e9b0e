// Host side of eviction by attention weight (include/leyline_weight.h): argument
// checks and the launches of kernels_weigh.hip and kernels_keep.hip.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <utility>
#include <vector>

#include "../../include/leyline_weight.h"
#include "step_host.h"
#include "weight_internal.h"

using namespace ll;

namespace {

ll_status check_floats(const void* p, const char* name) {
  if (!p) return fail(LL_EINVAL, "%s is NULL", name);
  if (reinterpret_cast<uintptr_t>(p) & 3) return fail(LL_EINVAL, "%s is not 4-byte aligned", name);
  return LL_OK;
}

constexpr int64_t kMaxWeightStride = int64_t{1} << 40;   // offsets stay in 64 bits

}  // namespace

extern "C" {

ll_status ll_step_weigh(ll_step* s, const ll_weigh_desc* d, void* stream) try {
  ll_status rc = check_step(s);
  if (rc) return rc;
  if (!d) return fail(LL_EINVAL, "NULL argument");
  ll_pool* p = s->pool;
  if ((rc = check_current(s))) return rc;
  hipStream_t st = static_cast<hipStream_t>(stream);
  ll::DeviceGuard g(s->device);
  bool capturing = false;
  if ((rc = is_capturing(st, &capturing))) return rc;
  if ((rc = check_room(s, d->tokens, capturing))) return rc;
  if ((rc = check_scores(p, d->layer, d->causal, d->window, d->scale, d->cap))) return rc;
  if (!(d->decay >= 0.f && d->decay <= 1.f)) return fail(LL_EINVAL, "decay must lie in [0, 1]");
  const int64_t T = capturing ? s->max_tokens : s->tokens;
  int64_t rows = 0;
  for (int64_t n : s->lens) rows = std::max(rows, n);
  if (capturing) rows = int64_t{p->desc.max_pages_per_seq} * p->P;
  if (d->weight_stride < rows || d->weight_stride > kMaxWeightStride)
    return fail(LL_EINVAL, "weight_stride must lie in %lld .. 2^40", (long long)rows);
  if (rows == 0) return LL_OK;
  if (T > 0) {
    if ((rc = check_plane(d->q, used(d->q_token_stride, T), used(d->q_head_stride, s->heads), "q"))) return rc;
    if (p->gqa) {
      if (d->q_pe) return fail(LL_EINVAL, "q_pe is for MLA pools only");
    } else if ((rc = check_plane(d->q_pe, used(d->q_pe_token_stride, T), used(d->q_pe_head_stride, s->heads), "q_pe"))) {
      return rc;
    }
    if ((rc = check_floats(d->lse, "lse"))) return rc;
  }
  if ((rc = check_floats(d->weights, "weights"))) return rc;
  WeighLaunch a{};
  a.counts = s->plans[0].d_counts;
  a.seqs = s->d_seqs;
  a.n_seqs = capturing ? s->max_seqs : static_cast<int32_t>(s->seqs.size());
  a.max_rows = rows;
  a.most = s->most * s->group;
  a.kv_heads = s->kv_heads;
  a.group = s->group;
  a.heads = s->heads;
  a.causal = d->causal;
  a.window = static_cast<int32_t>(std::min<int64_t>(d->window, INT32_MAX));
  a.scale = d->scale;
  a.cap = d->cap;
  a.decay = d->decay;
  a.dim = s->value_dim;
  a.k_plane = static_cast<const uint16_t*>(p->layer_ptrs[static_cast<size_t>(d->layer)]);
  a.page_table = p->desc.page_table;
  a.max_pages_per_seq = p->desc.max_pages_per_seq;
  a.num_pages = p->desc.num_pages;
  a.page_shift = p->page_shift;
  a.q = static_cast<const uint16_t*>(d->q);
  a.q_ts = d->q_token_stride;
  a.q_hs = d->q_head_stride;
  a.q_pe = static_cast<const uint16_t*>(d->q_pe);
  a.qp_ts = d->q_pe_token_stride;
  a.qp_hs = d->q_pe_head_stride;
  a.lse = d->lse;
  a.weights = d->weights;
  a.weight_stride = d->weight_stride;
  a.parts = s->d_part_o;
  a.part_values = s->part_values;
  if ((rc = start(s, st, capturing))) return rc;
  hipError_t e = ll::launch_weigh(a, p->gqa, st);
  if (e != hipSuccess) return ll::pool_device_fail(p, e, "weigh_kernel launch");
  finish(s, st, capturing);
  return LL_OK;
} catch (...) {
  return ll::pool_host_exception(s ? s->pool : nullptr);
}

ll_status ll_keep_heaviest(ll_pool* p, const int32_t* seq_ids, int32_t n, const int64_t* budgets, int64_t sinks,
                           int64_t recent, const float* weights, float* kept_weights, int64_t weight_stride,
                           uint8_t* keep_dev, const int64_t* keep_offsets, void* stream) try {
  ll_status rc = pool_check(p);
  if (rc) return rc;
  if (n < 0 || (n > 0 && (!seq_ids || !budgets || !keep_offsets))) return fail(LL_EINVAL, "bad sequence list");
  if (sinks < 0 || recent < 0 || sinks > INT32_MAX || recent > INT32_MAX)
    return fail(LL_EINVAL, "sinks and recent must lie in 0 .. 2^31 - 1");
  hipStream_t st = static_cast<hipStream_t>(stream);
  ll::DeviceGuard g(p->desc.device);
  bool capturing = false;
  if ((rc = is_capturing(st, &capturing))) return rc;
  if (capturing) return fail(LL_EUNSUPPORTED, "a selection depends on the sequences' lengths and cannot be captured");
  if ((rc = pool_enter(p))) return rc;
  if (n == 0) return LL_OK;
  if ((rc = check_floats(weights, "weights"))) return rc;
  if (reinterpret_cast<uintptr_t>(kept_weights) & 3) return fail(LL_EINVAL, "kept_weights is not 4-byte aligned");
  if (!keep_dev) return fail(LL_EINVAL, "keep masks are NULL");
  std::vector<char> seen(static_cast<size_t>(p->desc.max_seqs), 0);
  std::vector<KeepSeq> seqs(static_cast<size_t>(n));
  std::vector<std::pair<int64_t, int64_t>> masks;   // [begin, end) of each that is not empty
  int32_t most = 0;                                 // the highest row of the weights
  for (int32_t i = 0; i < n; ++i) {
    const int32_t q = seq_ids[i];
    if (q < 0 || q >= p->desc.max_seqs || !p->seqs[q].used) return fail(LL_EINVAL, "entry %d: unknown sequence %d", i, q);
    if (seen[q]) return fail(LL_EINVAL, "entry %d: sequence %d appears twice", i, q);
    seen[q] = 1;
    const int64_t rows = p->seqs[q].len;
    if (rows > INT32_MAX) return fail(LL_EUNSUPPORTED, "entry %d: %lld rows are too many", i, (long long)rows);
    if (budgets[i] < 0 || budgets[i] < sinks + recent)
      return fail(LL_EINVAL, "entry %d: a budget of %lld rows is below 0 or below sinks + recent", i, (long long)budgets[i]);
    if (rows > weight_stride || weight_stride > kMaxWeightStride)
      return fail(LL_EINVAL, "entry %d: weight_stride must lie in %lld .. 2^40", i, (long long)rows);
    if (keep_offsets[i] < 0) return fail(LL_EINVAL, "entry %d: negative mask offset", i);
    most = std::max(most, q);
    seqs[i] = KeepSeq{rows, std::min(budgets[i], rows), keep_offsets[i], q};
    if (rows > 0) masks.emplace_back(keep_offsets[i], keep_offsets[i] + rows);
  }
  std::sort(masks.begin(), masks.end());
  for (size_t i = 1; i < masks.size(); ++i)
    if (masks[i].first < masks[i - 1].second) return fail(LL_EINVAL, "keep masks overlap");
  if (kept_weights && kept_weights != weights) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(weights), b = reinterpret_cast<uintptr_t>(kept_weights);
    const uintptr_t bytes = static_cast<uintptr_t>(4 * (most * weight_stride + p->seqs[most].len));
    if (a < b + bytes && b < a + bytes) return fail(LL_EINVAL, "kept_weights overlaps weights");
  }
  if (masks.empty()) return LL_OK;
  // longest first: a workgroup takes one sequence
  std::stable_sort(seqs.begin(), seqs.end(), [](const KeepSeq& a, const KeepSeq& b) { return a.rows > b.rows; });
  if ((rc = pool_begin_call(p, st))) return rc;
  for (size_t at = 0; at < masks.size(); at += kKeepSeqs) {   // (sequences without rows come last)
    const int count = static_cast<int>(std::min<size_t>(kKeepSeqs, masks.size() - at));
    KeepLaunch a{};
    std::copy(seqs.begin() + at, seqs.begin() + at + count, a.seqs);
    a.sinks = sinks;
    a.recent = recent;
    a.weights = weights;
    a.kept_weights = kept_weights;
    a.weight_stride = weight_stride;
    a.keep = keep_dev;
    hipError_t e = ll::launch_keep(a, count, st);
    if (e != hipSuccess) return pool_device_fail(p, e, "keep_kernel launch");
  }
  p->last_stream = st;
  p->unevented = true;
  return LL_OK;
} catch (...) {
  return ll::pool_host_exception(p);
}

}  // extern "C"
