// Host side of the serving step (include/leyline_step.h): argument checks, the
// growth of the sequences, the step's plan (tokens, positions, the split of the
// attention) and the launches of its kernels.
//
// begin uploads the plan through the pool's staging ring and a kernel puts it
// where append and attend read it: those two then launch kernels only, touch no
// host or device memory of their own, and can be captured.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstring>
#include <memory>
#include <new>
#include <vector>

#include "../../include/leyline_step.h"
#include "host_common.h"
#include "pool_internal.h"
#include "step_internal.h"

namespace {

using ll::ceil_div;
using ll::fail;

constexpr int64_t kMaxStride = int64_t{1} << 32;
// Partial results of split tiles: values that the step's buffer holds (128 MiB),
// and shares (times KV heads) at most.
constexpr int64_t kPartValues = int64_t{1} << 25;
constexpr int64_t kMaxShares = 2048;

// A plan of the attention: the current begin's, in tiles of `tile` query rows.
struct Plan {
  int32_t tile = 16;
  int64_t items = 0;
  int64_t shares = 0;            // of them shares of split tiles, which a second kernel joins
  ll::StepCounts* d_counts = nullptr;
  ll::AttendItem* d_items = nullptr;
};

}  // namespace

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
  Plan plans[2];
  int eager = 0;
  // device: [counts, items, twice | rows | tab | theta | parts]
  char* d_buf = nullptr;
  int32_t* d_rows = nullptr;
  float* d_tab = nullptr;
  double* d_theta = nullptr;
  float* d_part_o = nullptr;
  float* d_part_ml = nullptr;
  // the step begun last
  bool begun = false;
  std::vector<int32_t> seqs;
  std::vector<uint64_t> gens;
  int64_t tokens = 0;
};

namespace {

int64_t tiles_of(int64_t q_rows, int tile) { return ceil_div(q_rows, tile); }

// Shares of split tiles that the partial results' buffer holds, per KV head.
int64_t max_slots(const ll_step* s, int tile) {
  return std::min(kMaxShares, kPartValues / s->value_dim / tile) / s->kv_heads;
}

// How many cached rows a workgroup takes at most.  `seen` holds the rows that each
// tile needs.  With few tiles a share is as short as the chip's workgroups allow,
// so that all run at once; with many, shorter shares even out the end, and cost
// their partial results.  Estimated in rows: a workgroup's own cost is about
// `kOverhead` rows.
int64_t pick_share(const ll_step* s, int tile, const std::vector<int64_t>& seen, int64_t groups) {
  constexpr int64_t kOverhead = 160, kGrain = 64;
  int64_t total = 0, longest = 1;
  for (int64_t w : seen) {
    total += w;
    longest = std::max(longest, w);
  }
  const int64_t slots = max_slots(s, tile);
  auto count = [&](int64_t share, int64_t* split) {   // workgroups per KV head, and those of split tiles
    int64_t n = 0;
    *split = 0;
    for (int64_t w : seen) {
      const int64_t k = ceil_div(w, share);
      n += k;
      if (k > 1) *split += k;
    }
    return n;
  };
  auto cost = [&](int64_t share, int64_t n) {
    const int64_t rounds = ceil_div(n * s->kv_heads, groups);
    if (rounds <= 1) return share + kOverhead;
    return total * s->kv_heads / groups + share / 2 + rounds * kOverhead;
  };
  int64_t split = 0, best = longest, best_cost = cost(longest, count(longest, &split));
  for (int rounds = 1; rounds <= 4; ++rounds) {
    int64_t lo = 1, hi = ceil_div(longest, kGrain);   // the shortest share (in grains) that fits
    while (lo < hi) {
      const int64_t mid = (lo + hi) / 2;
      const int64_t n = count(mid * kGrain, &split);
      if (n * s->kv_heads <= rounds * groups && split <= slots) hi = mid;
      else lo = mid + 1;
    }
    const int64_t share = hi * kGrain, n = count(share, &split);
    if (split > slots) continue;
    if (const int64_t c = cost(share, n); c < best_cost) {
      best = share;
      best_cost = c;
    }
  }
  return best;
}

// The attention's items: every sequence's query rows in tiles, the longest first;
// a tile that needs more cached rows than a share is split over several
// workgroups.  Shares of split tiles come before the others.
int64_t plan_items(const ll_step* s, int tile, const std::vector<ll::StepSeq>& seqs, std::vector<ll::AttendItem>* out) {
  struct Tile {
    int64_t seen;
    int32_t seq, index;
  };
  std::vector<Tile> tiles;
  std::vector<int64_t> seen;
  for (size_t i = 0; i < seqs.size(); ++i) {
    const int64_t q_rows = int64_t{seqs[i].count} * s->group;
    for (int64_t k = tiles_of(q_rows, tile) - 1; k >= 0; --k) {
      const int64_t last = std::min<int64_t>((k + 1) * tile, q_rows) - 1;
      seen.push_back(int64_t{seqs[i].row0} + last / s->group + 1);
      tiles.push_back(Tile{seen.back(), static_cast<int32_t>(i), static_cast<int32_t>(k)});
    }
  }
  std::stable_sort(tiles.begin(), tiles.end(), [](const Tile& a, const Tile& b) { return a.seen > b.seen; });
  const int64_t share = pick_share(s, tile, seen, ll::attend_groups(s->pool->gqa, s->value_dim, tile));
  int64_t slot = 0;
  for (const Tile& x : tiles) {
    const ll::StepSeq& q = seqs[x.seq];
    const int64_t shares = ceil_div(x.seen, share);
    ll::AttendItem it{};
    it.seq = q.seq;
    it.tok0 = q.tok0;
    it.q_rows = q.count * s->group;
    it.row0 = x.index * tile;
    it.first = q.row0;
    it.kv_len = q.row0 + q.count;
    for (int64_t c = 0; c < shares; ++c) {
      it.splits = static_cast<int32_t>(c | shares << 16);
      it.slot = static_cast<int32_t>(slot + c);
      out->push_back(it);
    }
    if (shares > 1) slot += shares;   // the longer tiles: all before the first whole one
  }
  return slot;
}

ll_status check_step(const ll_step* s) {
  if (!s) return fail(LL_EINVAL, "step is NULL");
  if (!s->pool) return fail(LL_EINVAL, "the step's pool has been destroyed");
  return ll::pool_check(s->pool);
}

// The step still fits its sequences.
ll_status check_current(const ll_step* s) {
  if (!s->begun) return fail(LL_EINVAL, "the step has not begun");
  for (size_t i = 0; i < s->seqs.size(); ++i)
    if (s->pool->seqs[s->seqs[i]].gen != s->gens[i])
      return fail(LL_EINVAL, "sequence %d has changed since the step began", s->seqs[i]);
  return LL_OK;
}

ll_status is_capturing(hipStream_t st, bool* out) {
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
int64_t used(int64_t stride, int64_t n) { return n > 1 ? stride : 0; }

ll_status check_plane(const void* p, int64_t ts, int64_t hs, const char* name) {
  if (!p) return fail(LL_EINVAL, "%s is NULL", name);
  if (reinterpret_cast<uintptr_t>(p) & 15) return fail(LL_EINVAL, "%s is not 16-byte aligned", name);
  if ((ts & 7) || (hs & 7) || ts < 0 || hs < 0 || ts > kMaxStride || hs > kMaxStride)
    return fail(LL_EINVAL, "%s: strides must be multiples of 8 values in [0, 2^32]", name);
  return LL_OK;
}

// Rows of an output may not overlap: either tokens lie outside heads or heads
// outside tokens.
ll_status check_output(int64_t ts, int64_t hs, int64_t tokens, int64_t heads, int64_t width, const char* name) {
  const int64_t t = tokens > 1 ? ts : INT64_MAX / 4, h = heads > 1 ? hs : INT64_MAX / 4;
  const bool token_major = h >= width && (heads == 1 ? t >= width : t >= (heads - 1) * hs + width);
  const bool head_major = t >= width && (tokens == 1 ? h >= width : h >= (tokens - 1) * ts + width);
  if (!token_major && !head_major) return fail(LL_EINVAL, "%s: rows overlap", name);
  return LL_OK;
}

// The caller's buffers hold every token that the call may touch: the step's, or
// under capture (later begins are replayed) as many as the step can have.
ll_status check_room(const ll_step* s, int64_t tokens, bool capturing) {
  const int64_t need = capturing ? s->max_tokens : s->tokens;
  if (tokens < need) return fail(LL_EINVAL, "buffers for %lld tokens, but the call may touch %lld", (long long)tokens, (long long)need);
  return LL_OK;
}

// Eager calls follow the pool's earlier work; a captured one is the caller's to
// order.
ll_status start(ll_step* s, hipStream_t st, bool capturing) {
  return capturing ? LL_OK : ll::pool_begin_call(s->pool, st);
}

void finish(ll_step* s, hipStream_t st, bool capturing) {
  if (capturing) return;
  s->pool->last_stream = st;
  s->pool->unevented = true;
}

}  // namespace

extern "C" {

ll_status ll_step_create(ll_pool* p, const ll_step_desc* d, ll_step** out) try {
  if (out) *out = nullptr;
  ll_status rc = ll::pool_check(p);
  if (rc) return rc;
  if (!d || !out) return fail(LL_EINVAL, "NULL argument");
  const int32_t kv_heads = p->gqa ? p->heads : 1;
  if (d->num_heads < 1 || d->num_heads % kv_heads)
    return fail(LL_EINVAL, "num_heads must be a positive multiple of the pool's %d KV heads", kv_heads);
  if (d->max_seqs < 1 || d->max_seqs > p->desc.max_seqs)
    return fail(LL_EINVAL, "max_seqs must lie in 1 .. %d", p->desc.max_seqs);
  // a launch over every token and head stays within one dispatch
  if (d->max_tokens < 1 || d->max_tokens > (1 << 22) || int64_t{d->max_tokens} * d->num_heads > (int64_t{1} << 25))
    return fail(LL_EINVAL, "max_tokens must lie in 1 .. 2^22, and max_tokens * num_heads in 1 .. 2^25");
  if (p->gqa && p->head_chunks * 8 > ll::kMaxHeadDim)
    return fail(LL_EUNSUPPORTED, "head_dim %d is above %d", p->head_chunks * 8, ll::kMaxHeadDim);
  // the kernels count cached rows in 32 bits, up to a tile past the last one
  if (int64_t{p->desc.max_pages_per_seq} * p->P > INT32_MAX - 1024)
    return fail(LL_EUNSUPPORTED, "a sequence may hold more than 2^31 - 1024 rows");
  std::unique_ptr<ll_step> s(new ll_step());
  s->device = p->desc.device;
  s->heads = d->num_heads;
  s->kv_heads = kv_heads;
  s->group = d->num_heads / kv_heads;
  s->max_seqs = d->max_seqs;
  s->max_tokens = d->max_tokens;
  s->value_dim = p->gqa ? p->head_chunks * 8 : ll::kKvLoraRank;
  s->seqs.reserve(static_cast<size_t>(d->max_seqs));
  s->gens.reserve(static_cast<size_t>(d->max_seqs));
  const int tile = ll::attend_tile(p->gqa, s->value_dim, int64_t{d->max_tokens} * s->group);
  s->max_items = int64_t{d->max_tokens} * s->group / 16 + d->max_seqs + kMaxShares / kv_heads;
  if (s->max_items * kv_heads > ll::kMaxDispatchItems / 512)   // of up to 512 threads
    return fail(LL_EUNSUPPORTED, "the step's attention would not fit one dispatch");
  const size_t pairs = p->theta.size();
  size_t at = 0;
  auto take = [&at](size_t bytes) {
    const size_t o = at;
    at = ll::align_up(at + bytes, 256);
    return o;
  };
  size_t o_counts[2], o_items[2];
  for (int k = 0; k < 2; ++k) {
    o_counts[k] = take(sizeof(ll::StepCounts));
    o_items[k] = take(sizeof(ll::AttendItem) * static_cast<size_t>(s->max_items));
  }
  const size_t o_rows = take(sizeof(int32_t) * static_cast<size_t>(d->max_tokens));
  const size_t o_tab = take(sizeof(float) * 2 * pairs * static_cast<size_t>(d->max_tokens));
  const size_t o_theta = take(sizeof(double) * pairs);
  const size_t part_rows = static_cast<size_t>(std::min(kMaxShares * tile, kPartValues / s->value_dim));
  const size_t o_po = take(part_rows * s->value_dim * sizeof(float));
  const size_t o_ml = take(part_rows * 2 * sizeof(float));
  ll::DeviceGuard g(s->device);
  if (!g.ok()) return fail(LL_EDEVICE, "hipSetDevice(%d) failed", s->device);
  if (hipMalloc(reinterpret_cast<void**>(&s->d_buf), at) != hipSuccess) {
    (void)hipGetLastError();
    return fail(LL_ENOMEM, "cannot allocate %zu bytes for the step", at);
  }
  for (int k = 0; k < 2; ++k) {
    s->plans[k].d_counts = reinterpret_cast<ll::StepCounts*>(s->d_buf + o_counts[k]);
    s->plans[k].d_items = reinterpret_cast<ll::AttendItem*>(s->d_buf + o_items[k]);
  }
  s->d_rows = reinterpret_cast<int32_t*>(s->d_buf + o_rows);
  s->d_tab = reinterpret_cast<float*>(s->d_buf + o_tab);
  s->d_theta = reinterpret_cast<double*>(s->d_buf + o_theta);
  s->d_part_o = reinterpret_cast<float*>(s->d_buf + o_po);
  s->d_part_ml = reinterpret_cast<float*>(s->d_buf + o_ml);
  const ll::StepCounts none{};
  hipError_t e = hipMemcpy(s->d_theta, p->theta.data(), pairs * sizeof(double), hipMemcpyHostToDevice);
  for (const Plan& x : s->plans)
    if (e == hipSuccess) e = hipMemcpy(x.d_counts, &none, sizeof none, hipMemcpyHostToDevice);
  if (e != hipSuccess) {
    (void)hipFree(s->d_buf);
    return fail(LL_EDEVICE, "step setup: %s", hipGetErrorString(e));
  }
  try {
    p->step_owners.push_back(&s->pool);
  } catch (...) {
    (void)hipFree(s->d_buf);
    throw;
  }
  s->pool = p;
  *out = s.release();
  return LL_OK;
} catch (...) {
  return ll::pool_host_exception(nullptr);
}

void ll_step_destroy(ll_step* s) try {
  if (!s) return;
  ll::DeviceGuard g(s->device);
  if (ll_pool* p = s->pool) {
    (void)ll::pool_wait_idle(p);
    p->step_owners.erase(std::remove(p->step_owners.begin(), p->step_owners.end(), &s->pool), p->step_owners.end());
  }
  (void)hipFree(s->d_buf);   // waits for the device
  delete s;
} catch (...) {
  return;
}

ll_status ll_step_begin(ll_step* s, const int32_t* seq_ids, const int32_t* counts, int32_t n, int32_t grow,
                        void* stream) try {
  ll_status rc = check_step(s);
  if (rc) return rc;
  ll_pool* p = s->pool;
  if (n < 0 || (n > 0 && (!seq_ids || !counts))) return fail(LL_EINVAL, "bad sequence list");
  if (n > s->max_seqs) return fail(LL_EINVAL, "%d sequences, but the step holds %d", n, s->max_seqs);
  if (grow != 0 && grow != 1) return fail(LL_EINVAL, "grow must be 0 or 1");
  hipStream_t st = static_cast<hipStream_t>(stream);
  ll::DeviceGuard g(s->device);
  bool capturing = false;
  if ((rc = is_capturing(st, &capturing))) return rc;
  if (capturing) return fail(LL_EUNSUPPORTED, "a step cannot begin on a capturing stream");
  if ((rc = ll::pool_enter(p))) return rc;
  const int64_t P = p->P;
  std::vector<char> seen(static_cast<size_t>(p->desc.max_seqs), 0);
  std::vector<int32_t> gain;   // the sequences that get pages
  int64_t tokens = 0, need = 0, most = 0;
  for (int32_t i = 0; i < n; ++i) {
    const int32_t q = seq_ids[i];
    if (q < 0 || q >= p->desc.max_seqs || !p->seqs[q].used) return fail(LL_EINVAL, "entry %d: unknown sequence %d", i, q);
    if (seen[q]) return fail(LL_EINVAL, "entry %d: sequence %d appears twice", i, q);
    seen[q] = 1;
    if (counts[i] < 0) return fail(LL_EINVAL, "entry %d: negative token count", i);
    const ll::SeqState& ss = p->seqs[q];
    if (grow) {
      const int64_t pages = ceil_div(ss.len + counts[i], P);
      if (pages > p->desc.max_pages_per_seq)
        return fail(LL_ERANGE, "entry %d: %lld rows exceed the page-table row", i, (long long)(ss.len + counts[i]));
      if (const int64_t more = pages - ceil_div(ss.len, P)) {
        need += more;
        gain.push_back(q);
      }
    } else if (counts[i] > ss.len) {
      return fail(LL_EINVAL, "entry %d: %d tokens, but sequence %d holds %lld rows", i, counts[i], q, (long long)ss.len);
    }
    tokens += counts[i];
    most = std::max<int64_t>(most, counts[i]);
  }
  if (tokens > s->max_tokens) return fail(LL_EINVAL, "%lld tokens, but the step holds %d", (long long)tokens, s->max_tokens);
  if (need > p->free.count())
    return fail(LL_ENOMEM, "need %lld fresh pages, %lld free", (long long)need, (long long)p->free.count());
  // Page lists that the commit below extends have to be up to date (behind an
  // eviction this waits for the device); the kernels read the device's own.
  if ((rc = ll::pool_fresh_tables(p, gain.data(), gain.size()))) return rc;

  // --- plan (host only, no state change yet)
  std::vector<int32_t> fresh;
  p->free.lowest(need, fresh);
  std::vector<ll::StepSeq> ss(static_cast<size_t>(n));
  std::vector<uint64_t> gens(static_cast<size_t>(n));
  int64_t tok = 0, at = 0;
  for (int32_t i = 0; i < n; ++i) {
    const ll::SeqState& q = p->seqs[seq_ids[i]];
    ll::StepSeq& x = ss[i];
    x.seq = seq_ids[i];
    x.tok0 = static_cast<int32_t>(tok);
    x.count = counts[i];
    x.row0 = static_cast<int32_t>(grow ? q.len : q.len - counts[i]);
    x.pos0 = grow ? q.next_pos : q.next_pos - counts[i];
    x.old_pages = static_cast<int32_t>(ceil_div(q.len, P));
    x.fresh_off = static_cast<int32_t>(at);
    x.new_pages = grow ? static_cast<int32_t>(ceil_div(q.len + counts[i], P) - x.old_pages) : 0;
    tok += counts[i];
    at += x.new_pages;
  }
  // a graph's plan keeps its tile; eager calls take the one for these tokens
  const int tile = ll::attend_tile(p->gqa, s->value_dim, most * s->group);
  const int graph_tile = s->captured ? s->plans[0].tile : tile;
  std::vector<ll::AttendItem> items, own;
  const int64_t shares = plan_items(s, graph_tile, ss, &items);
  const int64_t own_shares = tile == graph_tile ? 0 : plan_items(s, tile, ss, &own);
  if (const size_t n_items = std::max(items.size(), own.size()); static_cast<int64_t>(n_items) > s->max_items)
    return fail(LL_EINVAL, "the step's attention needs %zu items, more than %lld", n_items, (long long)s->max_items);
  // host memory that the commit below needs, before anything changes
  for (int32_t i = 0; i < n; ++i) {
    ll::SeqState& q = p->seqs[seq_ids[i]];
    const size_t pages = q.pages.size() + static_cast<size_t>(ss[i].new_pages);
    // reserve alone would make room for exactly these, and move the list every time
    if (pages > q.pages.capacity()) q.pages.reserve(std::max(pages, 2 * q.pages.capacity()));
  }

  // --- upload and lay out
  if ((rc = ll::pool_begin_call(p, st))) return rc;
  ll::Staging* sg = nullptr;
  const size_t b_seq = ll::align_up(ss.size() * sizeof(ll::StepSeq), 256);
  const size_t b_it = ll::align_up(items.size() * sizeof(ll::AttendItem), 256);
  const size_t b_pg = ll::align_up(fresh.size() * sizeof(int32_t), 256);
  const size_t b_own = ll::align_up(own.size() * sizeof(ll::AttendItem), 256);
  if ((rc = ll::pool_stage(p, b_seq + b_it + b_pg + b_own + 256, &sg))) return rc;
  if (!ss.empty()) std::memcpy(sg->host, ss.data(), ss.size() * sizeof(ll::StepSeq));
  if (!items.empty()) std::memcpy(sg->host + b_seq, items.data(), items.size() * sizeof(ll::AttendItem));
  if (!fresh.empty()) std::memcpy(sg->host + b_seq + b_it, fresh.data(), fresh.size() * sizeof(int32_t));
  if (!own.empty()) std::memcpy(sg->host + b_seq + b_it + b_pg, own.data(), own.size() * sizeof(ll::AttendItem));
  sg->used = b_seq + b_it + b_pg + b_own;
  if ((rc = ll::pool_upload(p, sg, st))) return rc;
  ll::StepSetupLaunch a{};
  a.counts.tokens = static_cast<int32_t>(tokens);
  a.counts.items = static_cast<int32_t>(items.size());
  a.counts.seqs = n;
  a.counts.shares = static_cast<int32_t>(shares);
  a.own_counts = a.counts;
  a.own_counts.items = static_cast<int32_t>(own.size());
  a.own_counts.shares = static_cast<int32_t>(own_shares);
  a.src_seqs = reinterpret_cast<const ll::StepSeq*>(sg->dev);
  a.src_items = reinterpret_cast<const ll::AttendItem*>(sg->dev + b_seq);
  a.fresh = reinterpret_cast<const int32_t*>(sg->dev + b_seq + b_it);
  a.src_own = reinterpret_cast<const ll::AttendItem*>(sg->dev + b_seq + b_it + b_pg);
  a.theta = s->d_theta;
  a.pairs = static_cast<int32_t>(p->theta.size());
  a.page_shift = p->page_shift;
  a.max_pages_per_seq = p->desc.max_pages_per_seq;
  a.num_pages = p->desc.num_pages;
  a.page_table = p->desc.page_table;
  a.dst_counts = s->plans[0].d_counts;
  a.dst_items = s->plans[0].d_items;
  a.dst_own_counts = s->plans[1].d_counts;
  a.dst_own_items = s->plans[1].d_items;
  a.rows = s->d_rows;
  a.tab = s->d_tab;
  hipError_t e = ll::launch_step_setup(a, st);
  if (e != hipSuccess) return ll::pool_device_fail(p, e, "step_setup_kernel launch");
  if ((rc = ll::pool_end_call(p, sg, st))) return rc;

  // --- commit host state
  for (int32_t pg : fresh) p->free.take(pg);
  p->free.advance_hint();
  s->seqs.assign(seq_ids, seq_ids + n);
  for (int32_t i = 0; i < n; ++i) {
    ll::SeqState& q = p->seqs[seq_ids[i]];
    if (grow && counts[i] > 0) {
      q.pages.insert(q.pages.end(), fresh.begin() + ss[i].fresh_off, fresh.begin() + ss[i].fresh_off + ss[i].new_pages);
      q.len += counts[i];
      q.next_pos += counts[i];
      q.gen = ++p->epoch;
    }
    gens[i] = q.gen;
  }
  s->gens = std::move(gens);
  s->plans[0].tile = graph_tile;
  s->plans[0].items = static_cast<int64_t>(items.size());
  s->plans[0].shares = shares;
  s->plans[1].tile = tile;
  s->plans[1].items = static_cast<int64_t>(own.size());
  s->plans[1].shares = own_shares;
  s->eager = tile == graph_tile ? 0 : 1;
  s->tokens = tokens;
  s->begun = true;
  return LL_OK;
} catch (...) {
  return ll::pool_host_exception(s ? s->pool : nullptr);
}

ll_status ll_step_append(ll_step* s, const ll_append_desc* d, void* stream) try {
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
  const int64_t T = capturing ? s->max_tokens : s->tokens, D = p->gqa ? s->value_dim : ll::kRopeDim;
  if (d->layer < 0 || d->layer >= p->desc.num_layers) return fail(LL_EINVAL, "layer %d out of range", d->layer);
  if (T == 0) return LL_OK;
  const bool rows = d->a || d->b, asks = d->q || d->q_out;
  if (!rows && !asks) return fail(LL_EINVAL, "neither cache rows nor queries are given");
  if (rows) {
    if ((rc = check_plane(d->a, used(d->a_token_stride, T), used(d->a_head_stride, s->kv_heads), p->gqa ? "K" : "c_kv"))) return rc;
    if ((rc = check_plane(d->b, used(d->b_token_stride, T), used(d->b_head_stride, s->kv_heads), p->gqa ? "V" : "k_pe"))) return rc;
  }
  if (asks) {
    if ((rc = check_plane(d->q, used(d->q_token_stride, T), used(d->q_head_stride, s->heads), "q"))) return rc;
    if ((rc = check_plane(d->q_out, used(d->q_out_token_stride, T), used(d->q_out_head_stride, s->heads), "q_out"))) return rc;
    if ((rc = check_output(d->q_out_token_stride, d->q_out_head_stride, T, s->heads, D, "q_out"))) return rc;
    if (d->q_out == d->q && (used(d->q_token_stride, T) != used(d->q_out_token_stride, T) ||
                             used(d->q_head_stride, s->heads) != used(d->q_out_head_stride, s->heads)))
      return fail(LL_EINVAL, "q_out is q, but its strides are others");
  }
  if (d->q_norm && !p->gqa) return fail(LL_EINVAL, "q_norm is for GQA / MHA pools only");
  if (d->norm || d->q_norm) {
    if (d->norm_type != LL_TYPE_BF16 && d->norm_type != LL_TYPE_F32) return fail(LL_EINVAL, "unknown norm_type %d", d->norm_type);
    if ((reinterpret_cast<uintptr_t>(d->norm) | reinterpret_cast<uintptr_t>(d->q_norm)) & 15)
      return fail(LL_EINVAL, "a norm weight is not 16-byte aligned");
    if (!(d->eps >= 0.f) || !std::isfinite(d->eps)) return fail(LL_EINVAL, "eps must be finite and not negative");
  }
  ll::AppendLaunch a{};
  a.counts = s->plans[0].d_counts;
  a.rows = s->d_rows;
  a.tab = s->d_tab;
  a.pairs = static_cast<int32_t>(p->theta.size());
  a.capacity = static_cast<int32_t>(T);
  a.heads = s->heads;
  a.kv_heads = s->kv_heads;
  a.head_chunks = static_cast<int32_t>(D / 8);
  a.group_shift = 0;
  while ((1 << a.group_shift) < a.head_chunks) ++a.group_shift;
  const int32_t per_wave = 64 >> a.group_shift;   // heads of a piece
  a.kv_pieces = !rows ? 0 : p->gqa ? 2 * static_cast<int32_t>(ceil_div(s->kv_heads, per_wave)) : 1;
  a.pieces = a.kv_pieces + (asks ? static_cast<int32_t>(ceil_div(s->heads, per_wave)) : 0);
  a.band_chunks = static_cast<int32_t>(p->theta.size() / 4);
  a.norm_f32 = d->norm_type == LL_TYPE_F32;
  a.eps = d->eps;
  a.a = static_cast<const uint16_t*>(d->a);
  a.a_ts = d->a_token_stride;
  a.a_hs = d->a_head_stride;
  a.b = static_cast<const uint16_t*>(d->b);
  a.b_ts = d->b_token_stride;
  a.b_hs = d->b_head_stride;
  a.norm = d->norm;
  a.q = static_cast<const uint16_t*>(d->q);
  a.q_ts = d->q_token_stride;
  a.q_hs = d->q_head_stride;
  a.q_out = static_cast<uint16_t*>(d->q_out);
  a.qo_ts = d->q_out_token_stride;
  a.qo_hs = d->q_out_head_stride;
  a.q_norm = d->q_norm;
  a.k_plane = static_cast<uint16_t*>(p->layer_ptrs[static_cast<size_t>(d->layer)]);
  a.v_plane = p->gqa ? static_cast<uint16_t*>(p->layer_ptrs[static_cast<size_t>(p->desc.num_layers + d->layer)]) : nullptr;
  if ((rc = start(s, st, capturing))) return rc;
  hipError_t e = ll::launch_append(a, p->gqa, p->desc.rope_pairing, st);
  if (e != hipSuccess) return ll::pool_device_fail(p, e, "append_kernel launch");
  finish(s, st, capturing);
  return LL_OK;
} catch (...) {
  return ll::pool_host_exception(s ? s->pool : nullptr);
}

ll_status ll_step_attend(ll_step* s, const ll_attend_desc* d, void* stream) try {
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
  if (d->layer < 0 || d->layer >= p->desc.num_layers) return fail(LL_EINVAL, "layer %d out of range", d->layer);
  if (d->causal != 0 && d->causal != 1) return fail(LL_EINVAL, "causal must be 0 or 1");
  if (d->window < 0 || (d->window > 0 && !d->causal)) return fail(LL_EINVAL, "window must be >= 0, and needs causal");
  // (the kernels keep scores in base 2)
  if (!std::isfinite(d->scale * ll::kLog2e)) return fail(LL_EINVAL, "scale, times log2 e, is not finite");
  const int64_t T = capturing ? s->max_tokens : s->tokens;
  if (T == 0) return LL_OK;
  if ((rc = check_plane(d->q, used(d->q_token_stride, T), used(d->q_head_stride, s->heads), "q"))) return rc;
  if (p->gqa) {
    if (d->q_pe) return fail(LL_EINVAL, "q_pe is for MLA pools only");
  } else if ((rc = check_plane(d->q_pe, used(d->q_pe_token_stride, T), used(d->q_pe_head_stride, s->heads), "q_pe"))) {
    return rc;
  }
  if ((rc = check_plane(d->out, used(d->out_token_stride, T), used(d->out_head_stride, s->heads), "out"))) return rc;
  if ((rc = check_output(d->out_token_stride, d->out_head_stride, T, s->heads, s->value_dim, "out"))) return rc;
  if (reinterpret_cast<uintptr_t>(d->lse) & 3) return fail(LL_EINVAL, "lse is not 4-byte aligned");
  ll::AttendLaunch a{};
  const Plan& plan = s->plans[capturing ? 0 : s->eager];
  a.counts = plan.d_counts;
  a.items = plan.d_items;
  a.n_items = static_cast<int32_t>(capturing ? s->max_items : plan.items);
  a.n_shares = static_cast<int32_t>(capturing ? max_slots(s, plan.tile) : plan.shares);
  a.join_blocks = static_cast<int32_t>(ceil_div(int64_t{plan.tile} * s->value_dim, 1024));
  a.kv_heads = s->kv_heads;
  a.group = s->group;
  a.tile = plan.tile;
  a.causal = d->causal;
  a.window = static_cast<int32_t>(std::min<int64_t>(d->window, INT32_MAX));
  a.scale = d->scale;
  a.dim = s->value_dim;
  a.k_plane = static_cast<const uint16_t*>(p->layer_ptrs[static_cast<size_t>(d->layer)]);
  a.v_plane = p->gqa ? static_cast<const uint16_t*>(p->layer_ptrs[static_cast<size_t>(p->desc.num_layers + d->layer)]) : nullptr;
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
  a.out = static_cast<uint16_t*>(d->out);
  a.o_ts = d->out_token_stride;
  a.o_hs = d->out_head_stride;
  a.lse = d->lse;
  a.heads = s->heads;
  a.part_o = s->d_part_o;
  a.part_ml = s->d_part_ml;
  if ((rc = start(s, st, capturing))) return rc;
  hipError_t e = ll::launch_attend(a, p->gqa, st);
  if (e != hipSuccess) return ll::pool_device_fail(p, e, "attend_kernel launch");
  if (capturing) s->captured = true;
  finish(s, st, capturing);
  return LL_OK;
} catch (...) {
  return ll::pool_host_exception(s ? s->pool : nullptr);
}

}  // extern "C"
