// The serving step's host side (step.cpp) on the CPU: built with pool.cpp and the
// HIP stand-ins under AddressSanitizer and UndefinedBehaviorSanitizer.  Random
// begins between allocations, splices, evictions and frees; every begin's books
// are predicted here, and its plan (token rows, page-table entries, attention
// items) is checked for what the kernels assume of it.  Refused calls must leave
// everything as it was.  Usage: step_driver mla|gqa page_size seed
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdio>
#include <cstdlib>
#include <map>
#include <random>
#include <set>
#include <string>
#include <vector>

#include "leyline_step.h"
#include "../../mla_paged_cache_amd/csrc/step_internal.h"

#define CHECK(x)                                                             \
  do {                                                                       \
    if (!(x)) {                                                              \
      std::fprintf(stderr, "line %d: %s (%s)\n", __LINE__, #x, ll_last_error()); \
      std::exit(1);                                                          \
    }                                                                        \
  } while (0)

namespace {
bool g_capturing = false, g_fail = false;
ll::StepSetupLaunch g_setup;
ll::AppendLaunch g_append;
ll::AttendLaunch g_attend;
int g_setups = 0, g_appends = 0, g_attends = 0;
}  // namespace

extern "C" hipError_t hipStreamIsCapturing(hipStream_t, hipStreamCaptureStatus* s) {
  *s = g_capturing ? hipStreamCaptureStatusActive : hipStreamCaptureStatusNone;
  return hipSuccess;
}

extern "C" hipError_t hipGetLastError() { return hipSuccess; }

namespace ll {
// What the kernel writes, in order.
hipError_t launch_step_setup(const StepSetupLaunch& a, hipStream_t) {
  if (g_fail) return hipErrorLaunchFailure;
  g_setup = a;
  ++g_setups;
  *a.dst_counts = a.counts;
  for (int i = 0; i < a.counts.items; ++i) a.dst_items[i] = a.src_items[i];
  for (int i = 0; i < a.counts.seqs; ++i) {
    const StepSeq& s = a.src_seqs[i];
    int32_t* table = a.page_table + int64_t{s.seq} * a.max_pages_per_seq;
    for (int k = 0; k < s.new_pages; ++k) {
      CHECK(s.old_pages + k < a.max_pages_per_seq);
      table[s.old_pages + k] = a.fresh[s.fresh_off + k];
    }
    for (int k = 0; k < s.count; ++k) {
      const int r = s.row0 + k;
      CHECK(r >= 0 && s.tok0 + k < a.counts.tokens);
      a.rows[s.tok0 + k] = (table[r >> a.page_shift] << a.page_shift) + (r & ((1 << a.page_shift) - 1));
      for (int j = 0; j < 2 * a.pairs; ++j) a.tab[(int64_t{s.tok0} + k) * 2 * a.pairs + j] = static_cast<float>(s.pos0 + k);
    }
  }
  return hipSuccess;
}
hipError_t launch_append(const AppendLaunch& a, bool, int, hipStream_t) {
  g_append = a;
  ++g_appends;
  return hipSuccess;
}
int attend_tile(bool, int, int64_t rows) { return rows <= 16 ? 16 : rows <= 32 ? 32 : rows <= 64 ? 64 : 128; }
int attend_groups(bool, int, int) { return 8; }
hipError_t launch_attend(const AttendLaunch& a, bool, hipStream_t) {
  g_attend = a;
  ++g_attends;
  return hipSuccess;
}
}  // namespace ll

namespace {

struct Seq {
  int64_t len = -1, pos = 0;
  std::vector<int32_t> pages;
  bool operator==(const Seq& o) const { return len == o.len && pos == o.pos && pages == o.pages; }
};

constexpr int kSeqs = 6, kPagesPerSeq = 40, kTokens = 90;

struct World {
  bool gqa;
  int P, num_pages, heads, kv_heads, dim;
  ll_pool* pool = nullptr;
  std::vector<std::vector<char>> planes;
  std::vector<int32_t> table;
  std::vector<char> buf;

  World(bool g, int page) : gqa(g), P(page), num_pages(150), heads(g ? 6 : 20), kv_heads(g ? 3 : 1), dim(g ? 64 : 512) {
    const size_t bytes = static_cast<size_t>(num_pages) * P * (gqa ? 3 * 64 * 2 : 576 * 2);
    std::vector<void*> k, v;
    for (int i = 0; i < 4; ++i) planes.emplace_back(bytes + 16);
    for (int i = 0; i < 2; ++i) {
      k.push_back(at16(planes[i]));
      v.push_back(at16(planes[2 + i]));
    }
    table.assign(static_cast<size_t>(kSeqs) * kPagesPerSeq, -1);
    buf.assign(1 << 16, 0);
    if (gqa) {
      ll_gqa_pool_desc d{};
      d.num_layers = 2, d.page_size = P, d.num_pages = num_pages, d.max_seqs = kSeqs, d.max_pages_per_seq = kPagesPerSeq;
      d.num_kv_heads = 3, d.head_dim = 64, d.rotary_dim = 32, d.rope_pairing = LL_ROPE_HALF, d.rope_base = 500000.0;
      d.k_layer_base = k.data(), d.v_layer_base = v.data(), d.page_table = table.data();
      CHECK(ll_pool_create_gqa(&d, &pool) == LL_OK);
    } else {
      ll_pool_desc d{};
      d.num_layers = 2, d.page_size = P, d.num_pages = num_pages, d.max_seqs = kSeqs, d.max_pages_per_seq = kPagesPerSeq;
      d.kv_lora_rank = 512, d.rope_dim = 64, d.rope_pairing = LL_ROPE_INTERLEAVED, d.rope_base = 10000.0;
      d.layer_base = k.data(), d.page_table = table.data();
      CHECK(ll_pool_create(&d, &pool) == LL_OK);
    }
  }
  static void* at16(std::vector<char>& v) {
    return reinterpret_cast<void*>((reinterpret_cast<uintptr_t>(v.data()) + 15) & ~uintptr_t{15});
  }
  std::map<int, Seq> books() const {
    std::map<int, Seq> out;
    for (int s = 0; s < kSeqs; ++s) {
      Seq q;
      q.pages.resize(kPagesPerSeq);
      int32_t n = 0;
      if (ll_seq_get(pool, s, &q.len, &q.pos, q.pages.data(), kPagesPerSeq, &n) != LL_OK) continue;
      q.pages.resize(static_cast<size_t>(n));
      out[s] = q;
    }
    return out;
  }
  std::vector<int32_t> free_pages(const std::map<int, Seq>& b) const {
    std::set<int32_t> used;
    for (auto& [s, q] : b) used.insert(q.pages.begin(), q.pages.end());
    std::vector<int32_t> out;
    for (int i = 0; i < num_pages; ++i)
      if (!used.count(i)) out.push_back(i);
    return out;
  }
};

struct StepModel {
  ll_step* h = nullptr;
  bool begun = false;
  std::vector<int> seqs, counts;
  std::map<int, Seq> as_begun;
  int tokens = 0, tile = 16;
};

// The plan covers every query row of every sequence against all its rows once.
void check_plan(const World& w, const StepModel& m, const std::map<int, Seq>& b) {
  const ll::StepSetupLaunch& a = g_setup;
  CHECK(a.counts.tokens == m.tokens && a.counts.seqs == static_cast<int>(m.seqs.size()));
  const int group = w.heads / w.kv_heads;
  int tok = 0;
  std::map<std::pair<int, int>, std::vector<ll::AttendItem>> by_tile;
  std::set<int> slots;
  for (int i = 0; i < a.counts.items; ++i) {
    const ll::AttendItem& it = a.dst_items[i];
    const int shares = it.splits >> 16;
    CHECK(shares >= 1 && (it.splits & 0xFFFF) < shares);
    CHECK((shares > 1) == (i < a.counts.shares));
    if (shares > 1) CHECK(slots.insert(it.slot).second && it.slot == i);
    by_tile[{it.seq, it.row0}].push_back(it);
  }
  // the partial results' buffer holds the slots
  CHECK(int64_t{a.counts.shares} * w.kv_heads <= 2048);
  CHECK(int64_t{a.counts.shares} * w.kv_heads * m.tile * w.dim <= int64_t{1} << 25);
  for (size_t i = 0; i < m.seqs.size(); ++i) {
    const Seq& q = b.at(m.seqs[i]);
    for (int k = 0; k < m.counts[i]; ++k, ++tok) {
      const int64_t r = q.len - m.counts[i] + k;
      CHECK(a.rows[tok] == q.pages[r / w.P] * w.P + r % w.P);
      CHECK(a.tab[int64_t{tok} * 2 * a.pairs] == static_cast<float>(q.pos - m.counts[i] + k));
    }
    const int q_rows = m.counts[i] * group;
    for (int r0 = 0; r0 < q_rows; r0 += m.tile) {
      auto f = by_tile.find({m.seqs[i], r0});
      CHECK(f != by_tile.end());
      const int shares = f->second[0].splits >> 16;
      CHECK(static_cast<int>(f->second.size()) == shares);
      for (int c = 0; c < shares; ++c) {
        const ll::AttendItem& it = f->second[c];
        CHECK((it.splits & 0xFFFF) == c && it.slot == f->second[0].slot + c);
        CHECK(it.tok0 == tok - m.counts[i] && it.q_rows == q_rows && it.kv_len == q.len);
        CHECK(it.first == q.len - m.counts[i]);
      }
      by_tile.erase(f);
    }
    for (size_t k = 0; k < q.pages.size(); ++k) CHECK(w.table[int64_t{m.seqs[i]} * kPagesPerSeq + k] == q.pages[k]);
  }
  CHECK(by_tile.empty() && tok == m.tokens);
}

ll_append_desc append_desc(World& w, int64_t tokens) {
  ll_append_desc d{};
  char* p = static_cast<char*>(World::at16(w.buf));
  d.tokens = tokens;
  d.a = d.b = d.q = p;
  d.q_out = p + 4096;
  d.a_token_stride = d.b_token_stride = w.gqa ? 192 : 512;
  d.a_head_stride = d.b_head_stride = 64;
  d.q_token_stride = d.q_out_token_stride = w.heads * 64;
  d.q_head_stride = d.q_out_head_stride = 64;
  d.eps = 1e-6f;
  return d;
}
ll_attend_desc attend_desc(World& w, int64_t tokens) {
  ll_attend_desc d{};
  char* p = static_cast<char*>(World::at16(w.buf));
  d.tokens = tokens;
  d.causal = 1;
  d.scale = 0.1f;
  d.q = p;
  d.q_token_stride = d.out_token_stride = w.heads * w.dim;
  d.q_head_stride = d.out_head_stride = w.dim;
  if (!w.gqa) {
    d.q_pe = p;
    d.q_pe_token_stride = w.heads * 64;
    d.q_pe_head_stride = 64;
  }
  d.out = p + 8192;
  return d;
}

void refusals(World& w, StepModel& m) {
  const int before = g_appends + g_attends;
  auto bad_append = [&](auto change) {
    ll_append_desc d = append_desc(w, m.tokens);
    change(d);
    CHECK(ll_step_append(m.h, &d, nullptr) == LL_EINVAL);
  };
  auto bad_attend = [&](auto change) {
    ll_attend_desc d = attend_desc(w, m.tokens);
    change(d);
    CHECK(ll_step_attend(m.h, &d, nullptr) == LL_EINVAL);
  };
  auto shift = [](const void* p) { return static_cast<const void*>(static_cast<const char*>(p) + 8); };
  CHECK(ll_step_append(m.h, nullptr, nullptr) == LL_EINVAL && ll_step_attend(m.h, nullptr, nullptr) == LL_EINVAL);
  bad_append([](auto& d) { d.layer = 2; });
  bad_append([](auto& d) { d.layer = -1; });
  bad_append([&](auto& d) { d.tokens = m.tokens - 1; });
  bad_append([](auto& d) { d.a = nullptr; });
  bad_append([](auto& d) { d.b = nullptr; });
  bad_append([](auto& d) { d.q = nullptr; });
  bad_append([](auto& d) { d.q_out = nullptr; });
  bad_append([](auto& d) { d.a = d.b = d.q = nullptr; d.q_out = nullptr; });
  bad_append([&](auto& d) { d.a = shift(d.a); });
  bad_append([&](auto& d) { d.b = shift(d.b); });
  bad_append([&](auto& d) { d.q = shift(d.q); });
  bad_append([&](auto& d) { d.norm = shift(d.a); });
  bad_append([](auto& d) { d.norm = d.a; d.norm_type = 2; });
  bad_append([](auto& d) { d.norm = d.a; d.eps = -1.f; });
  bad_append([](auto& d) { d.norm = d.a; d.eps = __builtin_nanf(""); });
  bad_append([](auto& d) { d.norm = d.a; d.eps = __builtin_inff(); });
  bad_append([](auto& d) { d.q_out_head_stride = 56; });
  bad_append([](auto& d) { d.q_out_head_stride = 0; });
  bad_append([](auto& d) { d.q_head_stride = 68; });
  bad_append([](auto& d) { d.q_head_stride = -64; });
  bad_append([](auto& d) { d.q_head_stride = (int64_t{1} << 32) + 8; });
  if (!w.gqa) bad_append([](auto& d) { d.q_norm = d.a; });
  bad_attend([](auto& d) { d.layer = 2; });
  bad_attend([&](auto& d) { d.tokens = m.tokens - 1; });
  bad_attend([](auto& d) { d.causal = 2; });
  bad_attend([](auto& d) { d.window = -1; });
  bad_attend([](auto& d) { d.causal = 0, d.window = 5; });
  bad_attend([](auto& d) { d.scale = __builtin_inff(); });
  bad_attend([](auto& d) { d.scale = __builtin_nanf(""); });
  bad_attend([](auto& d) { d.q = nullptr; });
  bad_attend([](auto& d) { d.out = nullptr; });
  bad_attend([&](auto& d) { d.q = shift(d.q); });
  bad_attend([&](auto& d) { d.out = const_cast<void*>(shift(d.out)); });
  bad_attend([](auto& d) { d.lse = reinterpret_cast<float*>(static_cast<char*>(d.out) + 2); });
  bad_attend([&](auto& d) { d.out_head_stride = w.dim - 8; });
  if (m.tokens > 1) bad_attend([&](auto& d) { d.out_token_stride = w.dim; });
  if (w.gqa) bad_attend([](auto& d) { d.q_pe = d.q; });
  else bad_attend([](auto& d) { d.q_pe = nullptr; });
  CHECK(g_appends + g_attends == before);
}

int run(bool gqa, int P, int seed) {
  World w(gqa, P);
  std::mt19937 rng(static_cast<unsigned>(seed));
  auto below = [&](int n) { return static_cast<int>(rng() % static_cast<unsigned>(n)); };
  {   // refused descriptors
    ll_step* h = reinterpret_cast<ll_step*>(8);
    auto bad = [&](int32_t heads, int32_t seqs, int32_t tokens) {
      const ll_step_desc d{heads, seqs, tokens};
      CHECK(ll_step_create(w.pool, &d, &h) == LL_EINVAL && !h);
    };
    bad(0, 1, 1), bad(-3, 1, 1), bad(w.heads, 0, 1), bad(w.heads, kSeqs + 1, 1), bad(w.heads, 1, 0);
    bad(w.heads, 1, (1 << 22) + 1), bad(3 << 20, 1, 100);
    if (gqa) bad(w.heads + 1, 1, 1);
    const ll_step_desc d{w.heads, 1, 1};
    CHECK(ll_step_create(nullptr, &d, &h) == LL_EINVAL);
    CHECK(ll_step_create(w.pool, nullptr, &h) == LL_EINVAL);
    CHECK(ll_step_create(w.pool, &d, nullptr) == LL_EINVAL);
    CHECK(ll_step_begin(nullptr, nullptr, nullptr, 0, 1, nullptr) == LL_EINVAL);
    CHECK(ll_step_append(nullptr, nullptr, nullptr) == LL_EINVAL && ll_step_attend(nullptr, nullptr, nullptr) == LL_EINVAL);
    ll_step_destroy(nullptr);
  }
  StepModel steps[2];
  const int room[2] = {4, kSeqs};
  for (int i = 0; i < 2; ++i) {
    const ll_step_desc d{w.heads, room[i], kTokens};
    CHECK(ll_step_create(w.pool, &d, &steps[i].h) == LL_OK);
    ll_append_desc ad = append_desc(w, kTokens);
    CHECK(ll_step_append(steps[i].h, &ad, nullptr) == LL_EINVAL);   // not begun
  }
  std::map<int, Seq> b = w.books();
  int begun = 0, refused = 0, stale = 0, behind = 0;
  for (int op = 0; op < 500; ++op) {
    const int kind = below(10);
    if (kind == 0) {
      int32_t s = -1;
      (void)ll_seq_alloc(w.pool, below(6 * P + 30), &s, nullptr);
    } else if (kind == 1 && !b.empty() && below(3) == 0) {
      CHECK(ll_seq_free(w.pool, std::next(b.begin(), below(static_cast<int>(b.size())))->first) == LL_OK);
    } else if (kind == 2 && !b.empty()) {
      const auto& [s, q] = *std::next(b.begin(), below(static_cast<int>(b.size())));
      if (q.len > 2) {
        ll_directive d{};
        d.seq_id = s, d.mode = LL_AMORTIZE, d.s_start = below(static_cast<int>(q.len)), d.s_end = d.s_start + 1;
        (void)leyline_splice(w.pool, &d, 1, nullptr);
      }
    } else if (kind == 3 && !b.empty()) {
      const auto& [s, q] = *std::next(b.begin(), below(static_cast<int>(b.size())));
      std::vector<uint8_t> keep(static_cast<size_t>(q.len) + 16);
      for (auto& k : keep) k = below(8) != 0;
      const int64_t off = 0;
      const int32_t id = s;
      const bool done = kv_evict_compact(w.pool, &id, 1, keep.data(), &off, nullptr) == LL_OK;
      // at page size 1 the books are still pending: a step refuses, whatever comes
      for (StepModel& m : steps) {
        ll_append_desc d = append_desc(w, kTokens);
        if (done && m.begun && std::find(m.seqs.begin(), m.seqs.end(), id) != m.seqs.end() && std::count(keep.begin(), keep.begin() + q.len, 0))
          CHECK(ll_step_append(m.h, &d, nullptr) == LL_EINVAL);
      }
      // and a begin right behind it settles them
      const int64_t kept = std::count(keep.begin(), keep.begin() + q.len, 1), pos = q.pos;
      const int32_t two = 2;
      StepModel& m = steps[1];
      if (done && below(2) && ll_step_begin(m.h, &id, &two, 1, 1, nullptr) == LL_OK) {
        m.begun = true;
        m.seqs = {id}, m.counts = {2}, m.tokens = 2;
        m.tile = ll::attend_tile(gqa, w.dim, 2 * (w.heads / w.kv_heads));
        m.as_begun = w.books();
        CHECK(m.as_begun[id].len == kept + 2 && m.as_begun[id].pos == pos + 2);
        check_plan(w, m, m.as_begun);
        ++behind;
      }
    } else {
      StepModel& m = steps[below(2)];
      std::vector<int32_t> seqs, counts;
      std::vector<int> ids;
      for (auto& [s, q] : b) ids.push_back(s);
      std::shuffle(ids.begin(), ids.end(), rng);
      const bool grow = below(3) != 0;
      const int n = ids.empty() ? 0 : below(static_cast<int>(ids.size()) + 1);
      int64_t total = 0, need = 0;
      bool over = false;
      for (int i = 0; i < n; ++i) {
        const Seq& q = b[ids[i]];
        int c = below(4) == 0 ? below(60) : below(3);
        if (!grow) c = static_cast<int>(std::min<int64_t>(c, q.len));
        seqs.push_back(ids[i]);
        counts.push_back(c);
        total += c;
        if (grow) {
          const int64_t pages = (q.len + c + P - 1) / P;
          over |= pages > kPagesPerSeq;
          need += pages - static_cast<int64_t>(q.pages.size());
        }
      }
      const std::vector<int32_t> fresh = w.free_pages(b);
      ll_status want = LL_OK;
      int32_t g = grow;
      void* st = nullptr;
      const int limit = &m == &steps[0] ? room[0] : room[1];
      switch (below(12)) {
        case 0:
          if (n >= 2) seqs[n - 1] = seqs[0], want = LL_EINVAL;
          break;
        case 1:
          if (n >= 1) seqs[below(n)] = below(2) ? -1 : kSeqs, want = LL_EINVAL;
          break;
        case 2:
          if (n >= 1) counts[below(n)] = -1, want = LL_EINVAL;
          break;
        case 3: g = 2, want = LL_EINVAL; break;
        case 4: g_capturing = true, want = LL_EUNSUPPORTED; break;
        case 5:
          if (n >= 1 && !grow) counts[0] = static_cast<int32_t>(b[seqs[0]].len + 1), want = LL_EINVAL;
          break;
        default: break;
      }
      if (want == LL_OK) {
        if (n > limit) want = LL_EINVAL;
        else if (over) want = LL_ERANGE;
        else if (total > kTokens) want = LL_EINVAL;
        else if (need > static_cast<int64_t>(fresh.size())) want = LL_ENOMEM;
      }
      const int setups = g_setups;
      const ll_status got = ll_step_begin(m.h, seqs.data(), counts.data(), n, g, st);
      g_capturing = false;
      const std::map<int, Seq> now = w.books();
      if (want != LL_OK) {
        // a wrong entry may be met after one that is too long
        CHECK(got == want || (got != LL_OK && (over || n > limit)));
        CHECK(now == b && g_setups == setups);
        ++refused;
      } else {
        CHECK(got == LL_OK && g_setups == setups + 1);
        size_t at = 0;
        std::map<int, Seq> model = b;
        if (grow)
          for (int i = 0; i < n; ++i) {
            Seq& q = model[seqs[i]];
            q.len += counts[i];
            q.pos += counts[i];
            while (static_cast<int64_t>(q.pages.size()) < (q.len + P - 1) / P) q.pages.push_back(fresh[at++]);
          }
        CHECK(now == model);
        m.begun = true;
        m.seqs.assign(seqs.begin(), seqs.end());
        m.counts.assign(counts.begin(), counts.end());
        m.tokens = static_cast<int>(total);
        const int most = n ? *std::max_element(counts.begin(), counts.end()) : 0;
        m.tile = ll::attend_tile(gqa, w.dim, int64_t{most} * (w.heads / w.kv_heads));
        m.as_begun = now;
        check_plan(w, m, now);
        ++begun;
      }
    }
    b = w.books();
    int64_t n_free = 0;
    CHECK(ll_pool_free_pages(w.pool, &n_free) == LL_OK && n_free == static_cast<int64_t>(w.free_pages(b).size()));
    for (StepModel& m : steps) {
      if (!m.begun) continue;
      bool changed = false;
      for (int s : m.seqs) changed |= !b.count(s) || !(b[s] == m.as_begun[s]);
      ll_append_desc ad = append_desc(w, m.tokens + below(2));
      ll_attend_desc td = attend_desc(w, m.tokens + below(2));
      const int na = g_appends, nt = g_attends;
      const ll_status ra = ll_step_append(m.h, &ad, nullptr), rt = ll_step_attend(m.h, &td, nullptr);
      CHECK(ra == rt);
      if (changed) {
        CHECK(ra == LL_EINVAL);
        ++stale;
      }
      if (ra != LL_OK) {   // refused; an operation may also have rewritten a sequence into the same books
        CHECK(ra == LL_EINVAL && g_appends == na && g_attends == nt);
        m.begun = false;
        continue;
      }
      const bool any = m.tokens > 0;
      CHECK(g_appends == na + any && g_attends == nt + any);
      if (any) {
        CHECK(g_append.capacity == m.tokens && g_attend.tile == m.tile);
        CHECK(g_attend.n_items == reinterpret_cast<const ll::StepCounts*>(g_attend.counts)->items);
        if (below(4) == 0) refusals(w, m);
      }
    }
  }
  CHECK(begun > 50 && refused > 30 && stale > 5 && behind > 3);
  // capture: the whole capacity, and the tile stays from then on
  StepModel& m = steps[1];
  const int32_t none = 0;
  for (auto& [s, q] : b) CHECK(ll_seq_free(w.pool, s) == LL_OK);
  int32_t s0 = -1;
  CHECK(ll_seq_alloc(w.pool, 30, &s0, nullptr) == LL_OK);
  int32_t one = 1, many = 10;
  CHECK(ll_step_begin(m.h, &s0, &one, 1, 0, nullptr) == LL_OK);
  g_capturing = true;
  ll_attend_desc td = attend_desc(w, 1);
  CHECK(ll_step_attend(m.h, &td, nullptr) == LL_EINVAL);   // room for one token only
  td.tokens = kTokens;
  CHECK(ll_step_attend(m.h, &td, nullptr) == LL_OK);
  ll_append_desc ad = append_desc(w, kTokens);
  CHECK(ll_step_append(m.h, &ad, nullptr) == LL_OK && g_append.capacity == kTokens);
  g_capturing = false;
  const ll::AttendLaunch cap = g_attend;
  m.tile = cap.tile;
  CHECK(ll_step_begin(m.h, &s0, &many, 1, 0, nullptr) == LL_OK);
  m.seqs = {s0}, m.counts = {many}, m.tokens = many;
  check_plan(w, m, w.books());
  CHECK(g_setup.counts.items <= cap.n_items && g_setup.counts.shares <= cap.n_shares);
  // nothing to do, and a begin of nothing
  CHECK(ll_step_begin(m.h, &none, &none, 0, 1, nullptr) == LL_OK);
  ad = append_desc(w, 0);
  CHECK(ll_step_append(m.h, &ad, nullptr) == LL_OK);
  // a failing launch poisons the pool, and its steps refuse from then on
  if (seed & 1) {
    g_fail = true;
    CHECK(ll_step_begin(m.h, &s0, &one, 1, 0, nullptr) == LL_EDEVICE);
    g_fail = false;
    CHECK(ll_step_begin(m.h, &s0, &one, 1, 0, nullptr) == LL_EPOISONED);
    CHECK(ll_step_append(m.h, &ad, nullptr) == LL_EPOISONED);
  }
  // either order of the ends
  if (seed & 2) {
    for (StepModel& x : steps) ll_step_destroy(x.h);
    ll_pool_destroy(w.pool);
  } else {
    ll_step_destroy(steps[0].h);
    ll_pool_destroy(w.pool);
    CHECK(ll_step_begin(m.h, &s0, &one, 1, 0, nullptr) == LL_EINVAL);
    CHECK(ll_step_append(m.h, &ad, nullptr) == LL_EINVAL && ll_step_attend(m.h, &td, nullptr) == LL_EINVAL);
    ll_step_destroy(m.h);
  }
  std::printf("begun %d refused %d stale %d\n", begun, refused, stale);
  return 0;
}

}  // namespace

int main(int argc, char** argv) {
  if (argc != 4) return 2;
  return run(std::string(argv[1]) == "gqa", std::atoi(argv[2]), std::atoi(argv[3]));
}
