// The serving step's host side at its limits, on the stand-ins and the small world
// of step_driver.cpp.  Usage: step_limits_driver <check> (see main).
#define main step_driver_main
#include "step_driver.cpp"
#undef main

#include "../../mla_paged_cache_amd/csrc/pool_internal.h"

namespace {

// Shares of a tile cover its rows in order, whole grains each, also at the longest
// sequence that a step takes and the most shares that a tile is split into.
void shares_of_long_tiles() {
  for (const int64_t rows : {int64_t{1}, int64_t{63}, int64_t{64}, int64_t{65}, int64_t{130816}, int64_t{INT32_MAX} - 1024})
    for (const int64_t shares : {1, 2, 3, 255, 1025, 2048})
      for (const int64_t grain : {32, 64}) {
        const int64_t per = ll::share_rows(rows, shares, grain);
        CHECK(per > 0 && per % grain == 0 && per * shares >= rows);
        CHECK(per == grain || (per - grain) * shares < rows);
      }
  // 2^31 - 1025 rows in 2048 shares: 1048575.5 rows each, in grains of 64
  CHECK(ll::share_rows(int64_t{INT32_MAX} - 1024, 2048, 64) == 1048576);
}

// Scores are kept in base 2: a scale whose product with log2 e is no number any more
// would make 0 times infinity of a score of 0.
void scales() {
  for (const bool gqa : {false, true}) {
    World w(gqa, 16);
    int32_t s0 = -1, one = 1;
    CHECK(ll_seq_alloc(w.pool, 30, &s0, nullptr) == LL_OK);
    const ll_step_desc d{w.heads, 1, kTokens};
    ll_step* s = nullptr;
    CHECK(ll_step_create(w.pool, &d, &s) == LL_OK && ll_step_begin(s, &s0, &one, 1, 0, nullptr) == LL_OK);
    for (const float sign : {1.f, -1.f}) {
      ll_attend_desc t = attend_desc(w, 1);
      t.scale = sign * 2.3e38f;
      CHECK(ll_step_attend(s, &t, nullptr) == LL_OK);
      t.scale = sign * 2.4e38f;   // * 1.4427 = 3.46e38, above 3.403e38
      CHECK(ll_step_attend(s, &t, nullptr) == LL_EINVAL);
    }
    ll_step_destroy(s);
    ll_pool_destroy(w.pool);
  }
}

// One token after another at page size 1: a begin's host work does not grow with
// the pages that the sequence holds, so its page list moves a few times only.
void growth() {
  constexpr int kPages = 6000;
  static char plane[32];
  void* p = reinterpret_cast<void*>((reinterpret_cast<uintptr_t>(plane) + 15) & ~uintptr_t{15});   // never touched
  std::vector<int32_t> table(kPages, -1);
  ll_gqa_pool_desc d{};
  d.num_layers = 1, d.page_size = 1, d.num_pages = kPages, d.max_seqs = 1, d.max_pages_per_seq = kPages;
  d.num_kv_heads = 1, d.head_dim = 16, d.rotary_dim = 16, d.rope_pairing = LL_ROPE_HALF, d.rope_base = 10000.0;
  d.k_layer_base = &p, d.v_layer_base = &p, d.page_table = table.data();
  ll_pool* pool = nullptr;
  CHECK(ll_pool_create_gqa(&d, &pool) == LL_OK);
  int32_t seq = -1, one = 1;
  CHECK(ll_seq_alloc(pool, 1000, &seq, nullptr) == LL_OK);
  const ll_step_desc sd{1, 1, 4};
  ll_step* s = nullptr;
  CHECK(ll_step_create(pool, &sd, &s) == LL_OK);
  int moves = 0;
  const int32_t* at = pool->seqs[seq].pages.data();
  for (int i = 0; i < 5000; ++i) {
    CHECK(ll_step_begin(s, &seq, &one, 1, 1, nullptr) == LL_OK);
    if (pool->seqs[seq].pages.data() != at) ++moves;
    at = pool->seqs[seq].pages.data();
  }
  CHECK(pool->seqs[seq].pages.size() == 6000 && moves <= 3);   // 1000 -> 2000 -> 4000 -> 8000
  ll_step_destroy(s);
  ll_pool_destroy(pool);
}

// A device-planned eviction leaves the host's page list of its sequences out of
// date.  A begin that gives a sequence no page has no use for it and waits for no
// copy; one that does brings it up to date, behind rows grown in between too.
void tables_behind_an_eviction() {
  for (const bool gqa : {false, true})
    for (const int P : {1, 4, 16}) {
      World w(gqa, P);
      int32_t id = -1;
      const int64_t n = std::min(16 * P + 5, 30 * P);
      CHECK(ll_seq_alloc(w.pool, n, &id, nullptr) == LL_OK);
      std::vector<uint8_t> keep(static_cast<size_t>(n), 1);
      keep[1] = 0;
      for (int64_t i = n - P / 2 - 1; i < n; ++i) keep[static_cast<size_t>(i)] = 0;   // leaves room in the last page
      const int64_t kept = std::count(keep.begin(), keep.end(), 1), off = 0;
      CHECK(kv_evict_compact(w.pool, &id, 1, keep.data(), &off, nullptr) == LL_OK);
      const ll_step_desc d{w.heads, 1, kTokens};
      ll_step* s = nullptr;
      CHECK(ll_step_create(w.pool, &d, &s) == LL_OK);
      int32_t three = 3, one = 1, none = 0, many = 2 * P;
      CHECK(ll_step_begin(s, &id, &three, 1, 0, nullptr) == LL_OK);
      const ll::SeqState& q = w.pool->seqs[id];
      CHECK(q.stale && q.len == kept);
      CHECK(ll_step_begin(s, &id, &none, 1, 1, nullptr) == LL_OK && q.stale);
      int64_t grown = 0;
      if ((kept + P - 1) / P == (kept + P) / P) {   // one row more is in a page that is there
        CHECK(ll_step_begin(s, &id, &one, 1, 1, nullptr) == LL_OK && q.stale && q.len == kept + 1);
        grown = 1;
      }
      CHECK(ll_step_begin(s, &id, &many, 1, 1, nullptr) == LL_OK && !q.stale);
      StepModel m;
      m.h = s, m.begun = true, m.seqs = {id}, m.counts = {many}, m.tokens = many;
      m.tile = ll::attend_tile(gqa, w.dim, int64_t{many} * (w.heads / w.kv_heads));
      const std::map<int, Seq> b = w.books();
      CHECK(b.at(id).len == kept + grown + many && b.at(id).pos == n + grown + many);
      check_plan(w, m, b);   // the list against the device's row, rows and items
      int64_t n_free = 0;
      CHECK(ll_pool_free_pages(w.pool, &n_free) == LL_OK && n_free == static_cast<int64_t>(w.free_pages(b).size()));
      ll_step_destroy(s);
      ll_pool_destroy(w.pool);
    }
}

// A graph keeps the tile that it was captured with; eager calls on the same step are
// planned for what they bring, before and after, and a later graph joins the first.
void eager_calls_beside_a_graph() {
  for (const bool gqa : {false, true}) {
    World w(gqa, 16);
    int32_t id = -1, one = 1, many = 70;
    CHECK(ll_seq_alloc(w.pool, 300, &id, nullptr) == LL_OK);
    const ll_step_desc d{w.heads, 1, kTokens};
    ll_step* s = nullptr;
    CHECK(ll_step_create(w.pool, &d, &s) == LL_OK);
    const int group = w.heads / w.kv_heads;
    const int small = ll::attend_tile(gqa, w.dim, group), big = ll::attend_tile(gqa, w.dim, int64_t{many} * group);
    CHECK(small != big);
    StepModel m;
    m.h = s, m.begun = true, m.seqs = {id};
    auto begin = [&](int32_t count) {
      CHECK(ll_step_begin(s, &id, &count, 1, 0, nullptr) == LL_OK);
      m.counts = {count}, m.tokens = count;
    };
    auto eager = [&](int tile) {
      const ll_attend_desc t = attend_desc(w, m.tokens);
      CHECK(ll_step_attend(s, &t, nullptr) == LL_OK && g_attend.tile == tile);
      return g_attend;
    };
    auto capture = [&](int tile) {
      g_capturing = true;
      const ll_attend_desc t = attend_desc(w, kTokens);
      CHECK(ll_step_attend(s, &t, nullptr) == LL_OK && g_attend.tile == tile);
      g_capturing = false;
      return g_attend;
    };
    begin(many);
    eager(big);
    begin(one);
    const ll::AttendLaunch first = eager(small), graph = capture(small);
    CHECK(graph.items == first.items && graph.counts == first.counts && graph.n_items > first.n_items);
    for (int turn = 0; turn < 2; ++turn) {
      begin(one);   // as the graph: one plan for both
      CHECK(g_setup.own_counts.items == 0);
      const ll::AttendLaunch same = eager(small);
      CHECK(same.items == graph.items && same.counts == graph.counts);
      m.tile = small;
      check_plan(w, m, w.books());
      begin(many);   // more than the graph's: a plan each
      m.tile = small;
      check_plan(w, m, w.books());
      CHECK(g_setup.counts.items <= graph.n_items && g_setup.counts.shares <= graph.n_shares);
      const ll::StepSetupLaunch both = g_setup;
      const ll::AttendLaunch own = eager(big), again = capture(small);
      CHECK(again.items == graph.items && again.counts == graph.counts && again.n_items == graph.n_items);
      CHECK(own.items == both.dst_own_items && own.counts == both.dst_own_counts && own.items != graph.items);
      CHECK(own.n_items == both.own_counts.items && own.n_shares == both.own_counts.shares);
      CHECK(both.own_counts.tokens == many && both.own_counts.seqs == 1);
      // the same checks of the eager plan
      std::vector<ll::AttendItem> items(both.src_own, both.src_own + both.own_counts.items);
      g_setup.counts = both.own_counts;
      g_setup.dst_items = items.data();
      m.tile = big;
      check_plan(w, m, w.books());
    }
    ll_step_destroy(s);
    ll_pool_destroy(w.pool);
  }
}

// q_out = q turns the queries in place, so both are laid out alike (a stride that no
// second token or head uses says nothing).
void queries_in_place() {
  for (const bool gqa : {false, true}) {
    World w(gqa, 16);
    int32_t id = -1, two = 2, one = 1;
    CHECK(ll_seq_alloc(w.pool, 30, &id, nullptr) == LL_OK);
    const ll_step_desc d{w.heads, 1, kTokens};
    ll_step* s = nullptr;
    CHECK(ll_step_create(w.pool, &d, &s) == LL_OK && ll_step_begin(s, &id, &two, 1, 0, nullptr) == LL_OK);
    ll_append_desc a = append_desc(w, 2);
    a.q_out = const_cast<void*>(a.q);
    CHECK(ll_step_append(s, &a, nullptr) == LL_OK);
    a.q_out_token_stride += 64;
    CHECK(ll_step_append(s, &a, nullptr) == LL_EINVAL);
    a.q_out_token_stride -= 64;
    a.q_head_stride = 0;   // one query for every head
    CHECK(ll_step_append(s, &a, nullptr) == LL_EINVAL);
    a.q_head_stride = a.q_out_head_stride;
    CHECK(ll_step_begin(s, &id, &one, 1, 0, nullptr) == LL_OK);
    a.q_out_token_stride += 64;   // of one token
    CHECK(ll_step_append(s, &a, nullptr) == LL_OK);
    ll_step_destroy(s);
    ll_pool_destroy(w.pool);
  }
}

}  // namespace

int main(int argc, char** argv) {
  const std::map<std::string, void (*)()> checks = {
      {"eager_calls_beside_a_graph", eager_calls_beside_a_graph},
      {"growth", growth},
      {"tables_behind_an_eviction", tables_behind_an_eviction},
      {"queries_in_place", queries_in_place},
      {"scales", scales},
      {"shares_of_long_tiles", shares_of_long_tiles},
  };
  const auto c = argc == 2 ? checks.find(argv[1]) : checks.end();
  if (c == checks.end()) return 2;
  c->second();
  return 0;
}
