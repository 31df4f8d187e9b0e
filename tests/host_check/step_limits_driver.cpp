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

}  // namespace

int main(int argc, char** argv) {
  const std::map<std::string, void (*)()> checks = {
      {"growth", growth},
      {"scales", scales},
      {"shares_of_long_tiles", shares_of_long_tiles},
  };
  const auto c = argc == 2 ? checks.find(argv[1]) : checks.end();
  if (c == checks.end()) return 2;
  c->second();
  return 0;
}
