// The pool's host types, shared by its own source (pool.cpp) and the serving
// step's (step.cpp), and the parts of the pool's call sequence that the step
// uses.  Not part of the C ABI.
#pragma once

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>
#include <cstring>
#include <deque>
#include <vector>

#include "../../include/leyline.h"
#include "host_common.h"
#include "leyline_internal.h"

namespace ll {

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

inline size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

// A dispatch packet counts its work-items in 32 bits.
constexpr int64_t kMaxDispatchItems = int64_t{0xFFFFFFFF};

// Lowest-free-first page allocator over a bitmap (bit set = free).
class FreePages {
 public:
  void init(int64_t n) {
    n_ = n;
    words_.assign(static_cast<size_t>(ceil_div(n, 64)), ~0ull);
    if (n % 64) words_.back() = (1ull << (n % 64)) - 1;
    count_ = n;
    hint_ = 0;
  }
  int64_t count() const { return count_; }
  bool is_free(int64_t p) const { return (words_[p >> 6] >> (p & 63)) & 1ull; }
  void take(int64_t p) {
    words_[p >> 6] &= ~(1ull << (p & 63));
    --count_;
  }
  void give(int64_t p) {
    words_[p >> 6] |= 1ull << (p & 63);
    ++count_;
    hint_ = std::min<int64_t>(hint_, p >> 6);
  }
  // The k lowest free pages, in increasing order (not taken).
  void lowest(int64_t k, std::vector<int32_t>& out) const {
    out.clear();
    out.reserve(static_cast<size_t>(k));
    for (size_t w = static_cast<size_t>(hint_); w < words_.size() && static_cast<int64_t>(out.size()) < k; ++w) {
      uint64_t bits = words_[w];
      while (bits && static_cast<int64_t>(out.size()) < k) {
        const int b = __builtin_ctzll(bits);
        out.push_back(static_cast<int32_t>(w * 64 + b));
        bits &= bits - 1;
      }
    }
  }
  // Pages marked in `bits` return to the free set, in one pass; false if one
  // of them was free already or is not a page (the caller then treats the
  // set as broken).
  bool give_bits_checked(const uint64_t* bits) {
    const size_t n = words_.size();
    if (n && (bits[n - 1] & ~tail_mask())) return false;
    // branch-free: freed words come in any order of zero and non-zero
    uint64_t clash = 0;
    int64_t added = 0;
    for (size_t w = 0; w < n; ++w) {
      const uint64_t b = bits[w];
      clash |= b & words_[w];
      words_[w] |= b;
      added += __builtin_popcountll(b);
    }
    size_t first = 0;
    while (first < n && !bits[first]) ++first;
    count_ += added;
    hint_ = std::min<int64_t>(hint_, static_cast<int64_t>(first));
    return clash == 0;
  }
  // Pages marked in `bits` (all taken now) return to the free set.
  void give_bits(const uint64_t* bits) {
    for (size_t w = 0; w < words_.size(); ++w) {
      if (!bits[w]) continue;
      count_ += __builtin_popcountll(bits[w] & ~words_[w]);
      words_[w] |= bits[w];
      hint_ = std::min<int64_t>(hint_, static_cast<int64_t>(w));
    }
  }
  size_t num_words() const { return words_.size(); }
  // The bitmap words (bit set = free), for the device's page plan.
  void copy_words(uint64_t* out) const { std::memcpy(out, words_.data(), words_.size() * sizeof(uint64_t)); }
  void advance_hint() {
    while (hint_ < static_cast<int64_t>(words_.size()) && words_[hint_] == 0) ++hint_;
  }

 private:
  // bits of the last word that are pages
  uint64_t tail_mask() const { return n_ % 64 ? (1ull << (n_ % 64)) - 1 : ~0ull; }

  int64_t n_ = 0, count_ = 0, hint_ = 0;
  std::vector<uint64_t> words_;
};

struct SeqState {
  bool used = false;
  int64_t len = 0;
  int64_t next_pos = 0;
  std::vector<int32_t> pages;
  // pages is out of date: the device page-table row (written by an eviction
  // the device planned) holds the sequence's table; copied back on demand
  bool stale = false;
  // the pool's epoch when the sequence last changed (a step made before then
  // no longer fits it)
  uint64_t gen = 0;
};

// The region of the staging ring one call fills on the host and sends to the
// device with one copy (pinned host memory and device memory at the same
// offsets).
struct Staging {
  char* host = nullptr;
  char* dev = nullptr;
  size_t start = 0;
  size_t cap = 0;
  size_t used = 0;
};

// A region still in use by device work, and the event that marks its end.
struct RingRegion {
  size_t start, end;
  hipEvent_t done;
};

struct ProfRec {
  hipEvent_t start, stop;
  int64_t bytes;
};

// Current-device guard.
class DeviceGuard {
 public:
  explicit DeviceGuard(int dev) {
    if (hipGetDevice(&old_) != hipSuccess) old_ = -1;
    if (old_ != dev) ok_ = hipSetDevice(dev) == hipSuccess;
  }
  ~DeviceGuard() {
    int cur = -1;
    if (old_ >= 0 && hipGetDevice(&cur) == hipSuccess && cur != old_) (void)hipSetDevice(old_);
  }
  bool ok() const { return ok_; }

 private:
  int old_ = -1;
  bool ok_ = true;
};

}  // namespace ll

struct ll_pool {
  ll_pool_desc desc{};       // GQA pools: kv_lora_rank 0, rope_dim = rotary_dim
  int page_shift = 0;
  int64_t P = 1;
  bool gqa = false;          // K and V planes with per-head RoPE bands
  int32_t num_planes = 0;    // MLA: num_layers; GQA: 2 * num_layers (K then V)
  int64_t row_bytes = 0;     // one row of one plane
  int64_t band_bytes = 0;    // RoPE bytes of one row of a rotated plane
  int32_t heads = 0, head_chunks = 0, rot_shift = 0;  // GQA row shape
  std::vector<void*> layer_ptrs;  // the planes
  void** d_layers = nullptr;
  // chunks from one plane to the next when every plane's base is the first
  // one's plus a multiple of one fixed stride (one caller allocation), else 0
  int64_t plane_stride_chunks = 0;
  std::vector<ll::SeqState> seqs;
  ll::FreePages free;
  // staging ring: one pinned + one device buffer; calls take consecutive
  // regions and a region is reused once its call's event has fired
  char* ring_host = nullptr;
  char* ring_dev = nullptr;
  size_t ring_cap = 0;
  size_t ring_head = 0;
  std::deque<ll::RingRegion> ring_inflight;
  std::vector<hipEvent_t> ring_events;  // idle events for new regions
  ll::Staging cur;                          // region of the call in progress
  hipEvent_t upload_ev = nullptr;
  // eviction scratch: device [counts | reuse | src_of_dst], pinned readback
  float* d_rowtab = nullptr;    // per-row cos/sin tables of ll_rope_rows
  size_t rowtab_cap = 0;        // floats
  char* d_scratch = nullptr;
  size_t scratch_cap = 0;
  char* h_readback = nullptr;
  size_t readback_cap = 0;
  hipEvent_t readback_ev = nullptr;
  hipStream_t copy_stream = nullptr;
  hipEvent_t last_done = nullptr;  // end of the last call's device work
  hipStream_t last_stream = nullptr;  // the stream that work ran on
  // Calls that take no staging (splices planned on the device) record no
  // event: last_done then lags, and last_work() records lazy_ev on
  // last_stream when a later step needs the end of all work issued so far.
  bool unevented = false;
  hipEvent_t lazy_ev = nullptr;
  int32_t splice_planner = LL_SPLICE_PLAN_AUTO;
  bool page_reuse = true;       // false: every new page of a rewritten sequence is fresh
  int64_t dispatch_items = ll::kMaxDispatchItems;  // work-items one row-kernel dispatch may hold
  char* d_direct = nullptr;     // tasks, tables and rotation tables of device-planned splices
  size_t direct_cap = 0;
  bool poisoned = false;
  uint64_t epoch = 0;           // counts changes of any sequence
  // the `pool` field of every step made on this pool: cleared when it ends
  std::vector<ll_pool**> step_owners;
  std::vector<double> theta;    // RoPE frequencies of the pool's band (float64)
  ll_plan_stats last{};
  int32_t prof_every = 0;       // time every n-th launch of each kernel (0: none)
  int64_t prof_tick[3] = {0, 0, 0};
  std::vector<ll::ProfRec> prof[3];  // row-moving kernel, keep scan, per-row rotation
  std::vector<hipEvent_t> spare_events;
  std::vector<int32_t> page_slot;  // per physical page: scratch marks of ll_seq_set_pages
  std::vector<int32_t> table_rows;     // host copy of device page-table rows (stale tables)
  // An eviction at page size 1 (no page is ever fresh): the call returns at
  // once and the host learns its result -- new lengths and the bitmap of
  // freed pages -- from a small readback that the next call on the pool
  // applies (settles) first.
  struct PendingEvict {
    bool active = false;
    hipEvent_t done = nullptr;   // the readback has landed
    std::vector<int32_t> seq_ids;
    size_t off_info = 0, off_freed = 0;  // in h_readback (counts at 0)
    int64_t n_words = 0;         // words of the freed bitmap
    int64_t prof_index = -1;     // prof[0] entry whose bytes are known only then
  } pending;
};

namespace ll {

// pool.cpp's own steps of a call, for step.cpp (see their definitions there).
ll_status pool_check(const ll_pool* p);
ll_status pool_enter(ll_pool* p);
ll_status pool_host_exception(ll_pool* p) noexcept;
ll_status pool_device_fail(ll_pool* p, hipError_t e, const char* what);
ll_status pool_begin_call(ll_pool* p, hipStream_t st);
ll_status pool_end_call(ll_pool* p, Staging* s, hipStream_t st);
ll_status pool_stage(ll_pool* p, size_t bytes, Staging** out);
ll_status pool_upload(ll_pool* p, Staging* s, hipStream_t st);
ll_status pool_fresh_tables(ll_pool* p, const int32_t* seqs, size_t n);
ll_status pool_wait_idle(ll_pool* p);

}  // namespace ll
