// Internal types shared by the host side of eviction by attention weight
// (weight.cpp) and its gfx950 kernels (kernels_weigh.hip, kernels_keep.hip).  Not
// part of the C ABI.
#pragma once

#include "step_internal.h"

namespace ll {

// One layer's weighing.
struct WeighLaunch {
  const StepCounts* counts;
  const StepSeq* seqs;
  int32_t n_seqs;                // sequences the grid covers
  int64_t max_rows;              // cached rows of a sequence that the grid covers
  int64_t most;                  // query rows that a sequence brings at most (the choice of a tile)
  int32_t kv_heads;
  int32_t group;                 // query heads per KV head
  int32_t heads;
  int32_t causal;
  int32_t window;                // 0: none
  float scale;                   // natural scores
  float cap;                     // 0: none
  float decay;
  int32_t dim;                   // GQA head_dim
  const uint16_t* k_plane;       // MLA: the layer's rows
  const int32_t* page_table;
  int32_t max_pages_per_seq;
  int32_t num_pages;
  int32_t page_shift;
  const uint16_t* q;
  int64_t q_ts, q_hs;
  const uint16_t* q_pe;
  int64_t qp_ts, qp_hs;
  const float* lse;              // [tokens][heads]
  float* weights;                // [page-table rows][stride]
  int64_t weight_stride;
  int32_t shares;                // workgroups that a tile of rows is cut over, set by the launch
  float* parts;                  // [shares][n_seqs][max_rows]: their sums, which a second kernel adds up
  int64_t part_values;           // room there
};

// One sequence's selection.
struct KeepSeq {
  int64_t rows;                  // below 2^31
  int64_t budget;                // rows to keep, at most `rows`
  int64_t keep_off;              // into the masks
  int64_t seq;                   // row of the weights
};

// A launch takes its sequences as kernel arguments.
constexpr int kKeepSeqs = 96;
struct KeepLaunch {
  KeepSeq seqs[kKeepSeqs];
  int64_t sinks, recent;
  const float* weights;
  float* kept_weights;           // or nullptr
  int64_t weight_stride;
  uint8_t* keep;
};
static_assert(sizeof(KeepLaunch) <= 4096, "kernel arguments");

hipError_t launch_weigh(const WeighLaunch& a, bool gqa, hipStream_t s);
hipError_t launch_keep(const KeepLaunch& a, int n, hipStream_t s);

}  // namespace ll
