// Internal types shared by the serving step's host side (step.cpp) and its
// gfx950 kernels (kernels_step.hip, kernels_attend.hip).  Not part of the C ABI.
#pragma once

#include "leyline_internal.h"

namespace ll {

// One sequence of a step's plan.
struct alignas(16) StepSeq {
  int32_t seq;          // page-table row
  int32_t tok0;         // its first token in the step
  int32_t count;        // its tokens
  int32_t row0;         // its first token's row in the sequence
  int64_t pos0;         // its first token's position
  int32_t old_pages;    // logical pages below this are in the page table already
  int32_t fresh_off;    // the others' physical pages: fresh[fresh_off ...]
  int32_t new_pages;    // how many
  int32_t pad[3];
};
static_assert(sizeof(StepSeq) == 48, "three 16-byte words");

// One workgroup's part of the attention (per KV head): `rows` query rows of one
// sequence against one share of the cached rows they see.  A query row is a
// token and a head of the KV head's group, row r: token r / group, head r % group.
struct alignas(16) AttendItem {
  int32_t seq;          // page-table row
  int32_t tok0;         // the sequence's first token in the step
  int32_t q_rows;       // query rows of the sequence (tokens * group)
  int32_t row0;         // first query row of the tile
  int32_t first;        // the first token's own cache row
  int32_t kv_len;       // cached rows
  int32_t splits;       // share | shares << 16
  int32_t slot;         // the share's place among the partial results, when shares > 1
};
static_assert(sizeof(AttendItem) == 32, "two 16-byte words");

// Rows of each of a tile's shares: equal, in multiples of `grain`.  (Rows may come
// within 1025 of 2^31, and shares are at most 2048: every sum here stays below 2^32,
// and a division of 64 bits would cost each workgroup about 150 instructions.)
constexpr uint32_t share_rows(uint32_t rows, uint32_t shares, uint32_t grain) {
  return ((rows + shares - 1) / shares + grain - 1) / grain * grain;
}

struct StepCounts {
  int32_t tokens;
  int32_t items;
  int32_t seqs;
  int32_t shares;       // the leading items that are shares of split tiles
};

// The plan as begin uploads it (src_*) and where the kernel puts it.
struct StepSetupLaunch {
  StepCounts counts;
  const StepSeq* src_seqs;
  const AttendItem* src_items;
  const int32_t* fresh;          // fresh pages of every sequence
  const double* theta;           // [pairs]
  int32_t pairs;
  int32_t page_shift;
  int32_t max_pages_per_seq;
  int32_t num_pages;
  int32_t* page_table;
  StepCounts* dst_counts;
  AttendItem* dst_items;
  StepCounts own_counts;         // the eager calls' own plan of the attention, where a graph holds
  const AttendItem* src_own;     // another tile (own_counts.items: 0 otherwise)
  StepCounts* dst_own_counts;
  AttendItem* dst_own_items;
  int32_t* rows;                 // [tokens] physical row, -1: none
  float* tab;                    // [tokens][2][pairs] float32 cos, then sin
};

// One layer's rows and queries.
struct AppendLaunch {
  const StepCounts* counts;
  const int32_t* rows;
  const float* tab;
  int32_t pairs;
  int32_t capacity;              // tokens the grid covers
  int32_t waves_per_token;       // set by the launch
  int32_t pieces;                // a token's pieces of 64 chunks: kv_pieces + those of the queries
  int32_t kv_pieces;             // of them for cache rows (GQA: K's, then V's; MLA: 1; 0: queries only)
  int32_t heads, kv_heads;
  int32_t head_chunks;           // GQA: head_dim / 8
  int32_t group_shift;           // log2 of the lanes a head takes
  int32_t band_chunks;           // rotary_dim / 8
  int32_t norm_f32;
  float eps;
  const uint16_t* a;
  int64_t a_ts, a_hs;
  const uint16_t* b;
  int64_t b_ts, b_hs;
  const void* norm;
  const uint16_t* q;
  int64_t q_ts, q_hs;
  uint16_t* q_out;
  int64_t qo_ts, qo_hs;
  const void* q_norm;
  uint16_t* k_plane;             // MLA: the layer's rows
  uint16_t* v_plane;
};

struct AttendLaunch {
  const StepCounts* counts;
  const AttendItem* items;
  int32_t n_items;               // items the grid covers
  int32_t n_shares;              // shares that the joining grid covers (0: nothing to join)
  int32_t join_blocks;           // workgroups that join one tile
  int32_t kv_heads;
  int32_t group;                 // query heads per KV head
  int32_t tile;                  // query rows of an item
  int32_t causal;
  int32_t window;                // 0: none
  float scale;                   // natural scores
  int32_t dim;                   // GQA head_dim
  const uint16_t* k_plane;       // MLA: the layer's rows
  const uint16_t* v_plane;
  const int32_t* page_table;
  int32_t max_pages_per_seq;
  int32_t num_pages;
  int32_t page_shift;
  const uint16_t* q;
  int64_t q_ts, q_hs;
  const uint16_t* q_pe;
  int64_t qp_ts, qp_hs;
  uint16_t* out;
  int64_t o_ts, o_hs;
  float* lse;                    // or nullptr
  int32_t heads;
  float* part_o;                 // [slot][kv head][tile][value width]
  float* part_ml;                // [slot][kv head][tile][2]: maximum (of scaled scores, base 2) and sum
};

constexpr int kMaxHeadDim = 256;
constexpr float kLog2e = 1.4426950408889634f;

hipError_t launch_step_setup(const StepSetupLaunch& a, hipStream_t s);
hipError_t launch_append(const AppendLaunch& a, bool gqa, int pairing, hipStream_t s);
// Query rows per item for a step whose sequences bring at most `rows` each.
int attend_tile(bool gqa, int dim, int64_t rows);
// Workgroups of that tile that the chip runs at once.
int attend_groups(bool gqa, int dim, int tile);
hipError_t launch_attend(const AttendLaunch& a, bool gqa, hipStream_t s);

}  // namespace ll
