// Device helpers shared by the trainer's attention, forward (kernels_train.hip) and
// backward (kernels_train_back.hip).
#pragma once

#include "matrix_common.h"
#include "step_internal.h"
#include "train_internal.h"

namespace ll {
namespace {

__device__ __forceinline__ const uint16_t* at(const Heads& x, int r, int t, int h) {
  return x.p + r * x.rs + t * x.ts + h * x.hs;
}
__device__ __forceinline__ uint16_t* place(const Heads& x, int r, int t, int h) {
  return x.p + r * x.rs + t * x.ts + h * x.hs;
}

__device__ __forceinline__ float wave_sum(float x) {
  for (int d = 32; d >= 1; d >>= 1) x += __shfl_xor(x, d);
  return x;
}

// A score in base 2 from its product, and the slope of the cap there.
struct Score {
  float x, slope;
};
__device__ __forceinline__ Score score_of(const TrainLaunch& a, float product) {
  if (a.cap == 0.f) return Score{product * (a.scale * kLog2e), 1.f};
  const float t = tanh_any(product * (a.scale / a.cap));
  return Score{a.cap * kLog2e * t, 1.f - t * t};
}

__device__ __forceinline__ void store8(uint16_t* p, const Vals& x, float by) {
  typedef float f32x8 __attribute__((ext_vector_type(8)));
  f32x8 y;
#pragma unroll
  for (int i = 0; i < 8; ++i) y[i] = x.v[i] * by;
  *reinterpret_cast<bf16x8*>(p) = __builtin_convertvector(y, bf16x8);
}
__device__ __forceinline__ void add8(Vals& o, float w, const Vals& x) {
#pragma unroll
  for (int i = 0; i < 8; ++i) o.v[i] = __builtin_fmaf(w, x.v[i], o.v[i]);
}

// Whether the query of this lane sees the keys of a product's values, as bits: key i has
// number first + product_row(i) and its death time in LDS (16-byte words of four).  Only
// for blocks that are seen in part: a branch around it, not a selection.
__device__ __forceinline__ uint32_t seen_bits(const char* deaths, int part, int first, int query, int lane) {
  typedef int i32x4 __attribute__((ext_vector_type(4)));
  uint32_t bits = 0;
#pragma unroll
  for (int i = 0; i < 16; i += 4) {
    const int k = part + product_row(i, lane);
    const i32x4 d = *reinterpret_cast<const i32x4*>(deaths + k * 4);
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (first + k + e <= query && query < d[e]) bits |= 1u << (i + e);
  }
  asm volatile("" : "+v"(bits));
  return bits;
}

// A row (of q, k, v or dout) as a lane's operand: KK steps of 16 values, this lane's 8
// of each; a row that is not there and chunks past `live` count as 0.
template <int KK>
__device__ __forceinline__ void load_operand(bf16x8 (&x)[KK], const uint16_t* row, bool there, int live, int lane) {
#pragma unroll
  for (int k = 0; k < KK; ++k) {
    const int c = 2 * k + (lane >> 5);
    chunk_t v{0u, 0u, 0u, 0u};
    if (there && c < live) v = *reinterpret_cast<const chunk_t*>(row + c * 8);
    x[k] = __builtin_bit_cast(bf16x8, v);
  }
}

// A negative scale turns the queries' signs; one too small to tell scores apart counts
// as 0, and so do the queries then.  Returns what a product is multiplied by: to base 2,
// or under a cap to the tanh's argument.
template <bool CAP, int KK>
__device__ __forceinline__ float fold_scale(bf16x8 (&q)[KK], float scale, float cap) {
  const float c = CAP ? scale / cap : scale * kLog2e;
  const bool nothing = !(fabsf(c) >= 1e-37f);
  if (c < 0.f || nothing) {
    const uint32_t keep = nothing ? 0u : ~0u, flip = nothing ? 0u : 0x80008000u;
#pragma unroll
    for (int k = 0; k < KK; ++k) {
      chunk_t v = __builtin_bit_cast(chunk_t, q[k]);
      v = (v & keep) ^ flip;
      q[k] = __builtin_bit_cast(bf16x8, v);
    }
  }
  return nothing ? 1.f : fabsf(c);
}

// The blocks of keys that queries [q0, q1] of one epoch see: first those of the epoch's
// list, then the epoch's own.  64 blocks are looked at together, lane x at block base + x;
// every wave of a workgroup goes through the same ones.
struct KeyWalk {
  const KeyBlock* keys;          // the epoch's own blocks
  const uint32_t* odd;           // which of them hold a value that is not finite
  const KeyBlock* list_blocks;
  const KeyEntry* list;
  const int32_t* death;          // from the epoch's first key on
  int q0, q1, k0;                // k0: the epoch's first key
  int n_pad;
  int listed, blocks;            // blocks of the list, and of the walk
  bool odd_list;                 // some key before k0 holds such a value
  int base;
  uint64_t seen, whole;
  bool rows_only;                // a block that is seen in part holds such a value

  __device__ __forceinline__ KeyWalk(const TrainLaunch& a, int r, int kvh, const uint32_t* odd_blocks, int q0_, int q1_, int lane)
      : q0(q0_), q1(q1_), n_pad(a.n_pad), odd_list(false), base(-64), seen(0), whole(0), rows_only(false) {
    const int e = q0 / a.epoch;
    k0 = e * a.epoch;
    const int64_t own = static_cast<int64_t>(r) * a.blocks, first = k0 / kTrainBlock;
    keys = a.keys + own + first;
    odd = odd_blocks + (static_cast<int64_t>(r) * a.kv_heads + kvh) * a.blocks;
    for (int b = lane; b < first; b += 64) odd_list |= odd[b] != 0;
    odd_list = __any(odd_list);
    odd += first;
    death = a.death + static_cast<int64_t>(r) * a.n_pad + k0;
    const int64_t at = static_cast<int64_t>(r) * a.list_keys() + a.list_at(e);
    list = a.list + at;
    list_blocks = a.list_blocks + at / kTrainBlock;
    listed = e == 0 ? 0 : (a.list_count[static_cast<int64_t>(r) * a.epochs + e] + kTrainBlock - 1) / kTrainBlock;
    blocks = listed + (q1 - k0) / kTrainBlock + 1;
  }
  __device__ __forceinline__ void look(int lane) {
    const int b = base + lane, own = b - listed;
    KeyBlock x{0, -1};
    if (b < listed) x = list_blocks[b];
    else if (b < blocks) x = keys[own];
    const bool some = x.last > q0;
    const bool all = some && x.first > q1 && (own < 0 || k0 + own * kTrainBlock + kTrainBlock - 1 <= q0);
    bool bad = false;
    if (some && !all) bad = own < 0 ? odd_list : odd[own] != 0;
    seen = __ballot(some);
    whole = __ballot(all);
    rows_only |= __any(bad);
  }
  // The next block, or -1; `all`: every query sees every key of it.
  __device__ __forceinline__ int next(bool* all, int lane) {
    while (seen == 0) {
      base += 64;
      if (base >= blocks) return -1;
      look(lane);
    }
    const int x = __builtin_ctzll(seen);
    seen &= seen - 1;
    *all = whole >> x & 1;
    return base + x;
  }
  // Key `lane` of block b and its death time (not above its number: nobody sees it).
  __device__ __forceinline__ KeyEntry key(int b, int lane) const {
    if (b < listed) return list[b * kTrainBlock + lane];
    const int i = (b - listed) * kTrainBlock + lane;
    return KeyEntry{k0 + i, k0 + i < n_pad ? death[i] : -1};
  }
  // The row to read for it.  A key that nobody sees may hold anything: its place reads
  // another key's row.
  static __device__ __forceinline__ int row_of(KeyEntry x, int lane) {
    const uint64_t some = __ballot(x.death > x.key);
    const int other = __shfl(x.key, some ? __builtin_ctzll(some) : 0);
    return some >> lane & 1 ? x.key : other;
  }
  // What the place of a block's key adds to its number for the comparison with a query:
  // listed keys come before every query of the epoch.
  __device__ __forceinline__ int first_key(int b) const { return b < listed ? -kTrainBlock : k0 + (b - listed) * kTrainBlock; }
};

}  // namespace
}  // namespace ll
