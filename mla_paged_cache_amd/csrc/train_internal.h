// Internal types shared by the trainer's attention's host side (train.cpp) and its
// gfx950 kernels (kernels_train.hip, kernels_train_back.hip).  Not part of the C ABI.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

namespace ll {

// A bf16 tensor [rollouts][tokens][heads][width]; strides in values.
struct Heads {
  uint16_t* p;
  int64_t rs, ts, hs;
};

// Keys and queries are taken in blocks of this many tokens.
constexpr int kTrainBlock = 64;
// Queries of one workgroup of the forward pass and of dq, keys of one of dk and dv.
constexpr int kTrainTile = 128;
// A rollout is cut into at most so many epochs of equal length, a multiple of
// kTrainTile.  The keys that are still seen when an epoch begins are listed, so that its
// queries go along those (and the epoch's own keys) instead of everything before them.
constexpr int kTrainEpochs = 64;

// Of a block of keys: the first and the last of its death times, each at most n_pad,
// a key that nobody sees counted as -1.  Queries [q0, q1] see all of keys [k0, k1] if
// k1 <= q0 and q1 < first, and none if q1 < k0 or last <= q0.
struct KeyBlock {
  int32_t first;
  int32_t last;
};

// The widths of the kernels' tiles that hold heads of dk and dv values.
struct HeadShape {
  int32_t dk, dv;
};
inline HeadShape head_shape(int32_t dk, int32_t dv) {
  if (dk <= 64 && dv <= 64) return HeadShape{64, 64};
  if (dk <= 128 && dv <= 128) return HeadShape{128, 128};
  if (dk <= 192 && dv <= 128) return HeadShape{192, 128};
  return HeadShape{256, 256};
}

// A key of an epoch's list, and its death time (at most n_pad); places behind the last
// key up to a multiple of kTrainBlock hold key 0 and -1.
struct KeyEntry {
  int32_t key;
  int32_t death;
};

struct TrainLaunch {
  int32_t n, heads, kv_heads, group;
  int32_t n_pad;
  int32_t blocks;                // ceil(n_pad / kTrainBlock)
  int32_t dk, dv;
  float scale, cap;
  const int32_t* death;
  Heads q, k, v, out, dout, dq, dk_, dv_;
  float* lse;                    // [n][n_pad][heads]
  int32_t epoch, epochs;         // length of an epoch, and how many there are
  int32_t shares;                // backward: workgroups that a tile of keys may be cut over
  // workspace
  KeyBlock* keys;                // [n][blocks]
  KeyEntry* list;                // [n][list_keys]: epoch e's at list_at(e), which holds up to e * epoch keys
  KeyBlock* list_blocks;         // of the lists' blocks, in the same way
  int32_t* list_count;           // [n][epochs] keys
  int32_t* order;                // [n][n_pad]: backward, the keys by the epoch that they die in, the last first, and
                                 // then by place; those that nobody sees behind them
  int32_t* seen_keys;            // [n]: how many are seen
  int64_t* work;                 // [n]: pairs of a query and a key that it sees
  uint32_t* odd_k;               // [n][kv_heads][blocks]: whether a key that is seen holds a value that is not finite;
  uint32_t* odd_v;               // the same of v
  uint32_t* odd_q;               // [n][heads][blocks]: of q and dout, any query
  uint32_t* odd_do;
  float* delta;                  // [n][heads][n_pad]: sum of dout * out; corrected by the kernel of dq
  float* ref;                    // [n][heads][n_pad]: lse in base 2; infinity where there is no weight

  int32_t* used;                 // [n * kv_heads * tiles]: shares that a tile of keys was cut into
  float* parts;                  // [n * kv_heads * tiles][shares]: their sums

  __host__ __device__ int64_t list_at(int64_t e) const { return e * (e - 1) / 2 * epoch; }
  __host__ __device__ int64_t list_keys() const { return list_at(epochs); }
};

hipError_t launch_train_scan(const TrainLaunch& a, bool backward, hipStream_t s);
hipError_t launch_train(const TrainLaunch& a, hipStream_t s);
hipError_t launch_train_back(const TrainLaunch& a, hipStream_t s);

}  // namespace ll
