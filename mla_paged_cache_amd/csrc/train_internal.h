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

// Keys and queries are taken in blocks of this many tokens for what the workspace
// says of them.
constexpr int kTrainBlock = 64;

// Of a block of keys: the first and the last of its death times, each at most n_pad,
// a key that nobody sees counted as -1.  Queries [q0, q1] see all of keys [k0, k1] if
// k1 <= q0 and q1 < first, and none if q1 < k0 or last <= q0.
struct KeyBlock {
  int32_t first;
  int32_t last;
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
  // workspace
  KeyBlock* keys;                // [n][blocks]
  uint32_t* odd_k;               // [n][kv_heads][blocks]: not 0 where a value of k is not finite; the same of v, q, dout
  uint32_t* odd_v;
  uint32_t* odd_q;               // [n][heads][blocks]
  uint32_t* odd_do;
  float* delta;                  // [n][heads][n_pad]: sum of dout * out
};

hipError_t launch_train_scan(const TrainLaunch& a, bool backward, hipStream_t s);
hipError_t launch_train(const TrainLaunch& a, hipStream_t s);
hipError_t launch_train_back(const TrainLaunch& a, hipStream_t s);

}  // namespace ll
