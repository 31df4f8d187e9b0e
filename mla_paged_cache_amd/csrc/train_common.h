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

}  // namespace
}  // namespace ll
