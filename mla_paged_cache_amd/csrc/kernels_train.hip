// gfx950 kernels of the trainer's attention (kvs_attend): query q sees key k iff
// k <= q < death[k];
//   s_k = scale * q . k  (or cap * tanh(scale * q . k / cap)),
//   out = sum_k softmax(s)_k v_k,  lse = log sum_k exp s_k,
// in one pass over the keys that keeps the running maximum, sum and weighted values in
// float32.  Scores are kept in base 2.
#include "train_common.h"

namespace ll {
namespace {

// One query row by one wave, one key at a time: a lane holds 8 values of a head.
// Reads exactly the keys that the query sees.
__device__ void train_row(const TrainLaunch& a, int r, int q, int h, int lane) {
  const int kvh = h / a.group;
  const bool lk = lane * 8 < a.dk, lv = lane * 8 < a.dv;
  const int32_t* const death = a.death + static_cast<int64_t>(r) * a.n_pad;
  const Vals x = load8(at(a.q, r, q, h) + lane * 8, lk);
  float m = -__builtin_inff(), l = 0.f;
  Vals o{};
  for (int k = 0; k <= q; ++k) {
    if (death[k] <= q) continue;
    const float s = score_of(a, wave_sum(dot8(x, load8(at(a.k, r, k, kvh) + lane * 8, lk)))).x;
    const float m2 = fmaxf(m, s);
    const float keep = m == m2 ? 1.f : exp2_(m - m2);
    const float p = s == -__builtin_inff() ? 0.f : exp2_(s - m2);
    l = l * keep + p;
    const Vals v = load8(at(a.v, r, k, kvh) + lane * 8, lv);
#pragma unroll
    for (int i = 0; i < 8; ++i) o.v[i] = __builtin_fmaf(p, v.v[i], o.v[i] * keep);
    m = m2;
  }
  if (l == 0.f) o = Vals{};   // no weight at all: 0, whatever the sum holds (0 times an infinity)
  if (lv) store8(place(a.out, r, q, h) + lane * 8, o, l == 0.f ? 0.f : 1.f / l);
  if (lane == 0)
    a.lse[(static_cast<int64_t>(r) * a.n_pad + q) * a.heads + h] = l == 0.f ? -__builtin_inff() : (m + __log2f(l)) * kLn2;
}

__global__ __launch_bounds__(256) void train_rows_kernel(TrainLaunch a) {
  int64_t unit = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 6);
  const int q = static_cast<int>(unit % a.n_pad);
  unit /= a.n_pad;
  const int r = static_cast<int>(unit / a.heads), h = static_cast<int>(unit % a.heads);
  if (r < a.n) train_row(a, r, q, h, threadIdx.x & 63);
}

}  // namespace

hipError_t launch_train(const TrainLaunch& a, hipStream_t s) {
  const int64_t waves = int64_t{a.n} * a.heads * a.n_pad;
  train_rows_kernel<<<dim3(static_cast<unsigned>((waves + 3) / 4)), dim3(256), 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace ll
