// gfx950 kernels of the gradients of the trainer's attention (kvs_attend_backward):
// with p = exp(s - lse) over the keys that a query sees,
//   delta = sum_d dout out,  ds = p (dout . v - delta) scale (1 - tanh^2),
//   dv = sum_q p dout,  dk = sum_q ds q,  dq = sum_k ds k,
// dk and dv summed over the heads that share a KV head.  Weights are worked out again
// from lse; one kernel goes along the keys of a query for dq, another along the queries
// of a key for dk and dv, so that each sum has one owner and one order.
#include "train_common.h"

namespace ll {
namespace {

// delta of every query and head, a wave each.
__global__ __launch_bounds__(256) void train_delta_kernel(TrainLaunch a) {
  const int lane = threadIdx.x & 63;
  int64_t unit = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 6);
  const int h = static_cast<int>(unit % a.heads);
  unit /= a.heads;
  const int r = static_cast<int>(unit / a.n_pad), q = static_cast<int>(unit % a.n_pad);
  if (r >= a.n) return;
  const bool lv = lane * 8 < a.dv;
  const float d = wave_sum(dot8(load8(at(a.dout, r, q, h) + lane * 8, lv), load8(at(a.out, r, q, h) + lane * 8, lv)));
  if (lane == 0) a.delta[(static_cast<int64_t>(r) * a.heads + h) * a.n_pad + q] = d;
}

// One pair that is seen: the weight p and the gradient ds of its product.
struct Pair {
  float p, ds;
};
__device__ __forceinline__ Pair pair_of(const TrainLaunch& a, float product, float dp, float lse, float delta) {
  const Score s = score_of(a, product);
  Pair x;
  x.p = exp2_(s.x - lse * kLog2e);
  x.ds = x.p * (dp - delta) * (a.scale * s.slope);
  return x;
}

// dq of one query row by one wave, one key at a time.
__device__ void train_dq_row(const TrainLaunch& a, int r, int q, int h, int lane) {
  const int kvh = h / a.group;
  const bool lk = lane * 8 < a.dk, lv = lane * 8 < a.dv;
  const int32_t* const death = a.death + static_cast<int64_t>(r) * a.n_pad;
  const Vals x = load8(at(a.q, r, q, h) + lane * 8, lk), g = load8(at(a.dout, r, q, h) + lane * 8, lv);
  const float lse = a.lse[(static_cast<int64_t>(r) * a.n_pad + q) * a.heads + h];
  const float delta = a.delta[(static_cast<int64_t>(r) * a.heads + h) * a.n_pad + q];
  Vals o{};
  if (lse != -__builtin_inff())
    for (int k = 0; k <= q; ++k) {
      if (death[k] <= q) continue;
      const Vals y = load8(at(a.k, r, k, kvh) + lane * 8, lk);
      const float s = wave_sum(dot8(x, y));
      const float dp = wave_sum(dot8(g, load8(at(a.v, r, k, kvh) + lane * 8, lv)));
      add8(o, pair_of(a, s, dp, lse, delta).ds, y);
    }
  if (lk) store8(place(a.dq, r, q, h) + lane * 8, o, 1.f);
}

// dk and dv of one key row by one wave, one query at a time.
__device__ void train_dkv_row(const TrainLaunch& a, int r, int k, int kvh, int lane) {
  const bool lk = lane * 8 < a.dk, lv = lane * 8 < a.dv;
  const int end = min(a.death[static_cast<int64_t>(r) * a.n_pad + k], a.n_pad);
  const Vals y = load8(at(a.k, r, k, kvh) + lane * 8, lk), v = load8(at(a.v, r, k, kvh) + lane * 8, lv);
  Vals gk{}, gv{};
  for (int h = kvh * a.group; h < (kvh + 1) * a.group; ++h)
    for (int q = k; q < end; ++q) {
      const float lse = a.lse[(static_cast<int64_t>(r) * a.n_pad + q) * a.heads + h];
      if (lse == -__builtin_inff()) continue;
      const Vals x = load8(at(a.q, r, q, h) + lane * 8, lk), g = load8(at(a.dout, r, q, h) + lane * 8, lv);
      const float s = wave_sum(dot8(x, y)), dp = wave_sum(dot8(g, v));
      const Pair w = pair_of(a, s, dp, lse, a.delta[(static_cast<int64_t>(r) * a.heads + h) * a.n_pad + q]);
      add8(gk, w.ds, x);
      add8(gv, w.p, g);
    }
  if (lk) store8(place(a.dk_, r, k, kvh) + lane * 8, gk, 1.f);
  if (lv) store8(place(a.dv_, r, k, kvh) + lane * 8, gv, 1.f);
}

__global__ __launch_bounds__(256) void train_dq_rows_kernel(TrainLaunch a) {
  int64_t unit = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 6);
  const int q = static_cast<int>(unit % a.n_pad);
  unit /= a.n_pad;
  const int r = static_cast<int>(unit / a.heads), h = static_cast<int>(unit % a.heads);
  if (r < a.n) train_dq_row(a, r, q, h, threadIdx.x & 63);
}
__global__ __launch_bounds__(256) void train_dkv_rows_kernel(TrainLaunch a) {
  int64_t unit = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 6);
  const int k = static_cast<int>(unit % a.n_pad);
  unit /= a.n_pad;
  const int r = static_cast<int>(unit / a.kv_heads), h = static_cast<int>(unit % a.kv_heads);
  if (r < a.n) train_dkv_row(a, r, k, h, threadIdx.x & 63);
}

}  // namespace

hipError_t launch_train_back(const TrainLaunch& a, hipStream_t s) {
  const int64_t rows = int64_t{a.n} * a.n_pad;
  auto grid = [&](int64_t waves) { return dim3(static_cast<unsigned>((waves + 3) / 4)); };
  train_delta_kernel<<<grid(rows * a.heads), dim3(256), 0, s>>>(a);
  train_dq_rows_kernel<<<grid(rows * a.heads), dim3(256), 0, s>>>(a);
  train_dkv_rows_kernel<<<grid(rows * a.kv_heads), dim3(256), 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace ll
