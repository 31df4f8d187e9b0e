// gfx950 kernel of the attention weight that cached rows get (ll_step_weigh):
//   W[j] = decay * W[j] + sum_t sum_h exp(s_thj - lse[t][h])
// over the step's tokens t that see row j, s the attention's scores (kernels_attend.hip).
#include "matrix_common.h"
#include "weight_internal.h"

namespace ll {
namespace {

// A wave per cached row, one query row after another.
template <bool GQA>
__global__ __launch_bounds__(256) void weigh_rows_kernel(WeighLaunch a) {
  const int lane = threadIdx.x & 63;
  const int64_t unit = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 6);
  const int i = static_cast<int>(unit / a.max_rows);
  const int j = static_cast<int>(unit % a.max_rows);
  if (i >= a.counts->seqs) return;
  const StepSeq s = a.seqs[i];
  const int kv_len = s.row0 + s.count;
  if (j >= kv_len) return;
  int page = a.page_table[static_cast<int64_t>(s.seq) * a.max_pages_per_seq + (j >> a.page_shift)];
  if (static_cast<uint32_t>(page) >= static_cast<uint32_t>(a.num_pages)) page = 0;
  const int64_t row = (static_cast<int64_t>(page) << a.page_shift) + (j & ((1 << a.page_shift) - 1));
  float sum = 0.f;
  for (int kvh = 0; kvh < a.kv_heads; ++kvh) {
    const bool live = !GQA || lane * 8 < a.dim;
    const uint16_t* kp = a.k_plane + (GQA ? (row * a.kv_heads + kvh) * a.dim : row * kRowElems) + lane * 8;
    const Vals k = load8(kp, live);
    Vals kpe{};
    if (!GQA) kpe = load8(kp + kKvLoraRank, lane < 8);
    for (int t = 0; t < s.count; ++t) {
      const int own = s.row0 + t;
      if (a.causal && (j > own || (a.window > 0 && j <= own - a.window))) continue;
      for (int g = 0; g < a.group; ++g) {
        const int64_t tok = s.tok0 + t, h = kvh * a.group + g;
        float x = dot8(k, load8(a.q + tok * a.q_ts + h * a.q_hs + lane * 8, live));
        if (!GQA) x += dot8(kpe, load8(a.q_pe + tok * a.qp_ts + h * a.qp_hs + lane * 8, lane < 8));
        for (int d = 32; d >= 1; d >>= 1) x += __shfl_xor(x, d);
        x = a.cap > 0.f ? a.cap * kLog2e * tanh_any(x * (a.scale / a.cap)) : x * (a.scale * kLog2e);
        const float lse = a.lse[tok * a.heads + h];
        if (lse != -__builtin_inff()) sum += exp2_(x - lse * kLog2e);
      }
    }
  }
  if (lane == 0) {
    float* w = a.weights + static_cast<int64_t>(s.seq) * a.weight_stride + j;
    *w = a.decay == 0.f ? sum : __builtin_fmaf(a.decay, *w, sum);
  }
}

}  // namespace

hipError_t launch_weigh(const WeighLaunch& a, bool gqa, hipStream_t s) {
  const int64_t waves = a.max_rows * a.n_seqs;
  void (*k)(WeighLaunch) = gqa ? weigh_rows_kernel<true> : weigh_rows_kernel<false>;
  k<<<dim3(static_cast<unsigned>((waves + 3) / 4)), dim3(256), 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace ll
