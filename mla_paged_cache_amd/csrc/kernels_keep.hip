// gfx950 kernel of the selection by weight (ll_keep_heaviest): of a sequence's rows
// the first `sinks` and the last `recent` ones, and of the others the heaviest, ties
// to the earlier row, as keep bytes; their weights moved together.
//
// One workgroup takes one sequence.  The weight that the last kept row has is found
// digit by digit, eight bits at a time from the top, by counting the rows of each
// digit among those that match so far; a last pass then keeps what is above it and,
// in row order, as many equal ones as there is room for.
#include "device_common.h"
#include "weight_internal.h"

namespace ll {
namespace {

constexpr int kKeepThreads = 1024;
constexpr int kKeepWaves = kKeepThreads / 64;
constexpr int kKeepRows = 8;                             // rows a thread takes at a time

// Order of the weights as unsigned numbers: NaN above infinity, -0 as 0.
__device__ __forceinline__ uint32_t order_of(float w) {
  if (w != w) return 0xFFFFFFFFu;
  const uint32_t u = __float_as_uint(w == 0.f ? 0.f : w);
  return u ^ (static_cast<uint32_t>(static_cast<int32_t>(u) >> 31) | 0x80000000u);
}

__global__ __launch_bounds__(kKeepThreads) void keep_kernel(KeepLaunch a) {
  const KeepSeq q = a.seqs[blockIdx.x];
  const int n = static_cast<int>(q.rows), tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
  const float* const w = a.weights + q.seq * a.weight_stride;
  float* const out = a.kept_weights ? a.kept_weights + q.seq * a.weight_stride : nullptr;
  uint8_t* const keep = a.keep + q.keep_off;
  // the rows to choose from
  const int lo = static_cast<int>(min(a.sinks, q.rows));
  const int hi = max(lo, n - static_cast<int>(min(a.recent, q.rows)));
  const int need = min(static_cast<int>(q.budget) - lo - (n - hi), hi - lo);   // of them to keep, >= 0

  __shared__ uint32_t bins[kKeepWaves][256];
  __shared__ uint32_t found[2];
  __shared__ uint32_t totals[2][kKeepWaves][2];
  uint32_t edge = 0, mask = 0;   // the digits found so far
  int left = need;               // rows to keep among those that match them
  for (int shift = 24; shift >= 0 && need > 0; shift -= 8) {
    for (int i = tid; i < kKeepWaves * 256; i += kKeepThreads) (&bins[0][0])[i] = 0;
    __syncthreads();
    for (int i = lo + tid; i < hi; i += kKeepThreads) {
      const uint32_t k = order_of(w[i]);
      if ((k & mask) == edge) atomicAdd(&bins[wave][k >> shift & 255], 1u);
    }
    __syncthreads();
    uint32_t sum = 0;
    if (tid < 256)
      for (int x = 0; x < kKeepWaves; ++x) sum += bins[x][tid];
    __syncthreads();
    if (tid < 256) bins[0][tid] = sum;
    __syncthreads();
    if (tid < 256) {
      uint32_t above = 0;
      for (int x = tid + 1; x < 256; ++x) above += bins[0][x];
      if (above < static_cast<uint32_t>(left) && above + sum >= static_cast<uint32_t>(left)) {
        found[0] = tid;
        found[1] = left - above;
      }
    }
    __syncthreads();
    edge |= found[0] << shift;
    mask |= 255u << shift;
    left = static_cast<int>(found[1]);
    __syncthreads();
  }

  // rows above the edge, and the first `left` that equal it
  int over = 0, ties = 0;        // of the chunks before this one
  int at = 0;
  for (int base = 0; base < n; base += kKeepThreads * kKeepRows, at ^= 1) {
    float v[kKeepRows];
    uint64_t is_over[kKeepRows], is_tie[kKeepRows];
    int my_over = 0, my_ties = 0;   // the wave's
#pragma unroll
    for (int e = 0; e < kKeepRows; ++e) {
      const int i = base + (wave * kKeepRows + e) * 64 + lane;
      v[e] = i < n ? w[i] : 0.f;
      const uint32_t k = order_of(v[e]);
      const bool inner = i >= lo && i < hi;
      is_over[e] = __ballot(i < n && (!inner || (need > 0 && k > edge)));
      is_tie[e] = __ballot(inner && need > 0 && k == edge);
      my_over += __popcll(is_over[e]);
      my_ties += __popcll(is_tie[e]);
    }
    if (lane == 0) {
      totals[at][wave][0] = my_over;
      totals[at][wave][1] = my_ties;
    }
    __syncthreads();   // (also: every weight of the chunk is read before any is written)
    int o = over, t = ties;
    for (int x = 0; x < kKeepWaves; ++x) {
      if (x < wave) {
        o += totals[at][x][0];
        t += totals[at][x][1];
      }
      over += totals[at][x][0];
      ties += totals[at][x][1];
    }
    const uint64_t before = (uint64_t{1} << lane) - 1;
#pragma unroll
    for (int e = 0; e < kKeepRows; ++e) {
      const int i = base + (wave * kKeepRows + e) * 64 + lane;
      const int rank = t + __popcll(is_tie[e] & before);
      const bool mine = (is_over[e] >> lane & 1) || ((is_tie[e] >> lane & 1) && rank < left);
      if (i < n) keep[i] = mine;
      if (mine && out) out[o + __popcll(is_over[e] & before) + min(rank, left)] = v[e];
      o += __popcll(is_over[e]);
      t += __popcll(is_tie[e]);
    }
  }
  if (out) {
    __syncthreads();
    for (int i = over + min(ties, left) + tid; i < n; i += kKeepThreads) out[i] = 0.f;
  }
}

}  // namespace

hipError_t launch_keep(const KeepLaunch& a, int n, hipStream_t s) {
  keep_kernel<<<dim3(static_cast<unsigned>(n)), dim3(kKeepThreads), 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace ll
