// gfx950 kernel of the selection by weight (ll_keep_heaviest): of a sequence's rows
// the first `sinks` and the last `recent` ones, and of the others the heaviest, ties
// to the earlier row, as keep bytes; their weights moved together.
//
// One workgroup takes one sequence.  The weight that the last kept row has is found
// digit by digit, eleven bits at a time from the top, by counting the rows of each
// digit among those that match so far; a last pass then keeps what is above it and,
// in row order, as many equal ones as there is room for.  Up to kKeepRows rows the
// weights are read once and stay in LDS; what is left is the passes' vector
// instructions (13 us for 4097 rows; 39 for 96 sequences of up to 32768 rows, whose 96 of the
// chip's 256 units spend 69% of their time on them).
#include "matrix_common.h"
#include "weight_internal.h"

namespace ll {
namespace {

constexpr int kKeepThreads = 1024;
constexpr int kKeepWaves = kKeepThreads / 64;
constexpr int kKeepBits = 11, kKeepBins = 1 << kKeepBits;
constexpr int kKeepCopies = 2;   // of the counts, against waves waiting for one another
constexpr int kKeepRows = 35 * kKeepThreads;   // whose weights fit LDS beside the counts

// Order of the weights as unsigned numbers: NaN above infinity, -0 as 0.
__device__ __forceinline__ uint32_t order_of(float w) {
  const uint32_t u = __float_as_uint(w + 0.f);
  const uint32_t k = u ^ (static_cast<uint32_t>(static_cast<int32_t>(u) >> 31) | 0x80000000u);
  return w != w ? 0xFFFFFFFFu : k;
}

// RESIDENT: the weights lie in LDS.
template <bool RESIDENT>
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

  __shared__ uint32_t bins[kKeepCopies][kKeepBins];
  __shared__ uint32_t found[2], sums[kKeepWaves];
  __shared__ int totals[2][kKeepWaves][2];
  extern __shared__ float held[];
  if (RESIDENT) {   // all on their way at once
    for (int i = wave * 64; i < n; i += kKeepThreads)
      if (i + lane < n) load_lds4((lds_ptr)held + i * 4, w + i + lane);
    __builtin_amdgcn_s_waitcnt(0x0F70);   // (and a barrier before another thread's are needed)
  }
  auto weight = [&](int i) { return order_of(RESIDENT ? held[i] : w[i]); };

  uint32_t edge = 0, mask = 0;   // the digits found so far
  int left = need;               // rows to keep among those that match them
  // (whoever keeps every row to choose from, or none, needs no edge)
  for (int shift = 32 - kKeepBits; need > 0 && need < hi - lo; shift = max(0, shift - kKeepBits)) {
    for (int i = tid; i < kKeepCopies * kKeepBins / 4; i += kKeepThreads) reinterpret_cast<chunk_t*>(bins)[i] = chunk_t{0u, 0u, 0u, 0u};
    __syncthreads();
    // Eight rows of a thread on their way at once.  A vector instruction takes four cycles,
    // and there are few waves: rows within bounds are not asked whether they are.
    for (int base = 0; base < hi; base += 8 * kKeepThreads) {
      uint32_t k[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) k[e] = weight(min(base + e * kKeepThreads + tid, n - 1));
      auto count = [&](auto inner) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int i = base + e * kKeepThreads + tid;
          if ((inner || (i >= lo && i < hi)) && ((k[e] ^ edge) & mask) == 0)
            atomicAdd(&bins[wave % kKeepCopies][k[e] >> shift & (kKeepBins - 1)], 1u);
        }
      };
      if (base >= lo && base + 8 * kKeepThreads <= hi)
        count(std::true_type{});
      else
        count(std::false_type{});
    }
    __syncthreads();
    // two digits a thread; how many rows lie above them
    uint32_t one = 0, two = 0;
#pragma unroll
    for (int c = 0; c < kKeepCopies; ++c) {
      one += bins[c][2 * tid];
      two += bins[c][2 * tid + 1];
    }
    uint32_t up = one + two;   // of this lane and those after it
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const uint32_t x = __shfl_down(up, d);
      if (lane + d < 64) up += x;
    }
    if (lane == 0) sums[wave] = up;
    __syncthreads();
    uint32_t above = up - one - two;
    for (int x = wave + 1; x < kKeepWaves; ++x) above += sums[x];
    const uint32_t room = static_cast<uint32_t>(left);
    if (above < room && above + two >= room) {
      found[0] = 2 * tid + 1;
      found[1] = room - above;
    } else if (above + two < room && above + two + one >= room) {
      found[0] = 2 * tid;
      found[1] = room - above - two;
    }
    __syncthreads();
    edge |= found[0] << shift;     // (the last digit covers bits that an earlier one has found: they are the same)
    mask |= (kKeepBins - 1u) << shift;
    left = static_cast<int>(found[1]);
    if (shift == 0) break;
  }
  const bool every = need > 0 && need == hi - lo;

  // Rows above the edge, and the first `left` that equal it: of 64 rows at a time as bits.
  // As numbers: above is whatever is not at or below the edge, NaN with it; where the edge
  // is NaN nothing is above, and NaN equals it.
  const bool odd = edge == 0xFFFFFFFFu;
  const float limit = __uint_as_float(edge & 0x80000000u ? edge ^ 0x80000000u : ~edge);
  const bool some = need > 0 && !every;
  auto look = [&](int i0, float x, uint64_t* overs, uint64_t* tied) {   // rows i0 + lane
    uint64_t o = __ballot(!(x <= limit)), t = __ballot(x == limit);
    if (odd) t = o & __ballot(x != x), o = 0;
    if (!some) t = 0, o = every ? ~uint64_t{0} : 0;
    if (i0 < lo || i0 + 64 > hi) {   // rows that are kept whatever they hold, and places behind the last row
      const uint64_t inner = __ballot(i0 + lane >= lo && i0 + lane < hi), there = __ballot(i0 + lane < n);
      o = ((o & inner) | ~inner) & there;
      t &= inner;
    }
    *overs = o;
    *tied = t;
  };
  const uint64_t before = (uint64_t{1} << lane) - 1;
  int over = 0, ties = 0;   // of all waves so far
  int o = 0, t = 0;         // of this wave's rows so far, and those before them
  auto put = [&](int i0, float x) {
    uint64_t overs, tied;
    look(i0, x, &overs, &tied);
    const int i = i0 + lane, rank = t + __popcll(tied & before);
    const bool mine = (overs >> lane & 1) || ((tied >> lane & 1) && rank < left);
    if (i < n) keep[i] = mine;
    if (mine && out) out[o + __popcll(overs & before) + min(rank, left)] = x;
    o += __popcll(overs);
    t += __popcll(tied);
  };
  auto share = [&](int my_over, int my_ties, int at) {   // where this wave's rows begin
    if (lane == 0) {
      totals[at][wave][0] = my_over;
      totals[at][wave][1] = my_ties;
    }
    __syncthreads();   // (also: every weight of the chunk is read before any is written)
    o = over, t = ties;
    for (int x = 0; x < kKeepWaves; ++x) {
      if (x < wave) {
        o += totals[at][x][0];
        t += totals[at][x][1];
      }
      over += totals[at][x][0];
      ties += totals[at][x][1];
    }
  };
  if constexpr (RESIDENT) {
    // each wave takes one run of rows
    const int run = ((n + kKeepWaves - 1) / kKeepWaves + 63) / 64 * 64, first = wave * run, last = min(first + run, n);
    int my_over = 0, my_ties = 0;
    __syncthreads();   // all weights are in LDS
    auto read = [&](int i0) { return held[min(i0 + lane, n - 1)]; };
    for (int i = first; i < last; i += 64) {
      uint64_t overs, tied;
      look(i, read(i), &overs, &tied);
      my_over += __popcll(overs);
      my_ties += __popcll(tied);
    }
    share(my_over, my_ties, 0);
    for (int i = first; i < last; i += 64) put(i, read(i));
  } else {
    // chunks of rows in registers, of which each wave has a run: weights that move within
    // their buffer only reach rows that have been read
    constexpr int E = 8;
    int at = 0;
    for (int base = 0; base < n; base += kKeepThreads * E, at ^= 1) {
      float v[E];
      int my_over = 0, my_ties = 0;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const int i = base + (wave * E + e) * 64 + lane;
        v[e] = i < n ? w[i] : 0.f;
      }
#pragma unroll
      for (int e = 0; e < E; ++e) {
        uint64_t overs, tied;
        look(base + (wave * E + e) * 64, v[e], &overs, &tied);
        my_over += __popcll(overs);
        my_ties += __popcll(tied);
      }
      share(my_over, my_ties, at);
#pragma unroll
      for (int e = 0; e < E; ++e) put(base + (wave * E + e) * 64, v[e]);
    }
  }
  if (out) {
    __syncthreads();
    for (int i = over + min(ties, left) + tid; i < n; i += kKeepThreads) out[i] = 0.f;
  }
}

}  // namespace

// The longest sequence of a launch comes first.
hipError_t launch_keep(const KeepLaunch& a, int n, hipStream_t s) {
  const dim3 g(static_cast<unsigned>(n)), b(kKeepThreads);
  const int64_t rows = a.seqs[0].rows;
  if (rows <= kKeepRows) {
    if (const hipError_t e = allow_lds<keep_kernel<true>>(kKeepRows * 4); e != hipSuccess) return e;
    keep_kernel<true><<<g, b, static_cast<size_t>(rows) * 4, s>>>(a);
  } else {
    keep_kernel<false><<<g, b, 0, s>>>(a);
  }
  return hipGetLastError();
}

}  // namespace ll
