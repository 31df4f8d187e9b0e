// gfx950 kernels of the serving step's attention over a paged cache.
//
// For a query row q (a token and a head) and the cached rows j it sees:
//   s_j = scale * q . k_j,  m = max_j s_j,  l = sum_j exp(s_j - m),
//   out = sum_j exp(s_j - m) v_j / l,       lse = m + log l.
// One pass over the rows keeps m, l and the unscaled sum of v, in float32; when m
// grows, l and the sum are scaled down.  Scores are kept in base 2 (times
// log2 e), so that each exponential is one instruction.
#include "device_common.h"
#include "step_internal.h"

namespace ll {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kAttendThreads = 256;

__device__ __forceinline__ float exp2_(float x) { return __builtin_amdgcn_exp2f(x); }

// The cached rows [lo, hi) that query row r of an item's sequence sees, and the
// item's share of the rows its whole tile needs.
struct Seen {
  int lo, hi;
};
__device__ __forceinline__ Seen rows_seen(const AttendLaunch& a, const AttendItem& it, int r) {
  if (r >= it.q_rows) return Seen{0, 0};
  const int own = it.first + r / a.group;   // the token's own row
  Seen s;
  s.hi = a.causal ? own + 1 : it.kv_len;
  s.lo = a.window > 0 && own + 1 > a.window ? own + 1 - a.window : 0;
  return s;
}

// Shares of the rows that some query of the tile sees are equal, in multiples of
// `grain` rows; the last ones may be empty.
__device__ __forceinline__ Seen item_share(const AttendLaunch& a, const AttendItem& it, int grain) {
  const int last = min(it.row0 + a.tile, it.q_rows) - 1;
  const Seen f = rows_seen(a, it, it.row0), l = rows_seen(a, it, last);
  const int shares = it.splits >> 16, c = it.splits & 0xFFFF;
  const int lo = f.lo - f.lo % grain;
  const int64_t per = (static_cast<int64_t>(l.hi - lo + shares - 1) / shares + grain - 1) / grain * grain;
  Seen s;
  s.lo = static_cast<int>(min(lo + c * per, static_cast<int64_t>(l.hi)));
  s.hi = static_cast<int>(min(lo + (c + 1) * per, static_cast<int64_t>(l.hi)));
  return s;
}

// Physical row of cached row j.  A page number outside the pool (only a page
// table that something else has written can hold one) reads page 0.
__device__ __forceinline__ int64_t physical_row(const AttendLaunch& a, int seq, int j) {
  int page = a.page_table[static_cast<int64_t>(seq) * a.max_pages_per_seq + (j >> a.page_shift)];
  if (static_cast<uint32_t>(page) >= static_cast<uint32_t>(a.num_pages)) page = 0;
  return (static_cast<int64_t>(page) << a.page_shift) + (j & ((1 << a.page_shift) - 1));
}

struct Vals {
  float v[8];
};
__device__ __forceinline__ Vals load8(const uint16_t* p, bool live) {
  chunk_t c{0u, 0u, 0u, 0u};
  if (live) c = *reinterpret_cast<const chunk_t*>(p);
  Vals r;
  const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    r.v[2 * i] = bf16_lo(w[i]);
    r.v[2 * i + 1] = bf16_hi(w[i]);
  }
  return r;
}
__device__ __forceinline__ float dot8(const Vals& x, const Vals& y) {
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) s = __builtin_fmaf(x.v[i], y.v[i], s);
  return s;
}

// One query row at a time per wave, one cached row at a time: a lane holds 8
// values of the head (MLA: of the latent part, and of k_pe in lanes 0..7).
// Reads exactly the rows that the query sees.
template <bool GQA>
__device__ void attend_rows(const AttendLaunch& a, const AttendItem& it, int kvh, int wave, int waves, int lane) {
  const int dv = GQA ? a.dim : kKvLoraRank;
  const bool live = lane * 8 < dv;
  const Seen share = item_share(a, it, 64);
  const int shares = it.splits >> 16;
  for (int rr = wave; rr < a.tile && it.row0 + rr < it.q_rows; rr += waves) {
    const int r = it.row0 + rr;
    const int t = it.tok0 + r / a.group, h = kvh * a.group + r % a.group;
    const Seen s = rows_seen(a, it, r);
    const Vals q = load8(a.q + t * a.q_ts + h * a.q_hs + lane * 8, live);
    Vals qp{};
    if (!GQA) qp = load8(a.q_pe + t * a.qp_ts + h * a.qp_hs + lane * 8, lane < 8);
    float m = -__builtin_inff(), l = 0.f;
    Vals o{};
    for (int j = max(s.lo, share.lo); j < min(s.hi, share.hi); ++j) {
      const int64_t row = physical_row(a, it.seq, j);
      Vals k, v;
      float x;
      if constexpr (GQA) {
        const int64_t off = (row * a.kv_heads + kvh) * a.dim + lane * 8;
        k = load8(a.k_plane + off, live);
        v = load8(a.v_plane + off, live);
        x = dot8(q, k);
      } else {
        const uint16_t* p = a.k_plane + row * kRowElems + lane * 8;
        k = load8(p, true);
        v = k;
        x = dot8(q, k) + dot8(qp, load8(p + kKvLoraRank, lane < 8));
      }
      for (int d = 32; d >= 1; d >>= 1) x += __shfl_xor(x, d);
      x *= a.scale * kLog2e;
      const float m2 = fmaxf(m, x);
      const float keep = m == m2 ? 1.f : exp2_(m - m2);
      const float p = x == -__builtin_inff() ? 0.f : exp2_(x - m2);
      l = l * keep + p;
#pragma unroll
      for (int i = 0; i < 8; ++i) o.v[i] = __builtin_fmaf(p, v.v[i], o.v[i] * keep);
      m = m2;
    }
    if (shares > 1) {
      const int64_t at = (static_cast<int64_t>(it.slot) * a.kv_heads + kvh) * a.tile + rr;
      if (live)
#pragma unroll
        for (int i = 0; i < 8; ++i) a.part_o[at * dv + lane * 8 + i] = o.v[i];
      if (lane == 0) {
        a.part_ml[at * 2] = m;
        a.part_ml[at * 2 + 1] = l;
      }
    } else {
      const float inv = l == 0.f ? 0.f : 1.f / l;
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = to_bf16(o.v[2 * i] * inv) | (to_bf16(o.v[2 * i + 1] * inv) << 16);
      if (live) *reinterpret_cast<chunk_t*>(a.out + t * a.o_ts + h * a.o_hs + lane * 8) = chunk_t{w[0], w[1], w[2], w[3]};
      if (a.lse && lane == 0) a.lse[static_cast<int64_t>(t) * a.heads + h] = l == 0.f ? -__builtin_inff() : (m + __log2f(l)) * kLn2;
    }
  }
}

template <bool GQA>
__global__ __launch_bounds__(kAttendThreads) void attend_rows_kernel(AttendLaunch a) {
  const int kvh = blockIdx.x % a.kv_heads;
  const int i = blockIdx.x / a.kv_heads;
  if (i >= a.counts->items) return;
  attend_rows<GQA>(a, a.items[i], kvh, threadIdx.x >> 6, 4, threadIdx.x & 63);
}

// The shares of a split tile put together: a wave per query row, each share
// weighed by how far its maximum lies below the largest.
template <bool GQA>
__global__ __launch_bounds__(kAttendThreads) void attend_join_kernel(AttendLaunch a) {
  const int lane = threadIdx.x & 63;
  const int rows4 = a.tile / 4;
  const int rr = (blockIdx.x % rows4) * 4 + (threadIdx.x >> 6);
  const int b = blockIdx.x / rows4;
  const int kvh = b % a.kv_heads;
  const int i = b / a.kv_heads;
  if (i >= a.counts->shares) return;
  const AttendItem it = a.items[i];
  const int shares = it.splits >> 16;
  const int r = it.row0 + rr;
  if ((it.splits & 0xFFFF) != 0 || r >= it.q_rows) return;
  const int dv = GQA ? a.dim : kKvLoraRank;
  const bool live = lane * 8 < dv;
  const int64_t at0 = (static_cast<int64_t>(it.slot) * a.kv_heads + kvh) * a.tile + rr;
  const int64_t step = static_cast<int64_t>(a.kv_heads) * a.tile;
  float m = -__builtin_inff();
  for (int c = lane; c < shares; c += 64) m = fmaxf(m, a.part_ml[(at0 + c * step) * 2]);
  for (int d = 32; d >= 1; d >>= 1) m = fmaxf(m, __shfl_xor(m, d));
  float l = 0.f;
  Vals o{};
  for (int c = 0; c < shares; ++c) {
    const int64_t at = at0 + c * step;
    const float lc = a.part_ml[at * 2 + 1];
    if (lc == 0.f) continue;   // an empty share
    const float w = exp2_(a.part_ml[at * 2] - m);
    l = __builtin_fmaf(lc, w, l);
    if (!live) continue;
#pragma unroll
    for (int k = 0; k < 8; ++k) o.v[k] = __builtin_fmaf(a.part_o[at * dv + lane * 8 + k], w, o.v[k]);
  }
  const int t = it.tok0 + r / a.group, h = kvh * a.group + r % a.group;
  const float inv = l == 0.f ? 0.f : 1.f / l;
  uint32_t w[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) w[k] = to_bf16(o.v[2 * k] * inv) | (to_bf16(o.v[2 * k + 1] * inv) << 16);
  if (live) *reinterpret_cast<chunk_t*>(a.out + t * a.o_ts + h * a.o_hs + lane * 8) = chunk_t{w[0], w[1], w[2], w[3]};
  if (a.lse && lane == 0) a.lse[static_cast<int64_t>(t) * a.heads + h] = l == 0.f ? -__builtin_inff() : (m + __log2f(l)) * kLn2;
}

}  // namespace

int attend_tile(bool gqa, int dim, int64_t rows) {
  (void)gqa;
  (void)dim;
  return rows <= 16 ? 16 : rows <= 32 ? 32 : rows <= 64 ? 64 : 128;
}

hipError_t launch_attend(const AttendLaunch& a, bool gqa, hipStream_t s) {
  const dim3 g(static_cast<unsigned>(int64_t{a.n_items} * a.kv_heads)), b(kAttendThreads);
  void (*k)(AttendLaunch) = gqa ? attend_rows_kernel<true> : attend_rows_kernel<false>;
  k<<<g, b, 0, s>>>(a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.n_shares == 0) return e;
  k = gqa ? attend_join_kernel<true> : attend_join_kernel<false>;
  k<<<dim3(static_cast<unsigned>(int64_t{a.n_shares} * a.kv_heads * (a.tile / 4))), b, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace ll
