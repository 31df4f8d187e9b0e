// gfx950 kernels of the serving step that run before its attention:
//
//  * step_setup_kernel: once per begin, the plan into the step's own buffers:
//    the counts and attention items, the page-table entries of the fresh pages,
//    each token's physical row, and the float32 cos / sin of its position's
//    float64 angles (computed once, read by every layer).
//  * append_kernel: once per layer, the tokens' new cache rows and queries.
#include "device_common.h"
#include "step_internal.h"

namespace ll {
namespace {

// The sequence of token t: the last one whose first token is not after t (a
// sequence without tokens shares its first token with the next one's).
__device__ __forceinline__ int seq_of_token(const StepSeq* seqs, int n, int t) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (seqs[mid].tok0 <= t) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// Thread = (token, pair) first, then the copies: items in 16-byte words, and one
// thread per sequence for its fresh pages.
__global__ __launch_bounds__(256) void step_setup_kernel(StepSetupLaunch a) {
  const int64_t t = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * 256;
  if (t == 0) *a.dst_counts = a.counts;
  for (int64_t i = t; i < int64_t{a.counts.tokens} * a.pairs; i += stride) {
    const int tok = static_cast<int>(i / a.pairs);
    const int j = static_cast<int>(i - int64_t{tok} * a.pairs);
    const StepSeq s = a.src_seqs[seq_of_token(a.src_seqs, a.counts.seqs, tok)];
    double sn, cs;
    sincos(static_cast<double>(s.pos0 + (tok - s.tok0)) * a.theta[j], &sn, &cs);
    float* row = a.tab + int64_t{tok} * 2 * a.pairs;
    row[j] = static_cast<float>(cs);
    row[a.pairs + j] = static_cast<float>(sn);
    if (j == 0) {
      const int r = s.row0 + (tok - s.tok0);
      const int lp = r >> a.page_shift;
      // the table's own entries for pages it has (other threads may be writing
      // the fresh ones), the uploaded list for the rest
      const int page = lp < s.old_pages ? a.page_table[int64_t{s.seq} * a.max_pages_per_seq + lp]
                                        : a.fresh[s.fresh_off + lp - s.old_pages];
      // a page number outside the pool (only a page table that something else has
      // written can hold one) is no row: append leaves it out
      const bool in_pool = static_cast<uint32_t>(page) < static_cast<uint32_t>(a.num_pages);
      a.rows[tok] = in_pool ? (page << a.page_shift) + (r & ((1 << a.page_shift) - 1)) : -1;
    }
  }
  const chunk_t* src = reinterpret_cast<const chunk_t*>(a.src_items);
  chunk_t* dst = reinterpret_cast<chunk_t*>(a.dst_items);
  for (int64_t i = t; i < int64_t{a.counts.items} * 2; i += stride) dst[i] = src[i];
  // a wave per sequence
  for (int64_t i = t >> 6; i < a.counts.seqs; i += stride >> 6) {
    const StepSeq s = a.src_seqs[i];
    for (int k = threadIdx.x & 63; k < s.new_pages; k += 64)
      a.page_table[int64_t{s.seq} * a.max_pages_per_seq + s.old_pages + k] = a.fresh[s.fresh_off + k];
  }
}

// 8 bf16 values as float32, and back.
struct Vals {
  float v[8];
};
__device__ __forceinline__ Vals widen(chunk_t c) {
  Vals r;
  const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    r.v[2 * i] = bf16_lo(w[i]);
    r.v[2 * i + 1] = bf16_hi(w[i]);
  }
  return r;
}
__device__ __forceinline__ chunk_t narrow(const Vals& r) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = to_bf16(r.v[2 * i]) | (to_bf16(r.v[2 * i + 1]) << 16);
  return chunk_t{w[0], w[1], w[2], w[3]};
}

// x * rsqrt(mean x^2 + eps) * w over the `lanes` (a power of two) lanes that hold
// one head, `values` values in all; lanes past the head hold zeros.
__device__ __forceinline__ void rms_norm(Vals& x, const void* weight, int f32, int chunk, bool live, int lanes,
                                         int values, float eps) {
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) s = __builtin_fmaf(x.v[i], x.v[i], s);
  for (int m = 1; m < lanes; m <<= 1) s += __shfl_xor(s, m);
  const float r = 1.f / sqrtf(s / static_cast<float>(values) + eps);
  if (!live) return;
  Vals w;
  if (f32) {
    const float* p = static_cast<const float*>(weight) + chunk * 8;
#pragma unroll
    for (int i = 0; i < 8; ++i) w.v[i] = p[i];
  } else {
    w = widen(static_cast<const chunk_t*>(weight)[chunk]);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) x.v[i] = x.v[i] * r * w.v[i];
}

// A head's RoPE band is its first `band` chunks, one lane each (a power of two).
// Interleaved pairs lie within a lane; half-split ones have their y half a band
// of lanes further on.  Every lane of the wave takes part.
template <int PAIRING>
__device__ __forceinline__ void rotate_band(Vals& x, const float* cs, int pairs, int chunk, int band) {
  if constexpr (PAIRING == 0) {
    if (chunk >= band) return;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float c = cs[4 * chunk + i], s = cs[pairs + 4 * chunk + i];
      const float a = x.v[2 * i], b = x.v[2 * i + 1];
      x.v[2 * i] = rot_x(a, b, c, s);
      x.v[2 * i + 1] = rot_y(a, b, c, s);
    }
  } else {
    const int half = band >> 1;
    Vals o;
#pragma unroll
    for (int i = 0; i < 8; ++i) o.v[i] = __shfl_xor(x.v[i], half);
    if (chunk >= band) return;
    const int p = (chunk & (half - 1)) * 8;
    const bool first = chunk < half;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float c = cs[p + i], s = cs[pairs + p + i];
      x.v[i] = first ? rot_x(x.v[i], o.v[i], c, s) : rot_y(o.v[i], x.v[i], c, s);
    }
  }
}

// A wave = some heads of one token (GQA: K, V or query heads; MLA: query heads,
// k_pe as a head, or the latent part), a 16-byte chunk per lane.  Bound by the
// bytes: every value is read once and written once.
template <bool GQA, int PAIRING>
__global__ __launch_bounds__(256) void append_kernel(AppendLaunch a) {
  const int64_t wave = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 6);
  const int lane = threadIdx.x & 63;
  const int64_t t = wave / a.waves_per_token;
  int w = static_cast<int>(wave - t * a.waves_per_token);
  if (t >= a.counts->tokens || t >= a.capacity) return;
  const float* cs = a.tab + t * 2 * a.pairs;
  if (!GQA && w == 0 && a.kv_waves) {   // the latent part: 64 chunks
    Vals x = widen(*reinterpret_cast<const chunk_t*>(a.a + t * a.a_ts + lane * 8));
    if (a.norm) rms_norm(x, a.norm, a.norm_f32, lane, true, 64, kKvLoraRank, a.eps);
    const int row = a.rows[t];
    if (row >= 0) reinterpret_cast<chunk_t*>(a.k_plane)[int64_t{row} * kRowChunks + lane] = narrow(x);
    return;
  }
  const int chunk = lane & ((1 << a.group_shift) - 1);
  const int sub = lane >> a.group_shift;
  const int per_wave = 64 >> a.group_shift;
  const bool in_head = chunk < a.head_chunks;
  const uint16_t* src = nullptr;
  uint16_t* dst = nullptr;
  const void* norm = nullptr;
  bool turn = true;
  if (w < a.kv_waves) {
    if constexpr (GQA) {
      const int half = a.kv_waves >> 1;
      const bool is_v = w >= half;
      const int h = (is_v ? w - half : w) * per_wave + sub;
      if (h < a.kv_heads && in_head) {
        src = is_v ? a.b + t * a.b_ts + h * a.b_hs : a.a + t * a.a_ts + h * a.a_hs;
        const int row = a.rows[t];
        if (row >= 0) dst = (is_v ? a.v_plane : a.k_plane) + (int64_t{row} * a.kv_heads + h) * (a.head_chunks * 8);
      }
      norm = is_v ? nullptr : a.norm;
      turn = !is_v;
    } else if (sub == 0) {
      const int row = a.rows[t];
      src = a.b + t * a.b_ts;
      if (row >= 0) dst = a.k_plane + int64_t{row} * kRowElems + kKvLoraRank;
    }
  } else {
    const int h = (w - a.kv_waves) * per_wave + sub;
    if (h < a.heads && in_head) {
      src = a.q + t * a.q_ts + h * a.q_hs;
      dst = a.q_out + t * a.qo_ts + h * a.qo_hs;
    }
    norm = GQA ? a.q_norm : nullptr;
  }
  chunk_t c{0u, 0u, 0u, 0u};
  if (src) c = *reinterpret_cast<const chunk_t*>(src + chunk * 8);
  if (turn) {
    Vals x = widen(c);
    if (norm) rms_norm(x, norm, a.norm_f32, chunk, in_head, 1 << a.group_shift, a.head_chunks * 8, a.eps);
    rotate_band<PAIRING>(x, cs, a.pairs, chunk, a.band_chunks);
    c = narrow(x);
  }
  if (dst) *reinterpret_cast<chunk_t*>(dst + chunk * 8) = c;
}

}  // namespace

hipError_t launch_step_setup(const StepSetupLaunch& a, hipStream_t s) {
  const int64_t work = std::max<int64_t>({int64_t{a.counts.tokens} * a.pairs, int64_t{a.counts.items} * 2,
                                          int64_t{a.counts.seqs} * 64, 1});
  const int64_t blocks = std::min<int64_t>((work + 255) / 256, 4096);
  step_setup_kernel<<<dim3(static_cast<unsigned>(blocks)), dim3(256), 0, s>>>(a);
  return hipGetLastError();
}

hipError_t launch_append(const AppendLaunch& a, bool gqa, int pairing, hipStream_t s) {
  const int64_t waves = int64_t{a.capacity} * a.waves_per_token;
  const dim3 g(static_cast<unsigned>((waves + 3) / 4)), b(256);
  void (*k)(AppendLaunch) = gqa ? (pairing == 0 ? append_kernel<true, 0> : append_kernel<true, 1>)
                                : (pairing == 0 ? append_kernel<false, 0> : append_kernel<false, 1>);
  k<<<g, b, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace ll
