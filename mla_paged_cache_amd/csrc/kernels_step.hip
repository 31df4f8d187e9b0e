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
  if (t == 0) {
    *a.dst_counts = a.counts;
    *a.dst_own_counts = a.own_counts;
  }
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
  auto copy = [&](const AttendItem* from, AttendItem* to, int n) {
    const chunk_t* src = reinterpret_cast<const chunk_t*>(from);
    chunk_t* dst = reinterpret_cast<chunk_t*>(to);
    for (int64_t i = t; i < int64_t{n} * 2; i += stride) dst[i] = src[i];
  };
  copy(a.src_items, a.dst_items, a.counts.items);
  copy(a.src_own, a.dst_own_items, a.own_counts.items);
  const chunk_t* seqs = reinterpret_cast<const chunk_t*>(a.src_seqs);
  for (int64_t i = t; i < int64_t{a.counts.seqs} * 3; i += stride) reinterpret_cast<chunk_t*>(a.dst_seqs)[i] = seqs[i];
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
  typedef float f32x8 __attribute__((ext_vector_type(8)));
  typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
  f32x8 x;
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = r.v[i];
  return __builtin_bit_cast(chunk_t, __builtin_convertvector(x, bf16x8));
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
// of lanes further on.  The cos and sin of this lane's pairs (chunks behind the
// band: of some others):
typedef float f32x4 __attribute__((ext_vector_type(4)));
template <int PAIRING>
struct Angles {
  f32x4 c[PAIRING == 0 ? 1 : 2], s[PAIRING == 0 ? 1 : 2];
};
template <int PAIRING>
__device__ __forceinline__ Angles<PAIRING> load_angles(const float* cs, int pairs, int chunk, int band) {
  const int p = PAIRING == 0 ? (chunk & (band - 1)) * 4 : (chunk & ((band >> 1) - 1)) * 8;
  Angles<PAIRING> r;
#pragma unroll
  for (int i = 0; i < (PAIRING == 0 ? 1 : 2); ++i) {
    r.c[i] = *reinterpret_cast<const f32x4*>(cs + p + 4 * i);
    r.s[i] = *reinterpret_cast<const f32x4*>(cs + pairs + p + 4 * i);
  }
  return r;
}
// Every lane of the wave takes part.
template <int PAIRING>
__device__ __forceinline__ void rotate_band(Vals& x, const Angles<PAIRING>& cs, int chunk, int band) {
  if constexpr (PAIRING == 0) {
    if (chunk >= band) return;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float a = x.v[2 * i], b = x.v[2 * i + 1];
      x.v[2 * i] = rot_x(a, b, cs.c[0][i], cs.s[0][i]);
      x.v[2 * i + 1] = rot_y(a, b, cs.c[0][i], cs.s[0][i]);
    }
  } else {
    const int half = band >> 1;
    Vals o;
#pragma unroll
    for (int i = 0; i < 8; ++i) o.v[i] = __shfl_xor(x.v[i], half);
    if (chunk >= band) return;
    const bool first = chunk < half;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float c = cs.c[i >> 2][i & 3], s = cs.s[i >> 2][i & 3];
      x.v[i] = first ? rot_x(x.v[i], o.v[i], c, s) : rot_y(o.v[i], x.v[i], c, s);
    }
  }
}

// A 16-byte chunk per lane; a piece = the heads of one token that 64 lanes hold
// (GQA: K, V or query heads; MLA: query heads).  A wave takes U pieces, or MLA's
// cache row (the latent part, and k_pe in lanes 0..7).  Lanes without a value read
// one that some other lane holds, so that all of a wave's loads are under way
// before the first is waited for.
//
// Bound by the bytes, every value is read once and written once: 24183 tokens of
// 128 MLA heads whose rotated parts lie in wider heads take 155 us (a plain copy of
// those parts 164, a dense one of as many bytes 153); 23705 tokens of 21 GQA heads
// of 96 take 33.5 us, 5.7 TB/s.
template <bool GQA, int PAIRING, int U, bool STREAM>
__global__ __launch_bounds__(256) void append_kernel(AppendLaunch a) {
  auto load = [](const uint16_t* p) { return *reinterpret_cast<const chunk_t*>(p); };
  auto store = [](chunk_t v, uint16_t* p) {
    chunk_t* c = reinterpret_cast<chunk_t*>(p);
    if constexpr (STREAM) __builtin_nontemporal_store(v, c);
    else *c = v;
  };
  const uint32_t wave = __builtin_amdgcn_readfirstlane(blockIdx.x * 4 + (threadIdx.x >> 6));
  const int lane = threadIdx.x & 63;
  const uint32_t tok = wave / static_cast<uint32_t>(a.waves_per_token);
  if (tok >= static_cast<uint32_t>(a.capacity)) return;
  const int64_t t = tok;
  int w = static_cast<int>(wave - tok * a.waves_per_token);
  const bool in_step = t < a.counts->tokens;   // under capture there may be fewer tokens than places
  const float* cs = a.tab + t * 2 * a.pairs;
  const int row = a.rows[t];
  if (!GQA && a.kv_pieces) {
    if (w == 0) {
      const int pe = lane & (kRopeDim / 8 - 1);
      const chunk_t c = load(a.a + t * a.a_ts + lane * 8);
      const chunk_t d = load(a.b + t * a.b_ts + pe * 8);
      const Angles<PAIRING> an = load_angles<PAIRING>(cs, a.pairs, pe, kRopeDim / 8);
      if (!in_step || row < 0) return;
      Vals x = widen(c), y = widen(d);
      if (a.norm) rms_norm(x, a.norm, a.norm_f32, lane, true, 64, kKvLoraRank, a.eps);
      rotate_band<PAIRING>(y, an, pe, kRopeDim / 8);
      uint16_t* dst = a.k_plane + int64_t{row} * kRowElems + lane * 8;
      store(narrow(x), dst);
      if (lane < kRopeDim / 8) store(narrow(y), dst + kKvLoraRank);
      return;
    }
    --w;
  }
  const int sub = lane >> a.group_shift;
  const int per_wave = 64 >> a.group_shift;
  const int place = lane & ((1 << a.group_shift) - 1);
  const bool in_head = place < a.head_chunks;
  const int chunk = in_head ? place : 0;
  const int kv = GQA ? a.kv_pieces : 0, half = kv >> 1;
  const Angles<PAIRING> an = load_angles<PAIRING>(cs, a.pairs, chunk, a.band_chunks);
  chunk_t c[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int p = min(w * U + u, a.pieces - 1);
    if (p < kv) {
      const int h = min((p < half ? p : p - half) * per_wave + sub, a.kv_heads - 1);
      const uint16_t* src = p < half ? a.a + t * a.a_ts + h * a.a_hs : a.b + t * a.b_ts + h * a.b_hs;
      c[u] = load(src + chunk * 8);
    } else {
      const int h = min((p - kv) * per_wave + sub, a.heads - 1);
      c[u] = load(a.q + t * a.q_ts + h * a.q_hs + chunk * 8);
    }
  }
  if (!in_step) return;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int p = w * U + u;
    if (p >= a.pieces) return;
    const bool is_v = p >= half && p < kv;
    if (!is_v) {
      const void* norm = p < kv ? a.norm : GQA ? a.q_norm : nullptr;
      Vals x = widen(in_head ? c[u] : chunk_t{0u, 0u, 0u, 0u});
      if (norm) rms_norm(x, norm, a.norm_f32, chunk, in_head, 1 << a.group_shift, a.head_chunks * 8, a.eps);
      rotate_band<PAIRING>(x, an, place, a.band_chunks);
      c[u] = narrow(x);
    }
    if (p < kv) {
      const int h = (is_v ? p - half : p) * per_wave + sub;
      uint16_t* dst = (is_v ? a.v_plane : a.k_plane) + (int64_t{row} * a.kv_heads + h) * (a.head_chunks * 8);
      if (h < a.kv_heads && in_head && row >= 0) store(c[u], dst + chunk * 8);
    } else {
      const int h = (p - kv) * per_wave + sub;
      uint16_t* dst = a.q_out + t * a.qo_ts + h * a.qo_hs;
      if (h < a.heads && in_head) store(c[u], dst + chunk * 8);
    }
  }
}

}  // namespace

hipError_t launch_step_setup(const StepSetupLaunch& a, hipStream_t s) {
  const int64_t work = std::max<int64_t>({int64_t{a.counts.tokens} * a.pairs, int64_t{a.counts.items} * 2,
                                          int64_t{a.own_counts.items} * 2, int64_t{a.counts.seqs} * 64, 1});
  const int64_t blocks = std::min<int64_t>((work + 255) / 256, 4096);
  step_setup_kernel<<<dim3(static_cast<unsigned>(blocks)), dim3(256), 0, s>>>(a);
  return hipGetLastError();
}

template <bool GQA, int U, bool STREAM>
hipError_t launch_pieces(AppendLaunch a, int pairing, hipStream_t s) {
  const int own = GQA ? 0 : a.kv_pieces;   // MLA: the cache row's wave
  a.waves_per_token = own + (a.pieces - own + U - 1) / U;
  const int64_t waves = int64_t{a.capacity} * a.waves_per_token;
  const dim3 g(static_cast<unsigned>((waves + 3) / 4)), b(256);
  void (*k)(AppendLaunch) = pairing == 0 ? append_kernel<GQA, 0, U, STREAM> : append_kernel<GQA, 1, U, STREAM>;
  k<<<g, b, 0, s>>>(a);
  return hipGetLastError();
}

// Once one piece a wave would fill the chip's 256 x 32 waves, four of them, and
// stores past the caches: 1152 pieces (96 tokens) take 4.1 us one by one and 4.8 us
// in pairs; 142 thousand take 50.1 us one by one, 38.2 in pairs, 36.6 by four, and
// 33.0 by four with streamed stores (streamed loads: 34.6).  MLA: one piece (its
// prompts 164.6 us, streamed stores 155.0, loads too 159.4, then in pairs 163.1).
hipError_t launch_append(const AppendLaunch& a, bool gqa, int pairing, hipStream_t s) {
  const bool many = int64_t{a.capacity} * a.pieces > 256 * 32;
  if (gqa) return many ? launch_pieces<true, 4, true>(a, pairing, s) : launch_pieces<true, 1, false>(a, pairing, s);
  return many ? launch_pieces<false, 1, true>(a, pairing, s) : launch_pieces<false, 1, false>(a, pairing, s);
}

}  // namespace ll
