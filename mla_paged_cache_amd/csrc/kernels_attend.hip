// gfx950 kernels of the serving step's attention over a paged cache.
//
// For a query row q (a token and a head) and the cached rows j it sees:
//   s_j = scale * q . k_j,  m = max_j s_j,  l = sum_j exp(s_j - m),
//   out = sum_j exp(s_j - m) v_j / l,       lse = m + log l.
// One pass over the rows keeps m, l and the unscaled sum of v, in float32; when m
// grows, l and the sum are scaled down.  Scores are kept in base 2 (times
// log2 e), so that each exponential is one instruction.
#include <atomic>
#include <type_traits>

#include "device_common.h"
#include "step_internal.h"

namespace ll {
namespace {

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
  const int64_t per = share_rows(l.hi - lo, shares, grain);
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
__device__ void attend_rows(const AttendLaunch& a, const AttendItem& it, const Seen& share, int kvh, int wave,
                            int waves, int lane) {
  const int dv = GQA ? a.dim : kKvLoraRank;
  const bool live = lane * 8 < dv;
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
      const float inv = 1.f / l;
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        w[i] = to_bf16(o.v[2 * i] * inv) | (to_bf16(o.v[2 * i + 1] * inv) << 16);
        if (l == 0.f) w[i] = 0u;   // no weight at all: 0, whatever the sum holds (0 times an infinity)
      }
      if (live) *reinterpret_cast<chunk_t*>(a.out + t * a.o_ts + h * a.o_hs + lane * 8) = chunk_t{w[0], w[1], w[2], w[3]};
      if (a.lse && lane == 0) a.lse[static_cast<int64_t>(t) * a.heads + h] = l == 0.f ? -__builtin_inff() : (m + __log2f(l)) * kLn2;
    }
  }
}

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) char* lds_ptr;

// A tile of cached rows in LDS: regions of ROWCH 16-byte chunks per row, chunk c
// of row r at place c ^ swizzle(r), so that both ways of reading it touch the 64
// banks evenly.  The scores' operand is one chunk of 16 rows per 16 lanes; the
// hardware serves lanes 0-3, 12-15, 20-27 of a 16-byte read together, i.e. rows
// 0-3, 12-15 at one chunk and rows 4-11 at the next.  The transposing reads of the
// values touch 8 consecutive rows at 2 neighbouring chunks per half wave.  Measured
// on 16-byte reads: 208 bytes a clock and CU, 121 with the plain rotation of r,
// 32 without a swizzle.
template <int ROWCH>
__device__ __forceinline__ int swizzle(int r) {
  if constexpr (ROWCH >= 16) {
    return (((r & 7) ^ ((r >> 1) & 4)) << 1) | ((r >> 3) & 1);
  } else {   // two rows per 256-byte line
    const int h = (r >> 1) & 7;
    return (((h & 3) ^ ((h >> 1) & 2)) << 1) | (h >> 2);
  }
}

__device__ __forceinline__ bf16x8 lds_chunk(lds_ptr p) {
  return *reinterpret_cast<__attribute__((address_space(3))) bf16x8*>(p);
}
// 16 lanes read 4 rows x 16 columns (8 bytes each) and get them transposed: lane
// i the 4 rows of column i.
__device__ __forceinline__ s16x4 lds_columns(lds_ptr p) {
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16(reinterpret_cast<__attribute__((address_space(3))) s16x4*>(p));
}

// Bits kNotFinite of the result are set where one of the chunk's values has all
// exponent bits set: one more in its lowest exponent bit then reaches the sign's.
constexpr uint32_t kNotFinite = 0x80008000u;
__device__ __forceinline__ uint32_t exponents(chunk_t c) {
  const chunk_t e = (c & 0x7F807F80u) + 0x00800080u;
  return e.x | e.y | e.z | e.w;
}

// How a workgroup does one item: QW waves side by side over the query rows (QN
// tiles of 16 each), KW over the cached rows of a tile of BN, DW over the columns
// of the values (each of these computes the scores for itself).
template <bool MLA_, int DP, int QN_, int QW_, int KW_, int DW_, int BN_, int STAGES_>
struct Shape {
  static constexpr bool MLA = MLA_;
  static constexpr int QN = QN_, QW = QW_, KW = KW_, DW = DW_, BN = BN_;
  static constexpr int WAVES = QW * KW * DW, THREADS = 64 * WAVES;
  static constexpr int DK = MLA ? kRowElems : DP, DV = MLA ? kKvLoraRank : DP;
  static constexpr int ROWCH = DV / 8;                       // chunks of a row of the main region
  static constexpr int MAIN = BN * DV * 2;                   // MLA: latent part; GQA: K
  static constexpr int SIDE = MLA ? BN * kRopeDim * 2 : MAIN;  // MLA: k_pe; GQA: V
  static constexpr int SIDE_ROWCH = MLA ? kRopeDim / 8 : ROWCH;
  static constexpr int STAGE = MAIN + SIDE;
  static constexpr int VALUES = MLA ? 0 : MAIN;              // where the values lie in a stage
  static constexpr int STAGES = STAGES_;                     // tiles in LDS
  static constexpr int AHEAD = STAGES - 1;                   // a tile is asked for this many tiles ahead
  static constexpr int PAGES = 2 * AHEAD + 1;                // tiles whose page numbers are in LDS
  // a tile's loads per wave, at least, and the pieces they come in
  static constexpr int LOADS = MLA ? BN / WAVES + BN / 8 / WAVES : 2 * BN * ROWCH / 64 / WAVES;
  static constexpr int PIECES = MLA ? BN / WAVES + (BN / 8 + WAVES - 1) / WAVES : BN * ROWCH / 64 / WAVES;
  static constexpr int KVT = BN / KW;                        // cached rows of a tile per wave
  static constexpr int TILE = 16 * QN * QW;                  // query rows
  // Below the largest tile a sequence is one tile (attend_tile; a graph that replays
  // more than it was captured behind is the exception), and its cached rows are read
  // once: past the caches 257, 90 and 413 us (64 MLA tokens over up to 32768
  // rows, one GQA token over 131072, 128 over up to 8192), otherwise 290, 101 and
  // 458.  Chunks of several tiles read rows again (2130 past the caches, 2004).
  static constexpr bool ONCE = TILE < (MLA || DP > 128 ? 128 : 256);
  // the sums fill the accumulation registers, which only assembly can ask for
  static constexpr bool ACC = QN * DV / 4 >= 256;
  // then the waves share the weights through LDS, and each sums the columns
  // [wave * DV / QW ...) of all queries: the values are read from LDS once, not by
  // every wave (MLA chunks of 2048 and 1917 tokens of 16 heads over up to 16384
  // rows: 1846 us with each wave summing its own queries, 1732 us so)
  static constexpr int WEIGHTS = STAGES * STAGE + WAVES * PAGES * BN * 4;   // where these lie in LDS
  static constexpr int KEEPS = WEIGHTS + TILE * BN * 2;                     // two tiles' scalings, and which waves have any
  static constexpr int LDS = ACC ? KEEPS + 2 * (TILE * 4 + 16) : WEIGHTS;
  static_assert(KVT % 16 == 0 && BN <= 64 && BN % WAVES == 0, "whole matrix tiles, a lane per row");
  static_assert(BN * ROWCH / 64 % WAVES == 0 && AHEAD >= 2, "as many loads for every wave; the next tile is there early");
  static_assert(LOADS * (AHEAD - 1) < 64, "the wait counter's range");
};

// The assembly below declares that it writes m0.  The compiler keeps no value there
// between its own uses (and warns that a reserved register is declared), but it may
// share one setting of m0 between several of those, which the declaration ends.
#pragma clang diagnostic ignored "-Winline-asm"

// 64 x 16 bytes from memory straight into LDS at `dst` + 16 * lane (base: uniform;
// off: the lane's byte offset).  As assembly, because the compiler otherwise waits
// for every such load before each transposing LDS read; it has no result
// register, and the kernel waits for it itself (`landed`, then a barrier).
// ONCE: nothing else of the launch reads the bytes, so that they need not stay in
// the caches.
template <bool ONCE>
__device__ __forceinline__ void load_lds(lds_ptr dst, const void* base, uint32_t off) {
  const uint32_t at = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(reinterpret_cast<uintptr_t>(dst)));
  // (five wait states between a vector instruction that writes `base` and the load)
  if constexpr (ONCE)
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tglobal_load_lds_dwordx4 %1, %2 nt" ::"s"(at), "v"(off), "s"(base) : "m0", "memory");
  else
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(at), "v"(off), "s"(base) : "m0", "memory");
}
template <bool ONCE>
__device__ __forceinline__ void load_lds(lds_ptr dst, const void* src) {
  const uint32_t at = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(reinterpret_cast<uintptr_t>(dst)));
  if constexpr (ONCE)
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off nt" ::"s"(at), "v"(src) : "m0", "memory");
  else
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(at), "v"(src) : "m0", "memory");
}

__device__ __forceinline__ void load_lds4(lds_ptr dst, const void* src) {
  const uint32_t at = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(reinterpret_cast<uintptr_t>(dst)));
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, off" ::"s"(at), "v"(src) : "m0", "memory");
}

// A tile from the cache to LDS: an instruction fills 64 consecutive places, so
// each lane fetches the chunk that the swizzle puts at its place.  Lane r holds
// the physical row of the tile's row r.  A wave's part comes in S::PIECES pieces,
// which the products of an earlier tile cover.
template <typename S>
__device__ __forceinline__ void load_mla_piece(int i, uint64_t row, lds_ptr dst, int wave, int lane) {
  const uint32_t lo = static_cast<uint32_t>(row), hi = static_cast<uint32_t>(row >> 32);
  if (i < S::BN / S::WAVES) {   // a row's latent part
    const int r = i * S::WAVES + wave;
    // (a lane's value comes back signed: without the casts its top bit would
    // spread over the upper half)
    const uint64_t at = static_cast<uint64_t>(static_cast<uint32_t>(__builtin_amdgcn_readlane(hi, r))) << 32 |
                        static_cast<uint32_t>(__builtin_amdgcn_readlane(lo, r));
    load_lds<S::ONCE>(dst + r * 1024, reinterpret_cast<const void*>(at), static_cast<uint32_t>(lane ^ swizzle<64>(r)) * 16);
  } else {                      // 8 rows' k_pe
    const int b = (i - S::BN / S::WAVES) * S::WAVES + wave;
    if (S::BN / 8 % S::WAVES != 0 && b >= S::BN / 8) return;
    const int r = b * 8 + (lane >> 3);
    const uint64_t at = static_cast<uint64_t>(static_cast<uint32_t>(__shfl(hi, r))) << 32 | static_cast<uint32_t>(__shfl(lo, r));
    load_lds<S::ONCE>(dst + S::MAIN + b * 1024, reinterpret_cast<const void*>(at + kKvLoraRank * 2 + ((lane & 7) ^ swizzle<8>(r)) * 16));
  }
}
// K and V of one KV head (k and v: its first value in row 0; row: the byte
// offset); chunks past `live` are left alone (they were zeroed once).
template <typename S>
__device__ __forceinline__ void load_gqa_piece(int i, const uint16_t* k, const uint16_t* v, int live, uint64_t row,
                                               lds_ptr dst, int wave, int lane) {
  const int b = i * S::WAVES + wave;
  const int place = b * 64 + lane;
  const int r = place / S::ROWCH;
  const int c = (place % S::ROWCH) ^ swizzle<S::ROWCH>(r);
  const uint32_t lo = static_cast<uint32_t>(row), hi = static_cast<uint32_t>(row >> 32);
  const uint64_t off = (static_cast<uint64_t>(static_cast<uint32_t>(__shfl(hi, r))) << 32 |
                        static_cast<uint32_t>(__shfl(lo, r))) + c * 16;
  if (c < live) {
    load_lds<S::ONCE>(dst + b * 1024, reinterpret_cast<const char*>(k) + off);
    load_lds<S::ONCE>(dst + S::MAIN + b * 1024, reinterpret_cast<const char*>(v) + off);
  }
}

// The flash kernel: scores and weighted sums on the matrix units.
//
// Scores are computed transposed (S^T = K Q^T: cached rows along the matrix
// instruction's rows, queries along its columns), so that a lane holds 4
// consecutive cached rows of one query: the softmax runs along a lane's own
// registers, and the weights, rounded to bf16, are already laid out as the operand
// of O^T = V^T P^T.  V^T comes from the transposing LDS reads.  Nothing but the
// cached rows goes through LDS.
//
// The running maximum is only a reference: it moves (and the sums are scaled)
// when a score (in base 2) exceeds it by more than 8, so weights stay below 2^8 and
// most tiles scale nothing.  Sums are float32; a weight is rounded to bf16 (relative
// 2^-9 on average) because the matrix units multiply bf16 by bf16.
//
// In a tile of which some query sees only a part, unseen weights are 0; since 0
// times a value that is not finite is not 0, such a tile is searched for those,
// and the item falls back to reading exactly the rows each query sees.
//
// One token per sequence is bound by reading the cache: 64 MLA sequences of up to
// 32768 rows 269 us (5.7 TB/s), 128 GQA ones of up to 8192 rows and 8 heads of 128
// 418 us (6.5 TB/s; a large read reaches 6.9).  Chunks are bound by the matrix units
// and what feeds them: 2048 and 1917 MLA tokens of 16 heads over up to 16384 rows
// 1683 us (43% busy), 4096 GQA tokens of 32 heads over 32768 rows 2148 us (44%).
// These are medians of the first twelve calls; the fastest took 250, 412, 1580 and
// 1970 us, for the chunks the last one, from which on they stay there.
template <typename S>
__global__ __launch_bounds__(S::THREADS) __attribute__((amdgpu_waves_per_eu(S::WAVES > 4 ? 2 : 1))) void attend_kernel(AttendLaunch a) {
  extern __shared__ __attribute__((aligned(16))) char smem[];
  constexpr int QN = S::QN, KT = S::KVT / 16, KK = S::DK / 32;
  constexpr int DT = S::DV / (S::ACC ? S::QW : S::DW) / 16;   // 16-column tiles of a wave's sums
  constexpr int ON = S::ACC ? QN * S::QW : QN;                // and their query tiles
  const int kvh = blockIdx.x % a.kv_heads;
  const int item = blockIdx.x / a.kv_heads;
  const AttendItem it = a.items[item];   // asked for together with the count
  if (item >= a.counts->items) return;
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
  const int qw = wave % S::QW, kw = wave / S::QW % S::KW, dw = wave / (S::QW * S::KW);
  const int li = lane & 15, g = lane >> 4;
  const Seen share = item_share(a, it, S::BN);
  const lds_ptr lds = (lds_ptr)smem;
  const int live = S::MLA ? S::ROWCH : a.dim / 8;   // chunks a cached head has

  // queries: this lane's 8 values of each 32 of the row
  bf16x8 q[QN][KK];
#pragma unroll
  for (int n = 0; n < QN; ++n) {
    const int r = it.row0 + (qw * QN + n) * 16 + li;
    const bool ok = r < it.q_rows;
    const int tt = ok ? r / a.group : 0;
    const int64_t t = it.tok0 + tt, h = kvh * a.group + (ok ? r - tt * a.group : 0);
    const uint16_t* p = a.q + t * a.q_ts + h * a.q_hs;
    const uint16_t* pe = S::MLA ? a.q_pe + t * a.qp_ts + h * a.qp_hs : nullptr;
#pragma unroll
    for (int k = 0; k < KK; ++k) {
      const int c = k * 4 + g;
      const bool in = ok && (S::MLA || c < live);
      // a place without a value reads the row's first one, and counts as 0
      chunk_t v = *reinterpret_cast<const chunk_t*>(S::MLA && k >= 16 ? pe + (c - 64) * 8 : p + (in ? c * 8 : 0));
      if (!in) v = chunk_t{0u, 0u, 0u, 0u};
      q[n][k] = __builtin_bit_cast(bf16x8, v);
    }
  }

  // A negative scale turns the queries' signs; one too small to tell scores apart
  // counts as 0, and so do the queries then.
  float c2 = a.scale * kLog2e;
  const bool nothing = !(fabsf(c2) >= 1e-37f);
  if (c2 < 0.f || nothing) {
    const uint32_t keep = nothing ? 0u : ~0u, flip = nothing ? 0u : 0x80008000u;
#pragma unroll
    for (int n = 0; n < QN; ++n)
#pragma unroll
      for (int k = 0; k < KK; ++k) {
        chunk_t v = __builtin_bit_cast(chunk_t, q[n][k]);
        v = (v & keep) ^ flip;
        q[n][k] = __builtin_bit_cast(bf16x8, v);
      }
  }
  c2 = nothing ? 1.f : fabsf(c2);

  f32x4 o[DT][ON];
  float m[QN], l[QN];
#pragma unroll
  for (int n = 0; n < QN; ++n) {
    m[n] = -__builtin_inff();
    l[n] = 0.f;
  }
#pragma unroll
  for (int n = 0; n < ON; ++n) {
#pragma unroll
    for (int d = 0; d < DT; ++d) {
      o[d][n] = f32x4{0.f, 0.f, 0.f, 0.f};
      if constexpr (S::ACC) asm volatile("" : "+a"(o[d][n]));
    }
  }

  const int tiles = (share.hi - share.lo + S::BN - 1) / S::BN;
  // every query of the item sees all of [full_lo, full_hi)
  const int last = min(it.row0 + S::TILE, it.q_rows) - 1;
  const int full_lo = rows_seen(a, it, last).lo;
  const int full_hi = min(rows_seen(a, it, it.row0).hi, share.hi);

  // A wave's own copy of the page numbers of the last few tiles' rows, asked for
  // AHEAD tiles before the tile itself.
  int* const pages = reinterpret_cast<int*>(smem + S::STAGES * S::STAGE) + wave * S::PAGES * S::BN;
  const int* const table = a.page_table + static_cast<int64_t>(it.seq) * a.max_pages_per_seq;
  auto load_pages = [&](int tile) {
    const int j = min(share.lo + tile * S::BN + lane, it.kv_len - 1);
    if (S::BN == 64 || lane < S::BN) load_lds4((lds_ptr)(pages + tile % S::PAGES * S::BN), table + (j >> a.page_shift));
  };
  // rows past the sequence's last one repeat it; a page number outside the pool
  // reads page 0 (see physical_row)
  const uint32_t row_bytes = S::MLA ? kRowBytes : a.kv_heads * a.dim * 2;
  auto tile_rows = [&](int tile) -> uint64_t {   // MLA: the row's address; GQA: its offset in a plane
    int page = pages[tile % S::PAGES * S::BN + (lane & (S::BN - 1))];
    if (static_cast<uint32_t>(page) >= static_cast<uint32_t>(a.num_pages)) page = 0;
    const int j = min(share.lo + tile * S::BN + (lane & (S::BN - 1)), it.kv_len - 1);
    const uint32_t row = (page << a.page_shift) + (j & ((1 << a.page_shift) - 1));
    return static_cast<uint64_t>(row) * row_bytes + (S::MLA ? reinterpret_cast<uint64_t>(a.k_plane) : 0);
  };
  auto load_piece = [&](int i, int tile, uint64_t row) {
    const lds_ptr dst = lds + tile % S::STAGES * S::STAGE;
    if constexpr (S::MLA) load_mla_piece<S>(i, row, dst, wave, lane);
    else load_gqa_piece<S>(i, a.k_plane + kvh * a.dim, a.v_plane + kvh * a.dim, live, row, dst, wave, lane);
  };
  // This wave's part of a tile has landed once only the loads of `later` tiles
  // after it are on their way: loads land in order, page numbers between them
  // only make the wait stricter.
  auto landed = [&](auto later, bool all_asked) {
    constexpr int n = S::LOADS * later.value;
    if (all_asked) __builtin_amdgcn_s_waitcnt(0x0F70 | (n & 15) | (n >> 4) << 14);
    else __builtin_amdgcn_s_waitcnt(0x0F70);   // near the end there are fewer: wait for all
  };

  if (!S::MLA && live < S::ROWCH) {
    for (int i = tid; i < S::STAGES * S::STAGE / 16; i += S::THREADS) reinterpret_cast<chunk_t*>(smem)[i] = chunk_t{0u, 0u, 0u, 0u};
    __syncthreads();
  }
  for (int i = 0; i < min(2 * S::AHEAD, tiles); ++i) load_pages(i);
  __builtin_amdgcn_s_waitcnt(0x0F70);   // vmcnt(0)
  for (int t = 0; t < min(S::AHEAD, tiles); ++t) {
    const uint64_t row = tile_rows(t);
#pragma unroll
    for (int i = 0; i < S::PIECES; ++i) load_piece(i, t, row);
  }

  // This lane's byte offsets within a stage, of the first chunks; the swizzle is
  // an exclusive or, so that other chunks are one more away.
  const int kr = kw * S::KVT + li, vr = kw * S::KVT + 4 * g + (li >> 2);
  const int k_at = kr * S::ROWCH * 16 + ((g ^ swizzle<S::ROWCH>(kr)) << 4);
  const int p_at = S::MAIN + kr * S::SIDE_ROWCH * 16 + ((g ^ swizzle<S::SIDE_ROWCH>(kr)) << 4);
  // this wave's first chunk of the values
  const int vc = S::ACC ? qw * (S::ROWCH / S::QW) : dw * (S::ROWCH / S::DW);
  const int v_at = S::VALUES + vr * S::ROWCH * 16 + (vc >> 4) * 256 +
                   ((((vc & 15) | ((li >> 1) & 1)) ^ swizzle<S::ROWCH>(vr)) << 4) + (li & 1) * 8;
  static_assert(S::STAGE % 256 == 0 && S::MAIN % 256 == 0, "the low bits of an address are the lane's");

  // Scores of a tile.  The operand of a step is read XD steps ahead, and `fill`
  // puts other work between the steps' products; the fences keep the compiler
  // from reading everything at once into registers it lacks.
  auto scores = [&](int tile, f32x4 (&s)[KT][QN], auto&& fill) {
    const int st = tile % S::STAGES * S::STAGE;
    const int main = st + k_at, side = st + p_at;
    auto chunk = [&](int kk, int k) -> bf16x8 {
      if (S::MLA && kk >= 16) return lds_chunk(lds + (side ^ ((kk & 1) << 6)) + k * 16 * S::SIDE_ROWCH * 16);
      if (S::ROWCH < 16) return lds_chunk(lds + (main ^ ((kk & 1) << 6)) + k * 16 * S::ROWCH * 16);
      return lds_chunk(lds + (main ^ ((kk & 3) << 6)) + (kk >> 2) * 256 + k * 16 * S::ROWCH * 16);
    };
    constexpr int XD = KK < 3 ? 1 : 2;
    bf16x8 x[XD + 1][KT];
#pragma unroll
    for (int kk = 0; kk < XD; ++kk)
#pragma unroll
      for (int k = 0; k < KT; ++k) x[kk][k] = chunk(kk, k);
#pragma unroll
    for (int kk = 0; kk < KK; ++kk) {
#pragma unroll
      for (int k = 0; k < KT; ++k)
#pragma unroll
        for (int n = 0; n < QN; ++n) {
          if (n == 0 && kk + XD < KK) x[(kk + XD) % (XD + 1)][k] = chunk(kk + XD, k);
          s[k][n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x[kk % (XD + 1)][k], q[n][kk],
                                                            kk == 0 ? f32x4{0.f, 0.f, 0.f, 0.f} : s[k][n], 0, 0, 0);
          fill((kk * KT + k) * QN + n);
          __builtin_amdgcn_sched_barrier(0);
        }
    }
  };

  f32x4 s[KT][QN];
  if (tiles > 0) {
    landed(std::integral_constant<int, S::AHEAD - 1>{}, tiles >= S::AHEAD);
    __syncthreads();
    scores(0, s, [](int) {});
  }
  float* const keeps = reinterpret_cast<float*>(smem + S::KEEPS);
  int* const moved = reinterpret_cast<int*>(smem + S::KEEPS + 2 * S::TILE * 4);
  bool rows_only = false;
  for (int tile = 0; tile < tiles; ++tile) {
    const int j0 = share.lo + tile * S::BN;
    if (j0 < full_lo || j0 + S::BN > full_hi) {   // some query does not see all of the tile
      uint32_t bits = 0;
#pragma unroll 8
      for (int i = tid; i < S::BN * S::ROWCH; i += S::THREADS)
        bits |= exponents(reinterpret_cast<const chunk_t*>(smem + tile % S::STAGES * S::STAGE + S::VALUES)[i]);
      rows_only = __syncthreads_or((bits & kNotFinite) != 0);
      if (rows_only) break;
#pragma unroll
      for (int n = 0; n < QN; ++n) {
        const Seen seen = rows_seen(a, it, it.row0 + (qw * QN + n) * 16 + li);
        const int lo = seen.lo, hi = min(seen.hi, share.hi);
#pragma unroll
        for (int k = 0; k < KT; ++k)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int j = j0 + kw * S::KVT + k * 16 + g * 4 + e;
            if (j < lo || j >= hi) s[k][n][e] = -__builtin_inff();
          }
      }
    }

    // the reference of the weights, in base 2
    float top[QN];
    bool grew = false;
#pragma unroll
    for (int n = 0; n < QN; ++n) {
      top[n] = -__builtin_inff();
#pragma unroll
      for (int k = 0; k < KT; ++k)
#pragma unroll
        for (int e = 0; e < 4; ++e) top[n] = fmaxf(top[n], s[k][n][e]);
      top[n] *= c2;
      grew |= top[n] > m[n] + 8.f;
    }
    if constexpr (S::ACC)   // the sums stay where they are, whatever follows reads
#pragma unroll
      for (int n = 0; n < ON; ++n)
#pragma unroll
        for (int d = 0; d < DT; ++d) asm volatile("" : "+a"(o[d][n]));
    const bool moves = __any(grew);
    if constexpr (S::ACC) moved[(tile & 1) * S::WAVES + wave] = moves;
    if (moves) {
#pragma unroll
      for (int n = 0; n < QN; ++n) {
        float x = fmaxf(top[n], m[n]);
        x = fmaxf(x, __shfl_xor(x, 16));
        x = fmaxf(x, __shfl_xor(x, 32));
        const float keep = x == m[n] ? 1.f : exp2_(m[n] - x);
        m[n] = x;
        l[n] *= keep;
        if constexpr (S::ACC) {
          if (g == 0) keeps[(tile & 1) * S::TILE + (qw * QN + n) * 16 + li] = keep;
        } else {
#pragma unroll
          for (int d = 0; d < DT; ++d) o[d][n] *= keep;
        }
      }
    }

    // the weights, a few at a time: value v of KT * QN * 4
    float ref[QN];
#pragma unroll
    for (int n = 0; n < QN; ++n) ref[n] = m[n] == -__builtin_inff() ? 0.f : m[n];   // nothing seen yet: every weight is 0
    constexpr int W = KT * QN * 4;
    bf16x4 p[KT][QN];
    auto weight = [&](int v) {
      const int k = v / 4 / QN, n = v / 4 % QN, e = v % 4;
      s[k][n][e] = exp2_(__builtin_fmaf(s[k][n][e], c2, -ref[n]));
      l[n] += s[k][n][e];
      if (e == 3) p[k][n] = __builtin_convertvector(s[k][n], bf16x4);
    };
    f32x4 next[KT][QN];
    if (tile + 1 < tiles) {
      // the next tile's scores, with this one's weights between the products
      landed(std::integral_constant<int, S::AHEAD - 2>{}, tile + S::AHEAD - 1 < tiles);
      __syncthreads();   // all of it has landed, and the stage of the tile before this one is free
      scores(tile + 1, next, [&](int i) {
        constexpr int PRODUCTS = KK * KT * QN;
#pragma unroll
        for (int v = i * W / PRODUCTS; v < (i + 1) * W / PRODUCTS; ++v) weight(v);
      });
    } else {
      if constexpr (S::ACC) __syncthreads();   // nobody reads the last tile's weights any more
#pragma unroll
      for (int v = 0; v < W; ++v) weight(v);
    }

    // the weighted values, with the loads of a later tile between the products
    const bool more = tile + S::AHEAD < tiles;
    uint64_t row = 0;
    if (more) {
      row = tile_rows(tile + S::AHEAD);
      if (tile + 2 * S::AHEAD < tiles) load_pages(tile + 2 * S::AHEAD);
    }
    const int values = tile % S::STAGES * S::STAGE + v_at;
    // step i: two 16-row tiles (or the only one) make one operand, rows
    // 32 (i / DT) on, columns d = i % DT
    constexpr int STEPS = (KT + 1) / 2 * DT, PIECES = S::PIECES;
    using operand = std::conditional_t<KT == 1, s16x4, bf16x8>;
    auto columns = [&](int i) -> operand {
      const int d = i % DT;
      const lds_ptr at = lds + (values ^ ((d & 7) << 5)) + (d >> 3) * 256 + (i / DT) * 32 * S::ROWCH * 16;
      const s16x4 x0 = lds_columns(at);
      if constexpr (KT == 1) {
        return x0;
      } else {
        const s16x4 x1 = lds_columns(at + 16 * S::ROWCH * 16);
        return __builtin_bit_cast(bf16x8, __builtin_shufflevector(x0, x1, 0, 1, 2, 3, 4, 5, 6, 7));
      }
    };
    auto weights = [&](int i, int n) -> operand {
      if constexpr (KT == 1) return __builtin_bit_cast(s16x4, p[0][n]);
      else return __builtin_shufflevector(p[i / DT * 2][n], p[i / DT * 2 + 1][n], 0, 1, 2, 3, 4, 5, 6, 7);
    };
    auto pieces = [&](int i, int steps) {   // piece x goes into step x steps / PIECES
      if (!more) return;
#pragma unroll
      for (int x = (i * PIECES + steps - 1) / steps; x < ((i + 1) * PIECES + steps - 1) / steps; ++x)
        load_piece(x, tile + S::AHEAD, row);
    };
    if constexpr (S::ACC) {
      // The weights go through LDS as they lie in the registers, and so do the
      // scalings of queries whose reference has moved.
      static_assert(!S::ACC || (QN == 2 && KT == 2 && S::QW == 4 && ON == 8), "the block below");
#pragma unroll
      for (int n = 0; n < QN; ++n)
        *reinterpret_cast<__attribute__((address_space(3))) bf16x8*>(lds + S::WEIGHTS + ((qw * QN + n) * 64 + lane) * 16) =
            weights(0, n);
      if (more) load_piece(PIECES - 1, tile + S::AHEAD, row);
      __syncthreads();
      typedef int i32x4 __attribute__((ext_vector_type(4)));
      const i32x4 moves = *reinterpret_cast<const i32x4*>(moved + (tile & 1) * S::WAVES);
      bf16x8 w[8], y[4];
#pragma unroll
      for (int n = 0; n < 8; ++n) w[n] = lds_chunk(lds + S::WEIGHTS + (n * 64 + lane) * 16);
      y[0] = columns(0), y[1] = columns(1);
      __builtin_amdgcn_sched_barrier(0);
      if (__builtin_amdgcn_readfirstlane(moves.x | moves.y | moves.z | moves.w))
#pragma unroll
        for (int n = 0; n < ON; ++n) {
          if (!__builtin_amdgcn_readfirstlane(moves[n / QN])) continue;
          const float keep = keeps[(tile & 1) * S::TILE + n * 16 + li];
#pragma unroll
          for (int d = 0; d < DT; ++d) {
            asm volatile("" : "+a"(o[d][n]));   // four at a time leave the accumulators
            o[d][n] *= keep;
            asm volatile("" : "+a"(o[d][n]));
            __builtin_amdgcn_sched_barrier(0);
          }
        }
      // Thirty-two columns and all query tiles at a time.  An operand that an ordinary
      // instruction has just written needs two wait states, and a sum is safe to
      // touch eight after its product: the block waits for both itself, since the
      // compiler does not see what it holds.  Two rows' loads go between its
      // products (outside they cost 100 clocks each, which no product covers); the
      // first is five wait states behind the instructions that wrote its address.
      static_assert(!S::ACC || (STEPS == 8 && PIECES == 9), "the loads of the block below");
      const uint32_t loads = __builtin_amdgcn_readfirstlane(more ? ~0u : 0u);
      const uint64_t lanes = static_cast<uint64_t>(loads) << 32 | loads;
      const uint32_t lo = static_cast<uint32_t>(row), hi = static_cast<uint32_t>(row >> 32);
#pragma unroll
      for (int i = 0; i < STEPS; i += 2) {
        const int b = i & 2;
        if (i + 2 < STEPS) y[b ^ 2] = columns(i + 2), y[(b ^ 2) + 1] = columns(i + 3);
        const int r0 = i * S::WAVES + wave, r1 = r0 + S::WAVES;   // pieces i and i + 1 (see load_mla_piece)
        const uint64_t at0 = static_cast<uint64_t>(static_cast<uint32_t>(__builtin_amdgcn_readlane(hi, r0))) << 32 |
                             static_cast<uint32_t>(__builtin_amdgcn_readlane(lo, r0));
        const uint64_t at1 = static_cast<uint64_t>(static_cast<uint32_t>(__builtin_amdgcn_readlane(hi, r1))) << 32 |
                             static_cast<uint32_t>(__builtin_amdgcn_readlane(lo, r1));
        const uint32_t to = __builtin_amdgcn_readfirstlane(
            static_cast<uint32_t>(reinterpret_cast<uintptr_t>(lds + (tile + S::AHEAD) % S::STAGES * S::STAGE + r0 * 1024)));
        const uint32_t off0 = static_cast<uint32_t>(lane ^ swizzle<64>(r0)) * 16;
        const uint32_t off1 = static_cast<uint32_t>(lane ^ swizzle<64>(r1)) * 16;
        uint64_t mask;   // the lanes that run, put back after each load
        asm volatile(
            "s_mov_b32 m0, %27\n\t"
            "s_nop 1\n\t"
            "v_mfma_f32_16x16x32_bf16 %0, %17, %19, %0\n\t"
            "v_mfma_f32_16x16x32_bf16 %1, %17, %20, %1\n\t"
            "v_mfma_f32_16x16x32_bf16 %2, %17, %21, %2\n\t"
            "v_mfma_f32_16x16x32_bf16 %3, %17, %22, %3\n\t"
            "s_and_saveexec_b64 %16, %33\n\t"
            "global_load_lds_dwordx4 %29, %31\n\t"
            "s_mov_b64 exec, %16\n\t"
            "v_mfma_f32_16x16x32_bf16 %4, %17, %23, %4\n\t"
            "v_mfma_f32_16x16x32_bf16 %5, %17, %24, %5\n\t"
            "v_mfma_f32_16x16x32_bf16 %6, %17, %25, %6\n\t"
            "v_mfma_f32_16x16x32_bf16 %7, %17, %26, %7\n\t"
            "s_mov_b32 m0, %28\n\t"
            "v_mfma_f32_16x16x32_bf16 %8, %18, %19, %8\n\t"
            "v_mfma_f32_16x16x32_bf16 %9, %18, %20, %9\n\t"
            "v_mfma_f32_16x16x32_bf16 %10, %18, %21, %10\n\t"
            "v_mfma_f32_16x16x32_bf16 %11, %18, %22, %11\n\t"
            "s_and_saveexec_b64 %16, %33\n\t"
            "global_load_lds_dwordx4 %30, %32\n\t"
            "s_mov_b64 exec, %16\n\t"
            "v_mfma_f32_16x16x32_bf16 %12, %18, %23, %12\n\t"
            "v_mfma_f32_16x16x32_bf16 %13, %18, %24, %13\n\t"
            "v_mfma_f32_16x16x32_bf16 %14, %18, %25, %14\n\t"
            "v_mfma_f32_16x16x32_bf16 %15, %18, %26, %15\n\t"
            "s_nop 9"
            : "+a"(o[i][0]), "+a"(o[i][1]), "+a"(o[i][2]), "+a"(o[i][3]), "+a"(o[i][4]), "+a"(o[i][5]), "+a"(o[i][6]),
              "+a"(o[i][7]), "+a"(o[i + 1][0]), "+a"(o[i + 1][1]), "+a"(o[i + 1][2]), "+a"(o[i + 1][3]), "+a"(o[i + 1][4]),
              "+a"(o[i + 1][5]), "+a"(o[i + 1][6]), "+a"(o[i + 1][7]), "=&s"(mask)
            : "v"(y[b]), "v"(y[b + 1]), "v"(w[0]), "v"(w[1]), "v"(w[2]), "v"(w[3]), "v"(w[4]), "v"(w[5]), "v"(w[6]),
              "v"(w[7]), "s"(to), "s"(to + S::WAVES * 1024), "v"(off0), "v"(off1), "s"(at0), "s"(at1), "s"(lanes)
            : "m0", "scc", "memory");
        __builtin_amdgcn_sched_barrier(0);
      }
    } else {
      constexpr int YD = 3;   // operands are read this many steps ahead
      operand y[YD + 1];
#pragma unroll
      for (int i = 0; i < YD; ++i) y[i] = columns(i);
#pragma unroll
      for (int i = 0; i < STEPS; ++i) {
        if (i + YD < STEPS) y[(i + YD) % (YD + 1)] = columns(i + YD);
        const int d = i % DT;
#pragma unroll
        for (int n = 0; n < QN; ++n) {
          if constexpr (KT == 1)
            o[d][n] = __builtin_amdgcn_mfma_f32_16x16x16bf16_1k(y[i % (YD + 1)], weights(i, n), o[d][n], 0, 0, 0);
          else
            o[d][n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(y[i % (YD + 1)], weights(i, n), o[d][n], 0, 0, 0);
        }
        pieces(i, STEPS);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
#pragma unroll
    for (int k = 0; k < KT; ++k)
#pragma unroll
      for (int n = 0; n < QN; ++n) s[k][n] = next[k][n];
  }

  if (rows_only) {
    __builtin_amdgcn_s_waitcnt(0x0F70);   // loads on their way into LDS
    attend_rows<!S::MLA>(a, it, share, kvh, wave, S::WAVES, lane);
    return;
  }

#pragma unroll
  for (int n = 0; n < QN; ++n) {
    l[n] += __shfl_xor(l[n], 16);
    l[n] += __shfl_xor(l[n], 32);
  }
  const int shares = it.splits >> 16;
  const int dv = S::MLA ? kKvLoraRank : a.dim;
  if constexpr (S::KW > 1) {
    // the waves' sums over their own cached rows, put together in LDS
    __shared__ float s_m[S::WAVES][16 * QN], s_l[S::WAVES][16 * QN];
    constexpr int OUT_ROWS = 16 * QN * S::QW;   // m and l are the same in the DW waves of a row: the first ones' count
    static_assert(S::KW * OUT_ROWS * S::DV * 4 <= S::STAGES * S::STAGE, "the sums fit where the tiles were");
    __syncthreads();   // the tiles are no longer read
    float* sums = reinterpret_cast<float*>(smem);
    if (g == 0)
#pragma unroll
      for (int n = 0; n < QN; ++n) {
        s_m[wave][n * 16 + li] = m[n];
        s_l[wave][n * 16 + li] = l[n];
      }
#pragma unroll
    for (int n = 0; n < QN; ++n)
#pragma unroll
      for (int d = 0; d < DT; ++d) {
        // 16-byte chunks rotated by the row, against bank conflicts
        const int row = (qw * QN + n) * 16 + li, ch = ((dw * DT + d) * 4 + g + row) % (S::DV / 4);
        *reinterpret_cast<f32x4*>(sums + (kw * OUT_ROWS + row) * S::DV + ch * 4) = o[d][n];
      }
    __syncthreads();
    static_assert(OUT_ROWS * (S::DV / 4) % S::THREADS == 0, "as many chunks for every thread");
#pragma unroll
    for (int x = 0; x < OUT_ROWS * (S::DV / 4) / S::THREADS; ++x) {
      const int i = x * S::THREADS + tid;
      const int row = i / (S::DV / 4), c = i % (S::DV / 4);
      const int r = it.row0 + row;
      if (r >= it.q_rows || c * 4 >= dv) continue;
      const int rw = row / (16 * QN), rn = row % (16 * QN);
      float top = -__builtin_inff(), total = 0.f;
      f32x4 sum{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int k = 0; k < S::KW; ++k) top = fmaxf(top, s_m[k * S::QW + rw][rn]);
#pragma unroll
      for (int k = 0; k < S::KW; ++k) {
        const float lk = s_l[k * S::QW + rw][rn];
        if (lk == 0.f) continue;
        const float w = exp2_(s_m[k * S::QW + rw][rn] - top);
        total = __builtin_fmaf(lk, w, total);
        sum += *reinterpret_cast<const f32x4*>(sums + (k * OUT_ROWS + row) * S::DV + (c + row) % (S::DV / 4) * 4) * w;
      }
      if (shares > 1) {
        const int64_t at = (static_cast<int64_t>(it.slot) * a.kv_heads + kvh) * a.tile + row;
        *reinterpret_cast<f32x4*>(a.part_o + at * dv + c * 4) = sum;
        if (c == 0) {
          a.part_ml[at * 2] = top;
          a.part_ml[at * 2 + 1] = total;
        }
      } else {
        const int tt = r / a.group, h = kvh * a.group + r - tt * a.group;
        const int64_t t = it.tok0 + tt;
        const float inv = total == 0.f ? 0.f : 1.f / total;
        *reinterpret_cast<bf16x4*>(a.out + t * a.o_ts + h * a.o_hs + c * 4) = __builtin_convertvector(sum * inv, bf16x4);
        if (a.lse && c == 0) a.lse[t * a.heads + h] = total == 0.f ? -__builtin_inff() : (top + __log2f(total)) * kLn2;
      }
    }
  } else {
    float* const ends = reinterpret_cast<float*>(smem + S::WEIGHTS);   // ACC: every query's m and l
    if constexpr (S::ACC) {
      __syncthreads();   // the weights are no longer read
      if (g == 0)
#pragma unroll
        for (int n = 0; n < QN; ++n) {
          ends[(qw * QN + n) * 16 + li] = m[n];
          ends[S::TILE + (qw * QN + n) * 16 + li] = l[n];
        }
      __syncthreads();
    }
#pragma unroll
    for (int n = 0; n < ON; ++n) {
      const int row = ((S::ACC ? 0 : qw * QN) + n) * 16 + li;
      const int r = it.row0 + row, col = (S::ACC ? qw : dw) * DT * 16 + g * 4;
      const float top = S::ACC ? ends[row] : m[S::ACC ? 0 : n], sum = S::ACC ? ends[S::TILE + row] : l[S::ACC ? 0 : n];
      if (r >= it.q_rows) continue;
      const int tt = r / a.group, h = kvh * a.group + r - tt * a.group;
      const int64_t t = it.tok0 + tt;
      if (shares > 1) {
        const int64_t at = (static_cast<int64_t>(it.slot) * a.kv_heads + kvh) * a.tile + row;
#pragma unroll
        for (int d = 0; d < DT; ++d) {
          if constexpr (S::ACC) asm volatile("" : "+a"(o[d][n]));
          if (col + d * 16 < dv) *reinterpret_cast<f32x4*>(a.part_o + at * dv + col + d * 16) = o[d][n];
          __builtin_amdgcn_sched_barrier(0);
        }
        if (col == 0) {
          a.part_ml[at * 2] = top;
          a.part_ml[at * 2 + 1] = sum;
        }
      } else {
        const float inv = 1.f / sum;
        uint16_t* out = a.out + t * a.o_ts + h * a.o_hs;
#pragma unroll
        for (int d = 0; d < DT; ++d) {
          if constexpr (S::ACC) asm volatile("" : "+a"(o[d][n]));
          // no weight at all: 0, whatever the sum holds (0 times an infinity)
          const f32x4 x = sum == 0.f ? f32x4{0.f, 0.f, 0.f, 0.f} : o[d][n] * inv;
          if (col + d * 16 < dv) *reinterpret_cast<bf16x4*>(out + col + d * 16) = __builtin_convertvector(x, bf16x4);
          __builtin_amdgcn_sched_barrier(0);
        }
        if (a.lse && col == 0) a.lse[t * a.heads + h] = sum == 0.f ? -__builtin_inff() : (top + __log2f(sum)) * kLn2;
      }
    }
  }
}

template <typename S>
hipError_t launch_shape(const AttendLaunch& a, hipStream_t s) {
  constexpr int lds = S::LDS;
  static std::atomic<bool> set[64];   // per device: hipFuncSetAttribute is not cheap
  int dev = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return e;
  if (dev < 0 || dev >= 64 || !set[dev]) {
    e = hipFuncSetAttribute(reinterpret_cast<const void*>(&attend_kernel<S>), hipFuncAttributeMaxDynamicSharedMemorySize, lds);
    if (e != hipSuccess) return e;
    if (dev >= 0 && dev < 64) set[dev] = true;
  }
  attend_kernel<S><<<dim3(static_cast<unsigned>(int64_t{a.n_items} * a.kv_heads)), dim3(S::THREADS), lds, s>>>(a);
  return hipGetLastError();
}

// The query rows a workgroup takes follow from how many the sequences bring
// (attend_tile); how its waves share them was measured:
//  * few rows: the waves split a tile's cached rows, and for MLA its values' columns
//    (one token of 16 heads over 1531 rows: 11.8 us, without the columns' split 16;
//    64 tokens over 32768: 280 and 286 us);
//  * many rows: two tiles of 16 queries a wave halve the reads of LDS per product.
// Four tiles in LDS: with three, single tokens wait for memory (those 64 MLA tokens
// 340 us against 280, 128 GQA tokens over up to 8192 rows 559 against 455); smaller
// tiles, more of them (32 rows, 7 or 9 tiles, GQA): 490 and 466 us.  (These with
// rows kept in the caches, see ONCE.)
template <bool MLA, int DP>
hipError_t launch_tile(const AttendLaunch& a, hipStream_t s) {
  constexpr bool WIDE = MLA || DP > 128;   // rows of 1 KiB: tiles of 32
  switch (a.tile) {
    case 16: return launch_shape<Shape<MLA, DP, 1, 1, WIDE ? 2 : 4, MLA ? 2 : 1, WIDE ? 32 : 64, 4>>(a, s);
    case 32: return launch_shape<Shape<MLA, DP, 1, 2, 2, MLA ? 2 : 1, WIDE ? 32 : 64, 4>>(a, s);
    case 64: return launch_shape<Shape<MLA, DP, 1, 4, 1, MLA ? 2 : 1, WIDE ? 32 : 64, 4>>(a, s);
    case 128: return launch_shape<Shape<MLA, DP, 2, 4, 1, 1, WIDE ? 32 : 64, 4>>(a, s);
    default:
      if constexpr (WIDE) return hipErrorInvalidValue;   // attend_tile never says so
      else return launch_shape<Shape<MLA, DP, 2, 8, 1, 1, WIDE ? 32 : 64, 4>>(a, s);
  }
}

// The shares of a split tile put together: 4 values of a query row per thread,
// each share weighed by how far its maximum lies below the largest.  Bound by the
// latency of its loads, so several shares are on their way at once.
template <bool GQA>
__global__ __launch_bounds__(kAttendThreads) void attend_join_kernel(AttendLaunch a) {
  const int dv = GQA ? a.dim : kKvLoraRank;
  const int per_row = dv / 4;
  const int unit = blockIdx.x % a.join_blocks * kAttendThreads + threadIdx.x;
  const int b = blockIdx.x / a.join_blocks;
  const int kvh = b % a.kv_heads;
  const int i = b / a.kv_heads;
  const AttendItem it = a.items[i];
  if (i >= a.counts->shares || (it.splits & 0xFFFF) != 0) return;
  const int rr = unit / per_row, c4 = unit - rr * per_row;
  const int r = it.row0 + rr;
  if (rr >= a.tile || r >= it.q_rows) return;
  const int shares = it.splits >> 16;
  const int64_t at0 = (static_cast<int64_t>(it.slot) * a.kv_heads + kvh) * a.tile + rr;
  const int64_t step = static_cast<int64_t>(a.kv_heads) * a.tile;
  const float* const ml = a.part_ml + at0 * 2;
  const f32x4* const po = reinterpret_cast<const f32x4*>(a.part_o + at0 * dv) + c4;
  constexpr int N = 8;
  float m = -__builtin_inff(), l = 0.f;
  f32x4 o{0.f, 0.f, 0.f, 0.f};
  for (int c = 0; c < shares; c += N) {
    float mc[N], lc[N];
    f32x4 oc[N];
#pragma unroll
    for (int k = 0; k < N; ++k) {   // past the last share: the last one again, weighing nothing
      const int64_t s = min(c + k, shares - 1) * step;
      mc[k] = ml[s * 2];
      lc[k] = c + k < shares ? ml[s * 2 + 1] : 0.f;
      oc[k] = po[s * per_row];
    }
    float top = m;
#pragma unroll
    for (int k = 0; k < N; ++k)
      if (lc[k] != 0.f) top = fmaxf(top, mc[k]);
    const float keep = top == m ? 1.f : exp2_(m - top);
    l *= keep;
    o *= keep;
    m = top;
#pragma unroll
    for (int k = 0; k < N; ++k) {
      if (lc[k] == 0.f) continue;   // an empty share
      const float w = mc[k] == m ? 1.f : exp2_(mc[k] - m);
      l = __builtin_fmaf(lc[k], w, l);
      o += oc[k] * w;
    }
  }
  const int tt = r / a.group, h = kvh * a.group + r - tt * a.group;
  const int64_t t = it.tok0 + tt;
  const float inv = l == 0.f ? 0.f : 1.f / l;
  *reinterpret_cast<bf16x4*>(a.out + t * a.o_ts + h * a.o_hs + c4 * 4) = __builtin_convertvector(o * inv, bf16x4);
  if (a.lse && c4 == 0) a.lse[t * a.heads + h] = l == 0.f ? -__builtin_inff() : (m + __log2f(l)) * kLn2;
}

}  // namespace

// The smallest tile that holds all rows a sequence brings, so that its cached rows
// are read once, up to what the registers hold (MLA and heads above 128: 128 rows).
// 4096 GQA tokens of 4 heads a KV head over 32768 rows: 2.23 ms in tiles of 256,
// 3.10 of 128, 4.96 of 64; seven chunks of up to 333 tokens, 5 heads a
// KV head, in a window of 1000: 52, 57, 78 us.
int attend_tile(bool gqa, int dim, int64_t rows) {
  return rows <= 16 ? 16 : rows <= 32 ? 32 : rows <= 64 ? 64 : rows <= 128 || !gqa || dim > 128 ? 128 : 256;
}

// One workgroup a CU, since its tiles fill LDS; two where rows of 64 values leave
// room.
int attend_groups(bool gqa, int dim, int tile) {
  return gqa && dim <= 64 && tile < 256 ? 512 : 256;
}

hipError_t launch_attend(const AttendLaunch& a, bool gqa, hipStream_t s) {
  hipError_t e;
  if (!gqa) e = launch_tile<true, 0>(a, s);
  else if (a.dim <= 64) e = launch_tile<false, 64>(a, s);
  else if (a.dim <= 128) e = launch_tile<false, 128>(a, s);
  else e = launch_tile<false, 256>(a, s);
  if (e != hipSuccess || a.n_shares == 0) return e;
  void (*k)(AttendLaunch) = gqa ? attend_join_kernel<true> : attend_join_kernel<false>;
  k<<<dim3(static_cast<unsigned>(int64_t{a.n_shares} * a.kv_heads * a.join_blocks)), dim3(kAttendThreads), 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace ll
