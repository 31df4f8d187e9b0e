// Device helpers shared by the trainer's attention, forward (kernels_train.hip) and
// backward (kernels_train_back.hip).
#pragma once

#include <atomic>

#include "matrix_common.h"
#include "step_internal.h"
#include "train_internal.h"

namespace ll {
namespace {

// Let a kernel take that much LDS; once per device and kernel, since it is not cheap.
template <void (*K)(TrainLaunch)>
hipError_t allow_lds(int bytes) {
  static std::atomic<bool> set[64];
  int dev = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess || (dev >= 0 && dev < 64 && set[dev])) return e;
  e = hipFuncSetAttribute(reinterpret_cast<const void*>(K), hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == hipSuccess && dev >= 0 && dev < 64) set[dev] = true;
  return e;
}

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

typedef float f32x16 __attribute__((ext_vector_type(16)));

// ---- a tile of rows in LDS, and the operands of 32x32x16 products out of it
//
// D values a row, in 16-byte chunks; chunk c of row r lies at place(r, c) of the row,
// so that both ways of reading a tile touch the 64 banks evenly:
//  * straight, 32 rows at one chunk per half wave; the hardware serves lanes 0-3,
//    12-15, 20-27 together, and those rows differ in their last four bits;
//  * transposing, 4 rows and 4 neighbouring chunks per half wave.
// Rows of 128 or 384 bytes start at every other multiple of 128 bytes, which is the
// fourth bit of difference there.
template <int D>
struct Rows {
  static constexpr int CH = D / 8, BYTES = D * 2;
  static_assert(CH == 8 || CH == 16 || CH == 24 || CH == 32, "the swizzles below");
  static __device__ __forceinline__ int place(int r, int c) {
    if constexpr (CH % 16 == 0) return c ^ ((r & 3) << 2 | (r >> 2 & 3));
    else return c ^ ((r >> 1 & 1) << 2 | (r >> 2 & 3));
  }
  // N rows of a head (x: its row 0, ts: values from row to row) into LDS, by WAVES
  // waves; lane r's `row` is the tile's row r (of the part from lane `from` on).  Chunks
  // past `live` and rows from `rows` on are left alone.
  template <int N, int WAVES>
  static __device__ __forceinline__ void load(lds_ptr dst, const uint16_t* x, int64_t ts, int row, int from, int live,
                                              int wave, int lane, int rows = N) {
    constexpr int LOADS = N * CH / 64;
    static_assert(LOADS % WAVES == 0, "as many for every wave");
#pragma unroll
    for (int i = 0; i < LOADS / WAVES; ++i) {
      const int b = i * WAVES + wave;
      const int r = (b * 64 + lane) / CH, c = place(r, (b * 64 + lane) % CH);
      const int64_t at = __shfl(row, from + r);   // (every lane takes part)
      if (c < live && r < rows) load_lds<false>(dst + b * 1024, x + at * ts + c * 8);
    }
  }
  // A lane's byte offsets in a tile, to which the tile's address in LDS (a multiple of 256)
  // is added; a step in k or d is then an exclusive or of the swizzled bits and a constant
  // above them, a step of 16 rows a constant.
  static constexpr int LOW = CH % 16 == 0 ? 16 : 8;   // chunks that the swizzle permutes
  static __device__ __forceinline__ int straight_at(int lane) {
    const int r = lane & 31;
    return r * BYTES + (place(r, lane >> 5) << 4);
  }
  static __device__ __forceinline__ int columns_at(int lane) {
    const int li = lane & 15, r = (lane >> 5) * 4 + (li >> 2);
    return r * BYTES + (place(r, (lane >> 4 & 1) * 2 + (li >> 1 & 1)) << 4) + (li & 1) * 8;
  }
  // Row r0 + (lane & 31), values 16 k + 8 (lane >> 5) on: an operand of S = X Y^T.
  static __device__ __forceinline__ bf16x8 straight(uint32_t at, int r0, int k) {
    return lds_chunk(reinterpret_cast<lds_ptr>(at ^ (2 * k % LOW) << 4) + r0 * BYTES + 2 * k / LOW * LOW * 16);
  }
  // Column 32 d + (lane & 31) of the rows that a lane of the 32x32 products holds:
  // r0 + 4 (lane >> 5) + {0 .. 3, 8 .. 11}.
  static __device__ __forceinline__ bf16x8 columns(uint32_t at, int r0, int d) {
    const uint32_t c = (4 * d % LOW) << 4, o = r0 * BYTES + 4 * d / LOW * LOW * 16;
    const s16x4 y0 = lds_columns(reinterpret_cast<lds_ptr>(at ^ c) + o);
    const s16x4 y1 = lds_columns(reinterpret_cast<lds_ptr>(at ^ c ^ 32) + o + 8 * BYTES);
    return __builtin_bit_cast(bf16x8, __builtin_shufflevector(y0, y1, 0, 1, 2, 3, 4, 5, 6, 7));
  }
};

// A lane's offset in the tile at x.  What follows from it is worked out where it is used,
// in one instruction, rather than kept in registers.
__device__ __forceinline__ uint32_t tile_at(lds_ptr x, int at) {
  uint32_t y = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(x)) + at;
  asm volatile("" : "+v"(y));
  return y;
}

// Row of a 32x32 product's value i in a lane.
__device__ __forceinline__ int product_row(int i, int lane) { return (i >> 2) * 8 + (lane >> 5) * 4 + (i & 3); }

// Whether the query of this lane sees the keys of a product's values, as bits: key i has
// number first + product_row(i) and its death time in LDS (16-byte words of four).  Only
// for blocks that are seen in part: a branch around it, not a selection.
__device__ __forceinline__ uint32_t seen_bits(const char* deaths, int part, int first, int query, int lane) {
  typedef int i32x4 __attribute__((ext_vector_type(4)));
  uint32_t bits = 0;
#pragma unroll
  for (int i = 0; i < 16; i += 4) {
    const int k = part + product_row(i, lane);
    const i32x4 d = *reinterpret_cast<const i32x4*>(deaths + k * 4);
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (first + k + e <= query && query < d[e]) bits |= 1u << (i + e);
  }
  asm volatile("" : "+v"(bits));
  return bits;
}

// Values 8 x .. 8 x + 7 of a product as the operand of the next one.
__device__ __forceinline__ bf16x8 operand(const f32x16& p, int x) {
  typedef float f32x8 __attribute__((ext_vector_type(8)));
  f32x8 y;
#pragma unroll
  for (int i = 0; i < 8; ++i) y[i] = p[8 * x + i];
  return __builtin_convertvector(y, bf16x8);
}

__device__ __forceinline__ f32x16 mfma(bf16x8 a, bf16x8 b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}

// N products whose operands are read a few steps ahead; the fences keep the compiler
// from reading everything at once into registers that it lacks.
template <int N, int AHEAD, typename Read, typename Use>
__device__ __forceinline__ void stream(Read&& read, Use&& use) {
  constexpr int A = AHEAD < N ? AHEAD : N;
  bf16x8 x[A + 1];
#pragma unroll
  for (int i = 0; i < A; ++i) x[i] = read(i);
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if (i + A < N) x[(i + A) % (A + 1)] = read(i + A);
    use(i, x[i % (A + 1)]);
    __builtin_amdgcn_sched_barrier(0);
  }
}

// A row (of q, k, v or dout) as a lane's operand: KK steps of 16 values, this lane's 8
// of each; a row that is not there and chunks past `live` count as 0.
template <int KK>
__device__ __forceinline__ void load_operand(bf16x8 (&x)[KK], const uint16_t* row, bool there, int live, int lane) {
#pragma unroll
  for (int k = 0; k < KK; ++k) {
    const int c = 2 * k + (lane >> 5);
    chunk_t v{0u, 0u, 0u, 0u};
    if (there && c < live) v = *reinterpret_cast<const chunk_t*>(row + c * 8);
    x[k] = __builtin_bit_cast(bf16x8, v);
  }
}

// A negative scale turns the queries' signs; one too small to tell scores apart counts
// as 0, and so do the queries then.  Returns what a product is multiplied by: to base 2,
// or under a cap to the tanh's argument.
template <bool CAP, int KK>
__device__ __forceinline__ float fold_scale(bf16x8 (&q)[KK], float scale, float cap) {
  const float c = CAP ? scale / cap : scale * kLog2e;
  const bool nothing = !(fabsf(c) >= 1e-37f);
  if (c < 0.f || nothing) {
    const uint32_t keep = nothing ? 0u : ~0u, flip = nothing ? 0u : 0x80008000u;
#pragma unroll
    for (int k = 0; k < KK; ++k) {
      chunk_t v = __builtin_bit_cast(chunk_t, q[k]);
      v = (v & keep) ^ flip;
      q[k] = __builtin_bit_cast(bf16x8, v);
    }
  }
  return nothing ? 1.f : fabsf(c);
}

// tanh of each product times c: all of a wave's in the short form where that holds.
__device__ __forceinline__ void tanh_all(f32x16& s, float c) {
  float most = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    s[i] *= c;
    most = fmaxf(most, fabsf(s[i]));
  }
  if (__any(most > 0.5f)) {
#pragma unroll
    for (int i = 0; i < 16; ++i) s[i] = tanh_any(s[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) s[i] = tanh_small(s[i]);
  }
}

// The blocks of keys that queries [q0, q1] of one epoch see: first those of the epoch's
// list, then the epoch's own.  64 blocks are looked at together, lane x at block base + x;
// every wave of a workgroup goes through the same ones.
struct KeyWalk {
  const KeyBlock* keys;          // the epoch's own blocks
  const uint32_t* odd;           // which of them hold a value that is not finite
  const KeyBlock* list_blocks;
  const KeyEntry* list;
  const int32_t* death;          // from the epoch's first key on
  int q0, q1, k0;                // k0: the epoch's first key
  int n_pad;
  int listed, blocks;            // blocks of the list, and of the walk
  bool odd_list;                 // some key before k0 holds such a value
  int base;
  uint64_t seen, whole;
  bool rows_only;                // a block that is seen in part holds such a value

  __device__ __forceinline__ KeyWalk(const TrainLaunch& a, int r, int kvh, const uint32_t* odd_blocks, int q0_, int q1_, int lane)
      : q0(q0_), q1(q1_), n_pad(a.n_pad), odd_list(false), base(-64), seen(0), whole(0), rows_only(false) {
    const int e = q0 / a.epoch;
    k0 = e * a.epoch;
    const int64_t own = static_cast<int64_t>(r) * a.blocks, first = k0 / kTrainBlock;
    keys = a.keys + own + first;
    odd = odd_blocks + (static_cast<int64_t>(r) * a.kv_heads + kvh) * a.blocks;
    for (int b = lane; b < first; b += 64) odd_list |= odd[b] != 0;
    odd_list = __any(odd_list);
    odd += first;
    death = a.death + static_cast<int64_t>(r) * a.n_pad + k0;
    const int64_t at = static_cast<int64_t>(r) * a.list_keys() + a.list_at(e);
    list = a.list + at;
    list_blocks = a.list_blocks + at / kTrainBlock;
    listed = e == 0 ? 0 : (a.list_count[static_cast<int64_t>(r) * a.epochs + e] + kTrainBlock - 1) / kTrainBlock;
    blocks = listed + (q1 - k0) / kTrainBlock + 1;
  }
  __device__ __forceinline__ void look(int lane) {
    const int b = base + lane, own = b - listed;
    KeyBlock x{0, -1};
    if (b < listed) x = list_blocks[b];
    else if (b < blocks) x = keys[own];
    const bool some = x.last > q0;
    const bool all = some && x.first > q1 && (own < 0 || k0 + own * kTrainBlock + kTrainBlock - 1 <= q0);
    bool bad = false;
    if (some && !all) bad = own < 0 ? odd_list : odd[own] != 0;
    seen = __ballot(some);
    whole = __ballot(all);
    rows_only |= __any(bad);
  }
  // The next block, or -1; `all`: every query sees every key of it.
  __device__ __forceinline__ int next(bool* all, int lane) {
    while (seen == 0) {
      base += 64;
      if (base >= blocks) return -1;
      look(lane);
    }
    const int x = __builtin_ctzll(seen);
    seen &= seen - 1;
    *all = whole >> x & 1;
    return base + x;
  }
  // Key `lane` of block b and its death time (not above its number: nobody sees it).
  __device__ __forceinline__ KeyEntry key(int b, int lane) const {
    if (b < listed) return list[b * kTrainBlock + lane];
    const int i = (b - listed) * kTrainBlock + lane;
    return KeyEntry{k0 + i, k0 + i < n_pad ? death[i] : -1};
  }
  // The row to read for it.  A key that nobody sees may hold anything: its place reads
  // another key's row.
  static __device__ __forceinline__ int row_of(KeyEntry x, int lane) {
    const uint64_t some = __ballot(x.death > x.key);
    const int other = __shfl(x.key, some ? __builtin_ctzll(some) : 0);
    return some >> lane & 1 ? x.key : other;
  }
  // What the place of a block's key adds to its number for the comparison with a query:
  // listed keys come before every query of the epoch.
  __device__ __forceinline__ int first_key(int b) const { return b < listed ? -kTrainBlock : k0 + (b - listed) * kTrainBlock; }
};

}  // namespace
}  // namespace ll
