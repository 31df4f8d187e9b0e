// gfx950 kernels of the trainer's attention (kvs_attend): query q sees key k iff
// k <= q < death[k];
//   s_k = scale * q . k  (or cap * tanh(scale * q . k / cap)),
//   out = sum_k softmax(s)_k v_k,  lse = log sum_k exp s_k,
// in one pass over the keys that keeps the running maximum, sum and weighted values in
// float32.  Scores are kept in base 2.
#include <algorithm>

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

constexpr int kScanThreads = 1024;
constexpr int kScanWaves = kScanThreads / 64;

// Keys chosen in order: each wave looks at 512 consecutive ones, `pick` says which go to
// which place.
struct Picked {
  int count = 0;   // so far, the same in every thread
};
template <typename Is, typename Put>
__device__ __forceinline__ void pick_in_order(int n, uint32_t (*totals)[kScanWaves], Picked& p, Is&& is, Put&& put) {
  constexpr int E = 8;
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  int at = 0;
  for (int base = 0; base < n; base += kScanThreads * E, at ^= 1) {
    uint64_t mine[E];
    int death[E], sum = 0;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int k = base + (wave * E + e) * 64 + lane;
      mine[e] = __ballot(k < n && is(k, &death[e]));
      sum += __popcll(mine[e]);
    }
    if (lane == 0) totals[at][wave] = sum;
    __syncthreads();
    int o = p.count;
#pragma unroll
    for (int x = 0; x < kScanWaves; ++x) {
      if (x < wave) o += totals[at][x];
      p.count += totals[at][x];
    }
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int k = base + (wave * E + e) * 64 + lane;
      if (mine[e] >> lane & 1) put(o + __popcll(mine[e] & ((uint64_t{1} << lane) - 1)), k, death[e]);
      o += __popcll(mine[e]);
    }
  }
  __syncthreads();   // the totals may be used again
}

// Epoch e's list of keys and what its blocks hold; for the backward pass the keys that
// die in the epoch in their places of the order (e = epochs: those that nobody sees).  A
// workgroup each, which goes through all death times of the rollout (a few microseconds).
template <bool BACKWARD>
__device__ void list_keys(const TrainLaunch& a, int r, int e, uint32_t (*totals)[kScanWaves]) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int32_t* const death = a.death + static_cast<int64_t>(r) * a.n_pad;
  const int64_t from64 = static_cast<int64_t>(e) * a.epoch, end64 = from64 + a.epoch;
  const int from = static_cast<int>(min(from64, static_cast<int64_t>(a.n_pad))), end = static_cast<int>(min(end64, static_cast<int64_t>(a.n_pad)));
  if (e > 0 && e < a.epochs) {
    const int64_t at = static_cast<int64_t>(r) * a.list_keys() + a.list_at(e);
    KeyEntry* const list = a.list + at;
    Picked p;
    pick_in_order(from, totals, p,
                  [&](int k, int* d) {
                    *d = min(death[k], a.n_pad);
                    return *d > from;
                  },
                  [&](int i, int k, int d) { list[i] = KeyEntry{k, d}; });
    const int blocks = (p.count + kTrainBlock - 1) / kTrainBlock;
    for (int i = p.count + threadIdx.x; i < blocks * kTrainBlock; i += kScanThreads) list[i] = KeyEntry{0, -1};
    if (threadIdx.x == 0) a.list_count[static_cast<int64_t>(r) * a.epochs + e] = p.count;
    __syncthreads();   // the list is written
    for (int b = wave; b < blocks; b += kScanWaves) {
      int first = list[b * kTrainBlock + lane].death, last = first;
      for (int x = 32; x >= 1; x >>= 1) {
        first = min(first, __shfl_xor(first, x));
        last = max(last, __shfl_xor(last, x));
      }
      if (lane == 0) a.list_blocks[at / kTrainBlock + b] = KeyBlock{first, last};
    }
  }
  if constexpr (BACKWARD) {
    int32_t* const order = a.order + static_cast<int64_t>(r) * a.n_pad;
    // those before: they die after this epoch (for the last place: all that are seen)
    const int after = e == a.epochs ? 0 : end;
    __shared__ int64_t pairs[kScanWaves];
    int before = 0;
    int64_t sees = 0;
    for (int k = threadIdx.x; k < a.n_pad; k += kScanThreads) {
      const int d = min(death[k], a.n_pad);
      before += d > k && d > after;
      sees += d > k ? d - k : 0;   // (a death time may lie 2^31 before its key)
    }
    for (int x = 32; x >= 1; x >>= 1) {
      before += __shfl_xor(before, x);
      sees += __shfl_xor(sees, x);
    }
    if (lane == 0) {
      totals[0][wave] = before;
      pairs[wave] = sees;
    }
    __syncthreads();
    Picked p;
    sees = 0;
    for (int x = 0; x < kScanWaves; ++x) {
      p.count += totals[0][x];
      sees += pairs[x];
    }
    __syncthreads();
    if (e == a.epochs && threadIdx.x == 0) {
      a.seen_keys[r] = p.count;
      a.work[r] = sees;
    }
    pick_in_order(e == a.epochs ? a.n_pad : end, totals, p,
                  [&](int k, int*) {
                    const int d = min(death[k], a.n_pad);
                    return e == a.epochs ? d <= k : d > k && d > from && d <= end;
                  },
                  [&](int i, int k, int) { order[i] = k; });
  }
}

// What the workspace says of keys and of blocks of 64 tokens, and for the backward pass
// delta.  Workgroups: first the epochs' lists; then a wave per block and unit: 0 the
// keys' death times; the KV heads' values; backward also their keys, every head's dout
// (with delta) and its queries.  This dispatch begins with workgroup `first_group`.
template <bool BACKWARD>
__global__ __launch_bounds__(kScanThreads) void train_scan_kernel(TrainLaunch a, int first_group) {
  __shared__ uint32_t totals[2][kScanWaves];
  const int lane = threadIdx.x & 63, group = first_group + static_cast<int>(blockIdx.x);
  const int lists = a.n * (a.epochs + BACKWARD);
  if (group < lists) {
    list_keys<BACKWARD>(a, group % a.n, a.epochs + BACKWARD - 1 - group / a.n, totals);
    return;
  }
  const int units = 1 + (BACKWARD ? 2 * a.kv_heads + 2 * a.heads : a.kv_heads);
  int64_t id = static_cast<int64_t>(group - lists) * kScanWaves + (threadIdx.x >> 6);
  const int b = static_cast<int>(id % a.blocks);
  id /= a.blocks;
  const int r = static_cast<int>(id / units);
  int unit = static_cast<int>(id % units);
  if (r >= a.n) return;
  const int t0 = b * kTrainBlock, rows = min(kTrainBlock, a.n_pad - t0);
  if (unit == 0) {
    int first = -1, last = -1;
    if (lane < rows) {
      const int d = min(a.death[static_cast<int64_t>(r) * a.n_pad + t0 + lane], a.n_pad);
      first = last = d > t0 + lane ? d : -1;
    }
    for (int x = 32; x >= 1; x >>= 1) {
      first = min(first, __shfl_xor(first, x));
      last = max(last, __shfl_xor(last, x));
    }
    if (lane == 0) a.keys[static_cast<int64_t>(r) * a.blocks + b] = KeyBlock{first, last};
    return;
  }
  --unit;
  const int64_t kv_at = static_cast<int64_t>(r) * a.kv_heads * a.blocks + b, at_ = static_cast<int64_t>(r) * a.heads * a.blocks + b;
  Heads x, y{};
  uint32_t* odd;
  int width = a.dv, h;
  bool sum = false, keys = true;
  if (unit < a.kv_heads) {
    x = a.v, h = unit, odd = a.odd_v + kv_at + static_cast<int64_t>(h) * a.blocks;
  } else if ((unit -= a.kv_heads) < a.kv_heads) {
    x = a.k, h = unit, odd = a.odd_k + kv_at + static_cast<int64_t>(h) * a.blocks, width = a.dk;
  } else if ((unit -= a.kv_heads) < a.heads) {
    x = a.dout, y = a.out, h = unit, odd = a.odd_do + at_ + static_cast<int64_t>(h) * a.blocks, sum = true, keys = false;
  } else {
    unit -= a.heads;
    x = a.q, h = unit, odd = a.odd_q + at_ + static_cast<int64_t>(h) * a.blocks, width = a.dk, keys = false;
  }
  // 8, 16 or 32 lanes a row, eight rows of a lane on their way at once (one at a time,
  // each waited for: 23 us instead of 18 for 3 x 389 tokens of 3 x 5 heads of 96)
  constexpr int AT_ONCE = 8;
  const int shift = width <= 64 ? 3 : width <= 128 ? 4 : 5, c = (lane & ((1 << shift) - 1)) * 8, per = 64 >> shift;
  uint32_t bits = 0;
  for (int g = lane >> shift; g < kTrainBlock; g += AT_ONCE * per) {   // (whole waves: the sums go across lanes)
    chunk_t v[AT_ONCE], w[AT_ONCE];
    int death[AT_ONCE];
    float lse[AT_ONCE];
#pragma unroll
    for (int i = 0; i < AT_ONCE; ++i) {
      const int t = t0 + min(g + i * per, rows - 1), at_c = c < width ? c : 0;
      v[i] = *reinterpret_cast<const chunk_t*>(at(x, r, t, h) + at_c);
      if (keys) death[i] = a.death[static_cast<int64_t>(r) * a.n_pad + t];
      if (BACKWARD && sum) {
        w[i] = *reinterpret_cast<const chunk_t*>(at(y, r, t, h) + at_c);
        lse[i] = a.lse[(static_cast<int64_t>(r) * a.n_pad + t) * a.heads + h];
      }
    }
#pragma unroll
    for (int i = 0; i < AT_ONCE; ++i) {
      const int t = g + i * per;
      const bool live = t < rows && c < width;
      if (live && !(keys && death[i] <= t0 + t)) bits |= exponents(v[i]);   // (a key that nobody sees may hold anything)
      if (BACKWARD && sum) {
        float d = live ? dot8(vals_of(v[i]), vals_of(w[i])) : 0.f;
        for (int k = 1 << shift >> 1; k >= 1; k >>= 1) d += __shfl_xor(d, k);
        if (c == 0 && t < rows) {
          const int64_t to = (static_cast<int64_t>(r) * a.heads + h) * a.n_pad + t0 + t;
          a.delta[to] = d;
          a.ref[to] = lse[i] == -__builtin_inff() ? __builtin_inff() : lse[i] * kLog2e;   // no weight: every p is 0
        }
      }
    }
  }
  const bool any = __any((bits & kNotFinite) != 0);
  if (lane == 0) *odd = any;
}

// The flash kernel.  A workgroup takes 32 * WAVES queries of a head, a wave 32 of them,
// and goes through the keys that some of them see, BN at a time, which it reads into LDS
// while it works on those before.  Scores are computed transposed (S^T = K Q^T), so that
// a lane holds 16 keys' scores of one query: the softmax runs along a lane's own
// registers (and the lane 32 further), and the weights, rounded to bf16, are the operand
// of O^T = V^T P^T as they lie.  V^T comes from the transposing LDS reads.
//
// The running maximum is only a reference: it moves when a score (in base 2) exceeds it
// by more than 8, so weights stay below 2^8 and most tiles scale nothing.
//
// Bound by the matrix and the vector instructions of the same waves (30% and 62% of the
// time), of which registers hold two a SIMD (one where heads are 256 wide): 2 x 8192 tokens,
// 8 KV heads, 32 of 128, cut every 2048 and capped, 1.00 ms, the call with its scan 1.02:
// 670 TFLOP/s of the pairs that are seen; 8192 tokens
// uncut 650 to 840 (500 where heads are 256 wide).  Tiles of 64 keys, 32 where heads are
// wider than 128, for two stages and two workgroups in LDS.
template <int DK, int DV, int BN, int WAVES, bool CAP>
__global__ __launch_bounds__(64 * WAVES) __attribute__((amdgpu_waves_per_eu(DK > 192 ? 1 : 2))) void train_kernel(TrainLaunch a) {
  extern __shared__ __attribute__((aligned(1024))) char smem[];
  using KR = Rows<DK>;
  using VR = Rows<DV>;
  constexpr int STAGE = BN * (KR::BYTES + VR::BYTES) + kTrainBlock * 4;   // keys, values, death times
  constexpr int KB = BN / 32, KK = DK / 16, DB = DV / 32, PARTS = kTrainBlock / BN;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  // the heads of one KV head and rollout side by side, the longest tiles first
  const int pairs = a.n * a.kv_heads, pair = blockIdx.x % pairs, rest = blockIdx.x / pairs;
  const int r = pair / a.kv_heads, kvh = pair % a.kv_heads, h = kvh * a.group + rest % a.group;
  const int tiles = (a.n_pad + 32 * WAVES - 1) / (32 * WAVES), tile = tiles - 1 - rest / a.group;
  const int q0 = tile * 32 * WAVES, q1 = min(q0 + 32 * WAVES, a.n_pad) - 1;
  const int mine = q0 + wave * 32 + (lane & 31);   // this lane's query
  const lds_ptr lds = (lds_ptr)smem;
  const int live_k = a.dk / 8, live_v = a.dv / 8;
  const uint16_t* const kp = at(a.k, r, 0, kvh);
  const uint16_t* const vp = at(a.v, r, 0, kvh);

  bf16x8 q[KK];
  load_operand(q, at(a.q, r, min(mine, a.n_pad - 1), h), mine < a.n_pad, live_k, lane);
  const float c = fold_scale<CAP>(q, a.scale, a.cap);
  const float c2 = CAP ? 1.f : c;
  const Tanh capped(c, a.cap * kLog2e);

  if (live_k < KR::CH || live_v < VR::CH) {
    for (int i = threadIdx.x; i < 2 * STAGE / 16; i += 64 * WAVES) reinterpret_cast<chunk_t*>(smem)[i] = chunk_t{0u, 0u, 0u, 0u};
    __syncthreads();
  }
  auto load = [&](KeyEntry key, int part, int stage) {
    const lds_ptr dst = lds + stage * STAGE;
    const int row = KeyWalk::row_of(key, lane);
    KR::template load<BN, WAVES>(dst, kp, a.k.ts, row, part * BN, live_k, wave, lane);
    VR::template load<BN, WAVES>(dst + BN * KR::BYTES, vp, a.v.ts, row, part * BN, live_v, wave, lane);
    if (wave == 0) reinterpret_cast<int*>(smem + stage * STAGE + BN * (KR::BYTES + VR::BYTES))[lane] = key.death;   // the whole block's
  };

  f32x16 o[DB];
#pragma unroll
  for (int d = 0; d < DB; ++d)
#pragma unroll
    for (int i = 0; i < 16; ++i) o[d][i] = 0.f;
  float m = -__builtin_inff(), l = 0.f;

  // tiles of a block's keys: this one, the next one (on its way), and the block after
  // that, whose keys are known a tile before they are asked for
  KeyWalk walk(a, r, kvh, a.odd_v, q0, q1, lane);
  bool all = false, next_all = false, then_all = false;
  int block = walk.next(&all, lane), next = -1, part = 0, stage = 0;
  KeyEntry key{}, next_key{};
  if (block >= 0) {
    key = walk.key(block, lane);
    load(key, 0, 0);
    next = walk.next(&next_all, lane);
    if (next >= 0) next_key = walk.key(next, lane);
  }
  const int k_at = KR::straight_at(lane), v_at = VR::columns_at(lane);
  while (block >= 0 && !walk.rows_only) {
    const bool ends = part == PARTS - 1;   // the block's last tile
    const int then = ends && next >= 0 ? walk.next(&then_all, lane) : -1;
    __builtin_amdgcn_s_waitcnt(0x0F70);   // vmcnt(0): this wave's part of the tile
    __syncthreads();                      // everyone's; and nobody reads the other stage any more
    KeyEntry then_key{};
    if (!ends) {
      load(key, part + 1, stage ^ 1);
    } else if (next >= 0) {
      load(next_key, 0, stage ^ 1);
      if (then >= 0) then_key = walk.key(then, lane);
    }
    const uint32_t ks = tile_at(lds + stage * STAGE, k_at), vs = tile_at(lds + stage * STAGE + BN * KR::BYTES, v_at);
    const int k0 = walk.first_key(block);

    f32x16 s[KB];
#pragma unroll
    for (int b = 0; b < KB; ++b) {
#pragma unroll
      for (int i = 0; i < 16; ++i) s[b][i] = 0.f;
#pragma unroll
      for (int k = 0; k < KK; ++k) s[b] = mfma(KR::straight(ks, b * 32, k), q[k], s[b]);
    }
#pragma unroll
    for (int b = 0; b < KB; ++b) {
      if constexpr (CAP) tanh_all(s[b], capped);
      if (!all) {
        const uint32_t seen = seen_bits(smem + stage * STAGE + BN * (KR::BYTES + VR::BYTES), part * BN + b * 32, k0, mine, lane);
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if (!(seen >> i & 1)) s[b][i] = -__builtin_inff();
      }
    }
    float top = -__builtin_inff();
#pragma unroll
    for (int b = 0; b < KB; ++b)
#pragma unroll
      for (int i = 0; i < 16; ++i) top = fmaxf(top, s[b][i]);
    top *= c2;
    if (__any(top > m + 8.f)) {
      const float x = fmaxf(fmaxf(top, m), __shfl_xor(fmaxf(top, m), 32));
      const float keep = x == m ? 1.f : exp2_(m - x);
      m = x;
      l *= keep;
#pragma unroll
      for (int d = 0; d < DB; ++d) o[d] *= keep;
    }
    const float ref = m == -__builtin_inff() ? 0.f : m;   // nothing seen yet: every weight is 0
#pragma unroll
    for (int b = 0; b < KB; ++b) {
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        s[b][i] = exp2_(__builtin_fmaf(s[b][i], c2, -ref));
        l += s[b][i];
      }
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const bf16x8 p = operand(s[b], x);
#pragma unroll
        for (int d = 0; d < DB; ++d) o[d] = mfma(VR::columns(vs, b * 32 + x * 16, d), p, o[d]);
      }
    }
    stage ^= 1;
    if (!ends) {
      ++part;
    } else {
      block = next, all = next_all, key = next_key, part = 0;
      next = then, next_all = then_all, next_key = then_key;
    }
  }
  __builtin_amdgcn_s_waitcnt(0x0F70);   // loads on their way into LDS
  if (walk.rows_only) {
    for (int i = q0 + wave; i <= q1; i += WAVES) train_row(a, r, i, h, lane);
    return;
  }
  l += __shfl_xor(l, 32);
  if (mine >= a.n_pad) return;
  const float inv = l == 0.f ? 0.f : 1.f / l;
  uint16_t* const out = place(a.out, r, mine, h);
#pragma unroll
  for (int d = 0; d < DB; ++d)
#pragma unroll
    for (int i = 0; i < 16; i += 4) {
      const int col = d * 32 + product_row(i, lane);
      f32x4 x{o[d][i], o[d][i + 1], o[d][i + 2], o[d][i + 3]};
      // no weight at all: 0, whatever the sum holds (0 times an infinity)
      x = l == 0.f ? f32x4{0.f, 0.f, 0.f, 0.f} : x * inv;
      if (col < a.dv) *reinterpret_cast<bf16x4*>(out + col) = __builtin_convertvector(x, bf16x4);
    }
  if (lane < 32)
    a.lse[(static_cast<int64_t>(r) * a.n_pad + mine) * a.heads + h] = l == 0.f ? -__builtin_inff() : (m + __log2f(l)) * kLn2;
}

template <int DK, int DV, int BN, int WAVES, bool CAP>
hipError_t launch_shape(const TrainLaunch& a, hipStream_t s) {
  constexpr int lds = 2 * (BN * (DK + DV) * 2 + kTrainBlock * 4);
  hipError_t e = allow_lds<train_kernel<DK, DV, BN, WAVES, CAP>>(lds);
  if (e != hipSuccess) return e;
  const int64_t groups = int64_t{a.n} * a.heads * ((a.n_pad + 32 * WAVES - 1) / (32 * WAVES));
  train_kernel<DK, DV, BN, WAVES, CAP><<<dim3(static_cast<unsigned>(groups)), dim3(64 * WAVES), lds, s>>>(a);
  return hipGetLastError();
}

template <int DK, int DV, int BN, int WAVES>
hipError_t launch_cap(const TrainLaunch& a, hipStream_t s) {
  return a.cap == 0.f ? launch_shape<DK, DV, BN, WAVES, false>(a, s) : launch_shape<DK, DV, BN, WAVES, true>(a, s);
}

}  // namespace

// As many dispatches as it takes: many short rollouts have more work-items than the 2^32 - 1
// that one holds.
hipError_t launch_train_scan(const TrainLaunch& a, bool backward, hipStream_t s) {
  constexpr int64_t most = 0xFFFFFFFFll / kScanThreads;
  const int64_t units = 1 + (backward ? 2 * a.kv_heads + 2 * a.heads : a.kv_heads);
  const int64_t lists = int64_t{a.n} * (a.epochs + (backward ? 1 : 0));
  const int64_t groups = lists + (a.n * units * a.blocks + kScanWaves - 1) / kScanWaves;
  for (int64_t at = 0; at < groups; at += most) {
    const dim3 g(static_cast<unsigned>(std::min(groups - at, most)));
    if (backward) train_scan_kernel<true><<<g, dim3(kScanThreads), 0, s>>>(a, static_cast<int>(at));
    else train_scan_kernel<false><<<g, dim3(kScanThreads), 0, s>>>(a, static_cast<int>(at));
    if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  }
  return hipSuccess;
}

hipError_t launch_train(const TrainLaunch& a, hipStream_t s) {
  hipError_t e = launch_train_scan(a, false, s);
  if (e != hipSuccess) return e;
  switch (head_shape(a.dk, a.dv).dk) {
    case 64: return launch_cap<64, 64, 64, 4>(a, s);
    case 128: return launch_cap<128, 128, 64, 4>(a, s);
    case 192: return launch_cap<192, 128, 32, 4>(a, s);
    default: return launch_cap<256, 256, 32, 4>(a, s);
  }
}

}  // namespace ll
