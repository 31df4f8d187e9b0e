// gfx950 kernels of the gradients of the trainer's attention (kvs_attend_backward):
// with p = exp(s - lse) over the keys that a query sees,
//   delta = sum_d dout out,  ds = p (dout . v - delta) scale (1 - tanh^2),
//   dv = sum_q p dout,  dk = sum_q ds q,  dq = sum_k ds k,
// dk and dv summed over the heads that share a KV head.  Weights are worked out again
// from lse; one kernel goes along the keys of a query for dq, another along the queries
// of a key for dk and dv, so that each sum has one owner and one order.
//
// The out that comes is rounded to bf16, and delta from it is off by as much; where few
// keys hold a query's weight, dout . v - delta cancels, and that error is what is left.
// Since the weights sum to 1, sum_k p (dout . v - delta) is what delta lacks: the dq kernel
// adds that sum, and dk and dv are worked out with the delta that it corrected.  dq itself
// takes the query's weighted mean key, sum_k p k, off its keys: sum_k ds k is the same for
// the ds of the formula, whose sum is 0 (under a cap only what the sum is off by is taken
// off), and neither an error of delta nor what ds is rounded by then counts with what the
// keys share, or with the one key that holds the weight.  ds and p are rounded to bf16 for
// the products after them, half a step (2^-8) of each.
#include "train_common.h"

namespace ll {
namespace {

// x's values and c.
__device__ __forceinline__ float sum8(bf16x8 x, float c) {
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  const bf16x2 ones = {static_cast<__bf16>(1.f), static_cast<__bf16>(1.f)};
#pragma unroll
  for (int i = 0; i < 8; i += 2) c = __builtin_amdgcn_fdot2_f32_bf16(bf16x2{x[i], x[i + 1]}, ones, c, false);
  return c;
}

constexpr int AH = 3;   // steps that a product's operands are read ahead (5: 2% slower)

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
  float* const at_delta = a.delta + (static_cast<int64_t>(r) * a.heads + h) * a.n_pad + q;
  float delta = *at_delta, lacks = 0.f;
  Vals o{};
  if (lse != -__builtin_inff())
    for (int pass = 0; pass < 2; ++pass) {   // the sum of p (dp - delta), then of ds k
      for (int k = 0; k <= q; ++k) {
        if (death[k] <= q) continue;
        const Vals y = load8(at(a.k, r, k, kvh) + lane * 8, lk);
        const float s = wave_sum(dot8(x, y));
        const float dp = wave_sum(dot8(g, load8(at(a.v, r, k, kvh) + lane * 8, lv)));
        const Pair w = pair_of(a, s, dp, lse, delta);
        if (pass == 0)
          lacks += w.p * (dp - delta);
        else
          add8(o, w.ds, y);
      }
      if (pass == 0) delta += lacks;
    }
  if (lane == 0) *at_delta = delta;
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

// A product's values as weights and their gradients: p from the score (s: scaled or
// under the cap's tanh already; c2 to base 2), ds from dp.  What is not seen counts 0.
//
// dq: a workgroup takes 32 * WAVES queries of a head and goes along the keys that they
// see, as the forward kernel does: S^T = K Q^T and dP^T = V dO^T with the queries in
// registers, then dQ^T += K^T dS^T and the weighted mean key's K^T W^T, K^T from the
// transposing LDS reads, once for both.
// GLDS: dO lies in LDS, where the registers of two waves a SIMD hold no more (keys are
// then taken 32 at a time, so that two workgroups fit).
// Bound by its registers: two waves a SIMD, one where heads are wider than 128 (2 x 4096
// tokens, 8 KV heads, 32 of 128, cut every 1024: 376 us, matrix units busy 43% and vector
// units 47% of the time; 4001 tokens of 16 heads of 192 / 128, capped: 274 us, 30% and
// 42%).  One wave a SIMD for heads of 128, 64 keys at a time: the whole call 8% slower.
// With w = p (under a cap p times its slope), rounded to w~, and ds from delta and rounded
// to ds~, what delta lacks is L = sum p (dp - delta), and
//   dq = sum ds~ k - (sum ds~ - sum ds + L sum w) / sum w~ * sum w~ k;
// without a cap sum ds is L and sum w is 1.  The rounded sums are those of the products'
// own operands, so that a key with nearly all weight drops out whatever it was rounded by.
// (Going along the keys again with the corrected delta instead leaves the rounding of ds
// times what the keys share: 0.005 of dq where each key value's mean is 3 standard
// deviations.)
template <int DK, int DV, int BN, int WAVES, bool GLDS, bool CAP>
__global__ __launch_bounds__(64 * WAVES) __attribute__((amdgpu_waves_per_eu(DK > 128 ? 1 : 2))) void train_dq_kernel(TrainLaunch a) {
  extern __shared__ __attribute__((aligned(1024))) char smem[];
  using KR = Rows<DK>;
  using VR = Rows<DV>;
  constexpr int STAGE = BN * (KR::BYTES + VR::BYTES) + kTrainBlock * 4;   // keys, values, death times
  constexpr int DOUT = 2 * STAGE;   // where dO lies
  constexpr int KB = BN / 32, KK = DK / 16, VK = DV / 16, DB = DK / 32, PARTS = kTrainBlock / BN;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) & (WAVES - 1);
  const int pairs = a.n * a.kv_heads, pair = blockIdx.x % pairs, rest = blockIdx.x / pairs;
  const int r = pair / a.kv_heads, kvh = pair % a.kv_heads, h = kvh * a.group + rest % a.group;
  const int tiles = (a.n_pad + 32 * WAVES - 1) / (32 * WAVES), tile = tiles - 1 - rest / a.group;
  const int q0 = tile * 32 * WAVES, q1 = min(q0 + 32 * WAVES, a.n_pad) - 1;
  const int mine = q0 + wave * 32 + (lane & 31), row = min(mine, a.n_pad - 1);
  const lds_ptr lds = (lds_ptr)smem;
  const int live_k = a.dk / 8, live_v = a.dv / 8;
  const uint16_t* const kp = at(a.k, r, 0, kvh);
  const uint16_t* const vp = at(a.v, r, 0, kvh);

  bf16x8 q[KK], g[GLDS ? 1 : VK];
  load_operand(q, at(a.q, r, row, h), mine < a.n_pad, live_k, lane);
  if constexpr (!GLDS) load_operand(g, at(a.dout, r, row, h), mine < a.n_pad, live_v, lane);
  const float c = fold_scale<CAP>(q, a.scale, a.cap);
  const float c2 = CAP ? a.cap * kLog2e : c;
  const Tanh capped(c, 1.f);
  const int64_t at_row = (static_cast<int64_t>(r) * a.heads + h) * a.n_pad + row;
  const float ref = a.ref[at_row], delta = a.delta[at_row];

  if (live_k < KR::CH || live_v < VR::CH) {
    for (int i = threadIdx.x; i < DOUT / 16; i += 64 * WAVES) reinterpret_cast<chunk_t*>(smem)[i] = chunk_t{0u, 0u, 0u, 0u};
    if (GLDS) for (int i = threadIdx.x; i < 32 * WAVES * VR::BYTES / 16; i += 64 * WAVES) reinterpret_cast<chunk_t*>(smem + DOUT)[i] = chunk_t{0u, 0u, 0u, 0u};
    __syncthreads();
  }
  if constexpr (GLDS) {   // (a wave reads its own rows: queries that are not there repeat the last one)
#pragma unroll
    for (int i = 0; i < WAVES / 2; ++i)
      VR::template load<64, WAVES>(lds + DOUT + i * 64 * VR::BYTES, at(a.dout, r, 0, h), a.dout.ts,
                                   min(q0 + i * 64 + lane, a.n_pad - 1), 0, live_v, wave, lane);
  }
  auto load = [&](KeyEntry key, int part, int stage) {
    const lds_ptr dst = lds + stage * STAGE;
    const int row = KeyWalk::row_of(key, lane);
    KR::template load<BN, WAVES>(dst, kp, a.k.ts, row, part * BN, live_k, wave, lane);
    VR::template load<BN, WAVES>(dst + BN * KR::BYTES, vp, a.v.ts, row, part * BN, live_v, wave, lane);
    if (wave == 0) reinterpret_cast<int*>(smem + stage * STAGE + BN * (KR::BYTES + VR::BYTES))[lane] = key.death;   // the whole block's
  };
  f32x16 o[DB], mean[DB];   // sums of ds~ k and of w~ k
  float lacks = 0.f, ds_sum = 0.f, w_sum = 0.f, ds_rounded = 0.f, w_rounded = 0.f;
#pragma unroll
  for (int d = 0; d < DB; ++d)
#pragma unroll
    for (int i = 0; i < 16; ++i) o[d][i] = mean[d][i] = 0.f;

  // tiles of a block's keys: this one, the next one (on its way), and the block after
  // that, whose keys are known a tile before they are asked for
  KeyWalk walk(a, r, kvh, a.odd_k, q0, q1, lane);
  bool all = false, next_all = false, then_all = false;
  int block = walk.next(&all, lane), next = -1, part = 0, stage = 0;
  KeyEntry key{}, next_key{};
  if (block >= 0) {
    key = walk.key(block, lane);
    load(key, 0, 0);
    next = walk.next(&next_all, lane);
    if (next >= 0) next_key = walk.key(next, lane);
  }
  const int k_at = KR::straight_at(lane), v_at = VR::straight_at(lane), c_at = KR::columns_at(lane);
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
    const lds_ptr keys = lds + stage * STAGE;
    const uint32_t ks = tile_at(keys, k_at), vs = tile_at(keys + BN * KR::BYTES, v_at), cs = tile_at(keys, c_at);
    const uint32_t gs = GLDS ? tile_at(lds + DOUT + wave * 32 * VR::BYTES, v_at) : 0u;
    const int k0 = walk.first_key(block);
#pragma unroll 1
    for (int b = 0; b < KB; ++b) {
      f32x16 s, dp;
#pragma unroll
      for (int i = 0; i < 16; ++i) s[i] = dp[i] = 0.f;
      stream<KK, AH>([&](int k) { return KR::straight(ks, b * 32, k); }, [&](int k, bf16x8 x) { s = mfma(x, q[k], s); });
      if constexpr (CAP) tanh_all(s, capped);
      if constexpr (GLDS) {
        bf16x8 z[2];
        stream<2 * VK, 4>([&](int x) { return x & 1 ? VR::straight(gs, 0, x / 2) : VR::straight(vs, b * 32, x / 2); },
                          [&](int x, bf16x8 y) {
                            z[x & 1] = y;
                            if (x & 1) dp = mfma(z[0], z[1], dp);
                          });
      } else {
        stream<VK, AH>([&](int k) { return VR::straight(vs, b * 32, k); }, [&](int k, bf16x8 x) { dp = mfma(x, g[k], dp); });
      }
      if (!all) {   // no weight and no ds for what is not seen (a tanh of -1 has no slope)
        const uint32_t seen = seen_bits(smem + stage * STAGE + BN * (KR::BYTES + VR::BYTES), part * BN + b * 32, k0, mine, lane);
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if (!(seen >> i & 1)) s[i] = CAP ? -1.f : -__builtin_inff(), dp[i] = delta;
      }
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        float p = exp2_(__builtin_fmaf(s[i], c2, -ref)), t = p * (dp[i] - delta);
        lacks += t;
        if constexpr (CAP) {
          const float slope = __builtin_fmaf(-s[i], s[i], 1.f);
          w_sum += p *= slope;
          ds_sum += t *= slope;
        }
        s[i] = p, dp[i] = t;
      }
      // (sums here and now: the compiler otherwise leaves them to the loop's end, and keeps what they add until then)
      asm volatile("" : "+v"(lacks));
      if constexpr (CAP) asm volatile("" : "+v"(w_sum), "+v"(ds_sum));
      const bf16x8 ds[2] = {operand(dp, 0), operand(dp, 1)}, w[2] = {operand(s, 0), operand(s, 1)};
#pragma unroll
      for (int x = 0; x < 2; ++x) ds_rounded = sum8(ds[x], ds_rounded), w_rounded = sum8(w[x], w_rounded);
      asm volatile("" : "+v"(ds_rounded), "+v"(w_rounded));
      __builtin_amdgcn_sched_barrier(0);
      stream<2 * DB, AH>([&](int x) { return KR::columns(cs, b * 32 + x / DB * 16, x % DB); },
                         [&](int x, bf16x8 y) {
                           o[x % DB] = mfma(y, ds[x / DB], o[x % DB]);
                           mean[x % DB] = mfma(y, w[x / DB], mean[x % DB]);
                         });
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
    for (int i = q0 + wave; i <= q1; i += WAVES) train_dq_row(a, r, i, h, lane);
    return;
  }
  auto both = [](float x) { return x + __shfl_xor(x, 32); };
  lacks = both(lacks), ds_rounded = both(ds_rounded), w_rounded = both(w_rounded);
  if constexpr (CAP) ds_rounded += lacks * both(w_sum) - both(ds_sum);
  const float by = w_rounded > 0.f ? ds_rounded / w_rounded : 0.f;   // (0: no key's weight is left)
  if (lane < 32 && mine < a.n_pad && ref < __builtin_inff()) a.delta[at_row] = delta + lacks;
  if (mine >= a.n_pad) return;
  uint16_t* const out = place(a.dq, r, mine, h);
#pragma unroll
  for (int d = 0; d < DB; ++d)
#pragma unroll
    for (int i = 0; i < 16; i += 4) {
      const int col = d * 32 + product_row(i, lane);
      f32x4 x = f32x4{o[d][i], o[d][i + 1], o[d][i + 2], o[d][i + 3]};
      x = (x - f32x4{mean[d][i], mean[d][i + 1], mean[d][i + 2], mean[d][i + 3]} * by) * a.scale;
      if (ref == __builtin_inff()) x = f32x4{0.f, 0.f, 0.f, 0.f};   // no weight at all, whatever the keys hold
      if (col < a.dk) *reinterpret_cast<bf16x4*>(out + col) = __builtin_convertvector(x, bf16x4);
    }
}

// dk and dv: a workgroup takes kTrainTile keys of a KV head in the order that the scan
// made, a wave 32 of them (K in registers, V in LDS or registers), and goes along the
// queries that see some of them, of each head that shares them, 32 * QW at a time through
// LDS, of which a wave takes 32: S = Q K^T and dP = dO V^T with a lane per key, then
// dV^T += dO^T P and dK^T += Q^T dS, dO^T and Q^T from the transposing LDS reads.  In the
// end the QW waves of the same keys add up.
// Matrix units busy 39% and vector units 55% of the time where two waves share a SIMD (2 x
// 4096 tokens, 8 KV heads, 32 of 128, cut every 1024: 559 us), 25% and 44% where registers
// hold one, whose exponentials nothing covers (4001 tokens of 16 heads of 192 / 128, capped:
// 310 us).
template <int DK, int DV, int QW, bool VLDS>
struct KeyShape {
  static constexpr int KW = kTrainTile / 32, WAVES = KW * QW, BN = 32 * QW;
  static constexpr int STAGE = BN * (DK + DV) * 2 + 2 * BN * 4;   // queries, dout, lse and delta
  static constexpr int VALUES = 2 * STAGE;                       // where V lies
  static constexpr int SUMS = QW > 1 ? KW * 32 * (DK > DV ? DK : DV) * 4 : 0;
  static constexpr int LDS = VALUES + (VLDS ? kTrainTile * DV * 2 : 0);
  static_assert(QW <= 2 && SUMS <= LDS && VALUES % 256 == 0, "the second wave's sums fit where the tiles were");
};

// Blocks of 64 queries that a share of a tile of keys takes.  A tile whose keys all live
// on goes along all queries of every head that shares them; where that is more than a
// compute unit's part of the whole work and a quarter, tiles are cut into shares of 0.6 of
// that part.  (2 x 4096 tokens, 8 KV heads, cut by evictions so that the longest tile is a
// third more than the part: whole 908 us, with shares 867.  4001 tokens of an MLA model,
// uncut, the longest as long as the part: whole 560, cut in two 605.)
constexpr int kUnits = 256, kShareBlocks = 6;   // compute units; blocks of a share at least
__device__ __forceinline__ int share_blocks(const TrainLaunch& a, int lane) {
  const int most = a.blocks * a.group;
  if (a.shares == 1) return most;
  int64_t pairs = 0;
  for (int r = lane; r < a.n; r += 64) pairs += a.work[r];
  for (int x = 32; x >= 1; x >>= 1) pairs += __shfl_xor(pairs, x);
  const float part = static_cast<float>(pairs) * a.heads / (kTrainTile * kTrainBlock * kUnits);
  if (most <= part * 1.25f) return most;
  const int chunk = max(max(static_cast<int>(part * 0.6f) + 1, kShareBlocks), (most + a.shares - 1) / a.shares);
  return __builtin_amdgcn_readfirstlane(min(chunk, most));
}

template <int DK, int DV, int QW, bool VLDS, int OCC, bool CAP>
__global__ __launch_bounds__(2 * kTrainTile * QW) __attribute__((amdgpu_waves_per_eu(OCC))) void train_dkv_kernel(TrainLaunch a) {
  extern __shared__ __attribute__((aligned(1024))) char smem[];
  using S = KeyShape<DK, DV, QW, VLDS>;
  using QR = Rows<DK>;
  using GR = Rows<DV>;
  constexpr int WAVES = S::WAVES, BN = S::BN, STAGE = S::STAGE;
  constexpr int KK = DK / 16, VK = DV / 16, KD = DK / 32, VD = DV / 32;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int kw = wave % S::KW, qw = wave / S::KW;
  const int pairs = a.n * a.kv_heads, pair = blockIdx.x % pairs;
  const int r = pair / a.kv_heads, kvh = pair % a.kv_heads;
  // (workgroups that a call does not need end before they look at anything else)
  const int chunk = share_blocks(a, lane);
  // The longest tiles first.  A tile's later shares may be short or empty; which of them
  // comes first changes from tile to tile, since workgroups go to the chip's parts in turn.
  const int tile = blockIdx.x / pairs / a.shares, share = (blockIdx.x / pairs + tile) % a.shares;
  if (share * chunk >= a.blocks * a.group) return;
  // places [p0, p0 + kTrainTile) of the keys' order: the first see the most queries
  const int p0 = tile * kTrainTile, place_ = p0 + kw * 32 + (lane & 31);
  const int32_t* const order = a.order + static_cast<int64_t>(r) * a.n_pad;
  const int32_t* const death = a.death + static_cast<int64_t>(r) * a.n_pad;
  const int mine = order[min(place_, a.n_pad - 1)];              // this lane's key
  const int some = min(a.n_pad, a.seen_keys[r]);                 // places of keys that somebody sees
  const bool there = place_ < some;
  const lds_ptr lds = (lds_ptr)smem;
  const int live_k = a.dk / 8, live_v = a.dv / 8;
  // of all keys of the workgroup: the last query that sees one, up to which all do, and
  // the first and last key
  int last = 0, first = INT32_MAX, k0 = INT32_MAX, k1 = 0, rows[kTrainTile / 64];
#pragma unroll
  for (int i = 0; i < kTrainTile / 64; ++i) {
    const int p = p0 + i * 64 + lane;
    const int key = order[min(p, a.n_pad - 1)], d = p < some ? min(death[key], a.n_pad) : 0;
    rows[i] = key;
    last = max(last, d);
    first = min(first, d);
    if (p < some) k0 = min(k0, key), k1 = max(k1, key);
  }
  for (int x = 32; x >= 1; x >>= 1) {
    last = max(last, __shfl_xor(last, x));
    first = min(first, __shfl_xor(first, x));
    k0 = min(k0, __shfl_xor(k0, x));
    k1 = max(k1, __shfl_xor(k1, x));
  }
  last = __builtin_amdgcn_readfirstlane(last);
  first = __builtin_amdgcn_readfirstlane(first);
  k0 = __builtin_amdgcn_readfirstlane(k0);
  k1 = __builtin_amdgcn_readfirstlane(k1);
  const int64_t slot = static_cast<int64_t>(pair) * ((a.n_pad + kTrainTile - 1) / kTrainTile) + tile;
  const int t0 = k0 - k0 % kTrainBlock, blocks = last > t0 ? (last - t0 + kTrainBlock - 1) / kTrainBlock : 0;
  const int cuts = max(1, (blocks * a.group + chunk - 1) / chunk);
  if (share >= cuts) return;
  const int end = there ? min(death[mine], a.n_pad) : mine;   // this lane's key is seen by queries [mine, end)

  bf16x8 k[KK], v[VLDS ? 1 : VK];
  load_operand(k, at(a.k, r, mine, kvh), there, live_k, lane);
  if constexpr (!VLDS) load_operand(v, at(a.v, r, mine, kvh), there, live_v, lane);
  const float c = fold_scale<CAP>(k, a.scale, a.cap);
  const float c2 = CAP ? a.cap * kLog2e : c;
  const Tanh capped(c, 1.f);
  if ((VLDS && p0 + kTrainTile > some) || live_k < QR::CH || live_v < GR::CH) {   // (V's places of keys that nobody sees stay 0)
    for (int i = threadIdx.x; i < S::LDS / 16; i += 64 * WAVES) reinterpret_cast<chunk_t*>(smem)[i] = chunk_t{0u, 0u, 0u, 0u};
    __syncthreads();
  }
  if constexpr (VLDS) {
#pragma unroll
    for (int i = 0; i < kTrainTile / 64; ++i)
      GR::template load<64, WAVES>(lds + S::VALUES + i * 64 * GR::BYTES, at(a.v, r, 0, kvh), a.v.ts, rows[i], 0, live_v, wave,
                                   lane, some - p0 - i * 64);
  }
  // a tile of queries that sees the keys in part, with a value that is not finite
  bool rows_only = false;
  for (int x = lane; x < a.group * blocks; x += 64) {
    const int b = t0 / kTrainBlock + x % blocks;
    const int64_t o = (static_cast<int64_t>(r) * a.heads + kvh * a.group + x / blocks) * a.blocks + b;
    const bool all = b * kTrainBlock >= k1 && b * kTrainBlock + kTrainBlock - 1 < first;
    if (!all && (a.odd_q[o] | a.odd_do[o])) rows_only = true;
  }
  rows_only = __any(rows_only);
  if (share == 0 && threadIdx.x == 0) a.used[slot] = rows_only ? 1 : cuts;
  if (rows_only) {
    __builtin_amdgcn_s_waitcnt(0x0F70);   // loads on their way into LDS
    if (share > 0) return;
    for (int i = p0 + wave; i < min(p0 + kTrainTile, a.n_pad); i += WAVES) train_dkv_row(a, r, order[i], kvh, lane);
    return;
  }
  // step i: queries [t0 + i % tiles * BN ...) of head i / tiles; this share's are
  // [begin, steps)
  const int per = kTrainBlock / BN, tiles = blocks * per, begin = share * chunk * per;
  const int steps = min(begin + chunk * per, tiles * a.group);
  auto load = [&](int i, int stage) {
    const lds_ptr dst = lds + stage * STAGE;
    const int h = kvh * a.group + i / tiles, row = min(t0 + i % tiles * BN + lane, a.n_pad - 1);
    QR::template load<BN, WAVES>(dst, at(a.q, r, 0, h), a.q.ts, row, 0, live_k, wave, lane);
    GR::template load<BN, WAVES>(dst + BN * QR::BYTES, at(a.dout, r, 0, h), a.dout.ts, row, 0, live_v, wave, lane);
    const int64_t q = (static_cast<int64_t>(r) * a.heads + h) * a.n_pad + row;
    if (wave < 2 && lane < BN) load_lds4(dst + BN * (QR::BYTES + GR::BYTES) + wave * BN * 4, (wave == 0 ? a.ref : a.delta) + q);
  };

  f32x16 gk[KD], gv[VD];
#pragma unroll
  for (int i = 0; i < 16; ++i) {
#pragma unroll
    for (int d = 0; d < KD; ++d) gk[d][i] = 0.f;
#pragma unroll
    for (int d = 0; d < VD; ++d) gv[d][i] = 0.f;
  }
  if (begin < steps) load(begin, 0);
  const int q_at = QR::straight_at(lane), g_at = GR::straight_at(lane), qc_at = QR::columns_at(lane), gc_at = GR::columns_at(lane);
  for (int i = begin; i < steps; ++i) {
    const int stage = (i - begin) & 1, q0 = t0 + i % tiles * BN;
    __builtin_amdgcn_s_waitcnt(0x0F70);
    __syncthreads();
    if (i + 1 < steps) load(i + 1, stage ^ 1);
    const lds_ptr qs = lds + stage * STAGE + qw * 32 * QR::BYTES, gs = lds + stage * STAGE + BN * QR::BYTES + qw * 32 * GR::BYTES;
    const uint32_t qa = tile_at(qs, q_at), ga = tile_at(gs, g_at), qc = tile_at(qs, qc_at), gc = tile_at(gs, gc_at);
    const uint32_t va = VLDS ? tile_at(lds + S::VALUES + kw * 32 * GR::BYTES, g_at) : 0u;
    const f32x4* const ls = reinterpret_cast<const f32x4*>(smem + stage * STAGE + BN * (QR::BYTES + GR::BYTES)) + qw * 8;
    const bool all = q0 >= k1 && q0 + BN - 1 < first;
    f32x16 s, dp;
#pragma unroll
    for (int x = 0; x < 16; ++x) s[x] = dp[x] = 0.f;
    stream<KK, AH>([&](int x) { return QR::straight(qa, 0, x); }, [&](int x, bf16x8 y) { s = mfma(y, k[x], s); });
    if constexpr (VLDS) {
      bf16x8 z[2];
      stream<2 * VK, 4>([&](int x) { return x & 1 ? GR::straight(va, 0, x / 2) : GR::straight(ga, 0, x / 2); },
                        [&](int x, bf16x8 y) {
                          z[x & 1] = y;
                          if (x & 1) dp = mfma(z[0], z[1], dp);
                        });
    } else {
      stream<VK, AH>([&](int x) { return GR::straight(ga, 0, x); }, [&](int x, bf16x8 y) { dp = mfma(y, v[x], dp); });
    }
    if constexpr (CAP) tanh_all(s, capped);
#pragma unroll
    for (int x = 0; x < 16; x += 4) {
      const f32x4 ref = ls[product_row(x, lane) / 4], delta = ls[BN / 4 + product_row(x, lane) / 4];
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        const float slope = CAP ? 1.f - s[x + y] * s[x + y] : 1.f;
        const float p = exp2_(__builtin_fmaf(s[x + y], c2, -ref[y]));
        dp[x + y] = p * (dp[x + y] - delta[y]) * slope;
        s[x + y] = p;
      }
    }
    if (!all) {
      uint32_t from = mine - q0 - qw * 32, n = end - mine;   // seen: queries [from, from + n) of the wave's 32
      asm volatile("" : "+v"(from), "+v"(n));                // (a branch around it, not a selection)
#pragma unroll
      for (int x = 0; x < 16; ++x)
        if (product_row(x, lane) - from >= n) s[x] = dp[x] = 0.f;
    }
    const bf16x8 p[2] = {operand(s, 0), operand(s, 1)}, ds[2] = {operand(dp, 0), operand(dp, 1)};
    __builtin_amdgcn_sched_barrier(0);
    stream<2 * (VD + KD), AH>(
        [&](int x) {
          return x < 2 * VD ? GR::columns(gc, x / VD * 16, x % VD)
                            : QR::columns(qc, (x - 2 * VD) / KD * 16, (x - 2 * VD) % KD);
        },
        [&](int x, bf16x8 y) {
          if (x < 2 * VD) gv[x % VD] = mfma(y, p[x / VD], gv[x % VD]);
          else gk[(x - 2 * VD) % KD] = mfma(y, ds[(x - 2 * VD) / KD], gk[(x - 2 * VD) % KD]);
        });
  }
  if constexpr (QW > 1) {
    // the other waves' sums through LDS, 16 bytes a lane at a time
    f32x4* const sums = reinterpret_cast<f32x4*>(smem) + kw * 32 * (DK > DV ? DK : DV) / 4;
    auto join = [&](auto& g) {
      constexpr int N = sizeof(g) / sizeof(f32x16);
      __syncthreads();
      if (qw == 1)
#pragma unroll
        for (int d = 0; d < N; ++d)
#pragma unroll
          for (int x = 0; x < 16; x += 4) sums[(d * 4 + x / 4) * 64 + lane] = f32x4{g[d][x], g[d][x + 1], g[d][x + 2], g[d][x + 3]};
      __syncthreads();
      if (qw == 0)
#pragma unroll
        for (int d = 0; d < N; ++d)
#pragma unroll
          for (int x = 0; x < 16; ++x) g[d][x] += sums[(d * 4 + x / 4) * 64 + lane][x & 3];
    };
    join(gk);
    join(gv);
  }
  if (qw > 0) return;
  if (cuts > 1) {
    // 16 bytes a lane at a time, which train_join_kernel adds up
    f32x4* const parts = reinterpret_cast<f32x4*>(a.parts) + (slot * a.shares + share) * (kTrainTile * (DK + DV) / 4);
    auto put = [&](f32x4* to, const f32x16& x) {
#pragma unroll
      for (int i = 0; i < 16; i += 4) __builtin_nontemporal_store(f32x4{x[i], x[i + 1], x[i + 2], x[i + 3]}, to + i / 4 * 64 + lane);
    };
#pragma unroll
    for (int d = 0; d < KD; ++d) put(parts + (kw * KD + d) * 256, gk[d]);
#pragma unroll
    for (int d = 0; d < VD; ++d) put(parts + kTrainTile * DK / 4 + (kw * VD + d) * 256, gv[d]);
    return;
  }
  if (place_ >= a.n_pad) return;
  auto store = [&](uint16_t* to, const f32x16& x, int d, int width, float by) {
#pragma unroll
    for (int i = 0; i < 16; i += 4) {
      const int col = d * 32 + product_row(i, lane);
      const f32x4 y{x[i], x[i + 1], x[i + 2], x[i + 3]};
      if (col < width) *reinterpret_cast<bf16x4*>(to + col) = __builtin_convertvector(y * by, bf16x4);
    }
  };
#pragma unroll
  for (int d = 0; d < KD; ++d) store(place(a.dk_, r, mine, kvh), gk[d], d, a.dk, a.scale);
#pragma unroll
  for (int d = 0; d < VD; ++d) store(place(a.dv_, r, mine, kvh), gv[d], d, a.dv, 1.f);
}

// The shares of a tile of keys added up in order, 4 values of a key per thread.
template <int DK, int DV>
__global__ __launch_bounds__(256) void train_join_kernel(TrainLaunch a) {
  constexpr int N = kTrainTile * (DK + DV) / 4, BLOCKS = N / 256;
  const int64_t slot = blockIdx.x / BLOCKS;
  const int cuts = a.used[slot];
  if (cuts <= 1) return;
  const int tiles = (a.n_pad + kTrainTile - 1) / kTrainTile, pair = static_cast<int>(slot / tiles);
  const int r = pair / a.kv_heads, kvh = pair % a.kv_heads;
  int i = blockIdx.x % BLOCKS * 256 + threadIdx.x;
  const f32x4* const p = reinterpret_cast<const f32x4*>(a.parts) + slot * a.shares * N + i;
  f32x4 sum = p[0];
  for (int c = 1; c < cuts; ++c) sum += p[static_cast<int64_t>(c) * N];
  const bool keys = i < kTrainTile * DK / 4;
  if (!keys) i -= kTrainTile * DK / 4;
  const int lane = i & 63, part = i >> 6, width = (keys ? DK : DV) / 8;   // parts of a wave's 32 keys
  const int at = static_cast<int>(slot % tiles) * kTrainTile + part / width * 32 + (lane & 31);
  const int col = part % width * 8 + (lane >> 5) * 4;
  if (at >= a.n_pad || col >= (keys ? a.dk : a.dv)) return;
  const int key = a.order[static_cast<int64_t>(r) * a.n_pad + at];
  if (keys) sum *= a.scale;
  *reinterpret_cast<bf16x4*>(place(keys ? a.dk_ : a.dv_, r, key, kvh) + col) = __builtin_convertvector(sum, bf16x4);
}

template <int DK, int DV, int BN, int QW, bool VLDS, int OCC, bool CAP>
hipError_t launch_shape(const TrainLaunch& a, hipStream_t s) {
  using K = KeyShape<DK, DV, QW, VLDS>;
  constexpr bool GLDS = DK == 128;
  constexpr int waves = kTrainTile / 32, lds = 2 * (BN * (DK + DV) * 2 + kTrainBlock * 4) + (GLDS ? kTrainTile * DV * 2 : 0);
  hipError_t e = allow_lds<train_dq_kernel<DK, DV, BN, waves, GLDS, CAP>>(lds);
  if (e == hipSuccess) e = allow_lds<train_dkv_kernel<DK, DV, QW, VLDS, OCC, CAP>>(K::LDS);
  if (e != hipSuccess) return e;
  const int64_t tiles = (a.n_pad + kTrainTile - 1) / kTrainTile;
  const dim3 queries(static_cast<unsigned>(a.n * a.heads * tiles));
  train_dq_kernel<DK, DV, BN, waves, GLDS, CAP><<<queries, dim3(64 * waves), lds, s>>>(a);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  train_dkv_kernel<DK, DV, QW, VLDS, OCC, CAP>
      <<<dim3(static_cast<unsigned>(a.n * a.kv_heads * tiles * a.shares)), dim3(64 * K::WAVES), K::LDS, s>>>(a);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (a.shares > 1) {
    constexpr int blocks = kTrainTile * (DK + DV) / 4 / 256;
    train_join_kernel<DK, DV><<<dim3(static_cast<unsigned>(a.n * a.kv_heads * tiles * blocks)), dim3(256), 0, s>>>(a);
    e = hipGetLastError();
  }
  return e;
}

template <int DK, int DV, int BN, int QW, bool VLDS, int OCC>
hipError_t launch_cap(const TrainLaunch& a, hipStream_t s) {
  return a.cap == 0.f ? launch_shape<DK, DV, BN, QW, VLDS, OCC, false>(a, s) : launch_shape<DK, DV, BN, QW, VLDS, OCC, true>(a, s);
}

}  // namespace

hipError_t launch_train_back(const TrainLaunch& a, hipStream_t s) {
  hipError_t e = launch_train_scan(a, true, s);
  if (e != hipSuccess) return e;
  switch (head_shape(a.dk, a.dv).dk) {
    case 64: return launch_cap<64, 64, 64, 2, false, 2>(a, s);
    case 128: return launch_cap<128, 128, 32, 2, true, 2>(a, s);
    case 192: return launch_cap<192, 128, 64, 1, true, 1>(a, s);
    default: return launch_cap<256, 256, 32, 1, true, 1>(a, s);
  }
}

}  // namespace ll
