// gfx950 kernel of the attention weight that cached rows get (ll_step_weigh):
//   W[j] = decay * W[j] + sum_t sum_h exp(s_thj - lse[t][h])
// over the step's tokens t that see row j, s the attention's scores (kernels_attend.hip).
#include <algorithm>

#include "matrix_common.h"
#include "weight_internal.h"

namespace ll {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));

constexpr int kWeighWaves = 4;
constexpr int kWeighRows = 32;   // query rows of a step
constexpr int64_t kWeighUnits = 1536;   // workgroups that long steps are cut into

// Bytes of a tile of query rows in LDS: the queries, their lse and what they see.
constexpr int weigh_stage(int d) { return (kWeighRows * (d * 2 + 12) + 255) / 256 * 256; }

// Bytes that a wave's keys pass through.
constexpr int weigh_keys(int d) { return kWeighRows * (d < 128 ? d : 128) * 2; }

// A wave takes 32 * KB cached rows, their keys of one KV head at a time in registers, and
// goes along the query rows that see some of them, 32 at a time through LDS, which the
// workgroup's waves share: S = Q K^T with a lane per cached row, so that the sum over
// query rows and heads stays in one register of the lane and one owner.  Single tokens
// are bound by reading the keys (the next head's are asked for before this one's are
// multiplied): 64 tokens over up to 16384 rows of 8 heads of 128 249 us, 5.4 TB/s.  Chunks
// are bound by the vector instructions of scores to weights, 27 for each matrix instruction
// with a cap: 3 x up to 1501 tokens over 8191 rows, 32 heads of 128, 470 us (vector units
// busy 69%, matrix units 21% of the time); without a cap and MLA, whose rows are longer, 657
// TFLOP/s.  Larger grids take several tiles a workgroup.
template <bool MLA, int DP, int KB, bool CAP>
__global__ __launch_bounds__(64 * kWeighWaves) __attribute__((amdgpu_waves_per_eu(!MLA && KB == 1 && DP <= 128 ? 3 : 2))) void weigh_kernel(WeighLaunch a) {
  constexpr int D = MLA ? kRowElems : DP, KK = D / 16, KEYS = 32 * KB * kWeighWaves;
  using R = Rows<D>;
  constexpr int LOADS = kWeighRows * R::CH / 64 / kWeighWaves;
  constexpr int TILE = kWeighRows * R::BYTES, STAGE = weigh_stage(D);
  extern __shared__ __attribute__((aligned(1024))) char smem[];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const lds_ptr lds = (lds_ptr)smem;
  const int live = MLA ? R::CH : a.dim / 8, seqs = a.counts->seqs;
  const int64_t tiles = (a.max_rows + KEYS - 1) / KEYS;
  const float c2 = CAP ? a.scale / a.cap : a.scale * kLog2e;
  const Tanh capped(c2, a.cap * kLog2e);
  const bool nothing = !(fabsf(c2) >= 1e-37f);   // a scale too small to tell scores apart counts as 0
  const int at = R::straight_at(lane);

  if (live < R::CH) {
    for (int i = threadIdx.x; i < 2 * STAGE / 16; i += 64 * kWeighWaves)
      reinterpret_cast<chunk_t*>(smem)[i] = chunk_t{0u, 0u, 0u, 0u};
    __syncthreads();
  }
  for (int64_t unit = blockIdx.x; unit < tiles * seqs * a.shares; unit += gridDim.x) {
    const int share = static_cast<int>(unit % a.shares), seq = static_cast<int>(unit / a.shares % seqs);
    const StepSeq s = a.seqs[seq];
    const int kv_len = s.row0 + s.count;
    const int64_t tile0 = unit / a.shares / seqs * KEYS;
    if (tile0 >= kv_len) continue;
    const int j0 = static_cast<int>(tile0), j1 = min(j0 + KEYS, kv_len) - 1;
    // the tokens that see some row of the tile, as query rows of a KV head
    const int t0 = a.causal ? max(0, j0 - s.row0) : 0;
    const int t1 = static_cast<int>(a.window > 0 ? min<int64_t>(s.count, int64_t{j1} + a.window - s.row0) : s.count);
    const int r0 = t0 * a.group, r1 = t1 * a.group;
    const int per = r1 > r0 ? (r1 - r0 + kWeighRows - 1) / kWeighRows : 0;
    // this share's steps: 32 query rows of a KV head each, one head after the other
    const int chunk = (per * a.kv_heads + a.shares - 1) / a.shares;
    const int begin = min(share * chunk, per * a.kv_heads), steps = min(begin + chunk, per * a.kv_heads);

    uint32_t row[KB];   // lane x of a half wave knows the physical row of a block's row x
#pragma unroll
    for (int b = 0; b < KB; ++b) {
      const int j = min(j0 + (wave * KB + b) * 32 + (lane & 31), kv_len - 1);
      int page = a.page_table[static_cast<int64_t>(s.seq) * a.max_pages_per_seq + (j >> a.page_shift)];
      if (static_cast<uint32_t>(page) >= static_cast<uint32_t>(a.num_pages)) page = 0;   // (see physical_row of the attention)
      row[b] = (static_cast<uint32_t>(page) << a.page_shift) + (j & ((1 << a.page_shift) - 1));
    }
    // A head's keys come from memory in whole rows (256 bytes of 4 rows an instruction, 128
    // of 8 at a row's end) and change lanes through LDS, 128 values of each row at a time;
    // a lane's operands straight from memory, 32 bytes of 32 rows an instruction, took 384
    // us instead of 289 (64 tokens over up to 16384 rows of 8 heads of 128).  They are read
    // once and go past the caches: 256 instead of 278 us there.  MLA rows are their own
    // operands' length, and the way through LDS costs more than it gives (64 tokens over up
    // to 32768 rows: 606 us, 360 without); past the caches, where each line is asked for
    // four times, 634.
    bf16x8 k[KB][KK], next[KB][KK];
    constexpr int WIDE = D / 128;
    auto fetch = [&](int kvh) {
      const uint16_t* const base = a.k_plane + (MLA ? 0 : kvh * a.dim);
      const uint32_t width = MLA ? kRowElems : a.kv_heads * a.dim;
      if constexpr (MLA) {
        const uint64_t of = static_cast<uint64_t>(row[0]) * kRowElems + (lane >> 5) * 8;
#pragma unroll
        for (int i = 0; i < KK; ++i) {
          chunk_t v = *reinterpret_cast<const chunk_t*>(base + of + i * 16);
          if (nothing) v = chunk_t{0u, 0u, 0u, 0u};
          k[0][i] = __builtin_bit_cast(bf16x8, v);
        }
        return;
      }
#pragma unroll
      for (int b = 0; b < KB; ++b)
#pragma unroll
        for (int i = 0; i < KK; ++i) {
          const int r = i < WIDE * 8 ? i % 8 * 4 + (lane >> 4) : (i - WIDE * 8) * 8 + (lane >> 3);
          const int c = i < WIDE * 8 ? i / 8 * 16 + (lane & 15) : WIDE * 16 + (lane & 7);
          const bool in = MLA || c < live;   // (a place without a value reads the row's first one, and counts as 0)
          const uint64_t of = static_cast<uint64_t>(static_cast<uint32_t>(__shfl(static_cast<int>(row[b]), r))) * width;
          chunk_t v = __builtin_nontemporal_load(reinterpret_cast<const chunk_t*>(base + of + (in ? c * 8 : 0)));
          if (!in || nothing) v = chunk_t{0u, 0u, 0u, 0u};
          next[b][i] = __builtin_bit_cast(bf16x8, v);
        }
    };
    const lds_ptr mine = lds + 2 * STAGE + wave * weigh_keys(D);   // a wave's own part of LDS
    const uint32_t wide_at = tile_at(mine, Rows<128>::straight_at(lane)), rest_at = tile_at(mine, Rows<64>::straight_at(lane));
    auto settle = [&]() {
      auto put = [&](int o, bf16x8 x) { *reinterpret_cast<__attribute__((address_space(3))) bf16x8*>(mine + o) = x; };
#pragma unroll
      for (int b = 0; b < KB; ++b) {
#pragma unroll
        for (int w = 0; w < WIDE; ++w) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int r = i * 4 + (lane >> 4);
            put(r * 256 + (Rows<128>::place(r, lane & 15) << 4), next[b][w * 8 + i]);
          }
#pragma unroll
          for (int i = 0; i < 8; ++i) k[b][w * 8 + i] = Rows<128>::straight(wide_at, 0, i);
        }
        if constexpr (D % 128 != 0) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int r = i * 8 + (lane >> 3);
            put(r * 128 + (Rows<64>::place(r, lane & 7) << 4), next[b][WIDE * 8 + i]);
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) k[b][WIDE * 8 + i] = Rows<64>::straight(rest_at, 0, i);
        }
      }
    };
    auto head_of = [&](int i) { return i / per; };
    // Step i: query rows [r0 + i % per * 32 ...) of KV head i / per.  Lane x of a half wave
    // knows row x, token `tok` and head `head` of the KV head's group; rows past the last one
    // repeat it and are seen by nothing.
    float ref = 0.f;
    int below = 0, from = 0;   // the cached rows that a lane's query row sees: [from, below)
    const int per_step = kWeighRows / a.group, over = kWeighRows % a.group;
    const int tok0 = (lane & 31) / a.group, head0 = (lane & 31) - tok0 * a.group;
    int tok = 0, head = 0;
    auto load = [&](int i, int stage, bool goes_on) {
      if (goes_on && i % per != 0) {   // 32 rows on
        tok += per_step, head += over;
        if (head >= a.group) head -= a.group, ++tok;
      } else {
        const int64_t r = int64_t{i % per} * kWeighRows + head0;
        tok = t0 + tok0 + static_cast<int>(r / a.group), head = static_cast<int>(r % a.group);
      }
      const int kvh = head_of(i);
      const bool there = tok < t1;
      const int t = there ? tok : t1 - 1, h = kvh * a.group + (there ? head : a.group - 1);
      if (wave == 0 && lane < kWeighRows) {
        ref = a.lse[static_cast<int64_t>(s.tok0 + t) * a.heads + h];
        const int own = s.row0 + t;
        below = !there ? 0 : a.causal ? own + 1 : kv_len;
        from = a.window > 0 && own + 1 > a.window ? own + 1 - a.window : 0;
      }
#pragma unroll
      for (int x = 0; x < LOADS; ++x) {
        const int b = x * kWeighWaves + wave, r = (b * 64 + lane) / R::CH, c = R::place(r, (b * 64 + lane) % R::CH);
        const int64_t of = s.tok0 + __shfl(t, r), hd = __shfl(h, r);
        const uint16_t* p = a.q + of * a.q_ts + hd * a.q_hs + c * 8;
        if constexpr (MLA)
          if (c >= kKvLoraRank / 8) p = a.q_pe + of * a.qp_ts + hd * a.qp_hs + (c - kKvLoraRank / 8) * 8;
        if (c < live) load_lds<false>(lds + stage * STAGE + b * 1024, p);
      }
    };
    float sum[KB] = {};
    if (begin < steps) {
      __syncthreads();   // nobody reads the last tile's queries any more
      fetch(head_of(begin));
      if (!MLA) settle();
      load(begin, 0, false);
    }
    for (int i = begin; i < steps; ++i) {
      const int stage = (i - begin) & 1, rows0 = r0 + i % per * kWeighRows;
      float* const info = reinterpret_cast<float*>(smem + stage * STAGE + TILE);
      __builtin_amdgcn_s_waitcnt(0x0F70);   // vmcnt(0): this wave's part of the queries
      if (wave == 0 && lane < kWeighRows) {
        info[lane] = ref == -__builtin_inff() ? __builtin_inff() : ref * kLog2e;   // sees nothing: every weight is 0
        reinterpret_cast<int*>(info)[kWeighRows + lane] = below;
        reinterpret_cast<int*>(info)[2 * kWeighRows + lane] = from;
      }
      __syncthreads();
      const bool last_of_head = (i + 1) % per == 0;
      if (!MLA && (i == begin || i % per == 0) && (i / per + 1) * per < steps) fetch(head_of(i + per));
      if (i + 1 < steps) load(i + 1, stage ^ 1, true);
      f32x16 x[KB];
      const f32x16 none = {};
      const uint32_t qa = tile_at(lds + stage * STAGE, at);
      stream<KK, 3>([&](int y) { return R::straight(qa, 0, y); },
                    [&](int y, bf16x8 q) {
#pragma unroll
                      for (int b = 0; b < KB; ++b) x[b] = mfma(q, k[b][y], y == 0 ? none : x[b]);
                    });
      const bool all = rows0 + kWeighRows <= r1 && (!a.causal || j1 <= s.row0 + rows0 / a.group) &&
                       (a.window == 0 || j0 > s.row0 + (rows0 + kWeighRows - 1) / a.group - a.window);
#pragma unroll
      for (int b = 0; b < KB; ++b) {
        float most = 0.f;
        if constexpr (CAP)
#pragma unroll
          for (int e = 0; e < 16; ++e) most = fmaxf(most, fabsf(x[b][e]));
        if (CAP && __any(most > capped.most)) {
#pragma unroll
          for (int e = 0; e < 16; ++e) x[b][e] = exp2_(capped.by * tanh_any(x[b][e] * capped.c) - info[product_row(e, lane)]);
        } else {
#pragma unroll
          for (int e = 0; e < 16; e += 4) {
            const f32x4 rf = *reinterpret_cast<const f32x4*>(info + product_row(e, lane));
#pragma unroll
            for (int y = 0; y < 4; ++y) {
              const float z = x[b][e + y];
              x[b][e + y] = exp2_(__builtin_fmaf(z, CAP ? capped.slope(z) : c2, -rf[y]));
            }
          }
        }
        if (!all) {
          int j = j0 + (wave * KB + b) * 32 + (lane & 31);
          asm volatile("" : "+v"(j));   // (a branch around it, not a selection)
#pragma unroll
          for (int e = 0; e < 16; e += 4) {
            const i32x4 lo = *reinterpret_cast<const i32x4*>(info + 2 * kWeighRows + product_row(e, lane));
            const i32x4 hi = *reinterpret_cast<const i32x4*>(info + kWeighRows + product_row(e, lane));
#pragma unroll
            for (int y = 0; y < 4; ++y)
              if (j < lo[y] || j >= hi[y]) x[b][e + y] = 0.f;
          }
        }
#pragma unroll
        for (int e = 0; e < 16; ++e) sum[b] += x[b][e];
      }
      if (!MLA && last_of_head && i + 1 < steps) settle();
    }
#pragma unroll
    for (int b = 0; b < KB; ++b) {
      const float total = sum[b] + __shfl_xor(sum[b], 32);
      const int j = j0 + (wave * KB + b) * 32 + lane;
      if (lane < 32 && j < kv_len && a.shares > 1) {
        a.parts[(static_cast<int64_t>(share) * seqs + seq) * a.max_rows + j] = total;
      } else if (lane < 32 && j < kv_len) {
        float* const w = a.weights + static_cast<int64_t>(s.seq) * a.weight_stride + j;
        *w = a.decay == 0.f ? total : __builtin_fmaf(a.decay, *w, total);
      }
    }
  }
}

// The shares' sums added up in order, a thread per cached row.
__global__ __launch_bounds__(256) void weigh_join_kernel(WeighLaunch a) {
  const int seqs = a.counts->seqs;
  const int64_t blocks = (a.max_rows + 255) / 256;
  for (int64_t unit = blockIdx.x; unit < blocks * seqs; unit += gridDim.x) {
    const int seq = static_cast<int>(unit % seqs);
    const StepSeq s = a.seqs[seq];
    const int64_t j = unit / seqs * 256 + threadIdx.x;
    if (j >= s.row0 + s.count) continue;
    float total = 0.f;
    for (int c = 0; c < a.shares; ++c) total += a.parts[(static_cast<int64_t>(c) * seqs + seq) * a.max_rows + j];
    float* const w = a.weights + static_cast<int64_t>(s.seq) * a.weight_stride + j;
    *w = a.decay == 0.f ? total : __builtin_fmaf(a.decay, *w, total);
  }
}

template <bool MLA, int DP, int KB, bool CAP>
hipError_t launch_cap(WeighLaunch a, hipStream_t s) {
  constexpr int lds = 2 * weigh_stage(MLA ? kRowElems : DP) + (MLA ? 0 : kWeighWaves * weigh_keys(DP));
  if (const hipError_t e = allow_lds<weigh_kernel<MLA, DP, KB, CAP>>(lds); e != hipSuccess) return e;
  // few tiles and many query rows: each tile is cut, into shares of 8 steps at least
  const int64_t units = (a.max_rows + 32 * KB * kWeighWaves - 1) / (32 * KB * kWeighWaves) * a.n_seqs;
  const int64_t steps = (a.most + kWeighRows - 1) / kWeighRows * a.kv_heads;
  a.shares = static_cast<int32_t>(std::max<int64_t>(
      1, std::min({(kWeighUnits + units - 1) / units, steps / 8, a.part_values / (a.max_rows * a.n_seqs)})));
  const dim3 g(static_cast<unsigned>(std::min<int64_t>(units * a.shares, 1 << 16)));
  weigh_kernel<MLA, DP, KB, CAP><<<g, dim3(64 * kWeighWaves), lds, s>>>(a);
  if (a.shares > 1) {
    if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
    const int64_t blocks = (a.max_rows + 255) / 256 * a.n_seqs;
    weigh_join_kernel<<<dim3(static_cast<unsigned>(std::min<int64_t>(blocks, 1 << 16))), dim3(256), 0, s>>>(a);
  }
  return hipGetLastError();
}
template <bool MLA, int DP, int KB>
hipError_t launch_shape(const WeighLaunch& a, hipStream_t s) {
  return a.cap == 0.f ? launch_cap<MLA, DP, KB, false>(a, s) : launch_cap<MLA, DP, KB, true>(a, s);
}

// Two blocks of cached rows a wave halve the reads of LDS per product, which chunks gain
// from; of single tokens, three waves of one block a SIMD ask for more at once (64 tokens
// over up to 16384 rows, through the caches: 278 us, 287 with two blocks; heads of 64 179
// and 195).
template <int DP>
hipError_t launch_dim(const WeighLaunch& a, hipStream_t s) {
  if (a.most >= 16 * kWeighRows) return launch_shape<false, DP, 2>(a, s);
  return launch_shape<false, DP, 1>(a, s);
}

}  // namespace

hipError_t launch_weigh(const WeighLaunch& a, bool gqa, hipStream_t s) {
  if (!gqa) return launch_shape<true, 0, 1>(a, s);
  if (a.dim <= 64) return launch_dim<64>(a, s);
  if (a.dim <= 128) return launch_dim<128>(a, s);
  return launch_shape<false, 256, 1>(a, s);
}

}  // namespace ll
