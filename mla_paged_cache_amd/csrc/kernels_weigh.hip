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

// Bytes of a tile of query rows in LDS: the queries, their lse and what they see.
constexpr int weigh_stage(int d) { return (kWeighRows * (d * 2 + 12) + 255) / 256 * 256; }

// A wave takes 32 * KB cached rows, their keys of one KV head at a time in registers, and
// goes along the query rows that see some of them, 32 at a time through LDS, which the
// workgroup's waves share: S = Q K^T with a lane per cached row, so that the sum over
// query rows and heads stays in one register of the lane and one owner.  Single tokens
// are bound by reading the keys (the next head's are asked for before this one's are
// multiplied); chunks by the matrix units.  Larger grids take several tiles a workgroup.
template <bool MLA, int DP, int KB, bool CAP>
__global__ __launch_bounds__(64 * kWeighWaves) __attribute__((amdgpu_waves_per_eu(2))) void weigh_kernel(WeighLaunch a) {
  constexpr int D = MLA ? kRowElems : DP, KK = D / 16, KEYS = 32 * KB * kWeighWaves;
  using R = Rows<D>;
  constexpr int TILE = kWeighRows * R::BYTES, STAGE = weigh_stage(D);
  extern __shared__ __attribute__((aligned(1024))) char smem[];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const lds_ptr lds = (lds_ptr)smem;
  const int live = MLA ? R::CH : a.dim / 8, seqs = a.counts->seqs;
  const int64_t tiles = (a.max_rows + KEYS - 1) / KEYS;
  const float c2 = CAP ? a.scale / a.cap : a.scale * kLog2e, cap2 = a.cap * kLog2e;
  const bool nothing = !(fabsf(c2) >= 1e-37f);   // a scale too small to tell scores apart counts as 0
  const int at = R::straight_at(lane);

  if (live < R::CH) {
    for (int i = threadIdx.x; i < 2 * STAGE / 16; i += 64 * kWeighWaves)
      reinterpret_cast<chunk_t*>(smem)[i] = chunk_t{0u, 0u, 0u, 0u};
    __syncthreads();
  }
  for (int64_t unit = blockIdx.x; unit < tiles * seqs; unit += gridDim.x) {
    const StepSeq s = a.seqs[unit % seqs];
    const int kv_len = s.row0 + s.count;
    const int64_t tile0 = unit / seqs * KEYS;
    if (tile0 >= kv_len) continue;
    const int j0 = static_cast<int>(tile0), j1 = min(j0 + KEYS, kv_len) - 1;
    // the tokens that see some row of the tile, as query rows of a KV head
    const int t0 = a.causal ? max(0, j0 - s.row0) : 0;
    const int t1 = static_cast<int>(a.window > 0 ? min<int64_t>(s.count, int64_t{j1} + a.window - s.row0) : s.count);
    const int r0 = t0 * a.group, r1 = t1 * a.group;
    const int per = r1 > r0 ? (r1 - r0 + kWeighRows - 1) / kWeighRows : 0, steps = per * a.kv_heads;

    const uint16_t* row[KB];   // this lane's keys: KV head 0
#pragma unroll
    for (int b = 0; b < KB; ++b) {
      const int j = min(j0 + (wave * KB + b) * 32 + (lane & 31), kv_len - 1);
      int page = a.page_table[static_cast<int64_t>(s.seq) * a.max_pages_per_seq + (j >> a.page_shift)];
      if (static_cast<uint32_t>(page) >= static_cast<uint32_t>(a.num_pages)) page = 0;   // (see physical_row of the attention)
      const int64_t r = (static_cast<int64_t>(page) << a.page_shift) + (j & ((1 << a.page_shift) - 1));
      row[b] = a.k_plane + r * (MLA ? kRowElems : a.kv_heads * a.dim);
    }
    bf16x8 k[KB][KK], next[KB][KK];
    auto keys = [&](bf16x8 (&x)[KB][KK], int kvh) {
#pragma unroll
      for (int b = 0; b < KB; ++b)
#pragma unroll
        for (int i = 0; i < KK; ++i) {
          const int c = 2 * i + (lane >> 5);
          const bool in = MLA || c < live;   // (a place without a value reads the row's first one, and counts as 0)
          chunk_t v = *reinterpret_cast<const chunk_t*>(row[b] + (MLA ? 0 : kvh * a.dim) + (in ? c * 8 : 0));
          if (!in || nothing) v = chunk_t{0u, 0u, 0u, 0u};
          x[b][i] = __builtin_bit_cast(bf16x8, v);
        }
    };
    // Step i: query rows [r0 + i % per * 32 ...) of KV head i / per.  Lane x of a half wave
    // knows row x; rows past the last one repeat it and are seen by nothing.
    float ref = 0.f;
    int below = 0, from = 0;   // the cached rows that a lane's query row sees: [from, below)
    auto load = [&](int i, int stage) {
      const int q = r0 + i % per * kWeighRows + (lane & 31), kvh = i / per;
      const bool there = q < r1;
      const int t = (there ? q : r1 - 1) / a.group, h = kvh * a.group + (there ? q : r1 - 1) - t * a.group;
      const int64_t tok = s.tok0 + t, off = tok * a.q_ts + h * a.q_hs, off_pe = MLA ? tok * a.qp_ts + h * a.qp_hs : 0;
      ref = a.lse[tok * a.heads + h];
      const int own = s.row0 + t;
      below = !there ? 0 : a.causal ? own + 1 : kv_len;
      from = a.window > 0 && own + 1 > a.window ? own + 1 - a.window : 0;
      auto of = [&](int64_t x, int r) {
        return static_cast<int64_t>(static_cast<uint64_t>(static_cast<uint32_t>(__shfl(static_cast<int>(x >> 32), r))) << 32 |
                                    static_cast<uint32_t>(__shfl(static_cast<int>(x), r)));
      };
#pragma unroll
      for (int x = 0; x < kWeighRows * R::CH / 64 / kWeighWaves; ++x) {
        const int b = x * kWeighWaves + wave, r = (b * 64 + lane) / R::CH, c = R::place(r, (b * 64 + lane) % R::CH);
        const uint16_t* p = a.q + of(off, r) + c * 8;
        if constexpr (MLA) {
          const uint16_t* pe = a.q_pe + of(off_pe, r) + (c - kKvLoraRank / 8) * 8;
          if (c >= kKvLoraRank / 8) p = pe;
        }
        if (c < live) load_lds<false>(lds + stage * STAGE + b * 1024, p);
      }
    };
    float sum[KB] = {};
    if (steps > 0) {
      __syncthreads();   // nobody reads the last tile's queries any more
      keys(k, 0);
      load(0, 0);
    }
    for (int i = 0; i < steps; ++i) {
      const int stage = i & 1, rows0 = r0 + i % per * kWeighRows;
      float* const info = reinterpret_cast<float*>(smem + stage * STAGE + TILE);
      __builtin_amdgcn_s_waitcnt(0x0F70);   // vmcnt(0): this wave's part of the queries
      if (wave == 0 && lane < kWeighRows) {
        info[lane] = ref == -__builtin_inff() ? __builtin_inff() : ref * kLog2e;   // sees nothing: every weight is 0
        reinterpret_cast<int*>(info)[kWeighRows + lane] = below;
        reinterpret_cast<int*>(info)[2 * kWeighRows + lane] = from;
      }
      __syncthreads();
      const bool last_of_head = (i + 1) % per == 0;
      if (!MLA && i % per == 0 && i / per + 1 < a.kv_heads) keys(next, i / per + 1);
      if (i + 1 < steps) load(i + 1, stage ^ 1);
      f32x16 x[KB];
#pragma unroll
      for (int b = 0; b < KB; ++b)
#pragma unroll
        for (int e = 0; e < 16; ++e) x[b][e] = 0.f;
      const uint32_t qa = tile_at(lds + stage * STAGE, at);
      stream<KK, 3>([&](int y) { return R::straight(qa, 0, y); },
                    [&](int y, bf16x8 q) {
#pragma unroll
                      for (int b = 0; b < KB; ++b) x[b] = mfma(q, k[b][y], x[b]);
                    });
      const bool all = rows0 + kWeighRows <= r1 && (!a.causal || j1 <= s.row0 + rows0 / a.group) &&
                       (a.window == 0 || j0 > s.row0 + (rows0 + kWeighRows - 1) / a.group - a.window);
#pragma unroll
      for (int b = 0; b < KB; ++b) {
        if constexpr (CAP) tanh_all(x[b], c2);
#pragma unroll
        for (int e = 0; e < 16; e += 4) {
          const f32x4 rf = *reinterpret_cast<const f32x4*>(info + product_row(e, lane));
#pragma unroll
          for (int y = 0; y < 4; ++y) x[b][e + y] = exp2_(__builtin_fmaf(x[b][e + y], CAP ? cap2 : c2, -rf[y]));
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
      if (!MLA && last_of_head) {
#pragma unroll
        for (int b = 0; b < KB; ++b)
#pragma unroll
          for (int y = 0; y < KK; ++y) k[b][y] = next[b][y];
      }
    }
#pragma unroll
    for (int b = 0; b < KB; ++b) {
      const float total = sum[b] + __shfl_xor(sum[b], 32);
      const int j = j0 + (wave * KB + b) * 32 + lane;
      if (lane < 32 && j < kv_len) {
        float* const w = a.weights + static_cast<int64_t>(s.seq) * a.weight_stride + j;
        *w = a.decay == 0.f ? total : __builtin_fmaf(a.decay, *w, total);
      }
    }
  }
}

template <bool MLA, int DP, int KB, bool CAP>
hipError_t launch_cap(const WeighLaunch& a, hipStream_t s) {
  constexpr int lds = 2 * weigh_stage(MLA ? kRowElems : DP);
  if (const hipError_t e = allow_lds<weigh_kernel<MLA, DP, KB, CAP>>(lds); e != hipSuccess) return e;
  const int64_t tiles = (a.max_rows + 32 * KB * kWeighWaves - 1) / (32 * KB * kWeighWaves);
  const dim3 g(static_cast<unsigned>(std::min<int64_t>(tiles * a.n_seqs, 1 << 16)));
  weigh_kernel<MLA, DP, KB, CAP><<<g, dim3(64 * kWeighWaves), lds, s>>>(a);
  return hipGetLastError();
}
template <bool MLA, int DP, int KB>
hipError_t launch_shape(const WeighLaunch& a, hipStream_t s) {
  return a.cap == 0.f ? launch_cap<MLA, DP, KB, false>(a, s) : launch_cap<MLA, DP, KB, true>(a, s);
}

// Two blocks of cached rows a wave halve the reads of LDS per product, where the rows
// still fill the chip.
template <int DP>
hipError_t launch_dim(const WeighLaunch& a, hipStream_t s) {
  if (a.max_rows * a.n_seqs >= 512 * 64 * kWeighWaves) return launch_shape<false, DP, 2>(a, s);
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
