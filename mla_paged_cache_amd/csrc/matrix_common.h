// Device helpers shared by the kernels on the matrix units (kernels_attend.hip,
// kernels_weigh.hip, kernels_train.hip): operand types, reads of LDS, asynchronous
// loads into it, and rows of bf16 as float32.
#pragma once

#include <atomic>

#include "device_common.h"

namespace ll {
namespace {

constexpr float kLn2 = 0.6931471805599453f;
__device__ __forceinline__ float exp2_(float x) { return __builtin_amdgcn_exp2f(x); }

struct Vals {
  float v[8];
};
__device__ __forceinline__ Vals vals_of(chunk_t c) {
  Vals r;
  const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    r.v[2 * i] = bf16_lo(w[i]);
    r.v[2 * i + 1] = bf16_hi(w[i]);
  }
  return r;
}
__device__ __forceinline__ Vals load8(const uint16_t* p, bool live) {
  chunk_t c{0u, 0u, 0u, 0u};
  if (live) c = *reinterpret_cast<const chunk_t*>(p);
  return vals_of(c);
}
__device__ __forceinline__ float dot8(const Vals& x, const Vals& y) {
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) s = __builtin_fmaf(x.v[i], y.v[i], s);
  return s;
}

// tanh of y = s * c, for scores that a cap bounds (cap * tanh(s * scale / cap)).
// Up to |y| = 1/2 a polynomial: tanh(y) / y interpolated in y^2 at Chebyshev points
// (off by 1.3e-8 of it, 1.1e-7 in float32), so that a small score keeps its
// relative precision; above, 1 - 2 / (exp(2 y) + 1), which is off by 1.5e-7 of 1.
__device__ __forceinline__ float tanh_small(float y) {
  const float u = y * y;
  float p = __builtin_fmaf(0.017141319f, u, -0.052989241f);
  p = __builtin_fmaf(p, u, 0.13324829f);
  p = __builtin_fmaf(p, u, -0.33333072f);
  p = __builtin_fmaf(p, u, 0.99999999f);
  return p * y;
}
__device__ __forceinline__ float tanh_any(float y) {
  // (an infinite y gives 1 or -1: exp2 gives infinity or 0, whose reciprocals do)
  const float t = __builtin_fmaf(-2.f, __builtin_amdgcn_rcpf(exp2_(y * 2.885390082f) + 1.f), 1.f);
  return fabsf(y) <= 0.5f ? tanh_small(y) : t;
}

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) char* lds_ptr;

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

typedef float f32x16 __attribute__((ext_vector_type(16)));

// ---- a tile of rows in LDS, and the operands of 32x32x16 products out of it
//
// D values a row, in 16-byte chunks; chunk c of row r lies at place(r, c) of the row,
// so that both ways of reading a tile touch the 64 banks evenly:
//  * straight, 32 rows at one chunk per half wave; the hardware serves lanes 0-3,
//    12-15, 20-27 together, and those rows differ in their last four bits;
//  * transposing, 4 rows and 4 neighbouring chunks per half wave.
// Rows of an odd multiple of 128 bytes start at every other multiple of 128, which is the
// fourth bit of difference there.
template <int D>
struct Rows {
  static constexpr int CH = D / 8, BYTES = D * 2;
  static_assert(CH % 8 == 0, "the swizzles below");
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

// by * tanh(c * s) of products s, without a multiplication by c or by: the polynomial's
// coefficients hold them, for c of a size where its powers do.
struct Tanh {
  float k[5];                    // s * sum k_i (s^2)^i
  float most;                    // |s| up to which that holds (-1: c is outside [2^-12, 2^12], or by above 2^120 / c^9)
  float c, by;
  static __device__ __forceinline__ float uniform(float x) { return __int_as_float(__builtin_amdgcn_readfirstlane(__float_as_int(x))); }
  __device__ __forceinline__ Tanh(float c_, float by_) : c(uniform(c_)), by(uniform(by_)) {
    const float w = c * c;
    const float b[5] = {0.99999999f, -0.33333072f, 0.13324829f, -0.052989241f, 0.017141319f};
    float x = c * by, last = x;
#pragma unroll
    for (int i = 0; i < 5; ++i) {
      k[i] = uniform(b[i] * x);
      last = x;
      x *= w;
    }
    // (an infinite coefficient times a score of 0 would be NaN; one that vanishes belongs to
    // scores below 2^-12, which it moves by 2^-26)
    most = uniform(fabsf(c) >= 0x1p-12f && fabsf(c) <= 0x1p12f && fabsf(last) <= 0x1p120f ? 0.5f / fabsf(c) : -1.f);
  }
  __device__ __forceinline__ float slope(float s) const {   // of the chord from 0
    const float w = s * s;
    float p = __builtin_fmaf(k[4], w, k[3]);
    p = __builtin_fmaf(p, w, k[2]);
    p = __builtin_fmaf(p, w, k[1]);
    return __builtin_fmaf(p, w, k[0]);
  }
  __device__ __forceinline__ float small(float s) const { return slope(s) * s; }
};
// All of a wave's products in the short form where that holds (a NaN takes either: both
// give NaN).
__device__ __forceinline__ void tanh_all(f32x16& s, const Tanh& f) {
  float most = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) most = fmaxf(most, fabsf(s[i]));
  if (__any(most > f.most)) {
#pragma unroll
    for (int i = 0; i < 16; ++i) s[i] = f.by * tanh_any(s[i] * f.c);
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) s[i] = f.small(s[i]);
  }
}

// Let a kernel take that much LDS; once per device and kernel, since it is not cheap.
template <auto* K>
hipError_t allow_lds(int bytes) {
  static std::atomic<bool> set[64];
  int dev = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess || (dev >= 0 && dev < 64 && set[dev])) return e;
  e = hipFuncSetAttribute(reinterpret_cast<const void*>(K), hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == hipSuccess && dev >= 0 && dev < 64) set[dev] = true;
  return e;
}

}  // namespace
}  // namespace ll
