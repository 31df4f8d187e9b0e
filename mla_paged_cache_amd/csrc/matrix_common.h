// Device helpers shared by the kernels on the matrix units (kernels_attend.hip,
// kernels_weigh.hip, kernels_train.hip): operand types, reads of LDS, asynchronous
// loads into it, and rows of bf16 as float32.
#pragma once

#include "device_common.h"

namespace ll {
namespace {

constexpr float kLn2 = 0.6931471805599453f;
__device__ __forceinline__ float exp2_(float x) { return __builtin_amdgcn_exp2f(x); }

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

}  // namespace
}  // namespace ll
