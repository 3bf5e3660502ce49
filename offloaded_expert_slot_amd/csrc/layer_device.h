// Device helpers shared by the kernels of the operators around the expert step.
#pragma once

#include <hip/hip_runtime.h>

#include "kv_pages.h"

namespace oes {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));

__device__ inline float bf16f(uint32_t bits16) { return __uint_as_float(bits16 << 16); }
__device__ inline float bf16_lo(uint32_t pair) { return __uint_as_float(pair << 16); }
__device__ inline float bf16_hi(uint32_t pair) { return __uint_as_float(pair & 0xffff0000u); }
// round to nearest even; NaN stays NaN
__device__ inline uint32_t f2bf16(float f) {
  uint32_t u = __float_as_uint(f);
  if ((u & 0x7f800000u) == 0x7f800000u) return (u >> 16) | ((u & 0xffffu) ? 0x40u : 0u);
  u += 0x7fffu + ((u >> 16) & 1u);
  return u >> 16;
}
// a, b -> packed bf16 pair (a low), round to nearest even: one conversion instruction
__device__ inline uint32_t f2bf16_pair(float a, float b) {
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  bf16x2 r;
  r.x = (__bf16)a;
  r.y = (__bf16)b;
  return __builtin_bit_cast(uint32_t, r);
}

// Sign bits of the bf16 of a pair that are infinite or NaN (exponents of all ones).
__device__ inline uint32_t odd_bits(uint32_t w) { return ((w & 0x7fff7fffu) + 0x00800080u) & 0x80008000u; }

// The value an e4m3 cache stores for x: clamped to +-448, rounded to nearest even,
// NaN kept.
__device__ inline uint32_t f2e4m3_pair(float a, float b) {
  const float ca = a != a ? a : fminf(fmaxf(a, -448.f), 448.f), cb = b != b ? b : fminf(fmaxf(b, -448.f), 448.f);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(ca, cb, 0, false) & 0xffffu;
}
template <bool HI>
__device__ inline f32x2 e4m3_pair(uint32_t w) {
  return __builtin_amdgcn_cvt_pk_f32_fp8(w, HI);
}

// 1 / (1 + exp(-v)); exp2 of a rounded argument is off by |v| half steps
__device__ inline float sigmoid(float v) { return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-1.44269504088896340736f * v)); }

// 16 bytes per lane from src + OFF to LDS base + 16 * lane; counted by vmcnt only.  (The instruction's offset counts
// for both addresses.)  ONCE: what no other workgroup will read.
template <int OFF = 0, bool ONCE = false>
__device__ inline void load_to_lds(const void *src, uint32_t lds) {
  if (ONCE)
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off offset:%2 nt" ::"s"(lds - OFF), "v"(src), "n"(OFF) : "memory");
  else
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off offset:%2" ::"s"(lds - OFF), "v"(src), "n"(OFF) : "memory");
}
// the same with a wave-uniform base and a 32-bit offset per lane
__device__ inline void load_to_lds(const void *base, uint32_t off, uint32_t lds) {
  const uint64_t b = (uint64_t)base;
  const uint64_t u = (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(b >> 32)) << 32 | (uint32_t)__builtin_amdgcn_readfirstlane((int)b);
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(lds), "v"(off), "s"(u) : "memory");
}
__device__ inline uint32_t lds_addr(const void *p) {
  return (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const void *)p;
}

__device__ inline void raise_status(const oes_kv &kv) {
  if (kv.status) *kv.status = OES_ERR_ARG;
}

}  // namespace oes
