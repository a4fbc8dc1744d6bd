// Helpers shared by the device translation units: vector types, bf16
// conversion, copies into LDS, the GELU, and the host-side argument and launch
// checks.
#pragma once

#include <hip/hip_runtime.h>

#include <algorithm>

#include "common.h"

typedef float v4f __attribute__((ext_vector_type(4)));
typedef float v16f __attribute__((ext_vector_type(16)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef _Float16 v8h __attribute__((ext_vector_type(8)));
typedef _Float16 v2h __attribute__((ext_vector_type(2)));
typedef unsigned v4u __attribute__((ext_vector_type(4)));
typedef unsigned v6u __attribute__((ext_vector_type(6)));
typedef int v8i __attribute__((ext_vector_type(8)));
typedef short v4s __attribute__((ext_vector_type(4)));   // four bf16 bit patterns

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// float -> bf16 bits, round to nearest even (finite values)
__device__ __forceinline__ uint32_t f32_to_bf16_rne(float f) {
  uint32_t u = __float_as_uint(f);
  u += 0x7FFFu + ((u >> 16) & 1u);
  return u >> 16;
}

__device__ __forceinline__ v8bf as_v8bf(uint4 u) { return __builtin_bit_cast(v8bf, u); }

// Global -> LDS copy of 16 bytes per lane by the load unit
// (global_load_lds_dwordx4): lane i writes LDS address lds_base + 16 i.
// lds_base must be uniform across the wavefront.  Written as inline asm so
// that the copy's completion is tracked by the caller's own vmcnt waits
// (the compiler would otherwise wait for every copy before any LDS read).
// The asm has no register outputs; M0 is set and used inside the block.
__device__ __forceinline__ void lds_dma16(const void *gsrc, uint32_t lds_base) {
  asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off"
               :: "v"(gsrc), "s"(lds_base) : "memory");
}
// The same copy with a wave-uniform base address in scalar registers and a
// 32-bit per-lane byte offset.  The base has to come from the scalar ALU (or from long before): a
// memory instruction must not read a scalar register within 5 wait states of the vector ALU's write
// (a readfirstlane), which the compiler does not see to inside asm.  tests/test_device_code.py looks
// at what was built.
__device__ __forceinline__ void lds_dma16_s(const void *sbase, uint32_t voff, uint32_t lds_base) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1"
               :: "v"(voff), "s"(sbase), "s"(lds_base) : "memory");
}
// and of 4 bytes per lane: lane i writes LDS address lds_base + 4 i
__device__ __forceinline__ void lds_dma4_s(const void *sbase, uint32_t voff, uint32_t lds_base) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dword %0, %1"
               :: "v"(voff), "s"(sbase), "s"(lds_base) : "memory");
}
// Of 16 bytes, with a base that a readfirstlane may have written just before: a move by the scalar ALU waits for it by
// itself, and is the wait state that the write of M0 needs.  (In place of lds_dma16_s everywhere it cost the
// 8-bit linear's tiles of 64 x 64 5 to 7%: 128 x 6144 x 4096 15.9 us and 15.1.)
__device__ __forceinline__ void lds_dma16_moved(const void *sbase, uint32_t voff, uint32_t lds_base) {
  uint64_t base;
  asm volatile("s_mov_b32 m0, %3\n\ts_mov_b64 %0, %2\n\tglobal_load_lds_dwordx4 %1, %0"
               : "=&s"(base) : "v"(voff), "s"(sbase), "s"(lds_base) : "memory");
}
template <int N>
__device__ __forceinline__ void vmcnt_wait() {
  asm volatile("s_waitcnt vmcnt(%0)" :: "n"(N) : "memory");
}
__device__ __forceinline__ void vmcnt_wait0() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }
// vmcnt(0) through the builtin (expcnt and lgkmcnt left at their maxima), so
// the compiler's own wait bookkeeping knows every load has landed
__device__ __forceinline__ void vmcnt_wait0_known() { __builtin_amdgcn_s_waitcnt(0x0F70); }

// tanh-form GELU, 0.5 y (1 + tanh u) with u = sqrt(2/pi) (y + 0.044715 y^3),
// evaluated as y / (1 + exp(-2u)) (the same function) so that large negative
// y keep their relative accuracy instead of cancelling in 1 + tanh(u).  With
// -2u log2(e) = y (c0 + c1 y^2) the exponential is one hardware exp2; exp2
// and the reciprocal (about 1 ulp of fp32 each) are far inside the half-ulp
// of the bf16 result; exp overflow gives 1/inf = 0, the right limit.
__device__ __forceinline__ float gelu_tanh_f32(float y) {
  constexpr float c0 = (float)(-2.0 * 0.7978845608028654 * 1.4426950408889634);
  constexpr float c1 = (float)(-2.0 * 0.7978845608028654 * 1.4426950408889634 * 0.044715);
  const float t = y * __builtin_fmaf(c1, y * y, c0);
  return y * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(t));
}

// ------------------------------------------------------------ host side
inline bool aligned16(const void *p) { return ((uintptr_t)p & 15u) == 0; }

// |scale| log2(e), for a softmax whose hidden scores are -inf before they are scaled.  A scale of zero becomes
// float32's smallest number: -inf stays what it is, and no other product, all below 2^128, gets above 2^-21.
// Subnormal bits are set by hand, as a host's thread may flush them.
inline float log2_scale(float scale) {
  const double c = fabs((double)scale) * 1.4426950408889634;
  return c < 0x1p-126 ? __builtin_bit_cast(float, std::max(1u, (uint32_t)(c * 0x1p149 + 0.5))) : (float)c;
}

inline svdq_status_t launch_status(const char *what) {
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return svdq::fail(SVDQ_ERR_HIP, "%s: %s", what, hipGetErrorString(e));
  return SVDQ_OK;
}
