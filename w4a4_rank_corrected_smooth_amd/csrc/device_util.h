// Helpers shared by the device translation units: vector types, bf16
// conversion, the GELU, and the host-side argument and launch checks.
#pragma once

#include <hip/hip_runtime.h>

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

inline svdq_status_t launch_status(const char *what) {
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return svdq::fail(SVDQ_ERR_HIP, "%s: %s", what, hipGetErrorString(e));
  return SVDQ_OK;
}
