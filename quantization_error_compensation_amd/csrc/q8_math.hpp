// Matrix steps and the gate of the 8-bit path's products.
#pragma once

#include "common.hpp"
#include "q8.hpp"

namespace spear {

typedef int32_t i32x4 __attribute__((ext_vector_type(4)));
typedef int32_t i32x16 __attribute__((ext_vector_type(16)));

// Operands: lane l holds row l % 16 (l % 32) and 16 bytes of K, K piece l / 16
// (l / 32).  Results: column l % 16, rows 4 (l / 16) + i; or column l % 32,
// rows 8 (v / 4) + 4 (l / 32) + v % 4.
__device__ __forceinline__ i32x4 mfma16x16x64_i8(u32x4 a, u32x4 b, i32x4 c) {
  return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, a),
                                               __builtin_bit_cast(i32x4, b), c, 0, 0, 0);
}
__device__ __forceinline__ i32x16 mfma32x32x32_i8(u32x4 a, u32x4 b, i32x16 c) {
  return __builtin_amdgcn_mfma_i32_32x32x32_i8(__builtin_bit_cast(i32x4, a),
                                               __builtin_bit_cast(i32x4, b), c, 0, 0, 0);
}

// The block of K at which workgroup i begins when all walk the same blocks of
// rows that lie a power of two apart: begun together, their loads meet the same
// memory channels (28672 -> 8192 at one token 47.3 us instead of 40.2; gated 8192
// -> 28672 at 72 tokens 109 instead of 83).  A third of the way further for each
// workgroup; sums of integers do not mind.
__device__ __forceinline__ int first_block(int i, int blocks) {
  return (int)((uint32_t)i * (uint32_t)(blocks / 3 | 1) % (uint32_t)blocks);
}

// Two fp32 -> bf16 pair, nearest even.
__device__ __forceinline__ uint32_t bf16_pair(float a, float b) {
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  bf16x2 r;
  r.x = (__bf16)a;
  r.y = (__bf16)b;
  return __builtin_bit_cast(uint32_t, r);
}

// act(a) * b, act(a) = a * sigmoid(z): z = a (SiLU), or for GELU's tanh form
// z = 2 sqrt(2 / pi) (a + 0.044715 a^3), since (1 + tanh(z / 2)) / 2 is
// sigmoid(z).  The exponential's argument is never positive, so nothing
// overflows.  z is off by 3.5 * 2^-24 of itself at most, times log2(e) by 1.25
// more, and 2^x turns that into |z| 2^-21.7 of the sigmoid: 2^-15 at |z| = 87,
// past which it is 0 or 1.
__device__ __forceinline__ float gate(bool gelu, float a, float b) {
  constexpr float kLog2e = 1.44269504088896340736f;
  const float z = gelu ? a * fmaf(0.0713548162726f, a * a, 1.59576912161f) : a;
  const float e = __builtin_amdgcn_exp2f(-fabsf(z) * kLog2e);
  const float sig = __builtin_amdgcn_rcpf(1.f + e) * (z < 0.f ? e : 1.f);
  return a * sig * b;
}

}  // namespace spear
