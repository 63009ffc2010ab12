// gated.hpp -- the activation of a gated product and its derivative, shared by the gated GEMM's
// epilogue and the gate's backward.
#pragma once

#include "common.hpp"

namespace fp8dyn {

// act(x) = x s, s = sigmoid(z): z = x for SiLU; z = sqrt(8 / pi) (x + 0.044715 x^3) for GELU in its tanh
// form, whose (1 + tanh(z / 2)) / 2 is sigmoid(z). The exponential is the exp2 instruction's of
// z log2(e), the quotient the reciprocal instruction's: both within some 1e-7 of the formula where s
// is not tiny, far below the half step of bf16 (2^-8) that results are rounded by; an s below 2^-126
// comes out as zero.
constexpr float kGeluC = 1.5957691216057308f, kGeluA = 0.044715f;

// GELU's cube and square would leave fp32 for gates past 10^12 and 10^19; beyond +-64 its s is 0 or 1 either way.
__device__ __forceinline__ float gelu_range(float x) { return __builtin_amdgcn_fmed3f(x, -64.0f, 64.0f); }

template <bool GELU>
__device__ __forceinline__ float gate_sigmoid(float x) {
  float z = x;
  if constexpr (GELU) {
    const float c = gelu_range(x);
    z = kGeluC * (c + kGeluA * c * c * c);
  }
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(z * -1.4426950408889634f));
}

template <bool GELU>
__device__ __forceinline__ float gate_act(float x) {
  return x * gate_sigmoid<GELU>(x);
}

// act(x) and d act / dx = s + x s (1 - s) dz/dx
template <bool GELU>
__device__ __forceinline__ void gate_act_d(float x, float& a, float& da) {
  const float s = gate_sigmoid<GELU>(x);
  float dz = 1.0f;
  if constexpr (GELU) {
    const float c = gelu_range(x);
    dz = kGeluC * (1.0f + 3.0f * kGeluA * c * c);
  }
  a = x * s;
  da = s + a * (1.0f - s) * dz;
}

typedef __bf16 gt_bf16x2 __attribute__((ext_vector_type(2)));

// two fp32 values as bf16 (RNE, NaN kept), the first in the low half
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const gt_bf16x2 h = {(__bf16)a, (__bf16)b};
  return __builtin_bit_cast(uint32_t, h);
}

}  // namespace fp8dyn
