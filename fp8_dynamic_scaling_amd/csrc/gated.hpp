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

template <bool GELU>
__device__ __forceinline__ float gate_sigmoid(float x) {
  const float z = GELU ? kGeluC * (x + kGeluA * x * x * x) : x;
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
  const float dz = GELU ? kGeluC * (1.0f + 3.0f * kGeluA * x * x) : 1.0f;
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
