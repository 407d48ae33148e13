// The activations of the gated block and their slopes, for epilogues that round to bf16: e^x and
// the quotient by the approximate instructions (a few units of 2^-22, next to bf16's 2^-8).
#pragma once

#include "common.cuh"

namespace mao {

// 1 / (1 + e^-x): 0 and 1 where e^-x leaves fp32's range.
__device__ __forceinline__ float fast_sigmoid(float x) {
  float e, s;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(x * -1.4426950408889634f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s) : "f"(1.0f + e));
  return s;
}

constexpr float kTanhA = 0.044715f;
constexpr float kTanhC = 0.7978845608028654f;  // sqrt(2 / pi)

// act(x), the form of the tanh through 1 + tanh(y) = 2 sigmoid(2 y): no cancellation far below 0.
// ACT is a template argument where it is applied many times over: with the three inline at each of
// them the code of an epilogue no longer stays in the instruction cache.
template <int ACT>
__device__ __forceinline__ float activate(float x) {
  if (ACT == MAO_SILU) return x * fast_sigmoid(x);
  if (ACT == MAO_GELU) return 0.5f * x * erfcf(x * -0.7071067811865476f);
  return x * fast_sigmoid(2.0f * kTanhC * (x + kTanhA * x * x * x));
}

// act(x) and its slope.
template <int ACT>
__device__ __forceinline__ void activate(float x, float& a, float& slope) {
  if (ACT == MAO_SILU) {
    const float s = fast_sigmoid(x);
    a = x * s;
    slope = s + a * (1.0f - s);
  } else if (ACT == MAO_GELU) {
    const float phi = 0.5f * erfcf(x * -0.7071067811865476f);
    a = x * phi;
    slope = phi + x * 0.3989422804014327f * __expf(-0.5f * x * x);
  } else {
    const float s = fast_sigmoid(2.0f * kTanhC * (x + kTanhA * x * x * x));
    a = x * s;
    slope = s + a * (1.0f - s) * (2.0f * kTanhC + 6.0f * kTanhC * kTanhA * x * x);
  }
}

}  // namespace mao
