// The activations of the gated block and their slopes, for epilogues that round to bf16: e^x and
// the quotient by the fast functions (a few units of 2^-22, next to bf16's 2^-9).
#pragma once

#include "common.cuh"

namespace mao {

__device__ __forceinline__ float fast_sigmoid(float x) {
  return __fdividef(1.0f, 1.0f + __expf(-x));
}

constexpr float kTanhA = 0.044715f;
constexpr float kTanhC = 0.7978845608028654f;  // sqrt(2 / pi)

// act(x), the form of the tanh through 1 + tanh(y) = 2 sigmoid(2 y): no cancellation far below 0.
__device__ __forceinline__ float activate(float x, int act) {
  if (act == MAO_SILU) return x * fast_sigmoid(x);
  if (act == MAO_GELU) return 0.5f * x * erfcf(x * -0.7071067811865476f);
  return x * fast_sigmoid(2.0f * kTanhC * (x + kTanhA * x * x * x));
}

// act(x) and its slope.
__device__ __forceinline__ void activate(float x, int act, float& a, float& slope) {
  if (act == MAO_SILU) {
    const float s = fast_sigmoid(x);
    a = x * s;
    slope = s * (1.0f + x * (1.0f - s));
  } else if (act == MAO_GELU) {
    const float phi = 0.5f * erfcf(x * -0.7071067811865476f);
    a = x * phi;
    slope = phi + x * 0.3989422804014327f * __expf(-0.5f * x * x);
  } else {
    const float s = fast_sigmoid(2.0f * kTanhC * (x + kTanhA * x * x * x));
    a = x * s;
    slope = s + 2.0f * x * s * (1.0f - s) * kTanhC * (1.0f + 3.0f * kTanhA * x * x);
  }
}

}  // namespace mao
