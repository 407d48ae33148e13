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
    // (where x^2 passes fp32's range, a or 1 - s is 0: not to be multiplied by an infinity)
    slope = s + a * (1.0f - s) * (2.0f * kTanhC + 6.0f * kTanhC * kTanhA * fminf(x * x, 1e30f));
  }
}

// Two values at a time: the packed fp32 instructions halve the arithmetic of an epilogue.
__device__ __forceinline__ uint64_t pair_of(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void split_pair(uint64_t p, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(p));
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
// act(x) and its slope, of two values.
template <int ACT>
__device__ __forceinline__ void activate2(uint64_t x, uint64_t& a, uint64_t& slope) {
  float x0, x1;
  if (ACT == MAO_SILU) {
    const uint64_t t = mul2(x, pair_of(-1.4426950408889634f, -1.4426950408889634f));
    float e0, e1, s0, s1;
    split_pair(t, x0, x1);
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e0) : "f"(x0));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e1) : "f"(x1));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s0) : "f"(1.0f + e0));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s1) : "f"(1.0f + e1));
    const uint64_t s = pair_of(s0, s1);
    a = mul2(x, s);
    slope = fma2(a, fma2(s, pair_of(-1.0f, -1.0f), pair_of(1.0f, 1.0f)), s);
  } else {
    float a0, a1, s0, s1;
    split_pair(x, x0, x1);
    activate<ACT>(x0, a0, s0);
    activate<ACT>(x1, a1, s1);
    a = pair_of(a0, a1);
    slope = pair_of(s0, s1);
  }
}

}  // namespace mao
