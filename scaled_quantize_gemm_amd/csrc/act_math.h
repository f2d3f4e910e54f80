// Activations and their derivatives in fp32, for the kernels that are bound by memory.
//
// GELU needs Phi(x) = erfc(-x / sqrt 2) / 2 and, backward, Phi(x) + x phi(x).  With z = |x| / sqrt 2,
// erfc(z) = e^(-z^2) erfcx(z); erfcx falls like 1/z, so erfcx(z) = t Q(t) with t = 1 / (1 + 0.3 z) and
// Q of degree 8, fitted here by reweighted least squares on 400 Chebyshev nodes for z in [0, 10] (relative
// error 2.0e-8; beyond 10, e^(-z^2) is 0 in fp32).  The relative error of the tail stays at fp32
// level where the 5-term form of the GEMM's epilogue (absolute error 1.5e-7) loses digits: a code
// next to a rounding border goes the right way.  The backward's density shares the exponential.
#pragma once

#include "common.h"

namespace sfp8 {

struct GeluParts {
  float tail;  // Phi(-|x|)
  float expo;  // e^(-x^2 / 2)
};

__device__ __forceinline__ GeluParts gelu_parts(float x) {
  // halved: the tail is erfc / 2
  constexpr float q[9] = {0.5f * 0.1691880060075352f,   0.5f * 0.17071521302100234f, 0.5f * 0.1483392729403964f,
                          0.5f * 0.21492564526538546f,  0.5f * -0.09464973146101112f, 0.5f * 0.547718557973177f,
                          0.5f * -0.5122767787999469f, 0.5f * 0.48556256570665635f,  0.5f * -0.12952277023763256f};
  const float t = __builtin_amdgcn_rcpf(fmaf(0.3f * 0.70710678118654752440f, fabsf(x), 1.0f));
  float p = q[8];
#pragma unroll
  for (int i = 7; i >= 0; --i) p = fmaf(p, t, q[i]);
  const float e = __builtin_amdgcn_exp2f(x * x * -0.72134752044448170368f);
  return {t * p * e, e};
}

// x Phi(x) = max(x, 0) - |x| Phi(-|x|) for either sign (|x| held finite: an infinity times the tail's 0 is no number)
__device__ __forceinline__ float act_gelu(float x) {
  const float a = fminf(fabsf(x), 3.40282346638528859812e+38f);
  const float h = fmaf(-a, gelu_parts(x).tail, fmaxf(x, 0.0f));
  return h;
}

// d gelu / dx = Phi(x) + x phi(x)
__device__ __forceinline__ float act_gelu_grad(float x) {
  const GeluParts g = gelu_parts(x);
  return fmaf(x * 0.39894228040143267794f, g.expo, x < 0.0f ? g.tail : 1.0f - g.tail);
}

// s = sigmoid(g) and c = 1 - s = sigmoid(-g), both to fp32 accuracy at either sign of g: from
// e = e^-|g| they are 1 / (1 + e) and e / (1 + e)
__device__ __forceinline__ void sigmoid_pair(float g, float& s, float& c) {
  const float e = __builtin_amdgcn_exp2f(fabsf(g) * -1.44269504088896340736f);
  const float r = __builtin_amdgcn_rcpf(1.0f + e);
  const float er = e * r;
  s = g < 0.0f ? er : r;
  c = g < 0.0f ? r : er;
}

__device__ __forceinline__ float act_swiglu(float g, float u) {
  float s, c;
  sigmoid_pair(g, s, c);
  return g * s * u;
}

// (d gate, d up) of silu(g) u for an output gradient d
__device__ __forceinline__ void act_swiglu_grad(float d, float g, float u, float& dg, float& du) {
  float s, c;
  sigmoid_pair(g, s, c);
  dg = d * u * s * fmaf(g, c, 1.0f);
  du = d * (g * s);
}

}  // namespace sfp8
