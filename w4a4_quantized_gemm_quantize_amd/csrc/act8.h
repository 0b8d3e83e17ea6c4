// Activations of the epilogues and of the experts' layer, in fp32.
#pragma once

#include "device.h"

namespace w4a4 {

enum { ACT_NONE = 0, ACT_RELU = 1, ACT_SILU = 2, ACT_GELU = 3, ACT_GELU_TANH = 4 };

// v sigmoid(z). The exponential's argument rounds once, so it is off by |z| 2^-24
// relative, where the sigmoid is small as well as where it is 1; an exponential
// past fp32's range gives a zero.
__device__ __forceinline__ float times_sigmoid(float v, float z) {
  return v * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(z * -1.44269504088896341f));
}
// silu(v) = v sigmoid(v), and GELU's tanh form v (1 + tanh u) / 2 = v sigmoid(2 u), u =
// sqrt(2 / pi) (v + 0.044715 v^3): v sigmoid(v (a + b v^2)). The square stops at
// 10^4, far beyond where the sigmoid is 0 or 1, so that it cannot overflow.
__device__ __forceinline__ float sigmoid_act(float v, float a, float b) {
  return times_sigmoid(v, v * fmaf(b, fminf(v * v, 1e4f), a));
}
// GELU: v Phi(v) = max(v, 0) - |v| Phi(-|v|), Phi the normal distribution function;
// Phi(-z) = exp(-z^2 / 2) t Q(t), t = 1 / (1 + 0.3 z), Q the polynomial of degree 7
// with the least largest relative error on 0 <= z <= 14 (1.3e-7, found by linear
// programming; fp32 rounding adds z^2 2^-24). Beyond, the product is zero in fp32. One
// chain without a branch, unlike the library's erf, whose temporaries made the
// largest tiles spill.
__device__ __forceinline__ float gelu_act(float v) {
  const float z = fminf(fabsf(v), 16.0f);
  const float t = __builtin_amdgcn_rcpf(fmaf(z, 0.3f, 1.0f));
  float q = 0.0355311483f;
  q = fmaf(q, t, -0.156623811f);
  q = fmaf(q, t, 0.205389827f);
  q = fmaf(q, t, -0.0528288148f);
  q = fmaf(q, t, 0.128126502f);
  q = fmaf(q, t, 0.100039937f);
  q = fmaf(q, t, 0.120734662f);
  q = fmaf(q, t, 0.119630486f);
  const float tail = z * t * q * __builtin_amdgcn_exp2f(z * z * -0.721347520444481704f);
  return (v < 0.0f ? 0.0f : v) - tail;                  // a NaN stays
}
__device__ __forceinline__ float sigmoid_a(int act) { return act == ACT_SILU ? 1.0f : 1.59576912f; }
__device__ __forceinline__ float sigmoid_b(int act) { return act == ACT_SILU ? 0.0f : 0.0713548162726009f; }

// The residual's addition: a rounding of its own on every path, so that all give the
// same bits. Without a residual +0 is added, which the tiles read for it: a zero is +0.
__device__ __forceinline__ float plus(float a, float r) {
#pragma clang fp contract(off)
  return a + r;
}

// One value; `act` is uniform.
__device__ __forceinline__ float activate(int act, float v) {
  if (act == ACT_NONE) return v;
  if (act == ACT_RELU) return v < 0.0f ? 0.0f : v;      // a NaN stays
  if (act == ACT_GELU) return gelu_act(v);
  return sigmoid_act(v, sigmoid_a(act), sigmoid_b(act));
}

}  // namespace w4a4
