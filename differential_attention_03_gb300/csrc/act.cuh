// The activations of the products and their slopes, in fp32.
//   relu       max(z, 0), slope 0 at 0
//   gelu       z Phi(z), Phi the normal distribution's integral
//   gelu_tanh  z / 2 (1 + tanh(c0 (z + c1 z^3)))  =  z sigma(2 c0 (z + c1 z^3))
//   silu       z sigma(z)
#pragma once

#include <cuda_runtime.h>

#include "diffattn.h"
#include "ptx.cuh"

namespace da {

// 1 / (1 + e^-z): e^-z = inf for z below -88 gives 0, as it should.
__device__ __forceinline__ float sigmoid(float z) { return __fdividef(1.f, 1.f + __expf(-z)); }

constexpr float kGeluC0 = 0.79788456080286536f;  // sqrt(2 / pi)
constexpr float kGeluC1 = 0.044715f;

// Phi(z), and e = exp(-z^2 / 2), by the rational approximation of erfc in Abramowitz and Stegun 7.1.26 (absolute error
// 1.5e-7; the tail below zero keeps its size, as nothing is subtracted from 1 there).  One exponential and one
// reciprocal: a kernel whose epilogue called erff was bound by it (8002 x 8192 x 2048, bias, stored z: 193 us; 177 so).
__device__ __forceinline__ float normal_integral(float z, float& e) {
  const float x = fabsf(z) * 0.70710678118654752f;
  const float t = __fdividef(1.f, 1.f + 0.3275911f * x);
  e = ex2(-0.72134752044448170f * z * z);  // (log2(e) / 2)
  const float tail = 0.5f * e * t *
                     (0.254829592f + t * (-0.284496736f + t * (1.421413741f + t * (-1.453152027f + t * 1.061405429f))));
  return z < 0.f ? tail : 1.f - tail;
}

template <int ACT>
__device__ __forceinline__ float act_of(float z) {
  if (ACT == DIFFATTN_ACT_RELU) return z > 0.f ? z : (z != z ? z : 0.f);
  if (ACT == DIFFATTN_ACT_GELU) {
    float e;
    return z * normal_integral(z, e);
  }
  if (ACT == DIFFATTN_ACT_GELU_TANH) return z * sigmoid(2.f * kGeluC0 * (z + kGeluC1 * z * z * z));
  if (ACT == DIFFATTN_ACT_SILU) return z * sigmoid(z);
  return z;
}

// act'(z), and act(z) beside it.
template <int ACT>
__device__ __forceinline__ float act_slope(float z, float& value) {
  if (ACT == DIFFATTN_ACT_RELU) {
    value = z > 0.f ? z : (z != z ? z : 0.f);
    return z > 0.f ? 1.f : (z != z ? z : 0.f);
  }
  if (ACT == DIFFATTN_ACT_GELU) {
    float e;
    const float phi = normal_integral(z, e);
    value = z * phi;
    return phi + z * e * 0.39894228040143268f;
  }
  if (ACT == DIFFATTN_ACT_GELU_TANH) {
    const float s = sigmoid(2.f * kGeluC0 * (z + kGeluC1 * z * z * z));
    value = z * s;
    return s + z * s * (1.f - s) * 2.f * kGeluC0 * (1.f + 3.f * kGeluC1 * z * z);
  }
  if (ACT == DIFFATTN_ACT_SILU) {
    const float s = sigmoid(z);
    value = z * s;
    return s * (1.f + z * (1.f - s));
  }
  value = z;
  return 1.f;
}

// f(integral_constant) for the activation `act`: one branch around a loop, none inside it.
template <int V>
struct ActTag {
  static constexpr int value = V;
};
template <class F>
__device__ __forceinline__ void with_act(int act, F&& f) {
  switch (act) {
    case DIFFATTN_ACT_RELU: f(ActTag<DIFFATTN_ACT_RELU>{}); break;
    case DIFFATTN_ACT_GELU: f(ActTag<DIFFATTN_ACT_GELU>{}); break;
    case DIFFATTN_ACT_GELU_TANH: f(ActTag<DIFFATTN_ACT_GELU_TANH>{}); break;
    case DIFFATTN_ACT_SILU: f(ActTag<DIFFATTN_ACT_SILU>{}); break;
    default: f(ActTag<DIFFATTN_ACT_NONE>{}); break;
  }
}

}  // namespace da
