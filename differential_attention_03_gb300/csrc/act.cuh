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

__device__ __forceinline__ float rcp_fast(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Two values at a time: sums and products of pairs are one instruction each.
__device__ __forceinline__ uint64_t pair_of(float x) { return f2pack(x, x); }
template <class F>
__device__ __forceinline__ uint64_t each(uint64_t x, F&& f) {
  float lo, hi;
  f2unpack(x, lo, hi);
  return f2pack(f(lo), f(hi));
}

// 1 / (1 + 2^-t): 2^-t = inf gives 0, as it should.
__device__ __forceinline__ uint64_t sigmoid2(uint64_t t) {
  return each(t, [](float x) { return rcp_fast(1.f + ex2(-x)); });
}

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kGeluC0 = 0.79788456080286536f;  // sqrt(2 / pi)
constexpr float kGeluC1 = 0.044715f;

// Phi(z), and e = exp(-z^2 / 2).  The smaller tail, Phi(-|z|), is e t P(t) with t = 1 / (1 + k |z|): erfc's scaled form is
// smooth in t, and P a polynomial fitted to it over |z| < 14.5 (least squares in the relative error, weighted until its
// extremes were level), so that small values keep their relative accuracy.  FINE, for what leaves in fp32: degree 8, 3e-7 in
// fp32, so Phi within 2^-20 + 1.5 z^2 2^-24 of itself, the second term from the rounding of the exponent.  Else degree 5, 5e-6,
// where the result's own rounding to bf16 is 2^-9 and more (the finer one takes 5 % more of a short contraction: 4096 x 4096
// x 512 30.7 and 32.5 us).  One exponential and one reciprocal: a kernel whose epilogue called erff was bound by it (8002 x
// 8192 x 2048, bias, stored z: 193 us when the product alone took 160; 156 so, the product alone 141).
template <bool FINE>
__device__ __forceinline__ uint64_t normal_integral2(uint64_t z, uint64_t& e) {
  e = each(mul2(mul2(z, z), pair_of(-0.5f * kLog2e)), [](float x) { return ex2(x); });
  const uint64_t a = each(z, [](float x) { return fabsf(x); });
  const uint64_t t = each(fma2(a, pair_of(FINE ? 0.34f : 0.31f), pair_of(1.f)), [](float x) { return rcp_fast(x); });
  uint64_t q;
  if (FINE) {
    q = fma2(t, pair_of(-0.025876413645322137f), pair_of(0.13835696513852064f));
    q = fma2(t, q, pair_of(-0.27087084145298024f));
    q = fma2(t, q, pair_of(0.1997173936819431f));
    q = fma2(t, q, pair_of(-0.04310615863072467f));
    q = fma2(t, q, pair_of(0.11471355380278708f));
    q = fma2(t, q, pair_of(0.11535171361673928f));
    q = fma2(t, q, pair_of(0.13609222657221123f));
    q = fma2(t, q, pair_of(0.13562157796838106f));
  } else {
    q = fma2(t, pair_of(-0.07392923137350546f), pair_of(0.18045061496190595f));
    q = fma2(t, q, pair_of(0.0157444093190871f));
    q = fma2(t, q, pair_of(0.13342994182106155f));
    q = fma2(t, q, pair_of(0.12044123862331163f));
    q = fma2(t, q, pair_of(0.12386070538132232f));
  }
  const uint64_t tail = mul2(mul2(q, t), e);
  float z0, z1, lo0, lo1, hi0, hi1;
  f2unpack(z, z0, z1);
  f2unpack(tail, lo0, lo1);
  f2unpack(fma2(tail, pair_of(-1.f), pair_of(1.f)), hi0, hi1);
  return f2pack(z0 < 0.f ? lo0 : hi0, z1 < 0.f ? lo1 : hi1);
}

// act(z) of a pair (FINE: as a result in fp32 needs it).
template <int ACT, bool FINE>
__device__ __forceinline__ uint64_t act_of2(uint64_t z) {
  if (ACT == DIFFATTN_ACT_RELU) return each(z, [](float x) { return x > 0.f ? x : (x != x ? x : 0.f); });
  if (ACT == DIFFATTN_ACT_GELU) {
    uint64_t e;
    return mul2(z, normal_integral2<FINE>(z, e));
  }
  if (ACT == DIFFATTN_ACT_GELU_TANH) {
    const uint64_t w = fma2(mul2(z, z), pair_of(2.f * kLog2e * kGeluC0 * kGeluC1), pair_of(2.f * kLog2e * kGeluC0));
    return mul2(z, sigmoid2(mul2(z, w)));
  }
  if (ACT == DIFFATTN_ACT_SILU) return mul2(z, sigmoid2(mul2(z, pair_of(kLog2e))));
  return z;
}

// act'(z) of a pair, and act(z) beside it.
template <int ACT, bool FINE>
__device__ __forceinline__ uint64_t act_slope2(uint64_t z, uint64_t& value) {
  if (ACT == DIFFATTN_ACT_RELU) {
    value = act_of2<ACT, FINE>(z);
    return each(z, [](float x) { return x > 0.f ? 1.f : (x != x ? x : 0.f); });
  }
  if (ACT == DIFFATTN_ACT_GELU) {
    uint64_t e;
    const uint64_t phi = normal_integral2<FINE>(z, e);
    value = mul2(z, phi);
    return fma2(mul2(z, e), pair_of(0.39894228040143268f), phi);
  }
  if (ACT == DIFFATTN_ACT_GELU_TANH) {
    // (a z beyond 1e4 has a slope of 0 or 1 either way; its square would not always be finite)
    const uint64_t zz = each(mul2(z, z), [](float x) { return fminf(x, 1e8f); });
    const uint64_t w = fma2(zz, pair_of(2.f * kLog2e * kGeluC0 * kGeluC1), pair_of(2.f * kLog2e * kGeluC0));
    const uint64_t s = sigmoid2(mul2(z, w));
    value = mul2(z, s);
    // s + value (1 - s) 2 c0 (1 + 3 c1 z^2)
    const uint64_t rest = fma2(s, mul2(value, pair_of(-1.f)), value);
    return fma2(rest, fma2(zz, pair_of(6.f * kGeluC0 * kGeluC1), pair_of(2.f * kGeluC0)), s);
  }
  if (ACT == DIFFATTN_ACT_SILU) {
    const uint64_t s = sigmoid2(mul2(z, pair_of(kLog2e)));
    value = mul2(z, s);
    return add2(s, fma2(s, mul2(value, pair_of(-1.f)), value));
  }
  value = z;
  return pair_of(1.f);
}

// v[0 .. N) = act(v); v = act(v) u.
template <int ACT, int N, bool FINE>
__device__ __forceinline__ void act_all(float* v) {
#pragma unroll
  for (int j = 0; j < N; j += 2) f2unpack(act_of2<ACT, FINE>(f2pack(v[j], v[j + 1])), v[j], v[j + 1]);
}
template <int ACT, int N>
__device__ __forceinline__ void act_times(float* v, const float* u) {
#pragma unroll
  for (int j = 0; j < N; j += 2) f2unpack(mul2(act_of2<ACT, false>(f2pack(v[j], v[j + 1])), f2pack(u[j], u[j + 1])), v[j], v[j + 1]);
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
