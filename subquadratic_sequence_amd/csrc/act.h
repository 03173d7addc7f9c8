// Activations of the gates and of the feed-forward and norm operators, with
// their derivatives, in fp32.
#pragma once

#include "../../include/hyena.h"
#include "common.h"

namespace hy {

// sigmoid(z) and 1 - sigmoid(z) = sigmoid(-z), both to a relative error of a few
// 2^-24: e = exp(-|z|) through the hardware exp2 of a product split in two words
// (the rounding error of |z| log2(e) is put back as a factor), one Newton step
// on the hardware reciprocal.
__device__ __forceinline__ void sigmoids(float z, float& s, float& c) {
  const float L2E = 1.44269504088896341f, L2E_LO = 1.92596299e-8f, LN2 = 0.693147180559945309f;
  const float x = -fabsf(z);
  const float hi = x * L2E;
  const float lo = fmaf(x, L2E_LO, fmaf(x, L2E, -hi));
  float e = __builtin_amdgcn_exp2f(hi);
  e = x < -200.f ? 0.f : fmaf(e, lo * LN2, e);  // below exp(-200) = 0 in fp32 (and lo of -inf is NaN)
  const float d = 1.f + e;
  float r = __builtin_amdgcn_rcpf(d);
  r = fmaf(r, fmaf(-d, r, 1.f), r);
  const float q = e * r;
  s = z >= 0.f ? r : q;
  c = z >= 0.f ? q : r;
}

// silu(g) and silu'(g) = s (1 + g (1 - s))
__device__ __forceinline__ float silu_f(float g) {
  float s, c;
  sigmoids(g, s, c);
  return g < -200.f ? 0.f : g * s;  // -inf * 0
}
__device__ __forceinline__ void silu_d(float g, float& y, float& d) {
  float s, c;
  sigmoids(g, s, c);
  const bool tail = fabsf(g) > 200.f;  // infinities: s c g is 0 there
  y = g < -200.f ? 0.f : g * s;
  d = tail ? s : fmaf(g * s, c, s);
}

// gelu(x) = x Phi(x) and its derivative Phi(x) + x phi(x); below -14 both are
// under 1e-43 in magnitude
__device__ __forceinline__ float gelu_f(float x) {
  return x < -14.f ? 0.f : 0.5f * x * (1.f + erff(x * 0.70710678118654752f));
}
__device__ __forceinline__ void gelu_d(float x, float& y, float& d) {
  const float phi = 0.5f * (1.f + erff(x * 0.70710678118654752f));
  const float e = 0.3989422804014327f * __builtin_amdgcn_exp2f(-0.72134752044448170f * x * x);
  const bool lo = x < -14.f, hi = x > 14.f;
  y = lo ? 0.f : x * phi;
  d = lo ? 0.f : (hi ? 1.f : fmaf(x, e, phi));
}

// The same for results that are rounded to bf16 (2^-8 of their value): relative
// errors of a few |x| 2^-24 cost nothing there, and fewer instructions count
// in an epilogue that runs beside no other work.
__device__ __forceinline__ float sigmoid_fast(float z) {
  return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-1.44269504088896341f * z));
}
// Phi(x) with erf from Abramowitz and Stegun 7.1.26 (absolute error 1.5e-7), and
// e = exp(-x^2 / 2)
__device__ __forceinline__ float phi_fast(float x, float& e) {
  const float a = fabsf(x) * 0.70710678118654752f;
  const float t = __builtin_amdgcn_rcpf(fmaf(0.3275911f, a, 1.f));
  e = __builtin_amdgcn_exp2f(-0.72134752044448170f * x * x);
  const float poly =
      t * fmaf(t, fmaf(t, fmaf(t, fmaf(t, 1.061405429f, -1.453152027f), 1.421413741f), -0.284496736f), 0.254829592f);
  const float half = 0.5f * poly * e;  // (1 - erf(a)) / 2
  return x < 0.f ? half : 1.f - half;
}

template <int ACT, typename T = float> __device__ __forceinline__ float act_f(float x) {
  if (ACT == HYENA_ACT_SILU) {
    if (sizeof(T) == 4) return silu_f(x);
    return x < -80.f ? 0.f : x * sigmoid_fast(x);  // (sigmoid(-80) < 2e-35, before exp2 overflows)
  }
  if (ACT == HYENA_ACT_GELU) {
    if (sizeof(T) == 4) return gelu_f(x);
    float e;
    const float p = phi_fast(x, e);
    return x < -14.f ? 0.f : x * p;
  }
  return x;
}
template <int ACT, typename T = float> __device__ __forceinline__ void act_d(float x, float& y, float& d) {
  if (ACT == HYENA_ACT_SILU) {
    if (sizeof(T) == 4) {
      silu_d(x, y, d);
    } else {
      const float s = sigmoid_fast(x);
      const bool lo = x < -80.f, hi = x > 80.f;
      y = lo ? 0.f : x * s;
      d = lo ? 0.f : (hi ? 1.f : fmaf(y, 1.f - s, s));
    }
  } else if (ACT == HYENA_ACT_GELU) {
    if (sizeof(T) == 4) {
      gelu_d(x, y, d);
    } else {
      float e;
      const float p = phi_fast(x, e);
      const bool lo = x < -14.f, hi = x > 14.f;
      y = lo ? 0.f : x * p;
      d = lo ? 0.f : (hi ? 1.f : fmaf(0.3989422804014327f * x, e, p));
    }
  } else {
    y = x;
    d = 1.f;
  }
}

}  // namespace hy
