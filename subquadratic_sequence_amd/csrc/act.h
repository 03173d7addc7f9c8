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

template <int ACT> __device__ __forceinline__ float act_f(float x) {
  if (ACT == HYENA_ACT_SILU) return silu_f(x);
  if (ACT == HYENA_ACT_GELU) return gelu_f(x);
  return x;
}
template <int ACT> __device__ __forceinline__ void act_d(float x, float& y, float& d) {
  if (ACT == HYENA_ACT_SILU) {
    silu_d(x, y, d);
  } else if (ACT == HYENA_ACT_GELU) {
    gelu_d(x, y, d);
  } else {
    y = x;
    d = 1.f;
  }
}

}  // namespace hy
