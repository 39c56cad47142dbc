// The activations of the dense layers and their derivatives, in fp32. Two precisions, by the bounds that hold for
// all finite z, in 2^-24 (measured over [-20, 20] and every bf16):
//   the device library's functions, for fp32 operands or results: activations within 3 max(1, |z|), derivatives
//   within 4. Of the value itself a few 2^-24 above -1; below, exponentials pass on the rounding of their arguments
//   (gelu and gelu_tanh near -5 up to 40)
//   short forms on the hardware's exp2 and reciprocal, 1 ulp each, for bf16 operands with results that are rounded to
//   2^-8: the same bounds (column sums of gradients stay fp32). gelu's tail is good to that bound, not to its own
//   digits: 0.2% at -5, half a bf16 step at -6, 1% at -8, where gelu is 5e-15
#pragma once
#include "common.h"

namespace tw {

enum Act { kActNone, kActRelu, kActSilu, kActGelu, kActGeluTanh };

template <bool FAST> TW_DEV float sigmoid_of(float z) {
  if constexpr (FAST) return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-1.44269504088896340736f * z));
  else return 1.f / (1.f + expf(-z));
}

// sigmoid(z) and t = 1 - sigmoid(z) = sigmoid(-z) from one exponential, each to its own last digits: the derivatives
// multiply t by z and more, so that the half step of 2^-24 which 1.f - s leaves where s is near 1 would be 16 and 33
// times 2^-24 in silu' at 16 and gelu_tanh' at 5 (so 4 at most). Gated backward of 16384 x 4096 x 14336: 8839 us with
// 1.f - s, 8866 so.
template <bool FAST> TW_DEV float sigmoid_pair(float z, float &t) {
  const float e = FAST ? __builtin_amdgcn_exp2f(-1.44269504088896340736f * fabsf(z)) : expf(-fabsf(z));
  const float r = FAST ? __builtin_amdgcn_rcpf(1.f + e) : 1.f / (1.f + e), q = e * r;
  t = z < 0.f ? r : q;
  return z < 0.f ? q : r;
}

// gelu(z) = z P(z), P the normal distribution function, and its density p: derivative P + z p.
// FAST: 1 - P(|z|) by Abramowitz and Stegun 7.1.26 (absolute error 0.75e-7), which shares the density's
// exponential.
template <bool FAST> TW_DEV float normal_cdf(float z, float &density) {
  const float e = FAST ? __builtin_amdgcn_exp2f(z * z * -0.72134752044448170368f) : expf(-0.5f * z * z);
  density = 0.39894228040143267794f * e;
  if constexpr (FAST) {
    const float t = __builtin_amdgcn_rcpf(fmaf(fabsf(z), 0.3275911f * 0.70710678118654752440f, 1.f));
    const float q = t * fmaf(t, fmaf(t, fmaf(t, fmaf(t, 0.5f * 1.061405429f, 0.5f * -1.453152027f), 0.5f * 1.421413741f),
                                     0.5f * -0.284496736f),
                             0.5f * 0.254829592f) * e;
    return z < 0.f ? q : 1.f - q;
  } else {
    return 0.5f * erfcf(-0.70710678118654752440f * z);
  }
}

// 2 a of gelu_tanh(z) = z (1 + tanh a) / 2 = z sigmoid(2 a)
constexpr float kTanhC = 1.59576912160573071176f, kTanhK = 0.044715f;
TW_DEV float tanh_arg(float z) { return kTanhC * fmaf(kTanhK * z * z, z, z); }

template <int ACT, bool FAST> TW_DEV float act_of(float z) {
  if constexpr (ACT == kActRelu) return z < 0.f ? 0.f : z;            // a NaN stays one
  else if constexpr (ACT == kActSilu) return z * sigmoid_of<FAST>(z);
  else if constexpr (ACT == kActGelu) {
    float density;
    return z * normal_cdf<FAST>(z, density);
  } else if constexpr (ACT == kActGeluTanh) return z * sigmoid_of<FAST>(tanh_arg(z));
  else return z;
}

// The activation, and its derivative in d.
template <int ACT, bool FAST> TW_DEV float act_grad(float z, float &d) {
  if constexpr (ACT == kActRelu) {
    d = z > 0.f ? 1.f : z <= 0.f ? 0.f : z;
    return z < 0.f ? 0.f : z;
  } else if constexpr (ACT == kActSilu) {
    float t;
    const float s = sigmoid_pair<FAST>(z, t);
    d = s * fmaf(z, t, 1.f);
    return z * s;
  } else if constexpr (ACT == kActGelu) {
    float density;
    const float p = normal_cdf<FAST>(z, density);
    d = fmaf(z, density, p);
    return z * p;
  } else if constexpr (ACT == kActGeluTanh) {
    float t;
    const float s = sigmoid_pair<FAST>(tanh_arg(z), t);
    // beyond 32 s t is zero, where z^2 would overflow against it
    const float c = __builtin_amdgcn_fmed3f(z, -32.f, 32.f);
    d = fmaf(c * s * t, kTanhC * fmaf(3.f * kTanhK * c, c, 1.f), s);
    return z * s;
  } else {
    d = 1.f;
    return z;
  }
}

// f(std::integral_constant<int, act>()): the activation is chosen once per workgroup, outside the
// unrolled loops over a tile's fragments.
template <typename F> TW_DEV void with_act(int act, F &&f) {
  switch (act) {
    case kActRelu: return f(std::integral_constant<int, kActRelu>());
    case kActSilu: return f(std::integral_constant<int, kActSilu>());
    case kActGelu: return f(std::integral_constant<int, kActGelu>());
    case kActGeluTanh: return f(std::integral_constant<int, kActGeluTanh>());
    default: return f(std::integral_constant<int, kActNone>());
  }
}

}  // namespace tw
