// Activations of the gated feed-forward block.
#pragma once
#include "dmuon.h"
#include "ptx.cuh"

namespace dm {

DM_DEV float fast_rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
DM_DEV float sigmoid(float x) { return fast_rcp(1.f + __expf(-x)); }

// act(x) and, for the gradient, act'(x), in fp32.  The tanh form is taken as
// x * sigmoid(2 sqrt(2/pi) (x + 0.044715 x^3)): (1 + tanh y) / 2 = sigmoid(2 y).
template <int ACT>
DM_DEV float act_value(float x) {
  if (ACT == DMUON_ACT_SILU) return x * sigmoid(x);
  if (ACT == DMUON_ACT_GELU) return 0.5f * x * (1.f + erff(x * 0.70710678f));
  return x * sigmoid(1.59576912f * fmaf(0.044715f * x * x, x, x));
}
template <int ACT>
DM_DEV void act_both(float x, float& a, float& da) {
  if (ACT == DMUON_ACT_SILU) {
    const float s = sigmoid(x);
    a = x * s;
    da = s * fmaf(x, 1.f - s, 1.f);
  } else if (ACT == DMUON_ACT_GELU) {
    const float phi = 0.5f * (1.f + erff(x * 0.70710678f));
    a = x * phi;
    da = fmaf(x * 0.39894228f, __expf(-0.5f * x * x), phi);
  } else {
    const float s = sigmoid(1.59576912f * fmaf(0.044715f * x * x, x, x));
    a = x * s;
    // the polynomial is bounded: past 1e19 it overflows where s (1 - s) is 0
    const float poly = fminf(fmaf(0.134145f * x, x, 1.f), 1e30f);
    da = fmaf(x * s * (1.f - s), 1.59576912f * poly, s);
  }
}

}  // namespace dm
