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

DM_DEV float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// The normal CDF, and e = exp(-x^2 / 2).  (1 + erf(x / sqrt 2)) / 2 cancels for negative x:
// 4% off at -5, nothing left at -5.6.  Phi(-a) = e g(a) with a smooth g, 1/2 at 0 and
// 1 / (a sqrt(2 pi)) far out: g = t P(t), t = 1 / (1 + 0.3 a), P a degree-7 fit to
// erfcx(a / sqrt 2) / 2 of least largest relative error (1.3e-7 up to a = 13.5, where e ends).
// In fp32 7e-7 up to a = 3, 5e-6 at 10, where rounding x^2 decides.  No branches, and the
// density's e for the gradient: 515 tokens forward through 3584/18944 164 us (166 with erff,
// 180 with erfcf), 301 back through 1536/8960 89 (93, 101).
DM_DEV float normal_cdf(float x, float& e) {
  const float a = fabsf(x);
  const float t = fast_rcp(fmaf(0.3f, a, 1.f));
  e = ex2(x * x * -0.72134752f);
  float p = 0.035931737f;
  p = fmaf(p, t, -0.15827599f);
  p = fmaf(p, t, 0.2082066f);
  p = fmaf(p, t, -0.055393815f);
  p = fmaf(p, t, 0.12946917f);
  p = fmaf(p, t, 0.0996375f);
  p = fmaf(p, t, 0.12079836f);
  p = fmaf(p, t, 0.11962639f);
  const float tail = e * (t * p);
  return x < 0.f ? tail : 1.f - tail;
}

// act(x) and, for the gradient, act'(x), in fp32.  The tanh form is taken as
// x * sigmoid(2 sqrt(2/pi) (x + 0.044715 x^3)): (1 + tanh y) / 2 = sigmoid(2 y).
template <int ACT>
DM_DEV float act_value(float x) {
  if (ACT == DMUON_ACT_SILU) return x * sigmoid(x);
  if (ACT == DMUON_ACT_GELU) {
    float e;
    return x * normal_cdf(x, e);
  }
  return x * sigmoid(1.59576912f * fmaf(0.044715f * x * x, x, x));
}
template <int ACT>
DM_DEV void act_both(float x, float& a, float& da) {
  if (ACT == DMUON_ACT_SILU) {
    const float s = sigmoid(x);
    a = x * s;
    da = s * fmaf(x, 1.f - s, 1.f);
  } else if (ACT == DMUON_ACT_GELU) {
    float e;
    const float phi = normal_cdf(x, e);
    a = x * phi;
    da = fmaf(x * 0.39894228f, e, phi);
  } else {
    const float s = sigmoid(1.59576912f * fmaf(0.044715f * x * x, x, x));
    a = x * s;
    // the polynomial is bounded: past 1e19 it overflows where s (1 - s) is 0
    const float poly = fminf(fmaf(0.134145f * x, x, 1.f), 1e30f);
    da = fmaf(x * s * (1.f - s), 1.59576912f * poly, s);
  }
}

}  // namespace dm
