// gated_act.cuh -- activations of the dense gated FFN.
#pragma once
#include "tw_common.cuh"

namespace tw {

// act(z) and act'(z).  exp and the division are the approximate instructions: the
// results are rounded to bf16.  For negative z no factor is a difference from 1, so that small
// values keep their digits too (0.5 (1 + erf) is 4% off at z = -5 and zero from -5.6 on).
template <int ACT>
TW_DEV void activate(float z, float& a, float& da) {
  if (ACT == TW_ACT_RELU) {
    a = z > 0.f ? z : 0.f;
    da = z > 0.f ? 1.f : 0.f;
    if (z != z) a = da = z;
  } else if (ACT == TW_ACT_SILU) {
    const float p = __fdividef(1.f, 1.f + __expf(-z));
    a = z * p;
    da = p * fmaf(z, 1.f - p, 1.f);
  } else if (ACT == TW_ACT_GELU) {
    // The normal distribution's tail is Phi(-t) = exp(-t^2/2) E(t), and E falls like 1/t: E is
    // s P(s), s = 1/(1 + 0.36 t), with the polynomial of least relative error on [0, 13.5]
    // (8e-7; beyond, Phi(-t) is below 2^-126).  One exp then serves Phi and its derivative: a
    // step of 1003 tokens at 1024 x 4096 takes 106 us, with erfcf 122.
    const float e = __expf(-0.5f * z * z), s = __fdividef(1.f, fmaf(0.36f, fabsf(z), 1.f));
    float q = 0.0473446f;
    q = fmaf(q, s, -0.180751756f);
    q = fmaf(q, s, 0.182297736f);
    q = fmaf(q, s, 0.0256237164f);
    q = fmaf(q, s, 0.140057474f);
    q = fmaf(q, s, 0.141710669f);
    q = fmaf(q, s, 0.143717438f) * s * e;
    const float cdf = z < 0.f ? q : 1.f - q;
    a = z * cdf;
    da = fmaf(z * 0.39894228f, e, cdf);
  } else {
    // 0.5 (1 + tanh(k)) = 1 / (1 + exp(-2k)) =: p, k = sqrt(2/pi) (z + 0.044715 z^3)
    const float p =
        __fdividef(1.f, 1.f + __expf(-1.5957691f * z * fmaf(0.044715f * z, z, 1.f)));
    a = z * p;
    // far out p (1 - p) is zero, and z^2 must not be infinite beside it
    const float t = fminf(fabsf(z), 1e9f);
    da = fmaf(z * p * (1.f - p), 1.5957691f * fmaf(0.134145f * t, t, 1.f), p);
  }
}

}  // namespace tw
