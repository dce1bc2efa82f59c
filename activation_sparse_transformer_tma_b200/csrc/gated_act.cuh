// gated_act.cuh -- activations of the dense gated FFN.
#pragma once
#include "tw_common.cuh"

namespace tw {

// act(z) and act'(z).  exp and the division are the approximate instructions: the
// results are rounded to bf16.
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
    const float cdf = 0.5f * (1.f + erff(z * 0.70710678f));
    a = z * cdf;
    da = fmaf(z * 0.39894228f, __expf(-0.5f * z * z), cdf);
  } else {
    // 0.5 (1 + tanh(k)) = 1 / (1 + exp(-2k)) =: p, k = sqrt(2/pi) (z + 0.044715 z^3)
    const float p =
        __fdividef(1.f, 1.f + __expf(-1.5957691f * z * fmaf(0.044715f * z, z, 1.f)));
    a = z * p;
    da = fmaf(z * p * (1.f - p), 1.5957691f * fmaf(0.134145f * z, z, 1.f), p);
  }
}

}  // namespace tw
