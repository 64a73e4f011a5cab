// Activations of the gated feed-forward block and their slopes, in float.
//   0  SiLU   x s(x), s the logistic function;  slope s (1 + x (1 - s))
//   1  GELU   x P(x), erf form;                 slope P + x p, p the normal density
// The normal distribution's tail comes from Hastings' rational approximation
// as printed in Abramowitz & Stegun, Handbook of Mathematical Functions,
// formula 7.1.26 (absolute error at most 1.5e-7, a thousandth of bf16's
// rounding at 1); its exponential, exp(-x^2 / 2), is the density's too.
#pragma once

namespace rtlynx {

template <int ACT>
__device__ __forceinline__ void act_both(float x, float& value, float& slope) {
    if constexpr (ACT == 0) {
        const float s = __fdividef(1.0f, 1.0f + __expf(-x));
        value = x * s;
        slope = s * fmaf(x, 1.0f - s, 1.0f);
    } else {
        const float z = fabsf(x) * 0.70710678118654752f;
        const float t = __fdividef(1.0f, fmaf(0.3275911f, z, 1.0f));
        float poly = fmaf(t, 1.061405429f, -1.453152027f);
        poly = fmaf(t, poly, 1.421413741f);
        poly = fmaf(t, poly, -0.284496736f);
        poly = fmaf(t, poly, 0.254829592f);
        const float e = __expf(-0.5f * x * x);
        const float tail = 0.5f * (poly * t) * e;
        const float p = x >= 0.0f ? 1.0f - tail : tail;
        value = x * p;
        slope = fmaf(x * 0.3989422804014327f, e, p);
    }
}

template <int ACT>
__device__ __forceinline__ float act_value(float x) {
    float value, slope;
    act_both<ACT>(x, value, slope);
    return value;
}

}  // namespace rtlynx
