// Activations of the gated feed-forward block and their slopes, in float.
//   0  SiLU   x s(x), s the logistic function;  slope s (1 + x (1 - s))
//   1  GELU   x P(x), erf form;                 slope P + x p, p the normal density
// The normal distribution's tail is e^(-z^2) t q(t), t = 1 / (1 + 0.49 z), z =
// |x| / sqrt 2: the scaled tail erfcx(z) / 2 goes to zero as t does, so a
// polynomial without constant term holds its relative error all the way out.
// q's seven coefficients are a fit of this project's own to erfcx in 64 bits
// (Lawson's iterated least squares) that keeps the tail to 2e-7 absolute and 1e-4
// relative, a fortieth of a bf16 half step: far out the value of GELU is the
// tail's, so the relative error is what reaches H.  Its exponential, exp(-x^2 / 2),
// is the density's too.
// SiLU goes to zero below -87.3, where its value is under 2^-118.
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
        const float t = __fdividef(1.0f, fmaf(0.49f, z, 1.0f));
        float poly = fmaf(t, 0.04136807471513748f, -0.1756596863269806f);
        poly = fmaf(t, poly, 0.20399731397628784f);
        poly = fmaf(t, poly, 0.018366925418376923f);
        poly = fmaf(t, poly, 0.136725053191185f);
        poly = fmaf(t, poly, 0.13695867359638214f);
        poly = fmaf(t, poly, 0.13824363052845f);
        const float e = __expf(-0.5f * x * x);
        const float tail = poly * t * e;
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
