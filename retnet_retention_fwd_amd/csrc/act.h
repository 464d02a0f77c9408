// Activations of the projections and their slopes.  All but the threshold are z P(z) with P a
// distribution function, and P is taken where it is small, so that large negative z keep a
// small value and not the difference of two large ones.
#pragma once

#include <hip/hip_runtime.h>

#include "../../include/retention.h"
#include "vec_io.h"

namespace retn {
namespace {

// |z| cut to `most`, beyond which P is 0 or 1 in fp32; a NaN stays one.
__device__ __forceinline__ float cut(float z, float most) { return fabsf(z) > most ? copysignf(most, z) : z; }

// Normal distribution function and e^(-z^2/2).  The complementary error function of |z|/sqrt(2)
// is Hastings' t (a1 + t (a2 + ...)) e^(-z^2/2), t = 1 / (1 + p |z|/sqrt(2)) (Abramowitz and
// Stegun 7.1.26, off by 1.5e-7 at most, 1.3 half steps of P in fp32).
__device__ __forceinline__ float normal_cdf(float z, float& e) {
    const float t = rcp(fmaf(fabsf(z), 0.3275911f * 0.70710678118654752f, 1.f));
    float p = fmaf(t, 1.061405429f, -1.453152027f);
    p = fmaf(t, p, 1.421413741f);
    p = fmaf(t, p, -0.284496736f);
    p = fmaf(t, p, 0.254829592f);
    e = __builtin_amdgcn_exp2f(z * z * (-0.5f * kLog2e));
    const float q = 0.5f * t * p * e;
    return z > 0.f ? 1.f - q : q;
}
// 2 sqrt(2/pi) (z + 0.044715 z^3): (1 + tanh(./2)) / 2 is its logistic function.
__device__ __forceinline__ float tanh_arg(float z) {
    return 1.5957691216057308f * fmaf(0.044715f * z * z, z, z);
}

__device__ __forceinline__ float act_value(float z, int act) {
    float e;
    switch (act) {
        case RETN_ACT_RELU: return z <= 0.f ? 0.f : z;
        case RETN_ACT_GELU: return z * normal_cdf(cut(z, 16.f), e);
        case RETN_ACT_GELU_TANH: return z * sigmoid_f(tanh_arg(cut(z, 16.f)));
        case RETN_ACT_SILU: return z * sigmoid_f(z);
        default: return z;
    }
}
// The value and its derivative.
__device__ __forceinline__ float act_slope(float z, int act, float& value) {
    switch (act) {
        case RETN_ACT_RELU: value = z <= 0.f ? 0.f : z; return z > 0.f ? 1.f : 0.f;
        case RETN_ACT_GELU: {
            const float c = cut(z, 16.f);
            float e;
            const float p = normal_cdf(c, e);
            value = z * p;
            return fmaf(c * 0.3989422804014327f, e, p);
        }
        case RETN_ACT_GELU_TANH: {
            const float c = cut(z, 16.f), p = sigmoid_f(tanh_arg(c));
            value = z * p;
            return fmaf(c * p * (1.f - p), 1.5957691216057308f * fmaf(3.f * 0.044715f * c, c, 1.f), p);
        }
        case RETN_ACT_SILU: {
            const float c = cut(z, 100.f), p = sigmoid_f(c);
            value = z * p;
            return fmaf(c * p, 1.f - p, p);
        }
        default: value = z; return 1.f;
    }
}

}  // namespace
}  // namespace retn
