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

// The normal distribution's weight beyond a >= 0, and e^(-a^2/2).  The weight is e^(-a^2/2) times a function
// that falls slowly, from 1/2 at 0 to 1 / (a sqrt(2 pi)), and that is t (c1 + t (c2 + ...)) with t = 1 / (1 + 0.305 a).
// The c are a fit of least relative error over 0 <= a <= 14 (1.6 half steps of fp32; 6.5 with the rounding of its
// terms), so the tail keeps its bits however small it is: in half steps of its own value it is off by 16 and,
// from the exponent's roundings, 1.5 a^2.  (Of seven terms the best is off by 15, of five by 589.)
__device__ __forceinline__ float normal_tail(float a, float& e) {
    const float t = rcp(fmaf(a, 0.305f, 1.f));
    float p = fmaf(t, 0.036698729f, -0.15298645f);
    p = fmaf(t, p, 0.1857138f);
    p = fmaf(t, p, -0.037974063f);
    p = fmaf(t, p, 0.12102026f);
    p = fmaf(t, p, 0.10342129f);
    p = fmaf(t, p, 0.12246675f);
    p = fmaf(t, p, 0.12163974f);
    e = __builtin_amdgcn_exp2f(a * a * (-0.5f * kLog2e));
    return t * p * e;
}
// The logistic function p of x, and p (1 - p).  Both from e^-|x|, which is one at most: 1 - p of a p next to one would
// lose its bits, and a slope takes them |z| times, or behind the cubic argument 30 times and more.
__device__ __forceinline__ float logistic(float x, float& pq) {
    const float e = __builtin_amdgcn_exp2f(fabsf(x) * -kLog2e), big = rcp(1.f + e), small = e * big;
    pq = big * small;
    return x > 0.f ? big : small;
}
// 2 sqrt(2/pi) (z + 0.044715 z^3): (1 + tanh(./2)) / 2 is its logistic function.
__device__ __forceinline__ float tanh_arg(float z) {
    return 1.5957691216057308f * fmaf(0.044715f * z * z, z, z);
}

template <int ACT>
__device__ __forceinline__ float act_value(float z) {
    if constexpr (ACT == RETN_ACT_RELU) {
        return z <= 0.f ? 0.f : z;
    } else if constexpr (ACT == RETN_ACT_GELU) {
        // z P(z) = max(z, 0) - |z| (1 - P(|z|))
        float e;
        const float a = fminf(fabsf(z), 16.f);
        return fmaf(-a, normal_tail(a, e), z <= 0.f ? 0.f : z);
    } else if constexpr (ACT == RETN_ACT_GELU_TANH) {
        return z * sigmoid_f(tanh_arg(z));
    } else {
        return z * sigmoid_f(z);
    }
}
// The derivative, and the value.
template <int ACT>
__device__ __forceinline__ float act_slope(float z, float& value) {
    if constexpr (ACT == RETN_ACT_RELU) {
        value = z <= 0.f ? 0.f : z;
        return z > 0.f ? 1.f : 0.f;
    } else if constexpr (ACT == RETN_ACT_GELU) {
        const float c = cut(z, 16.f);
        float e;
        const float a = fabsf(c), q = normal_tail(a, e), p = c > 0.f ? 1.f - q : q;
        value = fmaf(-a, q, z <= 0.f ? 0.f : z);     // as the forward's, also at the infinities
        return fmaf(c * 0.3989422804014327f, e, p);
    } else if constexpr (ACT == RETN_ACT_GELU_TANH) {
        float pq;
        const float c = cut(z, 16.f), p = logistic(tanh_arg(c), pq);
        value = z * p;
        return fmaf(c * pq, 1.5957691216057308f * fmaf(3.f * 0.044715f * c, c, 1.f), p);
    } else {
        float pq;
        const float c = cut(z, 100.f), p = logistic(c, pq);
        value = z * p;
        return fmaf(c, pq, p);
    }
}
template <int ACT>
__device__ __forceinline__ void act_values_as(float (&z)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) z[i] = act_value<ACT>(z[i]);
}
template <int ACT>
__device__ __forceinline__ void act_slopes_as(float (&z)[8], float (&value)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) z[i] = act_slope<ACT>(z[i], value[i]);
}
// z becomes its activation, in place.
__device__ __forceinline__ void act_values(float (&z)[8], int act) {
    switch (act) {
        case RETN_ACT_RELU: act_values_as<RETN_ACT_RELU>(z); break;
        case RETN_ACT_GELU: act_values_as<RETN_ACT_GELU>(z); break;
        case RETN_ACT_GELU_TANH: act_values_as<RETN_ACT_GELU_TANH>(z); break;
        case RETN_ACT_SILU: act_values_as<RETN_ACT_SILU>(z); break;
        default: break;
    }
}
// z becomes the slope at z, in place, and `value` the activation of z.
__device__ __forceinline__ void act_slopes(float (&z)[8], float (&value)[8], int act) {
    switch (act) {
        case RETN_ACT_RELU: act_slopes_as<RETN_ACT_RELU>(z, value); break;
        case RETN_ACT_GELU: act_slopes_as<RETN_ACT_GELU>(z, value); break;
        case RETN_ACT_GELU_TANH: act_slopes_as<RETN_ACT_GELU_TANH>(z, value); break;
        case RETN_ACT_SILU: act_slopes_as<RETN_ACT_SILU>(z, value); break;
        default:
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                value[i] = z[i];
                z[i] = 1.f;
            }
    }
}

}  // namespace
}  // namespace retn
