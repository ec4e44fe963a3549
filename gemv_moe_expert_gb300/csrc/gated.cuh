// gated.cuh -- the activations of the gated projection and their derivatives.
#pragma once

#include "../../include/gbmm.h"
#include "device_common.cuh"

namespace gbmm {

// 1 / (1 + e^-v); 0 and 1 at the far ends
__device__ __forceinline__ float sigmoid(float v) { return 1.f / (1.f + expf(-v)); }

// gelu's tanh form is v sigmoid(2 y), y = sqrt(2 / pi) (v + 0.044715 v^3), since
// (1 + tanh y) / 2 = sigmoid(2 y)
__device__ __forceinline__ float gelu_tanh_arg(float v) {
    return 1.5957691216057308f * v * fmaf(0.044715f, v * v, 1.f);
}

__device__ __forceinline__ float gate_act(int act, float v) {
    switch (act) {
    case GBMM_GATE_SILU: return v * sigmoid(v);
    case GBMM_GATE_GELU: return 0.5f * v * erfcf(-0.70710678118654752f * v);
    case GBMM_GATE_GELU_TANH: return v * sigmoid(gelu_tanh_arg(v));
    default: return fmaxf(v, 0.f) + (v != v ? v : 0.f);
    }
}

// The same for results of 16 bits: errors of a few 2^-22 relative to v, and 2^-14 of the result at the far ends.  The
// exponential and the quotient are the hardware's approximations.  erfc(z) / 2 = e^(-z z) t P(t), t = 1 / (1 + 0.37 z), z >=
// 0: P of degree 6 fitted to erfc(z) e^(z z) by weighted least squares until the relative error was even over 0..9.5
// (7.4e-7; with f32's roundings 1.2e-6).  An approximation that is even in absolute error, with two terms less, is off by
// 5e-4 of gelu(-4) and 1 % of gelu(-8), more than half a step of either type.
__device__ __forceinline__ float sigmoid_16(float v) { return __fdividef(1.f, 1.f + __expf(-v)); }
__device__ __forceinline__ float half_erfc_16(float z) {  // erfc(|z|) / 2
    const float y = fabsf(z), t = __fdividef(1.f, fmaf(0.37f, y, 1.f));
    float q = fmaf(-0.07127543f, t, 0.21782866f);
    q = fmaf(q, t, -0.09321387f);
    q = fmaf(q, t, 0.15870127f);
    q = fmaf(q, t, 0.07632857f);
    q = fmaf(q, t, 0.10744123f);
    q = fmaf(q, t, 0.10418995f);
    return q * t * __expf(-y * y);
}
__device__ __forceinline__ float gate_act_16(int act, float v) {
    switch (act) {
    case GBMM_GATE_SILU: return v * sigmoid_16(v);
    case GBMM_GATE_GELU: {
        const float c = half_erfc_16(0.70710678118654752f * v);
        return v * (v > 0.f ? 1.f - c : c);
    }
    case GBMM_GATE_GELU_TANH: return v * sigmoid_16(gelu_tanh_arg(v));
    default: return fmaxf(v, 0.f) + (v != v ? v : 0.f);
    }
}

// act(v), and its derivative (relu: 0 at 0)
__device__ __forceinline__ float gate_act_slope(int act, float v, float *slope) {
    switch (act) {
    case GBMM_GATE_SILU: {
        const float s = sigmoid(v);
        *slope = s * fmaf(v, 1.f - s, 1.f);
        return v * s;
    }
    case GBMM_GATE_GELU: {
        const float c = 0.5f * erfcf(-0.70710678118654752f * v);
        *slope = fmaf(v, 0.3989422804014327f * expf(-0.5f * v * v), c);
        return v * c;
    }
    case GBMM_GATE_GELU_TANH: {
        const float s = sigmoid(gelu_tanh_arg(v)), t = s * (1.f - s);
        // the second term ends where the sigmoid is flat
        const float d = t == 0.f ? 0.f : v * t * 1.5957691216057308f * fmaf(3.f * 0.044715f, v * v, 1.f);
        *slope = s + d;
        return v * s;
    }
    default:
        *slope = v > 0.f ? 1.f : (v != v ? v : 0.f);
        return fmaxf(v, 0.f) + (v != v ? v : 0.f);
    }
}

// the same for results of 16 bits
__device__ __forceinline__ float gate_act_slope_16(int act, float v, float *slope) {
    switch (act) {
    case GBMM_GATE_SILU: {
        const float s = sigmoid_16(v);
        *slope = s * fmaf(v, 1.f - s, 1.f);
        return v * s;
    }
    case GBMM_GATE_GELU: {
        const float h = half_erfc_16(0.70710678118654752f * v), c = v > 0.f ? 1.f - h : h;
        *slope = fmaf(v, 0.3989422804014327f * __expf(-0.5f * v * v), c);
        return v * c;
    }
    case GBMM_GATE_GELU_TANH: {
        const float s = sigmoid_16(gelu_tanh_arg(v)), t = s * (1.f - s);
        const float d = t == 0.f ? 0.f : v * t * 1.5957691216057308f * fmaf(3.f * 0.044715f, v * v, 1.f);
        *slope = s + d;
        return v * s;
    }
    default: return gate_act_slope(act, v, slope);
    }
}

}  // namespace gbmm
