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

}  // namespace gbmm
