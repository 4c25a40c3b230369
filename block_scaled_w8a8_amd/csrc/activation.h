// The gated product's activation and its slope, shared by the forward epilogues and the backward
// kernel.
#pragma once
#include "device_common.h"

namespace bfq {

// 1 / (1 + exp(-z)). exp2 of the rounded product z * log2(e), corrected by that product's rounding
// error (first order), so the relative error stays at a few 2^-24 for every z rather than growing
// with |z|; past |z| = 88 exp is 0 or Inf and the result exactly 1 or 0.
__device__ __forceinline__ float sigmoid_f32(float z) {
    constexpr float kLog2e = 1.44269504088896340736f, kLog2eLo = 1.92596299e-8f, kLn2 = 0.69314718056f;
    const float t = -z * kLog2e;
    const float r = __builtin_fmaf(-z, kLog2eLo, __builtin_fmaf(-z, kLog2e, -t));
    const float c = __builtin_fabsf(t) < 150.f ? __builtin_fmaf(r, kLn2, 1.f) : 1.f;
    return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(t) * c);
}

// Both activations are g * sigmoid(z) with z = g (c1 + c3 g^2): SILU c1 = 1, c3 = 0; the tanh form
// of GELU c1 = 2 sqrt(2/pi), c3 = 0.044715 c1, as 0.5 (1 + tanh t) = sigmoid(2t). g^2 is capped
// where z has long saturated, so that c3 = 0 never meets an infinity.
__device__ __forceinline__ float gate_sigmoid(float g, float c1, float c3, float& g2) {
    g2 = __builtin_fminf(g * g, 1e30f);
    return sigmoid_f32(g * __builtin_fmaf(c3, g2, c1));
}

__device__ __forceinline__ float act_f32(float g, float c1, float c3) {
    float g2;
    return g * gate_sigmoid(g, c1, c3, g2);
}

// act(g), and its slope sigmoid + g sigmoid (1 - sigmoid) (c1 + 3 c3 g^2).
__device__ __forceinline__ float act_slope_f32(float g, float c1, float c3, float& slope) {
    float g2;
    const float p = gate_sigmoid(g, c1, c3, g2), a = g * p;
    const float q = a * (1.f - p);
    slope = __builtin_fmaf(q, __builtin_fmaf(3.f * c3, g2, c1), p);
    return a;
}

}  // namespace bfq
