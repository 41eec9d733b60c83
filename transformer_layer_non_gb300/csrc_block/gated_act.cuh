// gated_act.cuh -- the activations of the gated block, and their slopes.
#pragma once

#include "../csrc_vocab/vec.cuh"
#include "block_internal.h"

namespace ls {
namespace {

// act(g), and its slope.
struct ActValue {
    float a, slope;
};
__device__ __forceinline__ float sigmoid(float x) {
    return __fdividef(1.f, 1.f + exp2_approx(-1.4426950408889634f * x));  // 0 where the exponential is infinite
}
template <int ACT> __device__ __forceinline__ ActValue act_of(float g) {
    if constexpr (ACT == LS_ACT_RELU) {
        return {g > 0.f ? g : g != g ? g : 0.f, g > 0.f ? 1.f : 0.f};
    } else if constexpr (ACT == LS_ACT_SILU) {
        const float s = sigmoid(g);
        return {g * s, s * (1.f + g * (1.f - s))};
    } else if constexpr (ACT == LS_ACT_GELU) {
        // Phi(-x) = erfc(x / sqrt(2)) / 2 = poly(t) exp(-x^2 / 2), t = 1 / (1 + p x), for x >= 0, which shares its
        // exponential with the slope.  poly: of degree 7 without a constant, as x Phi(-x) exp(x^2 / 2) has a limit; its
        // coefficients and p were fitted here for the least relative error up to x = 13.4, where the exponential ends:
        // 7.5e-7 of Phi, in FP32 1.2e-6 for x up to 3, growing with the rounding of x^2 / 2 to 8.3e-6 at 13.  (A
        // formula of degree 5 with an absolute bound was off by 5e-4 of Phi at -4 and 1e-2 at -8.)  One degree more:
        // 3.9e-7 next to 0, and 1.5 % of a step.  CUDA's normcdff took the epilogue longer than the products (forward
        // 4096 x 512 x 2048 BF16: 32 us, with this 17.6).
        const float t = __fdividef(1.f, fmaf(0.36062446f, fabsf(g), 1.f));
        const float e = exp2_approx(-0.7213475204444817f * g * g);
        float poly = fmaf(t, 0.04765733f, -0.18095501f);
        poly = fmaf(t, poly, 0.18110242f);
        poly = fmaf(t, poly, 0.026237981f);
        poly = fmaf(t, poly, 0.14000161f);
        poly = fmaf(t, poly, 0.14199094f);
        poly = fmaf(t, poly, 0.14396478f);
        const float tail = t * poly * e;  // of the side away from 0
        const float phi = g > 0.f ? 1.f - tail : tail;
        return {g * phi, fmaf(g * 0.3989422804014327f, e, phi)};
    } else {  // 0.5 (1 + tanh y) = sigmoid(2 y)
        const float k = 1.5957691216057308f, q = g * g;
        const float s = sigmoid(k * g * fmaf(0.044715f, q, 1.f));
        const float t = s * (1.f - s);
        return {g * s, s + (t > 0.f ? g * t * k * fmaf(0.134145f, q, 1.f) : 0.f)};
    }
}

}  // namespace
}  // namespace ls
