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
        // Phi(g) = erfc(-g / sqrt(2)) / 2 with erfc(x) = poly(t) exp(-x^2), t = 1 / (1 + p x), for x >= 0: Abramowitz
        // and Stegun, "Handbook of Mathematical Functions", 7.1.26 (off by 1.5e-7 at most, and by about 1e-6 of
        // itself far out), which shares its exponential with the slope.  CUDA's normcdff, exact to a few steps, took
        // the epilogue longer than the products (forward 4096 x 512 x 2048: 32 us, with this 16).
        const float x = 0.7071067811865476f * fabsf(g);
        const float t = __fdividef(1.f, fmaf(0.3275911f, x, 1.f));
        const float e = exp2_approx(-0.7213475204444817f * g * g);
        const float poly = t * fmaf(t, fmaf(t, fmaf(t, fmaf(t, 1.061405429f, -1.453152027f), 1.421413741f), -0.284496736f),
                                    0.254829592f);
        const float tail = 0.5f * poly * e;  // of the side away from 0
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
