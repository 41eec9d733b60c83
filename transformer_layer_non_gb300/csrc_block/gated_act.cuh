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
        const float phi = normcdff(g);
        return {g * phi, phi + g * 0.3989422804014327f * exp2_approx(-0.7213475204444817f * g * g)};
    } else {  // 0.5 (1 + tanh y) = sigmoid(2 y)
        const float k = 1.5957691216057308f, q = g * g;
        const float s = sigmoid(k * g * fmaf(0.044715f, q, 1.f));
        const float t = s * (1.f - s);
        return {g * s, s + (t > 0.f ? g * t * k * fmaf(0.134145f, q, 1.f) : 0.f)};
    }
}

}  // namespace
}  // namespace ls
