// act.cuh -- the activations of a product's epilogue and their derivatives.
#pragma once

#include <cuda_runtime.h>

#include "skinny_layer.h"

namespace skinny {

__host__ __device__ constexpr bool act_gated(int act) { return act == SKINNY_ACT_SWIGLU || act == SKINNY_ACT_GEGLU; }
__host__ __device__ constexpr bool act_gelu(int act) { return act == SKINNY_ACT_GELU || act == SKINNY_ACT_GEGLU; }

// Both are z * sigmoid(u): u = z (SiLU), or 2 sqrt(2 / pi) (z + 0.044715 z^3), where
// (1 + tanh(u / 2)) / 2 = sigmoid(u).
constexpr float kGelu2 = 1.5957691216057308f, kGeluCube = 0.044715f;

// The quotients are __fdividef's: within two steps, and 0 for divisors past 2^126, where the quotient has vanished.
__device__ __forceinline__ float act_value(int act, float z) {
    if (act == SKINNY_ACT_NONE) return z;
    const float u = act_gelu(act) ? kGelu2 * (z + kGeluCube * z * z * z) : z;
    return __fdividef(z, 1.f + expf(-u));
}

// act(z) and act'(z) = s + z s (1 - s) u'(z), s = sigmoid(u); where s (1 - s) has vanished, u' may have overflowed
// and the second term is none.
template <bool GELU>
__device__ __forceinline__ void act_both(float z, float &a, float &da) {
    float u = z, du = 1.f;
    if (GELU) {
        u = kGelu2 * (z + kGeluCube * z * z * z);
        du = kGelu2 * (1.f + 3.f * kGeluCube * z * z);
    }
    const float s = __fdividef(1.f, 1.f + expf(-u));
    a = z * s;
    const float t = s * (1.f - s);
    da = t == 0.f ? s : fmaf(a * (1.f - s), du, s);
}

}  // namespace skinny
