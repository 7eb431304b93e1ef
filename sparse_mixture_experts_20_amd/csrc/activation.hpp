// Activations, evaluated in fp32 (private; not part of the C ABI): the GELU
// formula of every expert and linear product, and the activations of the
// few-token layer and of the linear product.
#pragma once

#include "common.hpp"

namespace moe {

constexpr int kActNone = 2;   // MOE_ACT_NONE of the C ABI (linear product only)

// 1 - erf(u), u >= 0, and e^{-u^2}: Abramowitz and Stegun, Handbook of
// Mathematical Functions, formula 7.1.26: 1 - erf(u) = (a1 t + a2 t^2 + a3 t^3 +
// a4 t^4 + a5 t^5) e^{-u^2}, t = 1 / (1 + p u), with absolute error below 1.5e-7.
// The error is absolute: relative to 1 - erf(u) it grows along the tail (5e-5 at
// u sqrt 2 = 3, 1.6e-3 at 5, 1e-2 at 8).
__device__ __forceinline__ float erfc_as(float u, float &ex) {
    const float t = __builtin_amdgcn_rcpf(fmaf(0.3275911f, u, 1.0f));
    const float poly =
        t * fmaf(t, fmaf(t, fmaf(t, fmaf(t, 1.061405429f, -1.453152027f), 1.421413741f),
                         -0.284496736f),
                 0.254829592f);
    ex = __expf(-u * u);
    return poly * ex;
}

// GELU z Phi(z), Phi(z) = (1 + erf(z / sqrt 2)) / 2; for z < 0 from the complement,
// so that nothing cancels. In exact arithmetic the formula is within 2.2e-7 of
// the GELU for every z (far below the bf16 rounding that mostly follows, and a few
// fp32 steps of values of order one), but its far negative tail holds only the
// relative accuracy above.
__device__ __forceinline__ float gelu(float z) {
    float ex;
    const float q = erfc_as(fabsf(z) * 0.70710678118654752f, ex);
    return 0.5f * z * (z >= 0.f ? 2.0f - q : q);
}

// Its derivative Phi(z) + z phi(z): Phi from the same erf formula (within 1e-7),
// phi(z) = e^{-z^2 / 2} / sqrt(2 pi) from the same exponential.
__device__ __forceinline__ float gelu_grad(float z) {
    float ex;
    const float q = erfc_as(fabsf(z) * 0.70710678118654752f, ex);
    const float Phi = 0.5f * (z >= 0.f ? 2.0f - q : q);
    return fmaf(z * 0.39894228040143268f, ex, Phi);
}

// The same with the tails cut where the fp32 result has long been z or 0 (1 or 0):
// an infinite z gives its limit, where the formulas have 0 times infinity. (The
// grouped expert products use the formulas as they are: GELU of -inf is NaN there.)
__device__ __forceinline__ float act_gelu(float z) {
    const float r = gelu(z);
    return z < -16.f ? 0.f : r;
}
__device__ __forceinline__ float act_gelu_grad(float z) {
    const float r = gelu_grad(z);
    return fabsf(z) > 16.f ? (z > 0.f ? 1.f : 0.f) : r;
}

// ReLU keeps a NaN (fmaxf would turn it into 0 and hide it).
__device__ __forceinline__ float act_relu(float z) { return z < 0.f ? 0.f : z; }

__device__ __forceinline__ float activate(float z, int act) {
    return act == kActGelu ? act_gelu(z) : act == kActRelu ? act_relu(z) : z;
}

}  // namespace moe
