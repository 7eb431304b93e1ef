// Activations of the few-token layer and of the linear product, evaluated in
// fp32 (private; not part of the C ABI).
#pragma once

#include "common.hpp"

namespace moe {

constexpr int kActNone = 2;   // MOE_ACT_NONE of the C ABI (linear product only)

// 1 - erf(u), u >= 0, and e^{-u^2}: Abramowitz and Stegun, Handbook of
// Mathematical Functions, formula 7.1.26 (absolute error below 1.5e-7), the
// evaluation the grouped expert products use.
__device__ __forceinline__ float erfc_as(float u, float &ex) {
    const float t = __builtin_amdgcn_rcpf(fmaf(0.3275911f, u, 1.0f));
    const float poly =
        t * fmaf(t, fmaf(t, fmaf(t, fmaf(t, 1.061405429f, -1.453152027f), 1.421413741f),
                         -0.284496736f),
                 0.254829592f);
    ex = __expf(-u * u);
    return poly * ex;
}

// GELU z Phi(z); for z < 0 the complement is used directly, so small values
// keep their relative accuracy. -inf gives -0 * ... = NaN in the formula, so
// the tails are cut where the fp32 result has long been z or 0.
__device__ __forceinline__ float act_gelu(float z) {
    float ex;
    const float q = erfc_as(fabsf(z) * 0.70710678118654752f, ex);
    const float r = 0.5f * z * (z >= 0.f ? 2.0f - q : q);
    return z < -16.f ? 0.f : r;
}

// Its derivative Phi(z) + z phi(z).
__device__ __forceinline__ float act_gelu_grad(float z) {
    float ex;
    const float q = erfc_as(fabsf(z) * 0.70710678118654752f, ex);
    const float Phi = 0.5f * (z >= 0.f ? 2.0f - q : q);
    const float r = fmaf(z * 0.39894228040143268f, ex, Phi);
    return fabsf(z) > 16.f ? (z > 0.f ? 1.f : 0.f) : r;
}

// ReLU keeps a NaN (fmaxf would turn it into 0 and hide it).
__device__ __forceinline__ float act_relu(float z) { return z < 0.f ? 0.f : z; }

__device__ __forceinline__ float activate(float z, int act) {
    return act == kActGelu ? act_gelu(z) : act == kActRelu ? act_relu(z) : z;
}
__device__ __forceinline__ float activate_grad(float z, int act) {
    return act == kActGelu ? act_gelu_grad(z) : act == kActRelu ? (z > 0.f ? 1.f : 0.f) : 1.f;
}

}  // namespace moe
