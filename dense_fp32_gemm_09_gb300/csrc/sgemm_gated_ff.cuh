// The element-wise half of the gated feed-forward block: activations, and the form in which
// the pre-activations are kept.
#pragma once

#include "sgemm_act8.cuh"

namespace sgemm {
namespace ff {

using mx4::from_float;
using mx4::kBf16;
using mx4::to_float;

// act(g) = g s with s = 1 / (1 + e^-z): z = g for silu; for the tanh form of gelu,
// g (1 + tanh t) / 2 with t = c (g + 0.044715 g^3), c = sqrt(2 / pi), it is z = 2 t.  The
// approximate exponential and reciprocal are off by a few 2^-22 of s, far below the 2-byte
// rounding of what is made of it.
constexpr float kGeluC = 1.5957691216057308f;      // 2 sqrt(2 / pi)
constexpr float kGeluCube = 0.044715f;

struct Act {
    float s, slope_z, g, near;
    template <int ACT>
    __device__ __forceinline__ static Act of(float g) {
        Act a;
        a.g = a.near = g;
        float z = g;
        a.slope_z = 1.0f;
        if (ACT == kGeluTanh) {
            // From |g| = 30 on s is 0 or 1, and beyond 10^19 g^2 would overflow.  (A NaN stays one.)
            const float c = fabsf(g) > 30.0f ? copysignf(30.0f, g) : g, q = c * c;
            a.near = c;
            z = kGeluC * c * fmaf(kGeluCube, q, 1.0f);
            a.slope_z = kGeluC * fmaf(3.0f * kGeluCube, q, 1.0f);
        }
        a.s = __fdividef(1.0f, 1.0f + __expf(-z));
        return a;
    }
    __device__ __forceinline__ float value() const { return g * s; }
    // (With g itself, g slope_z is infinite from -1.8e36 down, and 0 times that NaN.)
    __device__ __forceinline__ float slope() const { return s * fmaf(near * (1.0f - s), slope_z, 1.0f); }
};
template <int ACT>
__device__ __forceinline__ float act(float g) { return Act::of<ACT>(g).value(); }

}  // namespace ff
}  // namespace sgemm
