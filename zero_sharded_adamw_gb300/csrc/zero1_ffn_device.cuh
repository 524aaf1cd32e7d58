// zero1_ffn_device.cuh -- the gated feed-forward block's activations, for its
// kernels.
#pragma once

#include <cuda_runtime.h>

namespace zero1 {

// act(g), and its derivative, in fp32.  The sigmoid from the approximate
// exponential and quotient: 2e-6 of itself at |g| = 20, a thousandth of a
// bf16 rounding.
__device__ __forceinline__ float sigmoid(float g) { return __fdividef(1.f, 1.f + __expf(-g)); }

constexpr float kRootHalf = 0.70710678118654752f, kDensity = 0.39894228040143268f;   // sqrt(1/2), 1/sqrt(2 pi)
constexpr float kRoot2Pi = 0.79788456080286536f, kCube = 0.044715f;                  // sqrt(2/pi)

template <bool SLOPE>
__device__ __forceinline__ void activate(int act, float g, float &a, float &slope)
{
    if (act == 0) {              // silu
        const float s = sigmoid(g);
        a = g * s;
        if (SLOPE) slope = s + a * (1.f - s);
    } else if (act == 1) {       // gelu
        const float cdf = 0.5f + 0.5f * erff(g * kRootHalf);
        a = g * cdf;
        if (SLOPE) slope = cdf + g * kDensity * __expf(-0.5f * g * g);
    } else if (act == 2) {       // gelu, its tanh form: (1 + tanh(z)) / 2 = sigmoid(2 z)
        const float s = sigmoid(2.f * kRoot2Pi * (g + kCube * g * g * g));
        a = g * s;
        if (SLOPE) slope = s + 2.f * a * (1.f - s) * kRoot2Pi * (1.f + 3.f * kCube * g * g);
    } else {                     // relu; NaN stays NaN
        a = g <= 0.f ? 0.f : g;
        if (SLOPE) slope = g <= 0.f ? 0.f : 1.f;
    }
}

}  // namespace zero1
