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

// ACT: ZERO1_ACT_SILU, _GELU, _GELU_TANH, _RELU.
template <int ACT, bool SLOPE>
__device__ __forceinline__ void activate(float g, float &a, float &slope)
{
    if (ACT == 0) {
        const float s = sigmoid(g);
        a = g * s;
        if (SLOPE) slope = s + a * (1.f - s);
    } else if (ACT == 1) {
        const float cdf = 0.5f + 0.5f * erff(g * kRootHalf);
        a = g * cdf;
        if (SLOPE) slope = cdf + g * kDensity * __expf(-0.5f * g * g);
    } else if (ACT == 2) {       // (1 + tanh(z)) / 2 = sigmoid(2 z)
        const float s = sigmoid(2.f * kRoot2Pi * (g + kCube * g * g * g));
        a = g * s;
        if (SLOPE) slope = s + 2.f * a * (1.f - s) * kRoot2Pi * (1.f + 3.f * kCube * g * g);
    } else {                     // NaN stays NaN
        a = g <= 0.f ? 0.f : g;
        if (SLOPE) slope = g <= 0.f ? 0.f : 1.f;
    }
}

// f(ActOf<ACT>{}): the activation is looked up once for many entries.
template <int ACT>
struct ActOf {
    static constexpr int value = ACT;
};
template <typename F>
__device__ __forceinline__ void with_activation(int act, F f)
{
    if (act == 0) f(ActOf<0>{});
    else if (act == 1) f(ActOf<1>{});
    else if (act == 2) f(ActOf<2>{});
    else f(ActOf<3>{});
}

}  // namespace zero1
