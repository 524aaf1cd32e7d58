// zero1_ffn_device.cuh -- the gated feed-forward block's activations, for its
// kernels.
#pragma once

#include <cuda_runtime.h>

namespace zero1 {

// act(g), and its derivative, in fp32.  The sigmoid from the approximate
// exponential and quotient: 2e-6 of itself at |g| = 20, a thousandth of a
// bf16 rounding; 0 where it is below fp32's normal range (g < -87.3).
__device__ __forceinline__ float sigmoid(float g) { return __fdividef(1.f, 1.f + __expf(-g)); }

constexpr float kDensity = 0.39894228040143268f;                                     // 1/sqrt(2 pi)
constexpr float kRoot2Pi = 0.79788456080286536f, kCube = 0.044715f;                  // sqrt(2/pi)

// Phi(g), and e = exp(-g^2/2).  (1 + erf(g sqrt(1/2))) / 2 cancels below zero:
// 10% off at -5.  For x = |g| the tail Phi(-x) is e times Mills' ratio over
// sqrt(2 pi), which falls from 1/2 like 1/x; a quotient of polynomials fitted
// to it (least squares, weighted towards the largest relative error, on [0,
// 14]; e is 0 beyond) is 4e-7 of it off at most, 6e-7 evaluated in fp32.  So
// Phi keeps its relative accuracy, to 1e-5 at g = -8 with e's.  GELU of 16,384
// x 768 x 2048: 125 us forward and 235 backward (erff 124 and 252, erfcf 144
// and 276).
__device__ __forceinline__ float normal_cdf(float g, float &e)
{
    const float x = fminf(fabsf(g), 14.f);
    e = __expf(-0.5f * g * g);
    const float over = ((0.017047782f * x + 0.119532058f) * x + 0.361971958f) * x + 0.49999981f;
    const float under = (((0.0427374538f * x + 0.299419798f) * x + 0.953441733f) * x + 1.52180965f) * x + 1.f;
    const float tail = __fdividef(e * over, under);
    return g < 0.f ? tail : 1.f - tail;
}

// ACT: ZERO1_ACT_SILU, _GELU, _GELU_TANH, _RELU.
template <int ACT, bool SLOPE>
__device__ __forceinline__ void activate(float g, float &a, float &slope)
{
    if (ACT == 0) {
        const float s = sigmoid(g);
        a = g * s;
        if (SLOPE) slope = s + a * (1.f - s);
    } else if (ACT == 1) {
        float e;
        const float cdf = normal_cdf(g, e);
        a = g * cdf;
        if (SLOPE) slope = cdf + g * kDensity * e;
    } else if (ACT == 2) {       // (1 + tanh(z)) / 2 = sigmoid(2 z)
        const float s = sigmoid(2.f * kRoot2Pi * (g + kCube * g * g * g));
        a = g * s;
        // past |g| = 1e15 1 - s or a is 0, and no factor beside it may leave fp32's range
        if (SLOPE) slope = s + a * (1.f - s) * (2.f * kRoot2Pi * (1.f + 3.f * kCube * fminf(g * g, 1e30f)));
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
