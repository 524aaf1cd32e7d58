// zero1_muon_device.cuh -- device code the matrix optimizer's kernels share:
// loads and stores of 8 neighbouring entries, the split into two f16 parts,
// the sum of squares, momentum, and the point the polynomial is taken about.
#pragma once

#include <cuda_fp16.h>

#include "zero1_muon.h"
#include "zero1_ptx.cuh"

namespace zero1 {

// A sum of squares in fp32 that moves to fp64 what would leave fp32's range.
struct SquareSum {
    float s = 0.f;
    double big = 0.0;
    template <int N>
    __device__ __forceinline__ void add(const float (&v)[N])
    {
        float q = 0.f;
#pragma unroll
        for (int i = 0; i < N; ++i) q += v[i] * v[i];
        if (q > 1e30f) outsized(v, N);
        else s += q;
    }
    __device__ __noinline__ void outsized(const float *v, int n)
    {
        for (int i = 0; i < n; ++i) big += (double)v[i] * (double)v[i];
    }
    __device__ __forceinline__ double total() const { return big + (double)s; }
};

__device__ __forceinline__ void load8(float v[8], const float *p)
{
    const float4 x = *reinterpret_cast<const float4 *>(p), y = *reinterpret_cast<const float4 *>(p + 4);
    v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w, v[4] = y.x, v[5] = y.y, v[6] = y.z, v[7] = y.w;
}

__device__ __forceinline__ void load8(float v[8], const uint16_t *p)
{
    ptx::set_widened(v, *reinterpret_cast<const uint4 *>(p));
}

__device__ __forceinline__ void store8(float *p, const float v[8])
{
    *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
    *reinterpret_cast<float4 *>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
}

__device__ __forceinline__ void store8(uint16_t *p, const float v[8])
{
    *reinterpret_cast<uint4 *>(p) = make_uint4(ptx::pack2(v[0], v[1]), ptx::pack2(v[2], v[3]), ptx::pack2(v[4], v[5]),
                                               ptx::pack2(v[6], v[7]));
}

__device__ __forceinline__ float load1(const float *p) { return *p; }
__device__ __forceinline__ float load1(const uint16_t *p) { return __uint_as_float((uint32_t)*p << 16); }
__device__ __forceinline__ void store1(float *p, float v) { *p = v; }
__device__ __forceinline__ void store1(uint16_t *p, float v) { *p = __bfloat16_as_ushort(__float2bfloat16_rn(v)); }

// hi + lo = v to 22 bits or to 2^-25, whichever is coarser, of two neighbours (one conversion of a pair takes
// the time of a quarter of one of a single value).
__device__ __forceinline__ void split(float v, float w, uint32_t &hi, uint32_t &lo)
{
    const __half2 h = __floats2half2_rn(v, w);
    const float2 f = __half22float2(h);
    const __half2 l = __floats2half2_rn(v - f.x, w - f.y);
    hi = *reinterpret_cast<const uint32_t *>(&h);
    lo = *reinterpret_cast<const uint32_t *>(&l);
}

// The momentum after a step whose rank-ordered gradient sum is `sum`, and the
// update it gives: m = mu m + (1-mu) g with g the mean, and
// u = mu m + (1-mu) g (nesterov) or m.
__device__ __forceinline__ float look_ahead(const MuonScalars &sc, float sum, float &mom)
{
    const float g = sum * sc.inv_w;
    mom = sc.momentum * mom + sc.one_minus_momentum * g;
    return sc.nesterov ? sc.momentum * mom + sc.one_minus_momentum * g : mom;
}

// In the last iterations A is near the identity and b A + c A A is a large
// term that nearly cancels a I: its errors count several times.  There the
// polynomial is taken about A = alpha I, an identity for any alpha: with
// A' = A - alpha I,
//   a + b A + c A A = (a + b alpha + c alpha^2) + (b + 2 c alpha) A' + c A' A',
// whose terms are small.  The iterations before keep alpha = 0, since
// directions still far below one would gain the error of terms that their
// part of b A + c A A does not have.
constexpr float kAlpha = 0.85f;
__device__ __forceinline__ float alpha_of(uint32_t iter, int steps) { return (int)iter + 2 >= steps ? kAlpha : 0.f; }
}  // namespace zero1
