// zero1_adamw.cu -- AdamW over a list of tensors, one step of all of them at
// once, with moments in fp32 or in 8 bits (include/zero1.h, zero1_adamw_*).
//
// The list's state is one flat run of blocks of 256 entries; a tensor starts
// at a block of its own, and a table names the tensor of every block.  One
// warp takes one block: its 8 entries a lane are 16 or 32 bytes of each
// operand, and the two largest values of a block (which its scales are formed
// from) are one warp reduction each.  So the grid is even whatever the
// tensors' sizes are, and a list of any length takes one pass.
//
// 8 bits.  With f(k, b) = (1 + (k mod 2^b)/2^b) 2^(k div 2^b):
//     m       = +-(f(k, 3) - 1) (max|m| / 61439),        7 bits and a sign,
//     sqrt(v) =   (f(k, 4) - 1) (max sqrt(v) / 63487),   8 bits:
// evenly spaced near zero and by octaves beyond, a fraction 2^-4 or 2^-5 of
// the value apart at most, over 2^-19 and 2^-20 of the block's largest.
// A running mean moves by a fraction 1-beta of itself a step, less than half
// a code's width (v with beta2 = 0.95 by 5% at most when it decays), so
// rounding to nearest would hold it where it is; every code is rounded up or
// down at random instead, by 16 bits of a hash of the seed, the step and the
// entry's place, with the exact value as its mean.  sqrt(v) > 0 is never
// rounded to zero: m may be rounded up where v vanishes, and m / sqrt(v)
// would have no bound.  The update uses the new moments before they are
// rounded.
//
// Every fp32 operation is rounded by itself (no fma), so master, parameters
// and codes are those of the written formulas bit for bit (but for the sign of
// a zero: a lane whose m and v are all zero moves by +0 where m is -0).  The
// norm's sum of squares is compensated in fp32 (each square and each addition
// with its error) and then fp64, so that the fp32 clip coefficient is its
// correct rounding but for values within 1e-12 of a tie.
//
// Measured on the GPT-2-small list (98 tensors, 124 million entries, bf16):
// norm 62 us (4.0 TB/s; half the issue slots, its loads and its arithmetic
// take turns), update with fp32 moments 505 us (28 bytes an entry at 6.9 TB/s,
// bound by HBM: a plain copy moves 6.7), with 8 bits 360 us (16 bytes at 5.5
// TB/s; 81% of the issue slots busy, 90 instructions an entry), reading 8-bit
// moments out 190 us (6.5 TB/s).  4,096 entries in one launch: 9.5 us, all latency.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstring>
#include <exception>
#include <memory>
#include <mutex>
#include <new>
#include <unordered_set>
#include <vector>

#include "zero1.h"
#include "zero1_adamw_plan.h"
#include "zero1_internal.h"
#include "zero1_launch.h"
#include "zero1_ptx.cuh"

namespace zero1 {
namespace {

constexpr uint32_t kUpdateBlocks = 4;     // blocks of a warp of the update, fp32 moments (they are unrolled)
constexpr uint32_t kStagedBlocks = 8;     // ... with 8 bits (16: 374 us in place of 366, 32: 392, all at once: 417)
constexpr float kMTop = 61439.f, kRTop = 63487.f;       // f(127, 3) - 1, f(255, 4) - 1
constexpr uint32_t kHeldLow = 27u << 23;                // 2^-100: a block whose largest value is smaller is all zeros
constexpr uint32_t kInf = 0x7F800000u;
constexpr uint64_t kMaxListTable = 1ull << 22;          // steps of the bias-correction table

// What the kernels share in device memory.
struct ListStatus {
    double nsq, norm, lr;
    unsigned long long t;     // steps taken
    float clip;
    float step_size, decay;   // of the next step
    unsigned ticket[2];       // blocks that have finished: of the norm, of the update; 0 between launches
};

struct ListTables {
    const uint32_t *blocks;         // of every block: its tensor, its entries less one above that, whether it decays
    ListStatus *status;
    double *partials;               // of the norm: one for each block of its grids
    const double *correction;       // sqrt(1 - beta2^t) / (1 - beta1^t) for t = 1 .. steps
    uint64_t steps;
    double weight_decay, max_norm;
};

// The scalars of step t + 1.
__device__ void form_scalars(const ListTables &d, unsigned long long t, double lr)
{
    const uint64_t i = t < d.steps ? t : d.steps - 1;   // both corrections are 1 from there on
    d.status->step_size = __double2float_rn(__dmul_rn(lr, d.correction[i]));
    d.status->decay = __double2float_rn(__dadd_rn(1.0, -__dmul_rn(lr, d.weight_decay)));
}

// which 1: the steps taken are `t`; 2: the learning rate is `lr`; 3: both.
__global__ void zero1_adamw_set_kernel(ListTables d, unsigned long long t, double lr, int which)
{
    if (which & 1) d.status->t = t;
    if (which & 2) d.status->lr = lr;
    form_scalars(d, d.status->t, d.status->lr);
}

// Two fp32 numbers in one instruction, products and sums each rounded by
// themselves: a paired product is contracted into the paired sum that takes
// it, .rn or not, so sums are written as a + b * one with a `one` that only
// the launch knows.
struct Two {
    unsigned long long v;
};
template <int CAP>
struct NormParams {
    const void *grads[CAP];
    uint32_t first[CAP];        // block that each tensor starts at
    ListTables d;
    uint64_t block0, nblocks;
    uint32_t tensor0, before;   // partial sums of earlier launches of this step
    float one;
    int last;
};

template <int CAP>
struct UpdateParams {
    const void *grads[CAP];
    void *params[CAP];
    uint32_t first[CAP];
    ListTables d;
    float *master;
    void *m, *v;
    float2 *scales;
    uint64_t block0, nblocks;
    uint64_t seed;
    Two beta1, omb1, beta2, omb2, eps2, one;   // each twice
    float eps;
    uint32_t tensor0, per_warp;   // blocks that a warp takes, one after another
    int clipped, decay_first, eps_easy, last;
};

constexpr uint32_t pack_block(uint32_t tensor, uint32_t count, bool decays) { return tensor | (count - 1) << 16 | (uint32_t)decays << 24; }
__device__ __forceinline__ uint32_t tensor_of(uint32_t word) { return word & 0xFFFFu; }
__device__ __forceinline__ uint32_t count_of(uint32_t word) { return ((word >> 16) & 0xFFu) + 1; }
__device__ __forceinline__ bool decays_of(uint32_t word) { return word >> 24; }

__device__ __forceinline__ bool whole16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Eight entries of a lane: neighbours (WHOLE: a full block whose tensor is
// 16-byte aligned) or every 32nd (its loads are then of one entry, side by
// side over the warp), with zeros past the block's count.
template <bool WHOLE>
__device__ __forceinline__ uint32_t entry_of(int j)
{
    const uint32_t lane = threadIdx.x & 31;
    return WHOLE ? lane * 8 + j : j * 32 + lane;
}
template <bool WHOLE>
__device__ __forceinline__ void get8(float v[8], const float *p, uint32_t count)
{
    if (WHOLE) {
        const float4 *q = reinterpret_cast<const float4 *>(p + entry_of<true>(0));
        const float4 a = q[0], b = q[1];
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = entry_of<false>(j) < count ? p[entry_of<false>(j)] : 0.f;
    }
}
template <bool WHOLE>
__device__ __forceinline__ void get8(float v[8], const uint16_t *p, uint32_t count)
{
    if (WHOLE) {
        ptx::set_widened(v, *reinterpret_cast<const uint4 *>(p + entry_of<true>(0)));
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            v[j] = entry_of<false>(j) < count ? __uint_as_float((uint32_t)p[entry_of<false>(j)] << 16) : 0.f;
    }
}
template <bool WHOLE>
__device__ __forceinline__ void put8(float *p, const float v[8], uint32_t count)
{
    if (WHOLE) {
        float4 *q = reinterpret_cast<float4 *>(p + entry_of<true>(0));
        q[0] = make_float4(v[0], v[1], v[2], v[3]);
        q[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (entry_of<false>(j) < count) p[entry_of<false>(j)] = v[j];
    }
}
template <bool WHOLE>
__device__ __forceinline__ void put8(uint16_t *p, const float v[8], uint32_t count)
{
    if (WHOLE) {
        *reinterpret_cast<uint4 *>(p + entry_of<true>(0)) =
            make_uint4(ptx::pack2(v[0], v[1]), ptx::pack2(v[2], v[3]), ptx::pack2(v[4], v[5]), ptx::pack2(v[6], v[7]));
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (entry_of<false>(j) < count) p[entry_of<false>(j)] = __bfloat16_as_ushort(__float2bfloat16_rn(v[j]));
    }
}
// Codes: one byte an entry.
template <bool WHOLE>
__device__ __forceinline__ void get8(uint32_t k[8], const uint8_t *p, uint32_t count)
{
    if (WHOLE) {
        const uint2 w = *reinterpret_cast<const uint2 *>(p + entry_of<true>(0));
#pragma unroll
        for (int j = 0; j < 8; ++j) k[j] = ((j < 4 ? w.x : w.y) >> (8 * (j & 3))) & 0xFFu;
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) k[j] = entry_of<false>(j) < count ? p[entry_of<false>(j)] : 0u;
    }
}
// ... which are the top bytes of k.
__device__ __forceinline__ uint32_t top_bytes(uint32_t a, uint32_t b, uint32_t c, uint32_t d)
{
    return __byte_perm(__byte_perm(a, b, 0x0073), __byte_perm(c, d, 0x0073), 0x5410);
}
template <bool WHOLE>
__device__ __forceinline__ void put8_top(uint8_t *p, const uint32_t k[8], uint32_t count)
{
    if (WHOLE) {
        *reinterpret_cast<uint2 *>(p + entry_of<true>(0)) =
            make_uint2(top_bytes(k[0], k[1], k[2], k[3]), top_bytes(k[4], k[5], k[6], k[7]));
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (entry_of<false>(j) < count) p[entry_of<false>(j)] = (uint8_t)(k[j] >> 24);
    }
}

__device__ __forceinline__ Two two(float a, float b)
{
    Two r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void apart(Two x, float &a, float &b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(x.v)); }
__device__ __forceinline__ Two mul(Two a, Two b)
{
    Two r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ Two fma(Two a, Two b, Two c)
{
    Two r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return r;
}
__device__ __forceinline__ Two add(Two a, Two b, Two one) { return fma(b, one, a); }

// ------------------------------------------------------------------ codes

// 32 well-mixed bits: two rounds of multiplication (by the first 32 bits of
// the fractions of sqrt 2 and sqrt 3) and shifted exclusive or.
__device__ __forceinline__ uint32_t mix_folded(uint32_t x)   // of x ^ (x >> 16)
{
    x *= 0x6A09E667u;
    x = (x ^ (x >> 15)) * 0xBB67AE85u;
    return x ^ (x >> 16);
}
__device__ __forceinline__ uint32_t mix(uint32_t x) { return mix_folded(x ^ (x >> 16)); }
// The key of a step's random bits; `high`: the upper half of an entry's place.
__device__ __forceinline__ uint32_t key_of(uint64_t seed, unsigned long long t, uint32_t high)
{
    const uint32_t k = mix(mix(mix((uint32_t)seed) ^ (uint32_t)(seed >> 32)) ^ (uint32_t)t);
    return high ? mix(k + high) : k;
}

// Correctly rounded square roots and quotients of two, without branches: from
// the approximate (reciprocal) root or reciprocal by one Newton step, then the
// exact remainder times the inverse added once (P. Markstein, "IA-64 and
// elementary functions", 2000, chapters 8 and 9).  For v = 0 or in [2^-100,
// 2^100], |m| = 0 or in [2^-60, 2^60] and d in [2^-50, 2^51], where nothing
// leaves fp32's normal range.  Compared with the IEEE instructions: all
// significands of two octaves at twelve exponents, and 1.7e10 quotients.
__device__ __forceinline__ Two roots(float v0, float v1)
{
    float y0, y1;
    asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y0) : "f"(v0));
    asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y1) : "f"(v1));
    const float most = 1.152921504606846976e18f;   // 2^60, for v = 0
    const Two v = two(v0, v1), y = two(fminf(y0, most), fminf(y1, most));
    Two g = mul(v, y), h = mul(y, two(-.5f, -.5f));           // sqrt(v), -1/(2 sqrt(v))
    const Two e = fma(g, h, two(.5f, .5f));
    g = fma(g, e, g);
    h = fma(h, e, h);
    return fma(fma(g, g, mul(v, two(-1.f, -1.f))), h, g);
}
__device__ __forceinline__ Two quotients(Two m, float d0, float d1)
{
    float y0, y1;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y0) : "f"(d0));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y1) : "f"(d1));
    Two y = two(y0, y1);
    const Two d = mul(two(d0, d1), two(-1.f, -1.f));
    y = fma(y, fma(d, y, two(1.f, 1.f)), y);
    const Two q = mul(m, y);
    return fma(fma(d, q, m), y, q);
}
constexpr float kMLow = 8.6736173798840355e-19f, kMHigh = 1.152921504606847e18f;     // 2^-60, 2^60
constexpr float kVLow = 7.8886090522101181e-31f, kVHigh = 1.2676506002282294e30f;    // 2^-100, 2^100

// f(k, b) - 1 of two codes; what their bytes stand for, times the scale.
__device__ __forceinline__ Two units(uint32_t y0, uint32_t y1)
{
    return two(__uint_as_float(y0 + (127u << 23)) - 1.f, __uint_as_float(y1 + (127u << 23)) - 1.f);
}
__device__ __forceinline__ void m_values(float &a, float &b, uint32_t k0, uint32_t k1, float scale)
{
    apart(mul(units((k0 & 127u) << 20, (k1 & 127u) << 20), two(scale, scale)), a, b);
    a = __uint_as_float(__float_as_uint(a) | (k0 & 128u) << 24);
    b = __uint_as_float(__float_as_uint(b) | (k1 & 128u) << 24);
}
__device__ __forceinline__ Two r_values(uint32_t k0, uint32_t k1, float scale)
{
    return mul(units(k0 << 19, k1 << 19), two(scale, scale));
}
__device__ __forceinline__ void decode8(float m[8], float v[8], const uint32_t km[8], const uint32_t kr[8], float2 s)
{
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
        m_values(m[j], m[j + 1], km[j], km[j + 1], s.x);
        const Two root = r_values(kr[j], kr[j + 1], s.y);
        apart(mul(root, root), v[j], v[j + 1]);
    }
}
// y = |x| / scale + 1 (below 2^16) as a code of 4 octave bits and BITS
// fraction bits, rounded at random, in the top bits of the result: the
// largest y, 2^16 less one code, and a few of its last places more do not
// carry, as a dither is 16 of them short of one code at least.
template <int BITS>
__device__ __forceinline__ uint32_t code_top(float y, uint32_t random16)
{
    return (__float_as_uint(y) + (random16 << (7 - BITS)) - (127u << 23)) << (5 + BITS - 4);
}
__device__ __forceinline__ void most_of(float &most, float a, float b)   // NaN stays
{
    asm("max.NaN.abs.f32 %0, %0, %1, %2;" : "+f"(most) : "f"(a), "f"(b));
}
__device__ __forceinline__ void least_of(float &least, float a, float b)
{
    asm("min.abs.f32 %0, %0, %1, %2;" : "+f"(least) : "f"(a), "f"(b));
}

// A block's scale and its inverse from the bits of its largest value; NaN
// where that is not finite (its codes are then all zero, and stand for NaN).
__device__ __forceinline__ bool scales_of(uint32_t largest, float top, float &scale, float &inv)
{
    const bool held = largest >= kHeldLow && largest < kInf;
    const float most = __uint_as_float(largest);
    scale = held ? __fdiv_rn(most, top) : largest < kHeldLow ? 0.f : __uint_as_float(0x7FC00000u);
    inv = held ? __fdiv_rn(top, most) : 0.f;
    return held;
}

// --------------------------------------------------------------- the norm

// A sum of squares to twice fp32's precision.
struct Squares {
    Two sum = two(0.f, 0.f), rest = two(0.f, 0.f);
    // Squares of two entries with the error of each addition and, where a
    // square may have one (fp32 entries: bf16's squares have 16 bits), of each square.
    template <bool EXACT>
    __device__ __forceinline__ void add2(Two g, Two one, Two minus)
    {
        const Two p = mul(g, g), s = add(sum, p, one);
        const Two back = fma(sum, minus, s);                              // s - sum
        Two lost = add(fma(fma(back, minus, s), minus, sum), fma(back, minus, p), one);
        if (!EXACT) lost = add(lost, fma(g, g, mul(p, minus)), one);
        rest = add(rest, lost, one);
        sum = s;
    }
    __device__ __forceinline__ float size() const
    {
        float a, b;
        apart(sum, a, b);
        return a + b;
    }
    __device__ __forceinline__ double total() const
    {
        float a, b, c, d;
        apart(sum, a, b);
        apart(rest, c, d);
        return ((double)a + (double)b) + ((double)c + (double)d);
    }
};
// Sums whose squares left fp32's range are taken again in fp64: entries from
// 2^60 on, or only ones below 2^-45 (a square that is cut off at 2^-149 counts
// in no larger sum).
constexpr float kSumHigh = 1.3292279957849159e36f, kSumLow = 8.0779356694631609e-28f;   // 2^120, 2^-90

// Sum over the block in a fixed order; valid on thread 0.
__device__ __forceinline__ double sum_block(double v)
{
    __shared__ double part[kWarps];
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
    __syncthreads();
    double s = 0.0;
    if (threadIdx.x == 0)
        for (uint32_t i = 0; i < kWarps; ++i) s += part[i];
    __syncthreads();
    return s;
}

// The norm of a sum of squares, and the clip coefficient it gives.
__device__ __forceinline__ float finish_norm(const ListTables &d, double squares)
{
    const double norm = sqrt(squares);
    float c = 1.f;
    if (isnan(norm))
        c = __int_as_float(0x7FC00000);
    else if (d.max_norm / norm < 1.0)
        c = (float)(d.max_norm / norm);
    d.status->nsq = squares;
    d.status->norm = norm;
    d.status->clip = c;
    return c;
}

// Whether this block is the last of its grid to get here (all threads).
__device__ __forceinline__ bool last_block(unsigned *ticket)
{
    __shared__ bool is_last;
    if (threadIdx.x == 0) {
        __threadfence();
        is_last = atomicAdd(ticket, 1u) + 1 == gridDim.x;
        if (is_last) {
            __threadfence();
            *ticket = 0;
        }
    }
    __syncthreads();
    return is_last;
}

// Every kNormBlocks blocks of 256 entries that this warp takes: visit(gradient, entries).
template <typename G, int CAP, typename F>
__device__ __forceinline__ void for_grads(const NormParams<CAP> &p, F visit)
{
    const uint64_t step = (uint64_t)gridDim.x * kWarps * kNormBlocks;
    for (uint64_t b0 = (uint64_t)blockIdx.x * kWarps * kNormBlocks + (threadIdx.x >> 5); b0 < p.nblocks; b0 += step) {
        uint32_t word[kNormBlocks];
#pragma unroll
        for (uint32_t u = 0; u < kNormBlocks; ++u)
            word[u] = b0 + u * kWarps < p.nblocks ? __ldg(p.d.blocks + p.block0 + b0 + u * kWarps) : 0u;
        const G *src[kNormBlocks];
        uint32_t count[kNormBlocks];
#pragma unroll
        for (uint32_t u = 0; u < kNormBlocks; ++u) {
            const bool there = b0 + u * kWarps < p.nblocks;
            const uint32_t i = there ? tensor_of(word[u]) - p.tensor0 : 0;
            src[u] = static_cast<const G *>(p.grads[i]) + (uint64_t)((uint32_t)(p.block0 + b0) + u * kWarps - p.first[i]) * kListBlock;
            count[u] = there ? count_of(word[u]) : 0;
        }
        visit(src, count);
    }
}

// Bound by HBM: one read of the gradients.  The last block of the step's last
// launch adds up all partial sums in order and forms the clip coefficient.
template <typename G, int CAP>
__global__ void __launch_bounds__(kListThreads, 4) zero1_adamw_norm_kernel(const __grid_constant__ NormParams<CAP> p)
{
    constexpr bool kExact = sizeof(G) == 2;
    ptx::launch_dependents();
    Squares ss;
    const Two one = two(p.one, p.one), minus = two(-p.one, -p.one);
    uint32_t any = 0;
    for_grads<G, CAP>(p, [&](const G *const src[kNormBlocks], const uint32_t count[kNormBlocks]) {
        bool all = true;
#pragma unroll
        for (uint32_t u = 0; u < kNormBlocks; ++u) all = all && count[u] == kListBlock && whole16(src[u]);
        if (all) {   // as they lie in memory: their bits are looked at by the word
            constexpr int kPieces = sizeof(G) / 2;
            uint4 raw[kNormBlocks][kPieces];
#pragma unroll
            for (uint32_t u = 0; u < kNormBlocks; ++u)
#pragma unroll
                for (int q = 0; q < kPieces; ++q) raw[u][q] = reinterpret_cast<const uint4 *>(src[u] + entry_of<true>(0))[q];
#pragma unroll
            for (uint32_t u = 0; u < kNormBlocks; ++u)
#pragma unroll
                for (int q = 0; q < kPieces; ++q) {
                    const uint32_t w[4] = {raw[u][q].x, raw[u][q].y, raw[u][q].z, raw[u][q].w};
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        any |= w[k];
                        if (kExact)
                            ss.add2<kExact>(two(__uint_as_float(w[k] << 16), __uint_as_float(w[k] & 0xFFFF0000u)), one, minus);
                        else if (k % 2 == 0)
                            ss.add2<kExact>(two(__uint_as_float(w[k]), __uint_as_float(w[k + 1])), one, minus);
                    }
                }
        } else {
#pragma unroll 1
            for (uint32_t u = 0; u < kNormBlocks; ++u) {
                float g[8];
                get8<false>(g, src[u], count[u]);
#pragma unroll
                for (int k = 0; k < 8; k += 2) {
                    any |= __float_as_uint(g[k]) | __float_as_uint(g[k + 1]);
                    ss.add2<kExact>(two(g[k], g[k + 1]), one, minus);
                }
            }
        }
    });
    double mine = ss.total();
    const float size = ss.size();
    // (a sign bit alone may send a thread there: a sum of zeros again)
    if (!(size < kSumHigh) || (size < kSumLow && any != 0)) {
        mine = 0.0;
        for_grads<G, CAP>(p, [&](const G *const src[kNormBlocks], const uint32_t count[kNormBlocks]) {
            bool all = true;   // the same entries as above
#pragma unroll
            for (uint32_t u = 0; u < kNormBlocks; ++u) all = all && count[u] == kListBlock && whole16(src[u]);
#pragma unroll 1
            for (uint32_t u = 0; u < kNormBlocks; ++u) {
                float g[8];
                if (all)
                    get8<true>(g, src[u], kListBlock);
                else
                    get8<false>(g, src[u], count[u]);
#pragma unroll 1
                for (int k = 0; k < 8; ++k) mine += (double)g[k] * (double)g[k];
            }
        });
    }
    const double sum = sum_block(mine);
    if (threadIdx.x == 0) p.d.partials[p.before + blockIdx.x] = sum;
    if (!last_block(&p.d.status->ticket[0]) || !p.last) return;
    double v = 0.0;
    for (uint32_t i = threadIdx.x; i < p.before + gridDim.x; i += kListThreads) v += __ldcg(p.d.partials + i);
    v = sum_block(v);
    if (threadIdx.x == 0) finish_norm(p.d, v);
}

// -------------------------------------------------------------- the update

// What a lane reads of a block.
template <int BITS>
struct Read {
    float g[8], w[8], m[8], v[8];
};
template <typename P, typename G, int BITS, bool WHOLE, int CAP>
__device__ __forceinline__ void read_block(Read<BITS> &x, const UpdateParams<CAP> &p, const G *grad, const P *param,
                                           uint32_t count, uint64_t block)
{
    const uint64_t flat = block * kListBlock;
    get8<WHOLE>(x.g, grad, count);
    if constexpr (sizeof(P) == 2)
        get8<WHOLE>(x.w, p.master + flat, count);
    else
        get8<WHOLE>(x.w, param, count);
    if constexpr (BITS == 32) {
        get8<WHOLE>(x.m, static_cast<const float *>(p.m) + flat, count);
        get8<WHOLE>(x.v, static_cast<const float *>(p.v) + flat, count);
    } else {
        uint32_t km[8], kr[8];
        get8<WHOLE>(km, static_cast<const uint8_t *>(p.m) + flat, count);
        get8<WHOLE>(kr, static_cast<const uint8_t *>(p.v) + flat, count);
        decode8(x.m, x.v, km, kr, p.scales[block]);
    }
}

// One block by one warp.
template <typename P, int BITS, bool WHOLE, int CAP>
__device__ __forceinline__ void update_block(Read<BITS> &x, const UpdateParams<CAP> &p, P *param, uint32_t count, bool decays,
                                             uint64_t block, float clip, float step_size, float decay, unsigned long long t)
{
    const uint64_t flat = block * kListBlock;
    constexpr bool kMaster = sizeof(P) == 2;
    float(&g)[8] = x.g, (&w)[8] = x.w, (&m)[8] = x.m, (&v)[8] = x.v, r[8];
    // (past the block's count all are zero: they change neither maximum)
    const float before = decays && p.decay_first ? decay : 1.f, after = decays && !p.decay_first ? decay : 1.f;
    float most_m = 0.f, most_v = 0.f, least_m = kMHigh, least_v = kVHigh;
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
        const Two c = mul(two(g[j], g[j + 1]), two(clip, clip));
        apart(add(mul(p.beta1, two(m[j], m[j + 1])), mul(p.omb1, c), p.one), m[j], m[j + 1]);
        apart(add(mul(p.beta2, two(v[j], v[j + 1])), mul(mul(p.omb2, c), c), p.one), v[j], v[j + 1]);
        most_of(most_m, m[j], m[j + 1]);
        most_of(most_v, v[j], v[j + 1]);
        least_of(least_m, m[j], m[j + 1]);
        least_of(least_v, v[j], v[j + 1]);
    }
    // zeros throughout (a row without gradients), or nothing near the ends of fp32's range
    const bool zeros = most_m == 0.f && most_v == 0.f;
    const bool easy = p.eps_easy && (zeros || (least_m >= kMLow && most_m <= kMHigh && least_v >= kVLow && most_v <= kVHigh));
    float q[8];
    if (easy) {
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
            const Two root = roots(v[j], v[j + 1]);
            apart(root, r[j], r[j + 1]);
            float d0, d1;
            apart(add(root, p.eps2, p.one), d0, d1);
            apart(quotients(two(m[j], m[j + 1]), d0, d1), q[j], q[j + 1]);
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            r[j] = __fsqrt_rn(v[j]);
            q[j] = __fdiv_rn(m[j], __fadd_rn(r[j], p.eps));
        }
    }
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
        const Two less = mul(two(-step_size, -step_size), two(q[j], q[j + 1]));
        const Two moved = add(mul(two(w[j], w[j + 1]), two(before, before)), less, p.one);
        apart(mul(moved, two(after, after)), w[j], w[j + 1]);
    }
    put8<WHOLE>(param, w, count);
    if constexpr (kMaster) put8<WHOLE>(p.master + flat, w, count);
    if constexpr (BITS == 32) {
        put8<WHOLE>(static_cast<float *>(p.m) + flat, m, count);
        put8<WHOLE>(static_cast<float *>(p.v) + flat, v, count);
    } else {
        float2 s;
        float inv_m, inv_r;
        const bool held_m = scales_of(__reduce_max_sync(~0u, __float_as_uint(most_m)), kMTop, s.x, inv_m);
        // the largest root is the root of the largest: a correctly rounded root does not decrease
        const float most_r = __fsqrt_rn(__uint_as_float(__reduce_max_sync(~0u, __float_as_uint(most_v))));
        const bool held_r = scales_of(__float_as_uint(most_r), kRTop, s.y, inv_r);
        // an entry's place differs from its lane's first in bits below 16 only, so their first folding is shared
        const uint32_t first = ((uint32_t)flat + entry_of<WHOLE>(0)) ^ key_of(p.seed, t, (uint32_t)(flat >> 32));
        const uint32_t folded = first ^ (first >> 16);
        uint32_t km[8], kr[8];
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
            float a[2], b[2];
            apart(mul(two(m[j], m[j + 1]), two(inv_m, inv_m)), a[0], a[1]);
            apart(add(mul(two(r[j], r[j + 1]), two(inv_r, inv_r)), p.one, p.one), b[0], b[1]);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const uint32_t random = mix_folded(folded ^ (WHOLE ? j + i : (j + i) * 32));
                km[j + i] = code_top<3>(__fadd_rn(fabsf(a[i]), 1.f), random & 0xFFFFu);
                kr[j + i] = code_top<4>(b[i], random >> 16);
            }
        }
        // a block of zeros has inverse 0 and codes 0 by itself; one that is not finite is held as codes 0
        if (!held_m) {
#pragma unroll
            for (int j = 0; j < 8; ++j) km[j] = 0;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            km[j] = (km[j] & 0x7FFFFFFFu) | (__float_as_uint(m[j]) & 0x80000000u);
            kr[j] = max(kr[j], min(__float_as_uint(r[j]), 1u) << 24);   // sqrt(v) > 0 never becomes 0
        }
        if (!held_r) {
#pragma unroll
            for (int j = 0; j < 8; ++j) kr[j] = 0;
        }
        put8_top<WHOLE>(static_cast<uint8_t *>(p.m) + flat, km, count);
        put8_top<WHOLE>(static_cast<uint8_t *>(p.v) + flat, kr, count);
        if ((threadIdx.x & 31) == 0) p.scales[block] = s;
    }
}

// Where a block's tensors are.
template <typename P, typename G>
struct Place {
    const G *grad;
    P *param;
    uint32_t count;
    bool decays;
    __device__ __forceinline__ bool whole() const { return count == kListBlock && whole16(grad) && whole16(param); }
};
template <typename P, typename G, int CAP>
__device__ __forceinline__ Place<P, G> place_of(const UpdateParams<CAP> &p, uint32_t word, uint64_t block)
{
    const uint32_t i = tensor_of(word) - p.tensor0;
    const uint64_t at = (uint64_t)((uint32_t)block - p.first[i]) * kListBlock;
    return {static_cast<const G *>(p.grads[i]) + at, static_cast<P *>(p.params[i]) + at, count_of(word), decays_of(word)};
}

__device__ __forceinline__ void copy_async16(uint32_t dst, const void *src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_async8(uint32_t dst, const void *src)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}

// A lane's part of a block on its way through shared memory (8-bit moments):
// every lane reads what it copied itself, so no barrier is needed.
template <typename P, typename G>
struct Staged {
    static constexpr uint32_t kGrad = 8 * sizeof(G) / 16, kBytes = 32 * (8 * sizeof(G) + 32 + 16);
    static __device__ __forceinline__ void copy(uint32_t at, const G *grad, const float *master, const void *m, const void *v, uint64_t flat)
    {
        const uint32_t lane = threadIdx.x & 31;
#pragma unroll
        for (uint32_t q = 0; q < kGrad; ++q) copy_async16(at + (q * 32 + lane) * 16, reinterpret_cast<const uint4 *>(grad) + lane * kGrad + q);
        at += kGrad * 512;
#pragma unroll
        for (uint32_t q = 0; q < 2; ++q) copy_async16(at + (q * 32 + lane) * 16, reinterpret_cast<const uint4 *>(master) + lane * 2 + q);
        at += 1024;
        copy_async8(at + lane * 8, static_cast<const uint8_t *>(m) + flat + lane * 8);
        copy_async8(at + 256 + lane * 8, static_cast<const uint8_t *>(v) + flat + lane * 8);
    }
    static __device__ __forceinline__ uint4 ld16(uint32_t at)
    {
        uint4 v;
        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
        return v;
    }
    static __device__ __forceinline__ void floats(float v[8], uint4 a, uint4 b)
    {
        const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = __uint_as_float(w[j]);
    }
    static __device__ __forceinline__ void read(Read<8> &x, uint32_t at, float2 scale)
    {
        const uint32_t lane = threadIdx.x & 31;
        if constexpr (kGrad == 1)
            ptx::set_widened(x.g, ld16(at + lane * 16));
        else
            floats(x.g, ld16(at + lane * 16), ld16(at + 512 + lane * 16));
        at += kGrad * 512;
        floats(x.w, ld16(at + lane * 16), ld16(at + 512 + lane * 16));
        at += 1024;
        uint32_t km[8], kr[8], a, b, c, d;
        asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(a), "=r"(b) : "r"(at + lane * 8) : "memory");
        asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(c), "=r"(d) : "r"(at + 256 + lane * 8) : "memory");
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            km[j] = ((j < 4 ? a : b) >> (8 * (j & 3))) & 0xFFu;
            kr[j] = ((j < 4 ? c : d) >> (8 * (j & 3))) & 0xFFu;
        }
        decode8(x.m, x.v, km, kr, scale);
    }
};

// Bound by HBM with fp32 moments; with 8-bit ones a block's arithmetic takes
// as long as its 2 KB, so the next block's are copied meanwhile.
template <typename P, typename G, int BITS, int CAP>
__global__ void __launch_bounds__(kListThreads, 4) zero1_adamw_update_kernel(const __grid_constant__ UpdateParams<CAP> p)
{
    const ListStatus *status = p.d.status;
    const float step_size = status->step_size, decay = status->decay;
    const unsigned long long t = status->t + 1;
    // After a norm the last blocks come first: their gradients are still in L2 (the GPT-2-small list 577 to 569 us;
    // with 8-bit moments, whose update waits for its arithmetic as much, 610 to 616).
    const auto place = [&](uint64_t b) { return p.block0 + (BITS == 32 && p.clipped ? p.nblocks - 1 - b : b); };
    if constexpr (BITS == 8) {
        extern __shared__ __align__(16) unsigned char raw[];
        using S = Staged<P, G>;
        const uint32_t mine = ptx::smem_u32(raw) + (threadIdx.x >> 5) * 2 * S::kBytes;
        const uint64_t stride = (uint64_t)gridDim.x * kWarps;
        uint64_t b = (uint64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
        const uint32_t *words = p.d.blocks;
        uint32_t word = b < p.nblocks ? __ldg(words + place(b)) : 0u, next = b + stride < p.nblocks ? __ldg(words + place(b + stride)) : 0u;
        float2 scale = make_float2(0.f, 0.f), next_scale = scale;
        const auto copy = [&](uint64_t which, uint32_t w, uint32_t buffer, float2 &s) {
            if (which < p.nblocks) {
                const uint64_t block = place(which);
                const Place<P, G> at = place_of<P, G, CAP>(p, w, block);
                s = p.scales[block];
                if (at.whole())
                    S::copy(mine + buffer * S::kBytes, at.grad, sizeof(P) == 2 ? p.master + block * kListBlock : reinterpret_cast<const float *>(at.param),
                            p.m, p.v, block * kListBlock);
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
        copy(b, word, 0, scale);       // none of this is the norm's
        ptx::grid_dependency_wait();   // for the norm
        const float clip = p.clipped ? __ldcg(&status->clip) : 1.f;
#pragma unroll 1
        for (uint32_t i = 0; b < p.nblocks; ++i, b += stride) {
            const uint32_t after = b + 2 * stride < p.nblocks ? __ldg(words + place(b + 2 * stride)) : 0u;
            copy(b + stride, next, (i + 1) & 1, next_scale);
            asm volatile("cp.async.wait_group 1;" ::: "memory");
            const uint64_t block = place(b);
            const Place<P, G> at = place_of<P, G, CAP>(p, word, block);
            Read<BITS> x;
            if (at.whole()) {
                S::read(x, mine + (i & 1) * S::kBytes, scale);
                update_block<P, BITS, true, CAP>(x, p, at.param, kListBlock, at.decays, block, clip, step_size, decay, t);
            } else {
                read_block<P, G, BITS, false, CAP>(x, p, at.grad, at.param, at.count, block);
                update_block<P, BITS, false, CAP>(x, p, at.param, at.count, at.decays, block, clip, step_size, decay, t);
            }
            word = next, next = after, scale = next_scale;
        }
    } else {
        const uint64_t b0 = (uint64_t)blockIdx.x * kWarps * p.per_warp + (threadIdx.x >> 5);
        uint32_t word[kUpdateBlocks];
#pragma unroll
        for (uint32_t u = 0; u < kUpdateBlocks; ++u)
            word[u] = u < p.per_warp && b0 + u * kWarps < p.nblocks ? __ldg(p.d.blocks + place(b0 + u * kWarps)) : 0u;
        ptx::grid_dependency_wait();   // for the norm
        const float clip = p.clipped ? __ldcg(&status->clip) : 1.f;
#pragma unroll
        for (uint32_t u = 0; u < kUpdateBlocks; ++u) {
            if (u >= p.per_warp || b0 + u * kWarps >= p.nblocks) break;
            const uint64_t block = place(b0 + u * kWarps);
            const Place<P, G> at = place_of<P, G, CAP>(p, word[u], block);
            Read<BITS> x;
            if (at.whole()) {
                read_block<P, G, BITS, true, CAP>(x, p, at.grad, at.param, kListBlock, block);
                update_block<P, BITS, true, CAP>(x, p, at.param, kListBlock, at.decays, block, clip, step_size, decay, t);
            } else {
                read_block<P, G, BITS, false, CAP>(x, p, at.grad, at.param, at.count, block);
                update_block<P, BITS, false, CAP>(x, p, at.param, at.count, at.decays, block, clip, step_size, decay, t);
            }
        }
    }
    __syncthreads();   // every warp has read the scalars
    if (last_block(&p.d.status->ticket[1]) && p.last && threadIdx.x == 0) {
        p.d.status->t = t;
        form_scalars(p.d, t, p.d.status->lr);
    }
}

// A clipped step of a short list in one launch: a block of 256 entries to a
// warp, which reads all of it before the norm is formed.
constexpr uint32_t kSmallWarps = 32;
template <typename P, typename G, int BITS>
__global__ void __launch_bounds__(32 * kSmallWarps) zero1_adamw_small_kernel(const __grid_constant__ UpdateParams<32> p)
{
    constexpr bool kExact = sizeof(G) == 2;
    __shared__ double sums[kSmallWarps];
    __shared__ float clip_of_all;
    const ListStatus *status = p.d.status;
    const float step_size = status->step_size, decay = status->decay;
    const unsigned long long t = status->t + 1;
    const uint32_t b = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const bool here = b < p.nblocks;
    Place<P, G> at{};
    Read<BITS> x;
#pragma unroll
    for (int k = 0; k < 8; ++k) x.g[k] = 0.f;
    if (here) {
        at = place_of<P, G, 32>(p, __ldg(p.d.blocks + b), b);
        if (at.whole())
            read_block<P, G, BITS, true, 32>(x, p, at.grad, at.param, kListBlock, b);
        else
            read_block<P, G, BITS, false, 32>(x, p, at.grad, at.param, at.count, b);
    }
    const Two minus = mul(p.one, two(-1.f, -1.f));
    Squares ss;
    uint32_t any = 0;
#pragma unroll
    for (int k = 0; k < 8; k += 2) {
        any |= __float_as_uint(x.g[k]) | __float_as_uint(x.g[k + 1]);
        ss.add2<kExact>(two(x.g[k], x.g[k + 1]), p.one, minus);
    }
    const float size = ss.size();
    double sum = ss.total();
    if (!(size < kSumHigh) || (size < kSumLow && any != 0)) {
        sum = 0.0;
#pragma unroll
        for (int k = 0; k < 8; ++k) sum += (double)x.g[k] * (double)x.g[k];
    }
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
    if (lane == 0) sums[b] = sum;
    __syncthreads();
    if (b == 0) {
        sum = sums[lane];
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
        if (lane == 0) clip_of_all = finish_norm(p.d, sum);
    }
    __syncthreads();   // (every warp has read the scalars, too)
    const float clip = clip_of_all;
    if (here) {
        if (at.whole())
            update_block<P, BITS, true, 32>(x, p, at.param, kListBlock, at.decays, b, clip, step_size, decay, t);
        else
            update_block<P, BITS, false, 32>(x, p, at.param, at.count, at.decays, b, clip, step_size, decay, t);
    }
    if (threadIdx.x == 0) {
        p.d.status->t = t;
        form_scalars(p.d, t, p.d.status->lr);
    }
}

// The moments that 8 bits hold, as fp32.
__global__ void __launch_bounds__(kListThreads) zero1_adamw_moments_kernel(ListTables d, uint64_t nblocks, const uint8_t *m,
                                                                           const uint8_t *v, const float2 *scales,
                                                                           float *m_out, float *v_out)
{
    const uint64_t block = (uint64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
    if (block >= nblocks) return;
    const uint32_t count = count_of(d.blocks[block]);
    const float2 s = scales[block];
    const uint64_t flat = block * kListBlock;
    const auto run = [&](auto whole) {
        constexpr bool WHOLE = decltype(whole)::value;
        uint32_t k[8];
        float x[8];
        if (m_out) {
            get8<WHOLE>(k, m + flat, count);
#pragma unroll
            for (int j = 0; j < 8; j += 2) m_values(x[j], x[j + 1], k[j], k[j + 1], s.x);
            put8<WHOLE>(m_out + flat, x, count);
        }
        if (v_out) {
            get8<WHOLE>(k, v + flat, count);
#pragma unroll
            for (int j = 0; j < 8; j += 2) {
                const Two root = r_values(k[j], k[j + 1], s.y);
                apart(mul(root, root), x[j], x[j + 1]);
            }
            put8<WHOLE>(v_out + flat, x, count);
        }
    };
    if (count == kListBlock)
        run(std::true_type{});
    else
        run(std::false_type{});
}

}  // namespace
}  // namespace zero1

// ------------------------------------------------------------------- host

struct zero1_adamw_ctx {
    zero1_hparams hp{};
    zero1_adamw_options opt{};
    std::vector<uint64_t> sizes;
    std::vector<uint64_t> first;              // block each tensor starts at; one more at the end
    std::vector<zero1::TensorRange> ranges;   // of a step's tensors, filled anew in every step
    int device = 0, num_sms = 0;
    void *block = nullptr;                    // one cudaMalloc: tables, status, partial sums
    uint64_t block_bytes = 0;
    uint64_t partials = 0;                    // partial sums of the norm that the tables have room for
    zero1::ListTables d{};
};

namespace {

using zero1::kCaps;
using zero1::kListBlock;

std::mutex g_adamw_mu;
std::unordered_set<zero1_adamw_ctx *> g_adamw_live;

int afail(int code, const char *fmt, ...)
{
    char msg[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(msg, sizeof msg, fmt, ap);
    va_end(ap);
    zero1::set_error_message(msg);
    return code;
}

int acuda(cudaError_t e, const char *what)
{
    cudaGetLastError();   // reported here, and not again by the caller's next launch
    return afail(e == cudaErrorMemoryAllocation ? ZERO1_ENOMEM : ZERO1_ECUDA, "%s: %s", what, cudaGetErrorString(e));
}

bool adamw_live(zero1_adamw_ctx *h)
{
    std::lock_guard<std::mutex> lk(g_adamw_mu);
    return h && g_adamw_live.count(h);
}

bool on16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool fine(double v) { return std::isfinite(v) && v >= 0.0; }
size_t bytes_of(int dtype) { return dtype == ZERO1_DTYPE_BF16 ? 2 : 4; }

struct AdamwDeviceGuard {
    int prev = -1;
    explicit AdamwDeviceGuard(int dev)
    {
        if (cudaGetDevice(&prev) != cudaSuccess) prev = -1;
        if (prev != dev) cudaSetDevice(dev);
    }
    ~AdamwDeviceGuard()
    {
        if (prev >= 0) cudaSetDevice(prev);
    }
};

struct FreeAdamw {
    void operator()(zero1_adamw_ctx *h) const
    {
        if (h->block) cudaFree(h->block);
        delete h;
    }
};

int create(const uint64_t *sizes, const uint8_t *decays, uint64_t count, const zero1_hparams *hp,
           const zero1_adamw_options *opts, zero1_adamw_handle *out)
{
    if (out == nullptr) return afail(ZERO1_EINVAL, "out is NULL");
    *out = nullptr;
    if (hp == nullptr || sizes == nullptr) return afail(ZERO1_EINVAL, "sizes or hparams is NULL");
    if (count == 0 || count > 65536) return afail(ZERO1_EINVAL, "count must be in [1, 65536]");
    zero1_adamw_options o{};
    o.state_bits = 32;
    if (opts) {
        if (opts->size != sizeof(zero1_adamw_options)) return afail(ZERO1_EINVAL, "options size does not match");
        o = *opts;
    }
    if (o.state_bits != 8 && o.state_bits != 32) return afail(ZERO1_EINVAL, "state_bits must be 8 or 32");
    for (const int t : {o.param_dtype, o.grad_dtype})
        if (t != ZERO1_DTYPE_BF16 && t != ZERO1_DTYPE_F32) return afail(ZERO1_EINVAL, "bad dtype");
    if (o.decay_before_update != 0 && o.decay_before_update != 1)
        return afail(ZERO1_EINVAL, "decay_before_update must be 0 or 1");
    if (o.reserved != 0) return afail(ZERO1_EINVAL, "reserved must be 0");
    if (!fine(hp->lr)) return afail(ZERO1_EINVAL, "lr must be finite and >= 0");
    if (!(hp->beta1 >= 0.0 && hp->beta1 < 1.0) || !(hp->beta2 >= 0.0 && hp->beta2 < 1.0))
        return afail(ZERO1_EINVAL, "betas must be in [0, 1)");
    if (!fine(hp->eps)) return afail(ZERO1_EINVAL, "eps must be finite and >= 0");
    if (!fine(hp->weight_decay)) return afail(ZERO1_EINVAL, "weight_decay must be finite and >= 0");
    if (!std::isfinite(hp->max_norm)) return afail(ZERO1_EINVAL, "max_norm must be finite");
    for (uint64_t i = 0; i < count; ++i)
        if (sizes[i] > (1ull << 40)) return afail(ZERO1_EINVAL, "tensor %llu has more than 2^40 entries", (unsigned long long)i);

    // ---- the plan
    std::vector<uint64_t> first(count + 1);
    uint64_t blocks = 0;
    for (uint64_t i = 0; i < count; ++i) {
        first[i] = blocks;
        blocks += (sizes[i] + kListBlock - 1) / kListBlock;
        // 2^40 entries of state are 4 TB: block numbers stay below 2^32
        if (blocks >= (1ull << 32)) return afail(ZERO1_EINVAL, "the list has more than 2^40 entries");
    }
    first[count] = blocks;
    if (blocks == 0) return afail(ZERO1_EINVAL, "every tensor is empty");
    std::vector<uint32_t> words(blocks);
    for (uint64_t i = 0; i < count; ++i) {
        const bool d = decays ? decays[i] != 0 : true;
        if (first[i] == first[i + 1]) continue;
        std::fill(words.begin() + first[i], words.begin() + first[i + 1], zero1::pack_block((uint32_t)i, kListBlock, d));
        const uint64_t rest = sizes[i] % kListBlock;
        if (rest) words[first[i + 1] - 1] = zero1::pack_block((uint32_t)i, (uint32_t)rest, d);
    }
    std::vector<double> correction;
    for (uint64_t t = 1;; ++t) {
        if (t > zero1::kMaxListTable)
            return afail(ZERO1_EINVAL, "the bias corrections do not reach 1.0 within %llu steps",
                         (unsigned long long)zero1::kMaxListTable);
        const double bc1 = 1.0 - std::pow(hp->beta1, (double)t), bc2 = 1.0 - std::pow(hp->beta2, (double)t);
        correction.push_back(std::sqrt(bc2) / bc1);
        if (bc1 == 1.0 && bc2 == 1.0) break;
    }

    // ---- the device
    int ndev = 0, dev = 0;
    cudaError_t e = cudaGetDeviceCount(&ndev);
    if (e != cudaSuccess || ndev == 0) {
        cudaGetLastError();
        return afail(ZERO1_ENODEV, "no CUDA device (%s)", cudaGetErrorString(e));
    }
    if ((e = cudaGetDevice(&dev)) != cudaSuccess) return acuda(e, "cudaGetDevice");
    int major = 0, minor = 0, sms = 0;
    if ((e = cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev)) != cudaSuccess ||
        (e = cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev)) != cudaSuccess ||
        (e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess)
        return acuda(e, "device query");
    if (major != 10 || minor != 3)
        return afail(ZERO1_ENODEV, "device %d is sm_%d%d; this library is built for sm_103a", dev, major, minor);

    // of the norm, over the launches a step takes (a list that takes launches of fewer tensors takes one)
    const uint64_t partials = zero1::norm_partials(first.data(), count, kCaps[2], sms);
    uint64_t at = 0;
    const auto take = [&](uint64_t bytes) {
        const uint64_t here = at;
        at += (bytes + 255) / 256 * 256;
        return here;
    };
    const uint64_t at_status = take(sizeof(zero1::ListStatus)), at_of = take(blocks * sizeof(uint32_t));
    const uint64_t at_corr = take(correction.size() * sizeof(double)), at_part = take(partials * sizeof(double));
    std::unique_ptr<zero1_adamw_ctx, FreeAdamw> h(new zero1_adamw_ctx);
    h->hp = *hp;
    h->opt = o;
    h->sizes.assign(sizes, sizes + count);
    h->first = first;
    h->ranges.resize(2 * count);
    h->device = dev;
    h->num_sms = sms;
    h->partials = partials;
    h->block_bytes = at;
    if ((e = cudaMalloc(&h->block, at)) != cudaSuccess) {
        h->block = nullptr;
        return acuda(e, "cudaMalloc of the list's tables");
    }
    unsigned char *base = static_cast<unsigned char *>(h->block);
    e = cudaMemset(h->block, 0, at);
    const auto put = [&](uint64_t to, const void *src, uint64_t bytes) {
        if (e == cudaSuccess) e = cudaMemcpy(base + to, src, bytes, cudaMemcpyHostToDevice);
    };
    put(at_of, words.data(), blocks * sizeof(uint32_t));
    put(at_corr, correction.data(), correction.size() * sizeof(double));
    zero1::ListTables &d = h->d;
    d.blocks = reinterpret_cast<const uint32_t *>(base + at_of);
    d.status = reinterpret_cast<zero1::ListStatus *>(base + at_status);
    d.partials = reinterpret_cast<double *>(base + at_part);
    d.correction = reinterpret_cast<const double *>(base + at_corr);
    d.steps = correction.size();
    d.weight_decay = hp->weight_decay;
    d.max_norm = hp->max_norm;
    if (e == cudaSuccess) e = zero1::launch(zero1::zero1_adamw_set_kernel, dim3(1), 1, 0, nullptr, d, 0ull, hp->lr, 3);
    if (e == cudaSuccess) e = cudaDeviceSynchronize();
    if (e != cudaSuccess) return acuda(e, "filling the list's tables");
    {
        std::lock_guard<std::mutex> lk(g_adamw_mu);
        g_adamw_live.insert(h.get());
    }
    *out = h.release();
    return ZERO1_OK;
}

struct StepCall {
    const void *const *grads;
    void *const *params;
    float *master;
    void *m, *v;
    float *scales;
    cudaStream_t stream;
};

template <typename G, int CAP>
cudaError_t norm_t(const zero1_adamw_ctx *h, const StepCall &c, uint64_t i0, uint64_t i1, uint32_t &before)
{
    zero1::NormParams<CAP> p;
    for (uint64_t i = i0; i < i1; ++i) p.grads[i - i0] = c.grads[i], p.first[i - i0] = (uint32_t)h->first[i];
    p.d = h->d;
    p.block0 = h->first[i0];
    p.nblocks = h->first[i1] - h->first[i0];
    p.tensor0 = (uint32_t)i0;
    p.before = before;
    p.one = 1.f;
    p.last = i1 == h->sizes.size();
    const uint32_t grid = zero1::norm_grid(p.nblocks, p.last, h->num_sms);
    if (grid == 0) return cudaSuccess;
    before += grid;
    if (before > h->partials) return cudaErrorInvalidConfiguration;
    return zero1::launch(zero1::zero1_adamw_norm_kernel<G, CAP>, dim3(grid), zero1::kListThreads, 0, c.stream, p);
}

template <int CAP>
void fill(zero1::UpdateParams<CAP> &p, const zero1_adamw_ctx *h, const StepCall &c, uint64_t i0, uint64_t i1)
{
    for (uint64_t i = i0; i < i1; ++i)
        p.grads[i - i0] = c.grads[i], p.params[i - i0] = c.params[i], p.first[i - i0] = (uint32_t)h->first[i];
    p.d = h->d;
    p.master = c.master;
    p.m = c.m;
    p.v = c.v;
    p.scales = reinterpret_cast<float2 *>(c.scales);
    p.block0 = h->first[i0];
    p.nblocks = h->first[i1] - h->first[i0];
    p.seed = h->opt.seed;
    const auto twice = [](double v) {
        const float f = (float)v;
        uint32_t bits;
        std::memcpy(&bits, &f, sizeof bits);
        return zero1::Two{(unsigned long long)bits << 32 | bits};
    };
    p.beta1 = twice(h->hp.beta1);
    p.omb1 = twice(1.0 - h->hp.beta1);
    p.beta2 = twice(h->hp.beta2);
    p.omb2 = twice(1.0 - h->hp.beta2);
    p.eps2 = twice(h->hp.eps);
    p.one = twice(1.0);
    p.eps = (float)h->hp.eps;
    p.tensor0 = (uint32_t)i0;
    p.clipped = h->hp.max_norm > 0.0;
    p.decay_first = h->opt.decay_before_update;
    p.eps_easy = p.eps >= 0x1p-50f && p.eps <= 0x1p50f;   // so that sqrt(v) + eps is never near the ends of fp32's range
    p.last = i1 == h->sizes.size();
}

template <typename P, typename G, int BITS, int CAP>
cudaError_t update_t(const zero1_adamw_ctx *h, const StepCall &c, uint64_t i0, uint64_t i1)
{
    zero1::UpdateParams<CAP> p;
    fill(p, h, c, i0, i1);
    p.per_warp = p.nblocks < 16ull * zero1::kWarps * (uint64_t)h->num_sms ? 1 : zero1::kUpdateBlocks;
    const uint64_t per = (uint64_t)zero1::kWarps * p.per_warp;
    uint64_t grid = (p.nblocks + per - 1) / per;
    uint32_t smem = 0;
    if (BITS == 8) {
        smem = zero1::kWarps * 2 * zero1::Staged<P, G>::kBytes;   // 32 or 40 KB
        p.per_warp = p.nblocks < 64ull * zero1::kWarps * (uint64_t)h->num_sms ? 1 : zero1::kStagedBlocks;
        grid = (p.nblocks + zero1::kWarps * p.per_warp - 1) / (zero1::kWarps * p.per_warp);
    }
    if (grid == 0) {
        if (!p.last) return cudaSuccess;
        grid = 1;
    }
    const auto kernel = zero1::zero1_adamw_update_kernel<P, G, BITS, CAP>;
    return p.clipped && i0 == 0 ? zero1::launch_early(kernel, dim3((unsigned)grid), zero1::kListThreads, smem, c.stream, p)
                                : zero1::launch(kernel, dim3((unsigned)grid), zero1::kListThreads, smem, c.stream, p);
}

template <typename P, typename G, int BITS, int CAP>
cudaError_t step_t(const zero1_adamw_ctx *h, const StepCall &c)
{
    const uint64_t count = h->sizes.size();
    cudaError_t e = cudaSuccess;
    uint32_t before = 0;
    if (CAP == kCaps[0] && h->hp.max_norm > 0.0 && h->first.back() <= zero1::kSmallWarps) {
        zero1::UpdateParams<kCaps[0]> p;
        fill(p, h, c, 0, count);
        return zero1::launch(zero1::zero1_adamw_small_kernel<P, G, BITS>, dim3(1), 32 * zero1::kSmallWarps, 0, c.stream, p);
    }
    if (h->hp.max_norm > 0.0)
        for (uint64_t i = 0; e == cudaSuccess && i < count; i += CAP)
            e = norm_t<G, CAP>(h, c, i, std::min<uint64_t>(i + CAP, count), before);
    for (uint64_t i = 0; e == cudaSuccess && i < count; i += CAP)
        e = update_t<P, G, BITS, CAP>(h, c, i, std::min<uint64_t>(i + CAP, count));
    return e;
}

template <typename P, typename G, int BITS>
cudaError_t step_cap(const zero1_adamw_ctx *h, const StepCall &c)
{
    const uint64_t count = h->sizes.size();
    if (count <= (uint64_t)kCaps[0]) return step_t<P, G, BITS, kCaps[0]>(h, c);
    if (count <= (uint64_t)kCaps[1]) return step_t<P, G, BITS, kCaps[1]>(h, c);
    return step_t<P, G, BITS, kCaps[2]>(h, c);
}

template <typename P, typename G>
cudaError_t step_bits(const zero1_adamw_ctx *h, const StepCall &c)
{
    return h->opt.state_bits == 8 ? step_cap<P, G, 8>(h, c) : step_cap<P, G, 32>(h, c);
}

struct Bytes {
    const void *p;
    uint64_t n;
};
bool apart(Bytes a, Bytes b)
{
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
    return !a.p || !b.p || x + a.n <= y || y + b.n <= x;
}

int check_state(const zero1_adamw_ctx *h, const void *master, const void *m, const void *v, const void *scales)
{
    if ((master != nullptr) != (h->opt.param_dtype == ZERO1_DTYPE_BF16))
        return afail(ZERO1_EINVAL, "master is the fp32 copy of bf16 parameters, and NULL for fp32 ones");
    if (!m || !v) return afail(ZERO1_EINVAL, "m or v is NULL");
    if ((scales != nullptr) != (h->opt.state_bits == 8)) return afail(ZERO1_EINVAL, "scales go with moments in 8 bits, and only with them");
    if (!on16(master) || !on16(m) || !on16(v) || !on16(scales))
        return afail(ZERO1_EALIGN, "master, m, v and scales must be 16-byte aligned");
    const uint64_t n = h->first.back() * kListBlock, each = h->opt.state_bits == 8 ? n : 4 * n;
    if (apart({master, 4 * n}, {m, each}) && apart({master, 4 * n}, {v, each}) && apart({m, each}, {v, each}) &&
        apart({scales, n / 32}, {m, each}) && apart({scales, n / 32}, {v, each}) && apart({scales, n / 32}, {master, 4 * n}))
        return ZERO1_OK;
    return afail(ZERO1_EINVAL, "two of master, m, v and scales share memory");
}

// No tensor may share memory with the state, and no parameter with another
// tensor: other blocks write them.
int check_tensors(zero1_adamw_ctx *h, const void *const *grads, void *const *params, const void *master, const void *m,
                  const void *v, const void *scales)
{
    const uint64_t n = h->first.back() * kListBlock, each = h->opt.state_bits == 8 ? n : 4 * n;
    const zero1::StateBuffer state[4] = {{master, 4 * n}, {m, each}, {v, each}, {scales, n / 32}};
    const zero1::ListTensors t{h->sizes.data(), h->sizes.size(), grads, params, bytes_of(h->opt.grad_dtype), bytes_of(h->opt.param_dtype)};
    int which = 0;
    bool param = false;
    size_t i = zero1::tensor_in_state(t, state, 4, &which, &param);
    const char *const names[4] = {"master", "m", "v", "scales"};
    if (i < t.count)
        return afail(ZERO1_EINVAL, "the %s of tensor %zu shares memory with %s", param ? "parameter" : "gradient", i, names[which]);
    i = zero1::shared_param(t, h->ranges.data());
    if (i < t.count) return afail(ZERO1_EINVAL, "parameter tensor %zu shares memory with another tensor of the call", i);
    return ZERO1_OK;
}

}  // namespace

extern "C" {

int zero1_adamw_create(const uint64_t *sizes, const uint8_t *decays, uint64_t count, const zero1_hparams *hp,
                       const zero1_adamw_options *opts, zero1_adamw_handle *out)
{
    try {
        return create(sizes, decays, count, hp, opts, out);
    } catch (const std::bad_alloc &) {
        return afail(ZERO1_ENOMEM, "host allocation failed");
    } catch (const std::exception &x) {
        return afail(ZERO1_EINVAL, "%s", x.what());
    }
}

int zero1_adamw_destroy(zero1_adamw_handle h)
{
    if (h == nullptr) return ZERO1_OK;
    {
        std::lock_guard<std::mutex> lk(g_adamw_mu);
        if (!g_adamw_live.erase(h)) return afail(ZERO1_EINVAL, "unknown or already destroyed handle");
    }
    AdamwDeviceGuard g(h->device);
    const cudaError_t e1 = cudaDeviceSynchronize(), e2 = cudaFree(h->block);
    delete h;
    if (e1 != cudaSuccess) return acuda(e1, "cudaDeviceSynchronize in destroy");
    if (e2 != cudaSuccess) return acuda(e2, "cudaFree");
    return ZERO1_OK;
}

int zero1_adamw_step(zero1_adamw_handle h, const void *const *grad_ptrs, void *const *param_ptrs, float *master, void *m,
                     void *v, float *scales, void *stream)
{
    if (!adamw_live(h)) return afail(ZERO1_EINVAL, "invalid handle");
    if (!grad_ptrs || !param_ptrs) return afail(ZERO1_EINVAL, "pointer array is NULL");
    if (const int rc = check_state(h, master, m, v, scales)) return rc;
    const size_t gb = bytes_of(h->opt.grad_dtype), pb = bytes_of(h->opt.param_dtype);
    for (size_t i = 0; i < h->sizes.size(); ++i) {
        if (h->sizes[i] == 0) continue;
        if (!grad_ptrs[i] || !param_ptrs[i]) return afail(ZERO1_EINVAL, "tensor %zu is NULL", i);
        if (reinterpret_cast<uintptr_t>(grad_ptrs[i]) % gb || reinterpret_cast<uintptr_t>(param_ptrs[i]) % pb)
            return afail(ZERO1_EALIGN, "tensor %zu is not aligned to its elements", i);
    }
    if (const int rc = check_tensors(h, grad_ptrs, param_ptrs, master, m, v, scales)) return rc;
    cudaError_t e;
    AdamwDeviceGuard g(h->device);
    const StepCall c{grad_ptrs, param_ptrs, master, m, v, scales, static_cast<cudaStream_t>(stream)};
    if (h->opt.param_dtype == ZERO1_DTYPE_BF16)
        e = h->opt.grad_dtype == ZERO1_DTYPE_BF16 ? step_bits<uint16_t, uint16_t>(h, c) : step_bits<uint16_t, float>(h, c);
    else
        e = h->opt.grad_dtype == ZERO1_DTYPE_BF16 ? step_bits<float, uint16_t>(h, c) : step_bits<float, float>(h, c);
    return e == cudaSuccess ? ZERO1_OK : acuda(e, "kernel launch");
}

int zero1_adamw_moments(zero1_adamw_handle h, const void *m, const void *v, const float *scales, float *m_out, float *v_out,
                        void *stream)
{
    if (!adamw_live(h)) return afail(ZERO1_EINVAL, "invalid handle");
    if (h->opt.state_bits != 8) return afail(ZERO1_EINVAL, "the moments of this handle are fp32 already");
    if (!m || !v || !scales) return afail(ZERO1_EINVAL, "NULL buffer");
    if (!on16(m) || !on16(v) || !on16(scales) || !on16(m_out) || !on16(v_out))
        return afail(ZERO1_EALIGN, "buffers must be 16-byte aligned");
    const uint64_t blocks = h->first.back(), n = blocks * kListBlock;
    for (const Bytes out : {Bytes{m_out, 4 * n}, Bytes{v_out, 4 * n}})
        if (!apart(out, {m, n}) || !apart(out, {v, n}) || !apart(out, {scales, n / 32}))
            return afail(ZERO1_EINVAL, "m_out or v_out shares memory with the moments");
    if (!apart({m_out, 4 * n}, {v_out, 4 * n})) return afail(ZERO1_EINVAL, "m_out and v_out share memory");
    AdamwDeviceGuard g(h->device);
    const cudaError_t e = zero1::launch(zero1::zero1_adamw_moments_kernel, dim3((unsigned)((blocks + zero1::kWarps - 1) / zero1::kWarps)),
                                        zero1::kListThreads, 0, static_cast<cudaStream_t>(stream), h->d, blocks,
                                        static_cast<const uint8_t *>(m), static_cast<const uint8_t *>(v),
                                        reinterpret_cast<const float2 *>(scales), m_out, v_out);
    return e == cudaSuccess ? ZERO1_OK : acuda(e, "kernel launch");
}

int zero1_adamw_set_steps(zero1_adamw_handle h, uint64_t t, void *stream)
{
    if (!adamw_live(h)) return afail(ZERO1_EINVAL, "invalid handle");
    AdamwDeviceGuard g(h->device);
    const cudaError_t e = zero1::launch(zero1::zero1_adamw_set_kernel, dim3(1), 1, 0, static_cast<cudaStream_t>(stream), h->d,
                                        (unsigned long long)t, 0.0, 1);
    return e == cudaSuccess ? ZERO1_OK : acuda(e, "kernel launch");
}

int zero1_adamw_set_lr(zero1_adamw_handle h, double lr, void *stream)
{
    if (!adamw_live(h)) return afail(ZERO1_EINVAL, "invalid handle");
    if (!fine(lr)) return afail(ZERO1_EINVAL, "lr must be finite and >= 0");
    AdamwDeviceGuard g(h->device);
    const cudaError_t e =
        zero1::launch(zero1::zero1_adamw_set_kernel, dim3(1), 1, 0, static_cast<cudaStream_t>(stream), h->d, 0ull, lr, 2);
    return e == cudaSuccess ? ZERO1_OK : acuda(e, "kernel launch");
}

static int read_status(zero1_adamw_ctx *h, zero1::ListStatus *s, void *stream)
{
    AdamwDeviceGuard g(h->device);
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaError_t e = cudaMemcpyAsync(s, h->d.status, sizeof *s, cudaMemcpyDeviceToHost, st);
    if (e == cudaSuccess) e = cudaStreamSynchronize(st);
    return e == cudaSuccess ? ZERO1_OK : acuda(e, "reading the status");
}

int zero1_adamw_get_steps(zero1_adamw_handle h, uint64_t *t, void *stream)
{
    if (!adamw_live(h)) return afail(ZERO1_EINVAL, "invalid handle");
    if (!t) return afail(ZERO1_EINVAL, "t is NULL");
    zero1::ListStatus s;
    if (const int rc = read_status(h, &s, stream)) return rc;
    *t = s.t;
    return ZERO1_OK;
}

int zero1_adamw_get_grad_norm(zero1_adamw_handle h, double *norm, float *clip_coef, void *stream)
{
    if (!adamw_live(h)) return afail(ZERO1_EINVAL, "invalid handle");
    if (!(h->hp.max_norm > 0.0)) return afail(ZERO1_EINVAL, "a handle that does not clip forms no norm");
    zero1::ListStatus s;
    if (const int rc = read_status(h, &s, stream)) return rc;
    if (norm) *norm = s.norm;
    if (clip_coef) *clip_coef = s.clip;
    return ZERO1_OK;
}

int zero1_adamw_layout(zero1_adamw_handle h, uint64_t *entries, uint64_t *starts, uint64_t *device_bytes)
{
    if (!adamw_live(h)) return afail(ZERO1_EINVAL, "invalid handle");
    if (entries) *entries = h->first.back() * kListBlock;
    if (starts)
        for (size_t i = 0; i < h->sizes.size(); ++i) starts[i] = h->first[i] * kListBlock;
    if (device_bytes) *device_bytes = h->block_bytes;
    return ZERO1_OK;
}

}  // extern "C"
