// zero1_layernorm.cu -- layer normalisation, forward and backward, with the
// sums over rows that give the weight's and the bias's gradients.
//
//   y = (x - mean) rstd gamma + beta,   rstd = 1/sqrt(var + eps) per row;
//   with h = (x - mean) rstd and g = dy gamma:
//   dx = rstd (g - mean(g) - h mean(g h)),
//   dgamma = sum over rows of dy h,  dbeta = sum over rows of dy.
//
// All sums are fp32, the variance from the deviations themselves.  Bound by
// HBM: forward reads x and writes y, backward reads x and dy and writes dx,
// each once.  A row is held in registers: by one warp while a lane's share
// fits (forward up to 2,048 aligned bf16, backward, with its column sums, up
// to 1,024), then by four to sixteen warps, up to 8,192 columns, or 16,384 of
// aligned bf16; wider rows are read again from the caches.  The column sums
// stay in registers over up to 512 rows of a thread, one partial row per block
// goes to the workspace, and a second kernel adds the partial rows in a fixed
// order (no atomics: the same inputs give the same bits).
//
// Measured, bf16: forward 16,384 x 768 in 12 us, 65,536 x 4,096 in 184 us
// (5.8 TB/s; 188 back to back); backward 65,536 x 4,096 in 279 us (5.8 TB/s,
// issue slots 57% busy) and 5 us for the column sums, 16,384 x 768 in 21 and
// 4 us; one row of 768 in 5 us, all latency.  Rows of single entries run at
// half the rate: 32,768 x 1,000 at a stride of 1,001 backward in 58 us (floor
// 29).  Past registers, two to five times the floor: 8,192 x 12,288 fp32
// forward in 211 us (119), backward in 460 (178); 8,192 x 18,432 bf16 in 270
// (89) and 616 (134).
#include <cstdarg>
#include <cstdio>

#include "zero1.h"
#include "zero1_internal.h"
#include "zero1_launch.h"
#include "zero1_ptx.cuh"

namespace zero1 {
namespace {

constexpr int kMaxPartials = 320;      // blocks of the backward pass, at most
constexpr int kLnThreads = 256;
constexpr uint32_t kWideTile = 1024;   // columns of one block of the wide column sums
// Rows whose column sums a thread adds up one after another.  Such a sum of n
// terms of one sign is off by up to n 2^-24 of itself (1e-4 measured at 13,800
// fp32 terms), so longer ones are taken in launches of 512 rows a thread
// (155,648 rows and more), each adding to the partial rows of those before.
constexpr uint64_t kRun = 512;
constexpr uint32_t kRowRun = 128 * 1024;   // columns of a wide row that are one run, 128 entries a thread

template <typename T, int V>
struct Piece;   // V neighbouring entries as they lie in memory
template <>
struct Piece<uint16_t, 8> {
    uint4 raw;
    __device__ __forceinline__ void get(float v[8]) const { ptx::set_widened(v, raw); }
    __device__ __forceinline__ void set(const float v[8])
    {
        raw = make_uint4(ptx::pack2(v[0], v[1]), ptx::pack2(v[2], v[3]), ptx::pack2(v[4], v[5]), ptx::pack2(v[6], v[7]));
    }
};
template <>
struct Piece<uint16_t, 1> {
    uint16_t raw;
    __device__ __forceinline__ void get(float v[1]) const { v[0] = __uint_as_float((uint32_t)raw << 16); }
    __device__ __forceinline__ void set(const float v[1]) { raw = __bfloat16_as_ushort(__float2bfloat16_rn(v[0])); }
};
template <>
struct Piece<float, 4> {
    float4 raw;
    __device__ __forceinline__ void get(float v[4]) const { v[0] = raw.x, v[1] = raw.y, v[2] = raw.z, v[3] = raw.w; }
    __device__ __forceinline__ void set(const float v[4]) { raw = make_float4(v[0], v[1], v[2], v[3]); }
};
template <>
struct Piece<float, 1> {
    float raw;
    __device__ __forceinline__ void get(float v[1]) const { v[0] = raw; }
    __device__ __forceinline__ void set(const float v[1]) { raw = v[0]; }
};

template <typename T, int V>
__device__ __forceinline__ Piece<T, V> fetch(const T *p)
{
    return *reinterpret_cast<const Piece<T, V> *>(p);
}

// Sums of a and b over the TPR threads of a row, on all of them.
template <int TPR, int THREADS>
__device__ __forceinline__ void row_sum(float &a, float &b, float2 (*shared)[THREADS / 32], int &turn)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        a += __shfl_xor_sync(~0u, a, o);
        b += __shfl_xor_sync(~0u, b, o);
    }
    if (TPR > 32) {   // two buffers in turn: one barrier a call, of the warps that share the row
        const uint32_t group = threadIdx.x / TPR;
        float2 *s = shared[turn];
        turn ^= 1;
        if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = make_float2(a, b);
        asm volatile("barrier.cta.sync.aligned %0, %1;" ::"r"(1 + group), "n"(TPR) : "memory");
        s += group * (TPR / 32);
        a = b = 0.f;
#pragma unroll
        for (int i = 0; i < TPR / 32; ++i) {
            a += s[i].x;
            b += s[i].y;
        }
    }
}

template <typename T>
struct FwdParams {
    const T *x, *gamma, *beta;
    T *y;
    float *mean, *rstd;
    uint64_t rows, ldx, ldy;
    uint32_t cols;
    float eps, inv_n;
};

// One row by TPR threads, each holding NV pieces of V entries.
template <typename T, int V, int TPR, int NV, int THREADS>
__global__ void __launch_bounds__(THREADS) zero1_layernorm_fwd_kernel(const __grid_constant__ FwdParams<T> p)
{
    __shared__ float2 shared[2][THREADS / 32];
    int turn = 0;
    const uint64_t row = (uint64_t)blockIdx.x * (THREADS / TPR) + threadIdx.x / TPR;
    if (row >= p.rows) return;   // whole warps, or the whole block
    const uint32_t t = threadIdx.x % TPR;
    const T *x = p.x + row * p.ldx;
    Piece<T, V> xs[NV];
    float sum = 0.f, none = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const uint32_t c = (j * TPR + t) * V;
        if (c < p.cols) xs[j] = fetch<T, V>(x + c);
    }
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        if ((j * TPR + t) * V < p.cols) {
            float v[V];
            xs[j].get(v);
#pragma unroll
            for (int i = 0; i < V; ++i) sum += v[i];
        }
    }
    row_sum<TPR, THREADS>(sum, none, shared, turn);
    const float mean = sum * p.inv_n;
    float ss = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        if ((j * TPR + t) * V < p.cols) {
            float v[V];
            xs[j].get(v);
#pragma unroll
            for (int i = 0; i < V; ++i) ss += (v[i] - mean) * (v[i] - mean);
        }
    }
    row_sum<TPR, THREADS>(ss, none, shared, turn);
    const float rstd = 1.0f / sqrtf(ss * p.inv_n + p.eps);
    if (t == 0) {
        p.mean[row] = mean;
        p.rstd[row] = rstd;
    }
    T *y = p.y + row * p.ldy;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const uint32_t c = (j * TPR + t) * V;
        if (c < p.cols) {
            float v[V], g[V], b[V];
            xs[j].get(v);
            fetch<T, V>(p.gamma + c).get(g);
            if (p.beta) fetch<T, V>(p.beta + c).get(b);
#pragma unroll
            for (int i = 0; i < V; ++i) v[i] = (v[i] - mean) * rstd * g[i] + (p.beta ? b[i] : 0.f);
            Piece<T, V> out;
            out.set(v);
            *reinterpret_cast<Piece<T, V> *>(y + c) = out;
        }
    }
}

// f(column, a, b) adds a column's terms to a and b, for every 1024th column
// of a row from this thread's on; RUNS: each run of columns to sums of its own
// first (the inner of two loops has fewer loads in flight: 3 to 6% slower at
// 12,288 to 50,001 columns, where one loop is exact enough).
template <bool RUNS, typename F>
__device__ __forceinline__ void over_row(uint32_t cols, float &a, float &b, F f)
{
    if (!RUNS) {
        for (uint32_t c = threadIdx.x; c < cols; c += 1024) f(c, a, b);
    } else {
        for (uint32_t first = 0; first < cols; first += kRowRun) {
            const uint32_t end = min(cols, first + kRowRun);
            float ra = 0.f, rb = 0.f;
            for (uint32_t c = first + threadIdx.x; c < end; c += 1024) f(c, ra, rb);
            a += ra;
            b += rb;
        }
    }
}

// Rows too wide for registers: one block a row, three passes over it.
template <typename T, bool RUNS>
__global__ void __launch_bounds__(1024) zero1_layernorm_fwd_wide_kernel(const __grid_constant__ FwdParams<T> p)
{
    __shared__ float2 shared[2][32];
    int turn = 0;
    const uint64_t row = blockIdx.x;
    const T *x = p.x + row * p.ldx;
    float sum = 0.f, none = 0.f, v[1], g[1], b[1] = {0.f};
    over_row<RUNS>(p.cols, sum, none, [&](uint32_t c, float &a, float &) {
        fetch<T, 1>(x + c).get(v);
        a += v[0];
    });
    row_sum<1024, 1024>(sum, none, shared, turn);
    const float mean = sum * p.inv_n;
    float ss = 0.f;
    over_row<RUNS>(p.cols, ss, none, [&](uint32_t c, float &a, float &) {
        fetch<T, 1>(x + c).get(v);
        a += (v[0] - mean) * (v[0] - mean);
    });
    row_sum<1024, 1024>(ss, none, shared, turn);
    const float rstd = 1.0f / sqrtf(ss * p.inv_n + p.eps);
    if (threadIdx.x == 0) {
        p.mean[row] = mean;
        p.rstd[row] = rstd;
    }
    T *y = p.y + row * p.ldy;
    for (uint32_t c = threadIdx.x; c < p.cols; c += 1024) {
        fetch<T, 1>(x + c).get(v);
        fetch<T, 1>(p.gamma + c).get(g);
        if (p.beta) fetch<T, 1>(p.beta + c).get(b);
        v[0] = (v[0] - mean) * rstd * g[0] + b[0];
        Piece<T, 1> out;
        out.set(v);
        *reinterpret_cast<Piece<T, 1> *>(y + c) = out;
    }
}

template <typename T>
struct BwdParams {
    const T *dy, *x, *gamma;
    const float *mean, *rstd;
    T *dx;
    float *partials;       // gridDim.x rows of dgamma, then of dbeta: [block][2][cols]
    uint64_t rows, lddy, ldx, lddx;
    uint32_t cols;
    float inv_n;
    int add;               // to what a launch over earlier rows left in the partials
};

// AHEAD: the next row's pieces are fetched while this one's are used, where
// 128 registers hold both and the column sums (blocks of 256, two an SM).
template <typename T, int V, int TPR, int NV, int THREADS, bool AHEAD>
__global__ void __launch_bounds__(THREADS, 512 / THREADS) zero1_layernorm_bwd_kernel(const __grid_constant__ BwdParams<T> p)
{
    constexpr int kRows = THREADS / TPR;      // rows at a time
    __shared__ float2 shared[2][THREADS / 32];
    extern __shared__ float fold[];           // kRows x cols, where a block holds several rows
    int turn = 0;
    ptx::launch_dependents();
    const uint32_t t = threadIdx.x % TPR, lane_row = threadIdx.x / TPR;
    float ag[NV * V], ab[NV * V];
#pragma unroll
    for (int i = 0; i < NV * V; ++i) ag[i] = ab[i] = 0.f;
    Piece<T, V> xs[NV], ds[NV];
    float mean = 0.f, rstd = 0.f;
    const uint64_t step = (uint64_t)gridDim.x * kRows;
    uint64_t row = (uint64_t)blockIdx.x * kRows + lane_row;
    const auto load = [&](uint64_t r) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const uint32_t c = (j * TPR + t) * V;
            if (c < p.cols) {
                xs[j] = fetch<T, V>(p.x + r * p.ldx + c);
                ds[j] = fetch<T, V>(p.dy + r * p.lddy + c);
            }
        }
        mean = p.mean[r];
        rstd = p.rstd[r];
    };
    // h and dy gamma of a row stay as they are computed while registers hold them, with the weights; else a row's
    // pieces stay and both are computed again.
    constexpr bool kKeep = AHEAD && NV * V <= (V == 8 ? 16 : 8);   // unpacked pieces take a register an entry
    constexpr int kKept = kKeep ? NV * V : 1;
    float gamma[kKept];
    if constexpr (kKeep) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const uint32_t c = (j * TPR + t) * V;
            if (c < p.cols) {
                float g[V];
                fetch<T, V>(p.gamma + c).get(g);
#pragma unroll
                for (int i = 0; i < V; ++i) gamma[j * V + i] = g[i];
            }
        }
    }
    if (AHEAD && row < p.rows) load(row);
    for (; row < p.rows; row += step) {
        if (!AHEAD) load(row);
        Piece<T, V> xc[NV], dc[NV];
        const float mc = mean, rc = rstd;
#pragma unroll
        for (int j = 0; j < NV; ++j) xc[j] = xs[j], dc[j] = ds[j];
        if (AHEAD && row + step < p.rows) load(row + step);
        float sg = 0.f, sh = 0.f, hs[kKept], ws[kKept];
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const uint32_t c = (j * TPR + t) * V;
            if (c < p.cols) {
                float x[V], d[V], g[V];
                xc[j].get(x);
                dc[j].get(d);
                if constexpr (!kKeep) fetch<T, V>(p.gamma + c).get(g);
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const float h = (x[i] - mc) * rc, w = d[i] * (kKeep ? gamma[(j * V + i) % kKept] : g[i]);
                    ag[j * V + i] += d[i] * h;
                    ab[j * V + i] += d[i];
                    sg += w;
                    sh += w * h;
                    if (kKeep) hs[(j * V + i) % kKept] = h, ws[(j * V + i) % kKept] = w;
                }
            }
        }
        row_sum<TPR, THREADS>(sg, sh, shared, turn);
        sg *= p.inv_n;
        sh *= p.inv_n;
        T *dx = p.dx + row * p.lddx;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const uint32_t c = (j * TPR + t) * V;
            if (c < p.cols) {
                float x[V], d[V], g[V];
                if constexpr (kKeep) {
#pragma unroll
                    for (int i = 0; i < V; ++i) d[i] = rc * (ws[(j * V + i) % kKept] - sg - hs[(j * V + i) % kKept] * sh);
                } else {
                    xc[j].get(x);
                    dc[j].get(d);
                    fetch<T, V>(p.gamma + c).get(g);
#pragma unroll
                    for (int i = 0; i < V; ++i) d[i] = rc * (d[i] * g[i] - sg - (x[i] - mc) * rc * sh);
                }
                Piece<T, V> out;
                out.set(d);
                *reinterpret_cast<Piece<T, V> *>(dx + c) = out;
            }
        }
    }
    float *part = p.partials + (uint64_t)blockIdx.x * 2 * p.cols;
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        const float *a = which ? ab : ag;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const uint32_t c = (j * TPR + t) * V;
            if (c < p.cols) {
                float *to = kRows > 1 ? fold + (uint64_t)lane_row * p.cols + c : part + c;
#pragma unroll
                for (int i = 0; i < V; ++i) to[i] = (kRows == 1 && p.add ? to[i] : 0.f) + a[j * V + i];
            }
        }
        if (kRows > 1) {
            __syncthreads();
            for (uint32_t c = threadIdx.x; c < p.cols; c += THREADS) {
                float s = 0.f;
#pragma unroll
                for (int r = 0; r < kRows; ++r) s += fold[(uint64_t)r * p.cols + c];
                part[c] = (p.add ? part[c] : 0.f) + s;
            }
            __syncthreads();
        }
        part += p.cols;
    }
}

// Rows too wide for registers: dx by one block a row in two passes.
template <typename T, bool RUNS>
__global__ void __launch_bounds__(1024) zero1_layernorm_bwd_wide_kernel(const __grid_constant__ BwdParams<T> p)
{
    __shared__ float2 shared[2][32];
    int turn = 0;
    const uint64_t row = blockIdx.x;
    const T *xr = p.x + row * p.ldx, *dr = p.dy + row * p.lddy;
    T *dx = p.dx + row * p.lddx;
    const float mean = p.mean[row], rstd = p.rstd[row];
    float sg = 0.f, sh = 0.f, x[1], d[1], g[1];
    over_row<RUNS>(p.cols, sg, sh, [&](uint32_t c, float &a, float &b) {
        fetch<T, 1>(xr + c).get(x);
        fetch<T, 1>(dr + c).get(d);
        fetch<T, 1>(p.gamma + c).get(g);
        a += d[0] * g[0];
        b += d[0] * g[0] * ((x[0] - mean) * rstd);
    });
    row_sum<1024, 1024>(sg, sh, shared, turn);
    sg *= p.inv_n;
    sh *= p.inv_n;
    for (uint32_t c = threadIdx.x; c < p.cols; c += 1024) {
        fetch<T, 1>(xr + c).get(x);
        fetch<T, 1>(dr + c).get(d);
        fetch<T, 1>(p.gamma + c).get(g);
        d[0] = rstd * (d[0] * g[0] - sg - (x[0] - mean) * rstd * sh);
        Piece<T, 1> out;
        out.set(d);
        *reinterpret_cast<Piece<T, 1> *>(dx + c) = out;
    }
}

// ... and the column sums by blocks of kWideTile columns over every
// gridDim.x-th row.  Reads dy before the kernel above may overwrite it
// (dx may be dy), so it goes first.
template <typename T>
__global__ void __launch_bounds__(kLnThreads) zero1_layernorm_cols_wide_kernel(const __grid_constant__ BwdParams<T> p)
{
    float *part = p.partials + (uint64_t)blockIdx.x * 2 * p.cols;
    for (uint32_t c = blockIdx.y * kWideTile + threadIdx.x; c < min(p.cols, (blockIdx.y + 1) * kWideTile); c += kLnThreads) {
        float ag = 0.f, ab = 0.f, x[1], d[1];
        for (uint64_t r = blockIdx.x; r < p.rows; r += gridDim.x) {
            fetch<T, 1>(p.x + r * p.ldx + c).get(x);
            fetch<T, 1>(p.dy + r * p.lddy + c).get(d);
            ag += d[0] * ((x[0] - p.mean[r]) * p.rstd[r]);
            ab += d[0];
        }
        part[c] = (p.add ? part[c] : 0.f) + ag;
        part[p.cols + c] = (p.add ? part[p.cols + c] : 0.f) + ab;
    }
}

// dgamma and dbeta: the partial rows added in order, 32 groups of them at
// once so that a thread's few reads are all in flight together.
template <typename G>
__global__ void __launch_bounds__(1024) zero1_layernorm_cols_kernel(const float *partials, int count, uint32_t cols,
                                                                    G *dgamma, G *dbeta)
{
    __shared__ float s[32][33];
    ptx::grid_dependency_wait();
    const uint32_t lane = threadIdx.x & 31, group = threadIdx.x >> 5;
    const uint64_t c = (uint64_t)blockIdx.x * 32 + lane;   // over dgamma's columns, then dbeta's
    const uint64_t width = 2ull * cols;
    float v = 0.f;
    if (c < width) {
        float x[kMaxPartials / 32];
#pragma unroll
        for (int i = 0; i < kMaxPartials / 32; ++i) {
            const int at = (int)group + 32 * i;
            x[i] = at < count ? partials[(uint64_t)at * width + c] : 0.f;
        }
#pragma unroll
        for (int i = 0; i < kMaxPartials / 32; ++i) v += x[i];
    }
    s[group][lane] = v;
    __syncthreads();
    v = s[lane][group];        // warp `group` adds up column `group`
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
    const uint64_t column = (uint64_t)blockIdx.x * 32 + group;
    if (lane == 0 && column < width) {
        G *out = column < cols ? dgamma + column : dbeta ? dbeta + (column - cols) : nullptr;
        if (out) {
            Piece<G, 1> w;
            w.set(&v);
            *reinterpret_cast<Piece<G, 1> *>(out) = w;
        }
    }
}

int lfail(int code, const char *fmt, ...)
{
    char msg[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(msg, sizeof msg, fmt, ap);
    va_end(ap);
    set_error_message(msg);
    return code;
}

int lcuda(cudaError_t e, const char *what)
{
    cudaGetLastError();   // reported here, and not again by the caller's next launch
    return lfail(ZERO1_ECUDA, "%s: %s", what, cudaGetErrorString(e));
}

template <typename T, int V, int TPR, int NV, int THREADS>
cudaError_t fwd(const FwdParams<T> &p, cudaStream_t st)
{
    constexpr uint64_t per = THREADS / TPR;
    return launch(zero1_layernorm_fwd_kernel<T, V, TPR, NV, THREADS>, (unsigned)((p.rows + per - 1) / per), THREADS, 0, st, p);
}

// The variants by pieces of a row: a warp while a lane holds at most 8 (32
// single entries), then a block of 256 threads.
template <typename T, int V>
cudaError_t fwd_pick(const FwdParams<T> &p, cudaStream_t st)
{
    const uint32_t n = (p.cols + V - 1) / V;
    if (n <= 32) return fwd<T, V, 32, 1, 256>(p, st);
    if (n <= 64) return fwd<T, V, 32, 2, 256>(p, st);
    if (n <= 96) return fwd<T, V, 32, 3, 256>(p, st);
    if (n <= 128) return fwd<T, V, 32, 4, 256>(p, st);
    if (n <= 256) return fwd<T, V, 32, 8, 256>(p, st);
    if constexpr (V == 1) {
        if (n <= 1024) return fwd<T, V, 32, 32, 256>(p, st);
    } else {
        if (n <= 512) return fwd<T, V, 128, 4, 256>(p, st);
        if (n <= 1024) return fwd<T, V, 256, 4, 256>(p, st);
    }
    if (n <= 2048) return fwd<T, V, 256, 8, 256>(p, st);
    if constexpr (V == 1)
        if (n <= 8192) return fwd<T, V, 512, 16, 512>(p, st);
    return cudaErrorNotSupported;
}

// Blocks of the backward pass (each leaves one partial row) where a block
// takes `at_once` rows at a time, and the most it may be for a size.
uint64_t partial_rows(uint64_t rows, uint64_t at_once)
{
    const uint64_t n = (rows + at_once - 1) / at_once;
    return n < 1 ? 1 : n < (uint64_t)kMaxPartials ? n : kMaxPartials;
}

// Launches over kRun rows a thread each, of `blocks` blocks that take
// `at_once` rows at a time.
template <typename T, typename F>
cudaError_t in_runs(const BwdParams<T> &p, int blocks, uint64_t at_once, F one)
{
    const uint64_t piece = kRun * blocks * at_once;
    cudaError_t e = cudaSuccess;
    for (uint64_t first = 0; e == cudaSuccess && (first == 0 || first < p.rows); first += piece) {
        BwdParams<T> q = p;
        q.dy += first * p.lddy;
        q.x += first * p.ldx;
        q.dx += first * p.lddx;
        q.mean += first;
        q.rstd += first;
        q.rows = p.rows - first < piece ? p.rows - first : piece;
        q.add = first > 0;
        e = one(q);
    }
    return e;
}

template <typename T, int V, int TPR, int NV, int THREADS = (TPR > 256 ? TPR : 256), bool AHEAD = true>
cudaError_t bwd(const BwdParams<T> &p, int *blocks, cudaStream_t st)
{
    const size_t fold = TPR < THREADS ? (size_t)(THREADS / TPR) * p.cols * sizeof(float) : 0;   // at most 32 KB
    const int n = (int)partial_rows(p.rows, THREADS / TPR);
    *blocks = n < *blocks ? n : *blocks;
    return in_runs(p, *blocks, THREADS / TPR, [&](const BwdParams<T> &q) {
        return launch(zero1_layernorm_bwd_kernel<T, V, TPR, NV, THREADS, AHEAD>, *blocks, THREADS, fold, st, q);
    });
}

// The variants by pieces of a row: a warp a row while its lanes hold the
// column sums (a row shared by more warps costs each of them the same
// shuffles: rows of 768 by three warps took twice the time of one), then
// blocks.  Single entries of unaligned rows: 8 a lane.
template <typename T, int V>
cudaError_t bwd_pick(const BwdParams<T> &p, int *blocks, cudaStream_t st)
{
    const uint32_t n = (p.cols + V - 1) / V;
    if (n <= 32) return bwd<T, V, 32, 1>(p, blocks, st);
    if (n <= 64) return bwd<T, V, 32, 2>(p, blocks, st);
    if (n <= 96) return bwd<T, V, 32, 3>(p, blocks, st);
    if (n <= 128) return bwd<T, V, 32, 4, 256, V < 8>(p, blocks, st);
    if constexpr (V == 1) {
        if (n <= 256) return bwd<T, V, 32, 8>(p, blocks, st);
        if (n <= 1024) return bwd<T, V, 128, 8>(p, blocks, st);
        if (n <= 2048) return bwd<T, V, 256, 8>(p, blocks, st);
        if (n <= 8192) return bwd<T, V, 512, 16, 512, false>(p, blocks, st);
        return cudaErrorNotSupported;
    } else {
        if (n <= 256) return bwd<T, V, 256, 1>(p, blocks, st);
        if (n <= 512) return bwd<T, V, 256, 2>(p, blocks, st);
        if (n <= 1024) return bwd<T, V, 512, 2>(p, blocks, st);
        if (n <= 2048) return bwd<T, V, 512, 4, 512, false>(p, blocks, st);
        return cudaErrorNotSupported;
    }
}

template <typename T, int V>
bool aligned_for(const T *p, uint64_t ld)
{
    return (reinterpret_cast<uintptr_t>(p) % 16) == 0 && ld % V == 0;
}

template <typename T, int V>
int forward(uint64_t rows, uint64_t cols, const void *x, uint64_t ldx, const void *gamma, const void *beta, double eps,
            void *y, uint64_t ldy, float *mean, float *rstd, cudaStream_t st)
{
    FwdParams<T> p{};
    p.x = static_cast<const T *>(x);
    p.gamma = static_cast<const T *>(gamma);
    p.beta = static_cast<const T *>(beta);
    p.y = static_cast<T *>(y);
    p.mean = mean;
    p.rstd = rstd;
    p.rows = rows;
    p.ldx = ldx;
    p.ldy = ldy;
    p.cols = (uint32_t)cols;
    p.eps = (float)eps;
    p.inv_n = (float)(1.0 / (double)cols);
    const bool vec = cols % V == 0 && aligned_for<T, V>(p.x, ldx) && aligned_for<T, V>(p.y, ldy) &&
                     aligned_for<T, V>(p.gamma, 0) && aligned_for<T, V>(p.beta, 0);
    cudaError_t e = vec ? fwd_pick<T, V>(p, st) : fwd_pick<T, 1>(p, st);
    if (e == cudaErrorNotSupported)   // wider than any
        e = launch(cols > kRowRun ? zero1_layernorm_fwd_wide_kernel<T, true> : zero1_layernorm_fwd_wide_kernel<T, false>,
                   (unsigned)rows, 1024, 0, st, p);
    return e == cudaSuccess ? ZERO1_OK : lcuda(e, "kernel launch");
}

template <typename T, int V>
int backward(uint64_t rows, uint64_t cols, const void *dy, uint64_t lddy, const void *x, uint64_t ldx, const void *gamma,
             const float *mean, const float *rstd, void *dx, uint64_t lddx, void *dgamma, void *dbeta, bool grad_bf16,
             float *partials, int sms, cudaStream_t st)
{
    BwdParams<T> p{};
    p.dy = static_cast<const T *>(dy);
    p.x = static_cast<const T *>(x);
    p.gamma = static_cast<const T *>(gamma);
    p.mean = mean;
    p.rstd = rstd;
    p.dx = static_cast<T *>(dx);
    p.partials = partials;
    p.rows = rows;
    p.lddy = lddy;
    p.ldx = ldx;
    p.lddx = lddx;
    p.cols = (uint32_t)cols;
    p.inv_n = (float)(1.0 / (double)cols);
    int blocks = (int)partial_rows(rows, 1);
    if (blocks > 2 * sms) blocks = 2 * sms;
    const bool vec = cols % V == 0 && aligned_for<T, V>(p.x, ldx) && aligned_for<T, V>(p.dy, lddy) &&
                     aligned_for<T, V>(p.dx, lddx) && aligned_for<T, V>(p.gamma, 0);
    cudaError_t e = vec ? bwd_pick<T, V>(p, &blocks, st) : bwd_pick<T, 1>(p, &blocks, st);
    if (e == cudaErrorNotSupported) {   // wider than any
        const dim3 grid(blocks, (unsigned)((cols + kWideTile - 1) / kWideTile));
        e = in_runs(p, blocks, 1, [&](const BwdParams<T> &q) {
            return launch(zero1_layernorm_cols_wide_kernel<T>, grid, kLnThreads, 0, st, q);
        });
        if (e == cudaSuccess && rows > 0)
            e = launch(cols > kRowRun ? zero1_layernorm_bwd_wide_kernel<T, true> : zero1_layernorm_bwd_wide_kernel<T, false>,
                       (unsigned)rows, 1024, 0, st, p);
    }
    if (e == cudaSuccess) {
        const unsigned grid = (unsigned)((2 * cols + 31) / 32);
        const float *src = partials;
        if (grad_bf16)
            e = launch_early(zero1_layernorm_cols_kernel<uint16_t>, grid, 1024, 0, st, src, blocks, p.cols,
                             static_cast<uint16_t *>(dgamma), static_cast<uint16_t *>(dbeta));
        else
            e = launch_early(zero1_layernorm_cols_kernel<float>, grid, 1024, 0, st, src, blocks, p.cols,
                             static_cast<float *>(dgamma), static_cast<float *>(dbeta));
    }
    return e == cudaSuccess ? ZERO1_OK : lcuda(e, "kernel launch");
}

bool on(const void *p, size_t bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; }

int check_sizes(uint64_t rows, uint64_t cols, int dtype)
{
    if (cols == 0 || cols > ((uint64_t)1 << 24)) return lfail(ZERO1_EINVAL, "cols must be in [1, 2^24]");
    if (rows > 0x7FFFFFFFull) return lfail(ZERO1_EINVAL, "rows must be below 2^31");
    if (dtype != ZERO1_DTYPE_BF16 && dtype != ZERO1_DTYPE_F32) return lfail(ZERO1_EINVAL, "bad dtype");
    return ZERO1_OK;
}

// Strides whose last row is past 2^50 entries name no memory (and, multiplied, could leave 64 bits).
bool stride_ok(uint64_t rows, uint64_t cols, uint64_t ld) { return ld >= cols && ld <= ((uint64_t)1 << 50) / (rows ? rows : 1); }

}  // namespace
}  // namespace zero1

extern "C" {

int zero1_layernorm_forward(uint64_t rows, uint64_t cols, int dtype, const void *x, uint64_t ldx, const void *gamma,
                            const void *beta, double eps, void *y, uint64_t ldy, float *mean, float *rstd, void *stream)
{
    using namespace zero1;
    const int rc = check_sizes(rows, cols, dtype);
    if (rc) return rc;
    if (!(eps >= 0.0 && eps < 1e30)) return lfail(ZERO1_EINVAL, "eps must be finite and >= 0");
    if (!stride_ok(rows, cols, ldx) || !stride_ok(rows, cols, ldy))
        return lfail(ZERO1_EINVAL, "row strides must be at least cols, and rows times one at most 2^50");
    if (x && x == y && ldx != ldy && rows > 1) return lfail(ZERO1_EINVAL, "y may be x with the same row stride only");
    if (rows == 0) return ZERO1_OK;
    if (!x || !gamma || !y || !mean || !rstd) return lfail(ZERO1_EINVAL, "NULL pointer argument");
    const size_t e = dtype == ZERO1_DTYPE_BF16 ? 2 : 4;
    if (!on(x, e) || !on(gamma, e) || !on(beta, e) || !on(y, e) || !on(mean, 4) || !on(rstd, 4))
        return lfail(ZERO1_EALIGN, "a buffer is not aligned to its elements");
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    return dtype == ZERO1_DTYPE_BF16 ? forward<uint16_t, 8>(rows, cols, x, ldx, gamma, beta, eps, y, ldy, mean, rstd, st)
                                     : forward<float, 4>(rows, cols, x, ldx, gamma, beta, eps, y, ldy, mean, rstd, st);
}

int zero1_layernorm_workspace(uint64_t rows, uint64_t cols, uint64_t *bytes)
{
    using namespace zero1;
    if (!bytes) return lfail(ZERO1_EINVAL, "bytes is NULL");
    const int rc = check_sizes(rows, cols, ZERO1_DTYPE_F32);
    if (rc) return rc;
    *bytes = partial_rows(rows, 1) * 2 * cols * sizeof(float);
    return ZERO1_OK;
}

int zero1_layernorm_backward(uint64_t rows, uint64_t cols, int dtype, const void *dy, uint64_t lddy, const void *x,
                             uint64_t ldx, const void *gamma, const float *mean, const float *rstd, void *dx,
                             uint64_t lddx, void *dgamma, void *dbeta, int grad_dtype, void *workspace,
                             uint64_t workspace_bytes, void *stream)
{
    using namespace zero1;
    int rc = check_sizes(rows, cols, dtype);
    if (rc) return rc;
    if (grad_dtype != ZERO1_DTYPE_BF16 && grad_dtype != ZERO1_DTYPE_F32) return lfail(ZERO1_EINVAL, "bad grad_dtype");
    if (!stride_ok(rows, cols, lddy) || !stride_ok(rows, cols, ldx) || !stride_ok(rows, cols, lddx))
        return lfail(ZERO1_EINVAL, "row strides must be at least cols, and rows times one at most 2^50");
    if (dx && dx == dy && lddx != lddy && rows > 1) return lfail(ZERO1_EINVAL, "dx may be dy with the same row stride only");
    if (!gamma || !dgamma || !workspace || (rows > 0 && (!dy || !x || !mean || !rstd || !dx)))
        return lfail(ZERO1_EINVAL, "NULL pointer argument");
    uint64_t need = 0;
    zero1_layernorm_workspace(rows, cols, &need);
    if (workspace_bytes < need)
        return lfail(ZERO1_EINVAL, "the workspace holds %llu bytes, the call needs %llu",
                     (unsigned long long)workspace_bytes, (unsigned long long)need);
    const size_t e = dtype == ZERO1_DTYPE_BF16 ? 2 : 4, g = grad_dtype == ZERO1_DTYPE_BF16 ? 2 : 4;
    if (!on(dy, e) || !on(x, e) || !on(gamma, e) || !on(dx, e) || !on(mean, 4) || !on(rstd, 4) || !on(dgamma, g) ||
        !on(dbeta, g) || !on(workspace, 16))
        return lfail(ZERO1_EALIGN, "a buffer is not aligned to its elements (workspace: 16 bytes)");
    int dev = 0, sms = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err == cudaSuccess) err = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (err != cudaSuccess) return lcuda(err, "device query");
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    float *w = static_cast<float *>(workspace);
    const bool gb = grad_dtype == ZERO1_DTYPE_BF16;
    return dtype == ZERO1_DTYPE_BF16
               ? backward<uint16_t, 8>(rows, cols, dy, lddy, x, ldx, gamma, mean, rstd, dx, lddx, dgamma, dbeta, gb, w, sms, st)
               : backward<float, 4>(rows, cols, dy, lddy, x, ldx, gamma, mean, rstd, dx, lddx, dgamma, dbeta, gb, w, sms, st);
}

}  // extern "C"
