// zero1_muon_kernels.cu -- kernels of the matrix optimizer: momentum and
// norm, the Newton-Schulz iteration on the tensor cores, and the update.
//
// The iteration (X of sides s <= l, A the s x s Gram matrix):
//     A = X X^T,  B = b A + c A A,  X <- a X + B X        (rows <= cols)
//     A = X^T X,  B = b A + c A A,  X <- a X + X B        (rows >  cols)
// Singular values far below one grow by a = 3.4 a step, 480-fold over five:
// an error that a rounding of X leaves there grows with them, and with X in
// bf16 (2^-9) the result of a matrix with a few strong directions is half
// noise.  So every operand is kept as two f16 parts, hi + lo = 22 bits, a
// product is hi*hi + hi*lo + lo*hi into one fp32 accumulator (the dropped
// lo*lo is 2^-24), and a X is added in fp32 outside the product.  The result
// is as exact as the iteration in fp32, for three tensor-core products in
// place of one.
#include "zero1_internal.h"
#include "zero1_muon.h"
#include "zero1_tc.cuh"

namespace zero1 {
namespace {

// ---------------------------------------------------------- elementwise

constexpr int kElemThreads = 256;

template <int CAP>
struct MomentumParams {
    const uint16_t *grads[CAP];
    MuonDev d;
    float *momentum;
    float inv_w, mu, omm;
    int world, nesterov;
};

template <int CAP>
struct ApplyParams {
    uint16_t *params[CAP];
    MuonDev d;
    float *master;
    float lr, decay;
    int world, region;
};

// One elementwise block: entries [begin, end) of its matrix in row order,
// visited by f(flat index, padded index) in steps of `step` entries that
// share a row.
template <typename F>
__device__ __forceinline__ void for_chunk(const MuonMat &m, uint32_t chunk, uint32_t step, F f)
{
    const uint64_t begin = (uint64_t)chunk * kChunk;
    const uint64_t size = (uint64_t)m.rows * m.cols;
    const uint32_t n = (uint32_t)min((uint64_t)kChunk, size - begin);
    const uint64_t r0 = begin / m.cols;
    const uint32_t c0 = (uint32_t)(begin - r0 * m.cols);
    for (uint32_t o = threadIdx.x * step; o < n; o += kElemThreads * step) {
        const uint32_t q = (c0 + o) / m.cols;
        const uint32_t c = c0 + o - q * m.cols;
        const uint64_t r = r0 + q;
        f(m.offset + r * m.ld + c, r * m.ldx + c);
    }
}

// A sum of squares in fp32 that moves to fp64 what would leave fp32's range.
struct SquareSum {
    float s = 0.f;
    double big = 0.0;
    __device__ __forceinline__ void add(float v)
    {
        const float q = v * v;
        if (q > 1e30f) big += (double)v * (double)v;
        else s += q;
    }
    __device__ __forceinline__ double total() const { return big + (double)s; }
};

// Sum over the block in a fixed order; valid on thread 0.
__device__ __forceinline__ double block_sum(double v)
{
    __shared__ double part[kElemThreads / 32];
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
    __syncthreads();
    double s = 0.0;
    if (threadIdx.x == 0)
        for (int i = 0; i < kElemThreads / 32; ++i) s += part[i];
    return s;
}

// Counters the iteration starts from.
__device__ __forceinline__ void reset_counters(const MuonDev &d)
{
    const uint32_t i = blockIdx.x * kElemThreads + threadIdx.x;
    if (i < d.count) d.done[i] = 0;
    if (i == 0) *d.ticket = 0;
}

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

// hi + lo = v to 22 bits.
__device__ __forceinline__ void split(float v, __half &hi, __half &lo)
{
    hi = __float2half_rn(v);
    lo = __float2half_rn(v - __half2float(hi));
}

__device__ __forceinline__ uint32_t pack(__half a, __half b)
{
    return (uint32_t)__half_as_ushort(a) | ((uint32_t)__half_as_ushort(b) << 16);
}

// Momentum and the update it gives, with the norm's partial sums:
// m = mu m + (1-mu) g for g the rank-ordered mean of the W gradients, and
// u = mu m + (1-mu) g (nesterov) or m, left as fp32 in region 1.
template <int CAP>
__global__ void __launch_bounds__(kElemThreads) muon_momentum_kernel(const __grid_constant__ MomentumParams<CAP> p)
{
    reset_counters(p.d);
    if (blockIdx.x >= p.d.nchunks) return;
    const MuonMat &m = p.d.mats[p.d.chunk_mat[blockIdx.x]];
    float *u = reinterpret_cast<float *>(m.region[1]);
    SquareSum ss;
    const auto one = [&](float sum, float &mom) {
        const float g = sum * p.inv_w;
        mom = p.mu * mom + p.omm * g;
        const float x = p.nesterov ? p.mu * mom + p.omm * g : mom;
        ss.add(x);
        return x;
    };
    if (m.vec) {
        for_chunk(m, blockIdx.x - m.chunk0, 8, [&](uint64_t f, uint64_t x) {
            float s[8], mom[8];
            load8(mom, p.momentum + f);
            load8(s, p.grads[0] + f);
#pragma unroll 8
            for (int r = 1; r < p.world; ++r) {
                float g[8];
                load8(g, p.grads[r] + f);
#pragma unroll
                for (int k = 0; k < 8; ++k) s[k] += g[k];
            }
#pragma unroll
            for (int k = 0; k < 8; ++k) s[k] = one(s[k], mom[k]);
            store8(p.momentum + f, mom);
            store8(u + x, s);
        });
    } else {
        for_chunk(m, blockIdx.x - m.chunk0, 1, [&](uint64_t f, uint64_t x) {
            float s = load1(p.grads[0] + f), mom = p.momentum[f];
            for (int r = 1; r < p.world; ++r) s += load1(p.grads[r] + f);
            u[x] = one(s, mom);
            p.momentum[f] = mom;
        });
    }
    const double sum = block_sum(ss.total());
    if (threadIdx.x == 0) p.d.partials[blockIdx.x] = sum;
}

// The norm's partial sums of a matrix given as it is.
template <typename T>
__global__ void __launch_bounds__(kElemThreads) muon_norm_kernel(MuonDev d, const T *in)
{
    reset_counters(d);
    if (blockIdx.x >= d.nchunks) return;
    const MuonMat &m = d.mats[d.chunk_mat[blockIdx.x]];
    SquareSum ss;
    if (m.vec) {
        for_chunk(m, blockIdx.x - m.chunk0, 8, [&](uint64_t f, uint64_t) {
            float v[8];
            load8(v, in + f);
#pragma unroll
            for (int k = 0; k < 8; ++k) ss.add(v[k]);
        });
    } else {
        for_chunk(m, blockIdx.x - m.chunk0, 1, [&](uint64_t f, uint64_t) {
            ss.add(load1(in + f));
        });
    }
    const double sum = block_sum(ss.total());
    if (threadIdx.x == 0) d.partials[blockIdx.x] = sum;
}

// X = U / (|U| + eps), as two f16 planes in region 0.
template <typename T>
__global__ void __launch_bounds__(kElemThreads) muon_split_kernel(MuonDev d, const T *in, float eps)
{
    const MuonMat &m = d.mats[d.chunk_mat[blockIdx.x]];
    __shared__ float factor;
    // the blocks' sums in a fixed order
    __shared__ double part[kElemThreads];
    double t = 0.0;
    for (uint32_t i = threadIdx.x; i < m.chunks; i += kElemThreads) t += d.partials[m.chunk0 + i];
    part[threadIdx.x] = t;
    __syncthreads();
    for (int o = kElemThreads / 2; o > 0; o >>= 1) {
        if (threadIdx.x < o) part[threadIdx.x] += part[threadIdx.x + o];
        __syncthreads();
    }
    if (threadIdx.x == 0) factor = (float)((double)kNsScale / (sqrt(part[0]) + (double)eps));
    __syncthreads();
    const float k = factor;
    __half *hi = reinterpret_cast<__half *>(m.region[0]), *lo = hi + m.xplane;
    const T *src = in ? in : reinterpret_cast<const T *>(m.region[1]);
    if (m.vec) {
        for_chunk(m, blockIdx.x - m.chunk0, 8, [&](uint64_t f, uint64_t x) {
            float v[8];
            __half h[8], l[8];
            load8(v, src + (in ? f : x));
#pragma unroll
            for (int i = 0; i < 8; ++i) split(v[i] * k, h[i], l[i]);
            *reinterpret_cast<uint4 *>(hi + x) = make_uint4(pack(h[0], h[1]), pack(h[2], h[3]), pack(h[4], h[5]), pack(h[6], h[7]));
            *reinterpret_cast<uint4 *>(lo + x) = make_uint4(pack(l[0], l[1]), pack(l[2], l[3]), pack(l[4], l[5]), pack(l[6], l[7]));
        });
    } else {
        for_chunk(m, blockIdx.x - m.chunk0, 1, [&](uint64_t f, uint64_t x) {
            __half h, l;
            split(load1(src + (in ? f : x)) * k, h, l);
            hi[x] = h;
            lo[x] = l;
        });
    }
}

// p = p (1 - lr wd) - lr scale X, and bf16(p) into the W replicas.
template <int CAP>
__global__ void __launch_bounds__(kElemThreads) muon_apply_kernel(const __grid_constant__ ApplyParams<CAP> p)
{
    const MuonMat &m = p.d.mats[p.d.chunk_mat[blockIdx.x]];
    const float *x = reinterpret_cast<const float *>(m.region[p.region]);
    const float step = p.lr * m.scale;
    if (m.vec) {
        for_chunk(m, blockIdx.x - m.chunk0, 8, [&](uint64_t f, uint64_t i) {
            float o[8], w[8];
            load8(o, x + i);
            load8(w, p.master + f);
#pragma unroll
            for (int k = 0; k < 8; ++k) w[k] = w[k] * p.decay - step * o[k];
            store8(p.master + f, w);
            for (int r = 0; r < p.world; ++r) store8(p.params[r] + f, w);
        });
    } else {
        for_chunk(m, blockIdx.x - m.chunk0, 1, [&](uint64_t f, uint64_t i) {
            const float w = p.master[f] * p.decay - step * x[i];
            p.master[f] = w;
            for (int r = 0; r < p.world; ++r) store1(p.params[r] + f, w);
        });
    }
}

template <typename T>
__global__ void __launch_bounds__(kElemThreads) muon_out_kernel(MuonDev d, T *out, int region)
{
    const MuonMat &m = d.mats[d.chunk_mat[blockIdx.x]];
    const float *x = reinterpret_cast<const float *>(m.region[region]);
    if (m.vec) {
        for_chunk(m, blockIdx.x - m.chunk0, 8, [&](uint64_t f, uint64_t i) {
            float v[8];
            load8(v, x + i);
            store8(out + f, v);
        });
    } else {
        for_chunk(m, blockIdx.x - m.chunk0, 1, [&](uint64_t f, uint64_t i) { store1(out + f, x[i]); });
    }
}

// ---------------------------------------------------------- the iteration

// Shared memory of one block: three stages of one K step (64) of its 128
// rows of A and its 64 rows of B, high and low parts, and for each of the
// two column halves of a tile 32 KB through which it enters and leaves.
constexpr int kStages = 3;
constexpr uint32_t kBox = 8192;                        // 64 x 64 f16
constexpr uint32_t kStageBytes = 6 * kBox;             // A hi, A lo (two boxes each), B hi, B lo
constexpr uint32_t kHalfBytes = 4 * kBox;              // 128 rows x 64 columns, hi and lo (or fp32)
constexpr int kSlots = 4;                              // tiles in flight between the roles
constexpr int kNsThreads = 384;                        // loads, products, 2 x stores, 2 x 4 epilogue warps
constexpr uint32_t kTmemCols = 512;                    // two accumulators of hi*hi, two of hi*lo + lo*hi
// K of one accumulator.  The tensor cores cut every addition of 16 products
// off below the sum's last place, so a sum of positive terms falls short by
// 8e-8 of itself for each (measured: 4e-6 over K = 1024, 9e-5 over 16384).
// Longer sums are gathered 256 at a time and added up in rounded fp32.
constexpr uint32_t kAccK = 256;
constexpr int kNsSmem = kStages * kStageBytes + 2 * kHalfBytes + 1024;

struct NsParams {
    MuonDev d;
    float a, b, c;
    uint32_t total;
    int steps;
};

// In the last iterations A is near the identity, and the sums A A and B X
// are large terms that nearly cancel a X: their errors count several times.
// There the polynomial is taken about A = alpha I, an identity for any
// alpha: with A' = A - alpha I,
//   a + b A + c A A = (a + b alpha + c alpha^2) + ((b + 2 c alpha) A' + c A' A'),
// whose products are small.  The iterations before keep alpha = 0, since
// directions still far below one would gain the error of a term that their
// B X does not have.
constexpr float kAlpha = 0.85f;
__device__ __forceinline__ float alpha_of(uint32_t iter, int steps) { return (int)iter + 2 >= steps ? kAlpha : 0.f; }

struct Tile {
    uint32_t mat, phase, iter, ti, tj;
};
constexpr uint32_t kNoMore = 3;                        // phase of the tile that ends the work

struct NsShared {
    uint4 slot[kSlots];
    uint64_t full[kStages], empty[kStages];            // operand ring
    uint64_t slot_full[kSlots], slot_empty[kSlots];    // tile ring
    uint64_t acc_full[2], acc_empty[2];                // accumulators
    uint64_t half_full[2], half_done[2];               // a half's memory: free, with the tile's term; written
    uint64_t drain;
    uint32_t tmem;
    int abort;
};

__device__ __forceinline__ uint4 pack_tile(const Tile &t) { return make_uint4(t.mat, t.phase | t.iter << 2, t.ti, t.tj); }
__device__ __forceinline__ Tile unpack_tile(uint4 v) { return Tile{v.x, v.y & 3u, v.y >> 2, v.z, v.w}; }

// The operands of a tile's product.  A Gram-sized matrix (A or B) is stored
// from its 256-row tiles' diagonal on; what lies below is read transposed
// from above, as an MN-major operand.
struct Product {
    const CUtensorMap *a, *b;
    uint32_t k;
    uint32_t a_turn, b_turn;   // K below which the operand is MN-major in memory

    __device__ __forceinline__ Product(const MuonDev &d, const Tile &t)
    {
        const MuonMat &m = d.mats[t.mat];
        const CUtensorMap *maps = d.maps + (uint64_t)t.mat * kMapsPerMat;
        const CUtensorMap *x = maps + (t.iter & 1 ? kMapX1 : kMapX0);
        constexpr uint32_t kAlways = 0xFFFFFFFFu;
        const uint32_t row_turn = t.ti * kNsTileM, col_turn = (t.tj >> 1) * kNsTileM;
        if (t.phase == 0) {          // X X^T, or X^T X
            a = b = x;
            k = m.tall ? m.rows : m.cols;
            a_turn = b_turn = m.tall ? kAlways : 0;
        } else if (t.phase == 1) {   // A A
            a = b = maps + kMapA;
            k = m.s;
            a_turn = row_turn;
            b_turn = col_turn;
        } else if (!m.tall) {        // B X
            a = maps + kMapB;
            b = x;
            k = m.s;
            a_turn = row_turn;
            b_turn = kAlways;
        } else {                     // X B
            a = x;
            b = maps + kMapB;
            k = m.s;
            a_turn = 0;
            b_turn = col_turn;
        }
    }
};

// Wait until `need` arrivals of the matrix have been made (bounded like the
// pipeline waits; gives up at once when any block of the grid has).
__device__ __forceinline__ bool wait_parts(const unsigned *done, unsigned need, volatile int *abort, unsigned *errors)
{
    const unsigned long long t0 = ptx::global_ns();
    for (uint32_t i = 1;; ++i) {
        if (tc::ld_acquire(done) >= need) return true;
        if ((i & 15u) == 0) {
            if (*abort) return false;
            if (*reinterpret_cast<volatile unsigned *>(errors) & kErrWaitTimeout) {
                *abort = 1;
                return false;
            }
            if (ptx::global_ns() - t0 > ptx::kWaitLimitNs) {
                *abort = 1;
                atomicOr(errors, kErrWaitTimeout);
                return false;
            }
        }
    }
}

// w[2i], w[2i+1] += k * (hi + lo) of eight entries.
__device__ __forceinline__ void add8(float *w, float k, uint4 hi, uint4 lo)
{
    const uint32_t x[4] = {hi.x, hi.y, hi.z, hi.w}, y[4] = {lo.x, lo.y, lo.z, lo.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 h = __half22float2(*reinterpret_cast<const __half2 *>(&x[i]));
        const float2 l = __half22float2(*reinterpret_cast<const __half2 *>(&y[i]));
        w[2 * i] += k * (h.x + l.x);
        w[2 * i + 1] += k * (h.y + l.y);
    }
}

// The whole iteration over all matrices in one launch, by pairs of blocks.
// Pairs draw tiles in an order in which every tile comes after those it
// depends on (all of the previous product of its matrix), so a pair that
// waits for a matrix's counter waits only for tiles that running pairs hold:
// none needs another to be resident, and the grid may be of any size.
// Within a pair, one thread of each block loads its operands (TMA), one
// thread of the first block issues the products, and in each block 2 x 4
// warps take its 128 x 128 half of the tile out of one accumulator while the
// other fills, 64 columns each four: through shared memory, into which a
// store thread loaded the term to be added (b A or a X) meanwhile and from
// which it stores the result and counts the tile as finished.
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kNsThreads, 1)
    muon_iterate_kernel(const __grid_constant__ NsParams p)
{
    extern __shared__ unsigned char raw[];
    __shared__ NsShared sh;
    const uint32_t ring = (tc::smem_u32(raw) + 1023u) & ~1023u;
    const uint32_t halves = ring + kStages * kStageBytes;
    const int warp = threadIdx.x >> 5;
    const uint32_t rank = tc::cluster_rank();
    unsigned *errors = p.d.errors;
    volatile int *abort = &sh.abort;

    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) ptx::mbar_init(&sh.full[i], 1), ptx::mbar_init(&sh.empty[i], 1);
        // a slot is read by the second block's loader, the first's products and, in both, 2 store and 8 epilogue warps
        for (int i = 0; i < kSlots; ++i) ptx::mbar_init(&sh.slot_full[i], 1), ptx::mbar_init(&sh.slot_empty[i], 22);
        for (int i = 0; i < 2; ++i) ptx::mbar_init(&sh.acc_full[i], 1), ptx::mbar_init(&sh.acc_empty[i], 16);
        for (int i = 0; i < 2; ++i) ptx::mbar_init(&sh.half_full[i], 1), ptx::mbar_init(&sh.half_done[i], 4);
        ptx::mbar_init(&sh.drain, 1);
        sh.abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) {
        __syncwarp();
        tc::tmem_alloc(&sh.tmem, kTmemCols);
    }
    tc::fence_before_sync();
    __syncthreads();
    ptx::cluster_sync();
    tc::fence_after_sync();
    const uint32_t tmem = sh.tmem;

    if (threadIdx.x == 0) {
        // ---- tiles (first block) and loads
        uint32_t issued = 0;
        for (uint32_t n = 0;; ++n) {
            const int slot = n % kSlots;
            Tile t{};
            if (rank == 0) {
                if (n >= kSlots && !tc::pair_wait(&sh.slot_empty[slot], (n / kSlots - 1) & 1u, abort, errors)) break;
                const uint32_t ticket = atomicAdd(p.d.ticket, 1u);
                t.phase = kNoMore;
                if (ticket < p.total) {
                    t.iter = ticket / p.d.work_per_iter;
                    const uint2 w = p.d.work[ticket - t.iter * p.d.work_per_iter];
                    t.mat = w.x & 0x3FFFFFFFu;
                    t.phase = w.x >> 30;
                    t.ti = w.y & 0xFFFFu;
                    t.tj = w.y >> 16;
                    const MuonMat &m = p.d.mats[t.mat];
                    uint32_t need = t.iter * (m.parts[0] + m.parts[1] + m.parts[2]);
                    if (t.phase > 0) need += m.parts[0];
                    if (t.phase > 1) need += m.parts[1];
                    if (!wait_parts(&p.d.done[t.mat], need, abort, errors)) break;
                }
                const uint4 v = pack_tile(t);
                sh.slot[slot] = v;
                tc::st_cluster(tc::map_to(tc::smem_u32(&sh.slot[slot]), 1), v);
                tc::arrive_cluster(tc::map_to(tc::smem_u32(&sh.slot_full[slot]), 1));
                tc::arrive_cluster(tc::map_to(tc::smem_u32(&sh.slot_full[slot]), 0));
            } else {
                if (!tc::pair_wait(&sh.slot_full[slot], (n / kSlots) & 1u, abort, errors)) break;
                t = unpack_tile(sh.slot[slot]);
                tc::arrive_cluster(tc::map_to(tc::smem_u32(&sh.slot_empty[slot]), 0));
            }
            if (t.phase == kNoMore) break;
            tc::fence_proxy_async_all();   // other blocks' results, before the loads below
            const Product w(p.d, t);
            const int row = (int)(t.ti * kNsTileM + rank * 128), col = (int)(t.tj * kNsTileN + rank * 64);
            bool ok = true;
            for (uint32_t k0 = 0; k0 < w.k; k0 += kNsTileK) {
                const uint32_t stage = issued % kStages;
                if (issued >= kStages) ok = tc::pair_wait(&sh.empty[stage], (issued / kStages - 1) & 1u, abort, errors);
                if (!ok) break;
                if (rank == 0) ptx::mbar_arrive_expect_tx(&sh.full[stage], 2 * kStageBytes);
                const uint32_t bar = tc::map_to(tc::smem_u32(&sh.full[stage]), 0);
                const uint32_t dst = ring + stage * kStageBytes;
                const bool a_mn = k0 < w.a_turn, b_mn = k0 < w.b_turn;
                const int k = (int)k0;
#pragma unroll
                for (int plane = 0; plane < 2; ++plane) {
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        tc::tma_box_pair(dst + (2 * plane + h) * kBox, w.a, a_mn ? row + 64 * h : k,
                                         a_mn ? k : row + 64 * h, plane, bar);
                    tc::tma_box_pair(dst + (4 + plane) * kBox, w.b, b_mn ? col : k, b_mn ? k : col, plane, bar);
                }
                ++issued;
            }
            if (!ok) break;
        }
        if (*abort && rank == 0) ptx::drain_loads<kStages>(sh.full, issued);
    } else if (threadIdx.x == 32 && rank == 0) {
        // ---- products
        uint32_t taken = 0, used = 0;   // stages, accumulators
        bool ok = true;
        for (uint32_t n = 0; ok; ++n) {
            const int slot = n % kSlots;
            if (!(ok = tc::pair_wait(&sh.slot_full[slot], (n / kSlots) & 1u, abort, errors))) break;
            const Tile t = unpack_tile(sh.slot[slot]);
            tc::arrive_cluster(tc::map_to(tc::smem_u32(&sh.slot_empty[slot]), 0));
            if (t.phase == kNoMore) break;
            const Product w(p.d, t);
            for (uint32_t k0 = 0; k0 < w.k; k0 += kNsTileK) {
                const uint32_t acc = used & 1u, d = tmem + acc * kNsTileN, e = tmem + (2 + (n & 1u)) * kNsTileN;
                const bool first = k0 % kAccK == 0;
                if (first && used >= 2) {
                    if (!(ok = tc::pair_wait(&sh.acc_empty[acc], (used / 2 - 1) & 1u, abort, errors))) break;
                    tc::fence_after_sync();
                }
                const uint32_t stage = taken % kStages;
                if (!(ok = tc::pair_wait(&sh.full[stage], (taken / kStages) & 1u, abort, errors))) break;
                tc::fence_after_sync();
                const bool a_mn = k0 < w.a_turn, b_mn = k0 < w.b_turn;
                const uint32_t idesc = tc::instr_desc(kNsTileM, kNsTileN, a_mn, b_mn);
                const uint64_t astep = tc::k16_step(a_mn), bstep = tc::k16_step(b_mn);
                const uint32_t src = ring + stage * kStageBytes;
                const uint64_t ah = tc::smem_desc(src, a_mn), al = tc::smem_desc(src + 2 * kBox, a_mn);
                const uint64_t bh = tc::smem_desc(src + 4 * kBox, b_mn), bl = tc::smem_desc(src + 5 * kBox, b_mn);
                // hi*hi and the two small products gather apart, which leaves a third as many additions to
                // the large sum
#pragma unroll
                for (int j = 0; j < kNsTileK / 16; ++j) {
                    tc::mma_f16(d, ah + j * astep, bh + j * bstep, idesc, !first || j > 0);
                    tc::mma_f16(e, ah + j * astep, bl + j * bstep, idesc, k0 + j > 0);
                    tc::mma_f16(e, al + j * astep, bh + j * bstep, idesc, true);
                }
                tc::mma_commit(&sh.empty[stage]);
                ++taken;
                if (k0 + kNsTileK >= w.k || (k0 + kNsTileK) % kAccK == 0) {
                    tc::mma_commit(&sh.acc_full[acc]);
                    ++used;
                }
            }
        }
        if (!ok) {   // let the products in flight end before the operands and TMEM go
            tc::mma_commit(&sh.drain);
            const unsigned long long t0 = ptx::global_ns();
            while (!ptx::mbar_test(&sh.drain, 0) && ptx::global_ns() - t0 < ptx::kWaitLimitNs) {
            }
        }
    } else if ((warp == 2 || warp == 3) && (threadIdx.x & 31) == 0) {
        // ---- a column half's memory: the term to be added in, the result out
        const int half = warp - 2;
        const uint32_t mem = halves + half * kHalfBytes;
        for (uint32_t n = 0;; ++n) {
            const int slot = n % kSlots;
            if (!tc::pair_wait(&sh.slot_full[slot], (n / kSlots) & 1u, abort, errors)) break;
            const Tile t = unpack_tile(sh.slot[slot]);
            tc::arrive_cluster(tc::map_to(tc::smem_u32(&sh.slot_empty[slot]), 0));
            if (t.phase == kNoMore) break;
            const MuonMat &m = p.d.mats[t.mat];
            const CUtensorMap *maps = p.d.maps + (uint64_t)t.mat * kMapsPerMat;
            const int row = (int)(t.ti * kNsTileM + rank * 128), col = (int)(t.tj * kNsTileN + half * 64);
            if (t.phase > 0) {
                const CUtensorMap *add = t.phase == 1 ? maps + kMapA : maps + (t.iter & 1 ? kMapX1 : kMapX0);
                tc::fence_proxy_async_all();
                ptx::mbar_arrive_expect_tx(&sh.half_full[half], kHalfBytes);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    tc::tma_box(mem + i * kBox, add, col, row + 64 * (i & 1), i >> 1, &sh.half_full[half]);
            } else {
                ptx::mbar_arrive(&sh.half_full[half]);
            }
            if (!tc::pair_wait(&sh.half_done[half], n & 1u, abort, errors)) break;
            const bool last = t.phase == 2 && (int)t.iter + 1 == p.steps;
            const int rows = (int)(t.phase < 2 ? m.s : m.rows), cols = (int)(t.phase < 2 ? m.s : m.cols);
            const CUtensorMap *out = maps + (t.phase == 0 ? kMapA : t.phase == 1 ? kMapB : last ? kMapOut
                                             : t.iter & 1 ? kMapX0 : kMapX1);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int y = row + 64 * (i & 1), x = last ? col + 32 * (i >> 1) : col;
                if (y < rows && x < cols) tc::tma_store_box(out, x, y, last ? 0 : i >> 1, mem + i * kBox);
            }
            ptx::tma_commit();
            ptx::tma_wait_all();
            tc::fence_proxy_async_all();
            tc::red_release_add(&p.d.done[t.mat], 1u);
        }
    } else if (warp >= 4) {
        // ---- finished tiles: this block's 128 rows, 64 columns to each half
        const int half = (warp - 4) >> 2;
        const uint32_t r = (uint32_t)(warp & 3) * 32 + (threadIdx.x & 31);
        const uint32_t line = halves + half * kHalfBytes + r * 128, turn = r & 7;   // this thread's row, its swizzle
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;
        const bool leader = (threadIdx.x & 31) == 0;
        uint32_t used = 0;   // accumulators
        for (uint32_t n = 0;; ++n) {
            const int slot = n % kSlots;
            if (!__all_sync(~0u, tc::pair_wait(&sh.slot_full[slot], (n / kSlots) & 1u, abort, errors))) break;
            const Tile t = unpack_tile(sh.slot[slot]);
            __syncwarp();
            if (leader) tc::arrive_cluster(tc::map_to(tc::smem_u32(&sh.slot_empty[slot]), 0));
            if (t.phase == kNoMore) break;
            const MuonMat &m = p.d.mats[t.mat];
            const uint32_t sums = ((t.phase == 0 ? (m.tall ? m.rows : m.cols) : m.s) + kAccK - 1) / kAccK;
            float w[64];
            bool ok = true;
            for (uint32_t i = 0; i < sums; ++i, ++used) {
                const uint32_t acc = used & 1u;
                ok = __all_sync(~0u, tc::pair_wait(&sh.acc_full[acc], (used / 2) & 1u, abort, errors));
                if (!ok) break;
                tc::fence_after_sync();
const uint32_t at = tmem + lanes + half * 64;
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    float x[16];
                    tc::tmem_load16(x, at + acc * kNsTileN + q * 16);
#pragma unroll
                    for (int j = 0; j < 16; ++j) w[16 * q + j] = i == 0 ? x[j] : w[16 * q + j] + x[j];
                }
                if (i + 1 == sums) {
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        float x[16];
                        tc::tmem_load16(x, at + (2 + (n & 1u)) * kNsTileN + q * 16);
#pragma unroll
                        for (int j = 0; j < 16; ++j) w[16 * q + j] += x[j];
                    }
                }
                tc::fence_before_sync();
                __syncwarp();
                if (leader) tc::arrive_cluster(tc::map_to(tc::smem_u32(&sh.acc_empty[acc]), 0));
            }
            if (!ok || !__all_sync(~0u, tc::pair_wait(&sh.half_full[half], n & 1u, abort, errors))) break;
            constexpr float inv = 1.0f / kNsScale;
            const float alpha = alpha_of(t.iter, p.steps);
            const float f = t.phase == 1 ? p.c * inv : inv;
            const float k = t.phase == 1 ? p.b + 2.f * p.c * alpha : p.a + alpha * (p.b + alpha * p.c);
#pragma unroll
            for (int q = 0; q < 64; ++q) w[q] *= f;
            if (t.phase > 0) {
#pragma unroll
                for (int q = 0; q < 8; ++q) {
                    const uint32_t piece = (q ^ turn) * 16;
                    add8(w + 8 * q, k, tc::ld_shared(line + piece), tc::ld_shared(line + 2 * kBox + piece));
                }
            } else if (alpha != 0.f) {   // A' = A - alpha I
                const uint32_t diagonal = t.ti * kNsTileM + rank * 128 + r - (t.tj * kNsTileN + half * 64);
#pragma unroll
                for (uint32_t q = 0; q < 64; ++q)
                    if (q == diagonal) w[q] -= alpha * kNsScale;
            }
            const bool last = t.phase == 2 && (int)t.iter + 1 == p.steps;
            if (!last) {
#pragma unroll
                for (int q = 0; q < 8; ++q) {
                    __half h[8], l[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) split(w[8 * q + i], h[i], l[i]);
                    const uint32_t piece = (q ^ turn) * 16;
                    tc::st_shared(line + piece, make_uint4(pack(h[0], h[1]), pack(h[2], h[3]), pack(h[4], h[5]), pack(h[6], h[7])));
                    tc::st_shared(line + 2 * kBox + piece,
                                  make_uint4(pack(l[0], l[1]), pack(l[2], l[3]), pack(l[4], l[5]), pack(l[6], l[7])));
                }
            } else {   // the result, fp32 and unscaled: 32 columns where the high parts were, 32 where the low parts were
#pragma unroll
                for (int q = 0; q < 16; ++q) {
                    const float *v = w + 4 * q;
                    tc::st_shared(line + (q >> 3) * 2 * kBox + ((q & 7) ^ turn) * 16,
                                  make_uint4(__float_as_uint(v[0] * inv), __float_as_uint(v[1] * inv),
                                             __float_as_uint(v[2] * inv), __float_as_uint(v[3] * inv)));
                }
            }
            ptx::fence_proxy_async_smem();
            __syncwarp();
            if (leader) ptx::mbar_arrive(&sh.half_done[half]);
        }
    }
    if (*abort) {   // give copies that nothing above waits for (the second block's loads, a half's term) 1 ms to land
        const unsigned long long t0 = ptx::global_ns();
        while (ptx::global_ns() - t0 < 1000000ull) {
        }
    }
    // Neither block leaves, nor gives up its tensor memory, while the other
    // may still reach into it.
    __syncwarp();
    tc::fence_before_sync();
    __syncthreads();
    ptx::cluster_sync();
    tc::fence_after_sync();
    if (warp == 1) tc::tmem_free(tmem, kTmemCols);
}

template <int CAP>
cudaError_t momentum_t(const MuonDev &d, const MuonScalars &sc, const void *const *grads, int world, float *momentum,
                       uint32_t grid, cudaStream_t stream)
{
    MomentumParams<CAP> p{};
    for (int r = 0; r < world; ++r) p.grads[r] = static_cast<const uint16_t *>(grads[r]);
    p.d = d;
    p.momentum = momentum;
    p.inv_w = sc.inv_w;
    p.mu = sc.momentum;
    p.omm = sc.one_minus_momentum;
    p.world = world;
    p.nesterov = sc.nesterov;
    muon_momentum_kernel<CAP><<<grid, kElemThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

template <int CAP>
cudaError_t apply_t(const MuonDev &d, const MuonScalars &sc, void *const *params, int world, float *master,
                    cudaStream_t stream)
{
    ApplyParams<CAP> p{};
    for (int r = 0; r < world; ++r) p.params[r] = static_cast<uint16_t *>(params[r]);
    p.d = d;
    p.master = master;
    p.lr = sc.lr;
    p.decay = sc.decay;
    p.world = world;
    p.region = sc.steps & 1;
    muon_apply_kernel<CAP><<<d.nchunks, kElemThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

// The first kernel of a call also clears one counter a matrix.
uint32_t first_grid(const MuonDev &d)
{
    const uint32_t need = (d.count + kElemThreads - 1) / kElemThreads;
    return d.nchunks > need ? d.nchunks : need;
}

}  // namespace

cudaError_t launch_muon_momentum(const MuonDev &d, const MuonScalars &sc, const void *const *grads, int world,
                                 float *momentum, cudaStream_t stream)
{
    const uint32_t grid = first_grid(d);
    if (world <= 8) return momentum_t<8>(d, sc, grads, world, momentum, grid, stream);
    if (world <= 64) return momentum_t<64>(d, sc, grads, world, momentum, grid, stream);
    return momentum_t<512>(d, sc, grads, world, momentum, grid, stream);
}

cudaError_t launch_muon_norm(const MuonDev &d, const void *in, bool bf16, cudaStream_t stream)
{
    if (bf16)
        muon_norm_kernel<<<first_grid(d), kElemThreads, 0, stream>>>(d, static_cast<const uint16_t *>(in));
    else
        muon_norm_kernel<<<first_grid(d), kElemThreads, 0, stream>>>(d, static_cast<const float *>(in));
    return cudaGetLastError();
}

cudaError_t launch_muon_split(const MuonDev &d, const MuonScalars &sc, const void *in, bool bf16, cudaStream_t stream)
{
    if (in && bf16)
        muon_split_kernel<<<d.nchunks, kElemThreads, 0, stream>>>(d, static_cast<const uint16_t *>(in), sc.eps);
    else
        muon_split_kernel<<<d.nchunks, kElemThreads, 0, stream>>>(d, static_cast<const float *>(in), sc.eps);
    return cudaGetLastError();
}

cudaError_t launch_muon_iterate(const MuonDev &d, const MuonScalars &sc, int num_sms, cudaStream_t stream)
{
    const cudaError_t e = allow_dynamic_smem(reinterpret_cast<const void *>(muon_iterate_kernel), kNsSmem);
    if (e != cudaSuccess) return e;
    NsParams p{};
    p.d = d;
    p.a = sc.a;
    p.b = sc.b;
    p.c = sc.c;
    p.steps = sc.steps;
    p.total = d.work_per_iter * (uint32_t)sc.steps;
    const uint32_t pairs = (uint32_t)num_sms / 2;
    const uint32_t grid = 2 * (p.total < pairs ? p.total : pairs);
    muon_iterate_kernel<<<grid, kNsThreads, kNsSmem, stream>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_muon_apply(const MuonDev &d, const MuonScalars &sc, void *const *params, int world, float *master,
                              cudaStream_t stream)
{
    if (world <= 8) return apply_t<8>(d, sc, params, world, master, stream);
    if (world <= 64) return apply_t<64>(d, sc, params, world, master, stream);
    return apply_t<512>(d, sc, params, world, master, stream);
}

cudaError_t launch_muon_out(const MuonDev &d, const MuonScalars &sc, void *out, bool bf16, cudaStream_t stream)
{
    if (bf16)
        muon_out_kernel<<<d.nchunks, kElemThreads, 0, stream>>>(d, static_cast<uint16_t *>(out), sc.steps & 1);
    else
        muon_out_kernel<<<d.nchunks, kElemThreads, 0, stream>>>(d, static_cast<float *>(out), sc.steps & 1);
    return cudaGetLastError();
}

}  // namespace zero1
