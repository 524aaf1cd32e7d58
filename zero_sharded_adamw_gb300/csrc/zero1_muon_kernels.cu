// zero1_muon_kernels.cu -- kernels of the matrix optimizer: momentum and
// norm, the Newton-Schulz iteration on the tensor cores, and the update.
//
// The iteration (X of sides s <= l, A the s x s Gram matrix, P the matrix
// that X is multiplied by):
//     A = X X^T,  P = a I + b A + c A A,  X <- P X        (rows <= cols)
//     A = X^T X,  P = a I + b A + c A A,  X <- X P        (rows >  cols)
// Singular values far below one grow by a = 3.4 a step, 480-fold over five:
// an error that a rounding of X leaves there grows with them, and with X in
// bf16 (2^-9) the result of a matrix with a few strong directions is half
// noise.  So every operand is kept as two f16 parts, hi + lo = 22 bits (fewer
// for entries far below the others, zero1_muon.h), and a product is hi*hi +
// hi*lo + lo*hi into one fp32 accumulator (the dropped lo*lo is 2^-24), for
// three tensor-core products in place of one.  Against 64 bits, by the
// matrix's norm, the result is off by 1.7e-6 at 768 x 768 (the iteration in
// plain fp32 by 2.5e-6), 4.4e-6 (7.2e-6) at 4096 x 16384, 2.9e-6 (2.5e-6) at
// 1031 x 257 and 1.4e-6 (1.0e-6) at 64 x 64; 0.28 to 2.6 times plain fp32's
// error over some 120 matrices, most where a side is at most 130 and few
// directions are strong or few entries not zero.  Half the rows of 768 x 2304,
// 1e-6 of the others in size, come out 1e-3 of themselves off (plain fp32:
// 5e-7).
//
// Bound by the tensor cores where tiles are many: five steps of 4096 x 4096
// take 2.41 to 2.49 ms, 1.74 PFLOP/s over the three products (tensor pipe 78%
// active, DRAM 10%), of 4096 x 16384 7.1 to 7.3 ms alone, 1.9 PFLOP/s, and
// 7.9 ms back to back, where the power limit holds the SMs at 1.4 to 1.6 GHz;
// all 48 matrices of the GPT-2-small blocks 2.2 to 2.3 ms, 1.6 PFLOP/s.  Bound
// by latency where they are few: three 768 x 768 take 0.23 ms, 15.5 us for
// each of fifteen products one after another, of which 8 us are products.
#include "zero1_internal.h"
#include "zero1_launch.h"
#include "zero1_muon.h"
#include "zero1_muon_device.cuh"
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
    int world;
    MuonScalars sc;
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
__device__ __forceinline__ void for_chunk(const MuonMat &m, uint32_t chunk, uint32_t size_of, uint32_t step, F f)
{
    const uint64_t begin = (uint64_t)chunk * size_of;
    const uint64_t size = (uint64_t)m.rows * m.cols;
    const uint32_t n = (uint32_t)min((uint64_t)size_of, size - begin);
    const uint64_t r0 = begin / m.cols;
    const uint32_t c0 = (uint32_t)(begin - r0 * m.cols);
    for (uint32_t o = threadIdx.x * step; o < n; o += kElemThreads * step) {
        const uint32_t q = (c0 + o) / m.cols;
        const uint32_t c = c0 + o - q * m.cols;
        const uint64_t r = r0 + q;
        f(m.offset + r * m.ld + c, r * m.ldx + c);
    }
}

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

// Bound by HBM: 2W + 12 bytes an entry (the update is read again by the split
// below).  85 million entries, W = 8: 420 us, 5.7 TB/s.
//
// Momentum and the update it gives, with the norm's partial sums:
// m = mu m + (1-mu) g for g the rank-ordered mean of the W gradients, and
// u = mu m + (1-mu) g (nesterov) or m, left as fp32 in region 1.
template <int CAP>
__global__ void __launch_bounds__(kElemThreads) muon_momentum_kernel(const __grid_constant__ MomentumParams<CAP> p)
{
    ptx::launch_dependents();
    reset_counters(p.d);
    if (blockIdx.x >= p.d.nchunks) return;
    const MuonMat &m = p.d.mats[p.d.chunk_mat[blockIdx.x]];
    float *u = reinterpret_cast<float *>(m.region[1]);
    SquareSum ss;
    if (m.vec) {
        for_chunk(m, blockIdx.x - m.chunk0, p.d.chunk, 8, [&](uint64_t f, uint64_t x) {
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
            for (int k = 0; k < 8; ++k) s[k] = look_ahead(p.sc, s[k], mom[k]);
            ss.add(s);
            store8(p.momentum + f, mom);
            store8(u + x, s);
        });
    } else {
        for_chunk(m, blockIdx.x - m.chunk0, p.d.chunk, 1, [&](uint64_t f, uint64_t x) {
            float s[1] = {load1(p.grads[0] + f)}, mom = p.momentum[f];
            for (int r = 1; r < p.world; ++r) s[0] += load1(p.grads[r] + f);
            u[x] = s[0] = look_ahead(p.sc, s[0], mom);
            ss.add(s);
            p.momentum[f] = mom;
        });
    }
    const double sum = block_sum(ss.total());
    if (threadIdx.x == 0) p.d.partials[blockIdx.x] = sum;
}

// The norm's partial sums of a matrix given as it is (67 million bf16: 60 us,
// 2.2 TB/s; few sums in flight a thread, 1% of the call).
template <typename T>
__global__ void __launch_bounds__(kElemThreads) muon_norm_kernel(MuonDev d, const T *in)
{
    ptx::launch_dependents();
    reset_counters(d);
    if (blockIdx.x >= d.nchunks) return;
    const MuonMat &m = d.mats[d.chunk_mat[blockIdx.x]];
    SquareSum ss;
    if (m.vec) {
        for_chunk(m, blockIdx.x - m.chunk0, d.chunk, 8, [&](uint64_t f, uint64_t) {
            float v[8];
            load8(v, in + f);
            ss.add(v);
        });
    } else {
        for_chunk(m, blockIdx.x - m.chunk0, d.chunk, 1, [&](uint64_t f, uint64_t) {
            const float v[1] = {load1(in + f)};
            ss.add(v);
        });
    }
    const double sum = block_sum(ss.total());
    if (threadIdx.x == 0) d.partials[blockIdx.x] = sum;
}

// X = U / (|U| + eps), as two f16 planes in region 0.  Every block forms the
// norm from all partial sums of its matrix itself, which saves a launch.
// 85 million entries: 109 us, 6.2 TB/s.
template <typename T>
__global__ void __launch_bounds__(kElemThreads) muon_split_kernel(MuonDev d, const T *in, float eps)
{
    ptx::launch_dependents();
    ptx::grid_dependency_wait();
    const MuonMat &m = d.mats[d.chunk_mat[blockIdx.x]];
    __shared__ float factor;
    // the blocks' sums in a fixed order
    __shared__ double part[kElemThreads / 32];
    double t = 0.0;
    for (uint32_t i = threadIdx.x; i < m.chunks; i += kElemThreads) t += d.partials[m.chunk0 + i];
    for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(~0u, t, o);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = t;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int i = 1; i < kElemThreads / 32; ++i) t += part[i];
        factor = (float)((double)kXScale / (sqrt(t) + (double)eps));
    }
    __syncthreads();
    const float k = factor;
    uint16_t *hi = reinterpret_cast<uint16_t *>(m.region[0]), *lo = hi + m.xplane;
    const T *src = in ? in : reinterpret_cast<const T *>(m.region[1]);
    if (m.vec) {
        for_chunk(m, blockIdx.x - m.chunk0, d.chunk, 8, [&](uint64_t f, uint64_t x) {
            float v[8];
            uint4 h, l;
            load8(v, src + (in ? f : x));
            split(v[0] * k, v[1] * k, h.x, l.x);
            split(v[2] * k, v[3] * k, h.y, l.y);
            split(v[4] * k, v[5] * k, h.z, l.z);
            split(v[6] * k, v[7] * k, h.w, l.w);
            *reinterpret_cast<uint4 *>(hi + x) = h;
            *reinterpret_cast<uint4 *>(lo + x) = l;
        });
    } else {
        for_chunk(m, blockIdx.x - m.chunk0, d.chunk, 1, [&](uint64_t f, uint64_t x) {
            uint32_t h, l;
            split(load1(src + (in ? f : x)) * k, 0.f, h, l);
            hi[x] = (uint16_t)h;
            lo[x] = (uint16_t)l;
        });
    }
}

// p = p (1 - lr wd) - lr scale X, and bf16(p) into the W replicas: 12 + 2W
// bytes an entry.  85 million entries, W = 8: 367 us, 6.5 TB/s.
template <int CAP>
__global__ void __launch_bounds__(kElemThreads) muon_apply_kernel(const __grid_constant__ ApplyParams<CAP> p)
{
    ptx::grid_dependency_wait();
    const MuonMat &m = p.d.mats[p.d.chunk_mat[blockIdx.x]];
    const float *x = reinterpret_cast<const float *>(m.region[p.region]);
    const float step = p.lr * m.scale;
    if (m.vec) {
        for_chunk(m, blockIdx.x - m.chunk0, p.d.chunk, 8, [&](uint64_t f, uint64_t i) {
            float o[8], w[8];
            load8(o, x + i);
            load8(w, p.master + f);
#pragma unroll
            for (int k = 0; k < 8; ++k) w[k] = w[k] * p.decay - step * o[k];
            store8(p.master + f, w);
            for (int r = 0; r < p.world; ++r) store8(p.params[r] + f, w);
        });
    } else {
        for_chunk(m, blockIdx.x - m.chunk0, p.d.chunk, 1, [&](uint64_t f, uint64_t i) {
            const float w = p.master[f] * p.decay - step * x[i];
            p.master[f] = w;
            for (int r = 0; r < p.world; ++r) store1(p.params[r] + f, w);
        });
    }
}

template <typename T>
__global__ void __launch_bounds__(kElemThreads) muon_out_kernel(MuonDev d, T *out, int region)
{
    ptx::grid_dependency_wait();
    const MuonMat &m = d.mats[d.chunk_mat[blockIdx.x]];
    const float *x = reinterpret_cast<const float *>(m.region[region]);
    if (m.vec) {
        for_chunk(m, blockIdx.x - m.chunk0, d.chunk, 8, [&](uint64_t f, uint64_t i) {
            float v[8];
            load8(v, x + i);
            store8(out + f, v);
        });
    } else {
        for_chunk(m, blockIdx.x - m.chunk0, d.chunk, 1, [&](uint64_t f, uint64_t i) { store1(out + f, x[i]); });
    }
}

// ---------------------------------------------------------- the iteration

// For tiles of TN columns.  Shared memory of one block: stages of one K step
// (64) of its 128 rows of A and its TN/2 rows of B, high and low parts, and
// 2 KB an epilogue warp.
constexpr uint32_t kBox = 8192;                        // 64 x 64 f16
constexpr int kSlots = 2;                              // tiles known to a pair: this one and the next
constexpr int kGroups = 4;                             // of 4 epilogue warps, TN/4 columns each
constexpr int kNsThreads = 64 + kGroups * 128;         // loads, products; epilogue
constexpr uint32_t kWarpOut = 2048;                    // 32 rows x 64 bytes on an epilogue warp's way out
template <int TN>
struct Shape {
    static constexpr int kBoxesB = TN / 128;           // of one part of B
    static constexpr uint32_t kStageBytes = (4 + 2 * kBoxesB) * kBox;   // A hi, A lo (two boxes each), B hi, B lo
    static constexpr int kStages = TN == 256 ? 3 : 4;
    // Two accumulators of 256 columns, all of TMEM.  A narrow tile's hold each
    // block's 64 columns of hi*hi + lo*hi and then of hi*lo + lo*lo: its B
    // parts lie one after the other, so one product takes both, at the rate
    // of a wide one (256 x 256 x 16 in 128 cycles, 256 x 128 x 16 in 105).
    static constexpr int kAccs = 2;
    static constexpr uint32_t kAccCols = 256;
    static constexpr int kSmem = kStages * kStageBytes + 4 * kGroups * kWarpOut + 1024;
    static_assert(kSmem >= kAloneSmem, "two pairs could wait for each other's tensor memory");
};
// K of one accumulator.  The tensor cores cut every addition of 16 products
// off below the sum's last place, so a sum of positive terms falls short by
// 8e-8 of itself for each (measured with one product: 4e-6 over K = 1024,
// 9e-5 over 16384).  Longer sums are gathered 128 at a time and added up in
// rounded fp32.  A wide tile's first two sums are of 256, which keeps the
// products busy while the tile before is written.
template <int TN>
__device__ __forceinline__ bool starts_sum(uint32_t k)
{
    return k % (TN == 256 && k < 512 ? 256 : 128) == 0;
}
template <int TN>
__device__ __forceinline__ uint32_t sums_of(uint32_t k)
{
    return TN == 128 ? (k + 127) / 128 : k <= 512 ? (k + 255) / 256 : 2 + (k - 512 + 127) / 128;
}

struct NsParams {
    MuonDev d;
    float a, b, c;
    uint32_t total;
    int steps, stall;
};

// The linear and the square term come from one product, c A' (A' + v I) with
// v = (b + 2 c alpha)/c; A' + v I differs from A' in its diagonal tiles only.

// A tile, as it is described to all roles of both blocks of a pair: they meet
// the plan in shared memory only.
struct __align__(16) Tile {
    uint32_t mat, phase;
    uint32_t map_a, map_b;     // tensor maps of the operands
    uint32_t k;
    uint32_t a_turn, b_turn;   // K below which an operand is MN-major in memory
    uint32_t diag;             // tensor map of B for the 256 of K from b_turn on, or 0
    uint32_t row, col;         // of the tile in its matrix
    uint32_t rows, cols;       // of the matrix
    unsigned char *out;        // first entry of the matrix: f16 parts, or fp32 in the last product
    uint64_t plane;            // bytes from the high to the low parts
    unsigned char *also;       // diagonal blocks of A' + v I, or null: a copy with v more on the diagonal
    uint64_t also_plane;
    uint32_t pitch;            // bytes of a row
    uint32_t last;             // results in fp32
    float factor, on_diagonal; // result = factor * product, plus this on the diagonal
    float v;
    uint32_t pad[3];
};
constexpr uint32_t kNoMore = 3;                        // phase of the tile that ends the work
constexpr int kTileWords = sizeof(Tile) / 16;

struct NsShared {
    Tile slot[kSlots];
    uint64_t full[4], empty[4];                        // operand ring
    uint64_t slot_full[kSlots], slot_empty[kSlots];    // tile ring
    uint64_t slot_go[kSlots];                          // a tile's operands are there to be loaded
    uint64_t acc_full[2], acc_empty[2];                // accumulators
    uint64_t drain;
    uint32_t tmem;
    int abort;
};

// The products:
//   phase 0: A' = X X^T (or X^T X) - alpha I,
//   phase 1: P = c A' (A' + v I) + (a + b alpha + c alpha^2) I,
//   phase 2: X <- P X (or X P).
// A Gram-sized matrix (A' or P) is stored from its diagonal 256 x 256 blocks
// on; what lies below is read transposed from above, as an MN-major operand.
__device__ __forceinline__ void describe(const NsParams &p, uint32_t ticket, Tile &t, uint32_t &need)
{
    const uint32_t iter = ticket / p.d.work_per_iter;
    const uint2 w = p.d.work[ticket - iter * p.d.work_per_iter];
    t.mat = w.x & 0x3FFFFFFFu;
    t.phase = w.x >> 30;
    const MuonMat &m = p.d.mats[t.mat];
    const uint32_t ti = w.y & 0xFFFFu, tj = w.y >> 16;
    need = iter * (m.parts[0] + m.parts[1] + m.parts[2]) + (t.phase > 0 ? m.parts[0] : 0) + (t.phase > 1 ? m.parts[1] : 0);
    const uint32_t maps = t.mat * kMapsPerMat, x = maps + (iter & 1 ? kMapX1 : kMapX0);
    constexpr uint32_t kAlways = 0xFFFFFFFFu;
    constexpr float inv = 1.0f / kGramScale;
    t.row = ti * kNsRows;
    t.col = tj * p.d.tile;
    const uint32_t block = t.col / kNsRows * kNsRows;   // the diagonal block beside the tile's columns
    const float alpha = alpha_of(iter, p.steps);
    t.v = (p.b + 2.f * p.c * alpha) / p.c * kGramScale;
    t.diag = 0;
    t.also = nullptr;
    t.also_plane = (uint64_t)m.s * (kNsRows * 2);
    t.last = t.phase == 2 && (int)iter + 1 == p.steps;
    t.factor = t.phase == 0 ? kGramScale / (kXScale * kXScale) : t.phase == 1 ? p.c * inv : t.last ? inv / kXScale : inv;
    t.on_diagonal = 0.f;
    if (t.phase < 2) {
        t.rows = t.cols = m.s;
        t.pitch = m.lds * 2;
        t.plane = m.splane * 2;
        t.out = t.phase == 0 ? m.gram : m.poly;
        if (t.phase == 0) {
            t.map_a = t.map_b = x;
            t.k = m.tall ? m.rows : m.cols;
            t.a_turn = t.b_turn = m.tall ? kAlways : 0;
            t.on_diagonal = -alpha * kGramScale;
            if (t.row == block) t.also = m.diag;
        } else {
            t.map_a = t.map_b = maps + kMapA;
            t.k = m.s;
            t.a_turn = t.row;
            t.b_turn = block;
            t.diag = maps + kMapD;
            t.on_diagonal = (p.a + alpha * (p.b + alpha * p.c)) * kGramScale;
        }
    } else {
        t.rows = m.rows;
        t.cols = m.cols;
        t.pitch = m.ldx * (t.last ? 4 : 2);
        t.plane = m.xplane * 2;
        t.out = m.region[(iter + 1) & 1];
        t.k = m.s;
        t.map_a = m.tall ? x : maps + kMapP;
        t.map_b = m.tall ? maps + kMapP : x;
        t.a_turn = m.tall ? 0 : t.row;
        t.b_turn = m.tall ? block : kAlways;
    }
}

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

// A warp's 32 rows of 64 bytes: lane r gives row r, and 4 lanes write each
// row, 16 bytes at a time.  `mem`: the warp's 2 KB; row r keeps its pieces
// exchanged by (r >> 1) & 3, free of bank conflicts both ways.
__device__ __forceinline__ uint32_t turned(uint32_t mem, uint32_t row, uint32_t piece)
{
    return mem + row * 64 + ((piece ^ ((row >> 1) & 3u)) * 16);
}
__device__ __forceinline__ void turn_in(uint32_t mem, const uint32_t x[16])
{
    const uint32_t lane = threadIdx.x & 31;
#pragma unroll
    for (uint32_t j = 0; j < 4; ++j)
        tc::st_shared(turned(mem, lane, j), make_uint4(x[4 * j], x[4 * j + 1], x[4 * j + 2], x[4 * j + 3]));
    __syncwarp();
}
__device__ __forceinline__ void turn_out(uint32_t mem, unsigned char *dst, uint64_t pitch, uint32_t rows)
{
    const uint32_t lane = threadIdx.x & 31;
#pragma unroll
    for (uint32_t i = 0; i < 4; ++i) {
        const uint32_t row = 8 * i + (lane >> 2);
        const uint4 v = tc::ld_shared(turned(mem, row, lane & 3));
        if (row < rows) *reinterpret_cast<uint4 *>(dst + row * pitch + (lane & 3) * 16) = v;
    }
    __syncwarp();
}

// The whole iteration over all matrices in one launch, by pairs of blocks.
// Pairs draw tiles in an order in which every tile comes after those it
// depends on (all of the previous product of its matrix), so a pair that
// waits for a matrix's counter waits only for tiles that running pairs hold:
// none needs another to be resident, and the grid may be of any size.
// Within a pair, one thread of the second block draws tiles and waits for
// what they depend on, one thread of each block loads its operands (TMA), one
// thread of the first block issues the products, and in each block 4 x 4
// warps take its 128 x 256 half of the tile out of one accumulator while the
// other fills, write it and count it as finished.  Each warp turns its 32
// rows in 2 KB of shared memory so that a store covers 8 rows of 64 bytes;
// straight from the registers, a row a lane, writing took 4.5 us a tile, and
// through TMA, 64 columns at a time in the 32 KB that the stages leave, 7.4.
// Eighteen warps put five on one of an SM's four schedulers, which leaves a
// thread 96 registers: a wide tile's 64 results beside the 16 just read spill
// 72 bytes of stores and 108 of loads.
template <int TN>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kNsThreads, 1)
    muon_iterate_kernel(const __grid_constant__ NsParams p)
{
    using S = Shape<TN>;
    constexpr int kStages = S::kStages, kBoxesB = S::kBoxesB, kAccs = S::kAccs;
    constexpr uint32_t kStageBytes = S::kStageBytes;
    constexpr int kCols = TN / kGroups;                // columns of an epilogue warp
    extern __shared__ unsigned char raw[];
    __shared__ NsShared sh;
    const uint32_t ring = (tc::smem_u32(raw) + 1023u) & ~1023u;
    const int warp = threadIdx.x >> 5;
    const uint32_t rank = tc::cluster_rank();
    unsigned *errors = p.d.errors;
    volatile int *abort = &sh.abort;

    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) ptx::mbar_init(&sh.full[i], 1), ptx::mbar_init(&sh.empty[i], 1);
        // a slot is read by both loaders, the first block's products and, in both, 16 epilogue warps
        for (int i = 0; i < kSlots; ++i) {
            ptx::mbar_init(&sh.slot_full[i], 1), ptx::mbar_init(&sh.slot_go[i], 1);
            ptx::mbar_init(&sh.slot_empty[i], 3 + 2 * 4 * kGroups);
        }
        for (int i = 0; i < kAccs; ++i) ptx::mbar_init(&sh.acc_full[i], 1), ptx::mbar_init(&sh.acc_empty[i], 2 * 4 * kGroups);
        ptx::mbar_init(&sh.drain, 1);
        sh.abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) {
        __syncwarp();
        tc::tmem_alloc(&sh.tmem, 512);
    }
    tc::fence_before_sync();
    __syncthreads();
    ptx::cluster_sync();
    tc::fence_after_sync();
    const uint32_t tmem = sh.tmem;
    ptx::launch_dependents();
    ptx::grid_dependency_wait();

    if (threadIdx.x == 32 && rank == 1) {
        // ---- tiles, one ahead: drawing and describing one takes 2 us of dependent reads
        for (uint32_t n = 0; !p.stall; ++n) {
            const int slot = n % kSlots;
            if (n >= kSlots && !tc::pair_wait(&sh.slot_empty[slot], (n / kSlots - 1) & 1u, abort, errors)) break;
            const uint32_t ticket = atomicAdd(p.d.ticket, 1u);
            Tile t{};
            uint32_t need = 0;
            t.phase = kNoMore;
            if (ticket < p.total) describe(p, ticket, t, need);
            const uint32_t there = tc::map_to(tc::smem_u32(&sh.slot[slot]), 0);
            sh.slot[slot] = t;
#pragma unroll
            for (int i = 0; i < kTileWords; ++i) tc::st_cluster(there + 16 * i, reinterpret_cast<const uint4 *>(&t)[i]);
            tc::arrive_cluster(tc::map_to(tc::smem_u32(&sh.slot_full[slot]), 0));
            tc::arrive_cluster(tc::map_to(tc::smem_u32(&sh.slot_full[slot]), 1));
            if (t.phase == kNoMore || !wait_parts(&p.d.done[t.mat], need, abort, errors)) break;
            tc::arrive_cluster(tc::map_to(tc::smem_u32(&sh.slot_go[slot]), 0));
            tc::arrive_cluster(tc::map_to(tc::smem_u32(&sh.slot_go[slot]), 1));
        }
    } else if (threadIdx.x == 0) {
        // ---- loads
        uint32_t issued = 0;
        for (uint32_t n = 0;; ++n) {
            const int slot = n % kSlots;
            if (!tc::pair_wait(&sh.slot_full[slot], (n / kSlots) & 1u, abort, errors)) break;
            const Tile &t = sh.slot[slot];
            if (t.phase == kNoMore) break;
            tc::prefetch_map(p.d.maps + t.map_a);
            tc::prefetch_map(p.d.maps + t.map_b);
            if (!tc::pair_wait(&sh.slot_go[slot], (n / kSlots) & 1u, abort, errors)) break;
            tc::fence_proxy_async_all();   // other blocks' results, before the loads below
            const int row = (int)(t.row + rank * 128), col = (int)(t.col + rank * (TN / 2));
            const uint32_t k_end = t.k, a_turn = t.a_turn, b_turn = t.b_turn, diag = t.diag;
            const CUtensorMap *map_a = p.d.maps + t.map_a, *map_b = p.d.maps + t.map_b, *map_d = p.d.maps + diag;
            tc::arrive_cluster(tc::map_to(tc::smem_u32(&sh.slot_empty[slot]), 1));
            bool ok = true;
            for (uint32_t k0 = 0; k0 < k_end; k0 += kNsTileK) {
                const uint32_t stage = issued % kStages;
                if (issued >= kStages) ok = tc::pair_wait(&sh.empty[stage], (issued / kStages - 1) & 1u, abort, errors);
                if (!ok) break;
                if (rank == 0) ptx::mbar_arrive_expect_tx(&sh.full[stage], 2 * kStageBytes);
                const uint32_t bar = tc::map_to(tc::smem_u32(&sh.full[stage]), 0);
                const uint32_t dst = ring + stage * kStageBytes;
                const bool a_mn = k0 < a_turn, b_mn = k0 < b_turn;
                const int k = (int)k0;
                const bool on_diag = diag != 0 && k0 - b_turn < kNsRows;
                const CUtensorMap *mb = on_diag ? map_d : map_b;
                const int kb = on_diag ? (int)(k0 - b_turn) : k;
#pragma unroll
                for (int plane = 0; plane < 2; ++plane) {
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int r = row + 64 * i;
                        tc::tma_box_pair(dst + (2 * plane + i) * kBox, map_a, a_mn ? r : k, a_mn ? k : r, plane, bar);
                    }
#pragma unroll
                    for (int i = 0; i < kBoxesB; ++i) {
                        const int c = col + 64 * i;
                        tc::tma_box_pair(dst + (4 + kBoxesB * plane + i) * kBox, mb, b_mn ? c : kb, b_mn ? kb : c, plane, bar);
                    }
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
            const uint32_t phase = sh.slot[slot].phase, k_end = sh.slot[slot].k;
            const uint32_t a_turn = sh.slot[slot].a_turn, b_turn = sh.slot[slot].b_turn;
            tc::arrive_cluster(tc::map_to(tc::smem_u32(&sh.slot_empty[slot]), 1));
            if (phase == kNoMore) break;
            for (uint32_t k0 = 0; k0 < k_end; k0 += kNsTileK) {
                const uint32_t acc = used % kAccs, d = tmem + acc * S::kAccCols;
                const bool first = starts_sum<TN>(k0);
                if (first && used >= kAccs) {
                    if (!(ok = tc::pair_wait(&sh.acc_empty[acc], (used / kAccs - 1) & 1u, abort, errors))) break;
                    tc::fence_after_sync();
                }
                const uint32_t stage = taken % kStages;
                if (!(ok = tc::pair_wait(&sh.full[stage], (taken / kStages) & 1u, abort, errors))) break;
                tc::fence_after_sync();
                const bool a_mn = k0 < a_turn, b_mn = k0 < b_turn;
                const uint32_t idesc = tc::instr_desc(kNsRows, 256, a_mn, b_mn);
                const uint64_t astep = tc::k16_step(a_mn), bstep = tc::k16_step(b_mn);
                const uint32_t src = ring + stage * kStageBytes;
                const uint64_t ah = tc::smem_desc(src, a_mn), al = tc::smem_desc(src + 2 * kBox, a_mn);
                const uint64_t bh = tc::smem_desc(src + 4 * kBox, b_mn), bl = tc::smem_desc(src + (4 + kBoxesB) * kBox, b_mn);
                // the small products first: what is cut off goes by the size of the sum so far
#pragma unroll
                for (int j = 0; j < kNsTileK / 16; ++j) {
                    if (TN == 256) tc::mma_f16(d, ah + j * astep, bl + j * bstep, idesc, !first || j > 0);
                    tc::mma_f16(d, al + j * astep, bh + j * bstep, idesc, TN == 256 || !first || j > 0);
                }
#pragma unroll
                for (int j = 0; j < kNsTileK / 16; ++j) tc::mma_f16(d, ah + j * astep, bh + j * bstep, idesc, true);
                tc::mma_commit(&sh.empty[stage]);
                ++taken;
                if (k0 + kNsTileK >= k_end || starts_sum<TN>(k0 + kNsTileK)) {
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
    } else if (warp >= 2) {
        // ---- finished tiles: this block's 128 rows, kCols columns to each group
        const int group = (warp - 2) >> 2;
        const uint32_t r = (uint32_t)(warp & 3) * 32 + (threadIdx.x & 31);
        const uint32_t at = tmem + ((uint32_t)(warp & 3) << 21) + group * kCols + (TN == 128 && group >= 2 ? 64 : 0);
        const uint32_t mem = ring + kStages * kStageBytes + (warp - 2) * kWarpOut;
        const bool leader = (threadIdx.x & 31) == 0;
        uint32_t used = 0;            // accumulators
        unsigned *owed = nullptr;     // a tile's counter that this warp has not added to yet
        // this warp's results, then its arrival: ordered for loads (TMA) by any block
        const auto settle = [&]() {
            if (owed) {
                tc::fence_proxy_async_all();
                __syncwarp();
                if (leader) tc::red_release_add(owed, 1u);
                owed = nullptr;
            }
        };
        for (uint32_t n = 0;; ++n) {
            const int slot = n % kSlots;
            // Waiting for the writes to land may come in the next tile's time if its operands are there already;
            // else that tile may be waiting for this one.
            if (!__all_sync(~0u, tc::pair_peek(&sh.slot_go[slot], (n / kSlots) & 1u))) settle();
            if (!__all_sync(~0u, tc::pair_wait(&sh.slot_full[slot], (n / kSlots) & 1u, abort, errors))) break;
            const Tile &t = sh.slot[slot];
            const uint32_t phase = t.phase, sums = sums_of<TN>(t.k);
            if (phase == kNoMore) break;
            float w[kCols];
#pragma unroll
            for (int q = 0; q < kCols; ++q) w[q] = 0.f;
            bool ok = true;
            for (uint32_t i = 0; i < sums; ++i, ++used) {
                const uint32_t acc = used % kAccs;
                ok = __all_sync(~0u, tc::pair_wait(&sh.acc_full[acc], (used / kAccs) & 1u, abort, errors));
                if (!ok) break;
                tc::fence_after_sync();
#pragma unroll
                for (int q = 0; q < kCols / 16; ++q) {
                    float x[16];
                    tc::tmem_load16(x, at + acc * S::kAccCols + q * 16);
#pragma unroll
                    for (int j = 0; j < 16; ++j) w[16 * q + j] += x[j];
                    if (TN == 128) {
                        tc::tmem_load16(x, at + acc * S::kAccCols + 64 + q * 16);
#pragma unroll
                        for (int j = 0; j < 16; ++j) w[16 * q + j] += x[j];
                    }
                }
                tc::fence_before_sync();
                __syncwarp();
                if (leader) tc::arrive_cluster_relaxed(tc::map_to(tc::smem_u32(&sh.acc_empty[acc]), 0));
                if (i == 1 || sums == 1) settle();
            }
            if (!ok) break;
            const uint32_t col = t.col + group * kCols, row = t.row + rank * 128 + r, row0 = row - (r & 31);
            const uint32_t here = t.rows - row0;   // this warp's rows, 32 or the last of the matrix
            const uint32_t pitch = t.pitch, diagonal = row - col;
            const bool any = col < t.cols && row0 < t.rows, last = t.last;
            const bool meets = phase < 2 && t.row == t.col / kNsRows * kNsRows;
            unsigned char *out = t.out + (uint64_t)row0 * pitch + col * (last ? 4 : 2);
            unsigned char *also = t.also ? t.also + (uint64_t)row0 * (kNsRows * 2) + (col - t.row) * 2 : nullptr;
            const uint64_t plane = t.plane, also_plane = t.also_plane;
            const float f = t.factor, more = t.on_diagonal, v = t.v;
            owed = &p.d.done[t.mat];
            __syncwarp();
            // before the writes: the arrival would wait for them
            if (leader) tc::arrive_cluster(tc::map_to(tc::smem_u32(&sh.slot_empty[slot]), 1));
            if (any) {
#pragma unroll
                for (uint32_t q = 0; q < kCols; ++q) w[q] *= f;
                float own = 0.f;   // where this row meets the diagonal
                if (meets) {
#pragma unroll
                    for (uint32_t q = 0; q < kCols; ++q) {
                        w[q] += q == diagonal ? more : 0.f;
                        own = q == diagonal ? w[q] : own;
                    }
                }
                if (last) {
#pragma unroll
                    for (int q = 0; q < kCols / 16; ++q) {
                        turn_in(mem, reinterpret_cast<const uint32_t *>(w + 16 * q));
                        turn_out(mem, out + 64 * q, pitch, here);
                    }
                } else {
#pragma unroll
                    for (int q = 0; q < kCols / 32; ++q) {
                        uint32_t hi[16], lo[16];
#pragma unroll
                        for (int i = 0; i < 16; ++i) split(w[32 * q + 2 * i], w[32 * q + 2 * i + 1], hi[i], lo[i]);
#pragma unroll
                        for (int part = 0; part < 2; ++part) {
                            turn_in(mem, part ? lo : hi);
                            turn_out(mem, out + part * plane + 64 * q, pitch, here);
                            if (also) {
                                if ((diagonal >> 5) == (uint32_t)q) {
                                    uint32_t own_hi, own_lo;
                                    split(own + v, 0.f, own_hi, own_lo);
                                    tc::st_shared16(turned(mem, r & 31, (diagonal & 31) >> 3) + (diagonal & 7) * 2,
                                                    (uint16_t)(part ? own_lo : own_hi));
                                }
                                __syncwarp();
                                turn_out(mem, also + part * also_plane + 64 * q, kNsRows * 2, here);
                            }
                        }
                    }
                }
            }
        }
        if (!*abort) settle();
    }
    if (*abort) {   // give copies that nothing above waits for (the second block's loads) 1 ms to land
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
    if (warp == 1) tc::tmem_free(tmem, 512);
}

template <int CAP>
cudaError_t momentum_t(const MuonDev &d, const MuonScalars &sc, const void *const *grads, int world, float *momentum,
                       uint32_t grid, cudaStream_t stream)
{
    MomentumParams<CAP> p{};
    for (int r = 0; r < world; ++r) p.grads[r] = static_cast<const uint16_t *>(grads[r]);
    p.d = d;
    p.momentum = momentum;
    p.world = world;
    p.sc = sc;
    return launch(muon_momentum_kernel<CAP>, grid, kElemThreads, 0, stream, p);
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
    return launch_early(muon_apply_kernel<CAP>, d.nchunks, kElemThreads, 0, stream, p);
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
        return launch(muon_norm_kernel<uint16_t>, first_grid(d), kElemThreads, 0, stream, d, static_cast<const uint16_t *>(in));
    return launch(muon_norm_kernel<float>, first_grid(d), kElemThreads, 0, stream, d, static_cast<const float *>(in));
}

cudaError_t launch_muon_split(const MuonDev &d, const MuonScalars &sc, const void *in, bool bf16, cudaStream_t stream)
{
    if (in && bf16)
        return launch_early(muon_split_kernel<uint16_t>, d.nchunks, kElemThreads, 0, stream, d, static_cast<const uint16_t *>(in), sc.eps);
    return launch_early(muon_split_kernel<float>, d.nchunks, kElemThreads, 0, stream, d, static_cast<const float *>(in), sc.eps);
}

template <int TN>
static cudaError_t iterate_t(const NsParams &p, uint32_t grid, cudaStream_t stream)
{
    const cudaError_t e = allow_dynamic_smem(reinterpret_cast<const void *>(muon_iterate_kernel<TN>), Shape<TN>::kSmem);
    if (e != cudaSuccess) return e;
    return launch_early(muon_iterate_kernel<TN>, grid, kNsThreads, Shape<TN>::kSmem, stream, p);
}

cudaError_t launch_muon_iterate(const MuonDev &d, const MuonScalars &sc, int num_sms, cudaStream_t stream)
{
    NsParams p{};
    p.d = d;
    p.a = sc.a;
    p.b = sc.b;
    p.c = sc.c;
    p.steps = sc.steps;
    p.stall = sc.stall;
    p.total = d.work_per_iter * (uint32_t)sc.steps;
    const uint32_t pairs = (uint32_t)num_sms / 2;
    const uint32_t grid = 2 * (p.total < pairs ? p.total : pairs);
    return d.tile == 256 ? iterate_t<256>(p, grid, stream) : iterate_t<128>(p, grid, stream);
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
        return launch_early(muon_out_kernel<uint16_t>, d.nchunks, kElemThreads, 0, stream, d, static_cast<uint16_t *>(out), sc.steps & 1);
    return launch_early(muon_out_kernel<float>, d.nchunks, kElemThreads, 0, stream, d, static_cast<float *>(out), sc.steps & 1);
}

}  // namespace zero1
