// zero1_ffn_gemm.cu -- the matrix products of the gated feed-forward block on
// the tensor cores, with its activation and that one's gradient as their
// epilogues.
//
//   forward:  gate = x Wg, up = x Wu, h = act(gate) up       (one launch)
//             y = h Wd
//   backward: dh = dy Wd^T, dup = dh act(gate),
//             dgate = dh up act'(gate)                       (one launch)
//             dWg = x^T dgate, dWu = x^T dup, dWd = h^T dy,
//             dx = dgate Wg^T + dup Wu^T                     (one launch)
//
// Operands are bf16 as they lie in memory (K- or MN-major, no transposed
// copies), sums fp32 in tensor memory.  What is written between the launches
// (h; dgate and dup) is bf16: the next product takes bf16, and a rounding of
// 2^-9 of each of its K terms adds up to one of 2^-9 of the result, as much
// as the result's own.
#include "zero1_ffn.h"
#include "zero1_ffn_device.cuh"
#include "zero1_internal.h"
#include "zero1_launch.h"
#include "zero1_muon.h"
#include "zero1_tc.cuh"

namespace zero1 {
namespace {

constexpr uint32_t kBox = 8192;                     // 64 x 64 bf16
constexpr uint32_t kStageBytes = 4 * kBox;          // one block's 128 rows of A and 128 of B
constexpr uint32_t kWarpTurn = 4096;                // 32 rows x 32 fp32 of an epilogue warp
// Eight epilogue warps have registers for what is in flight (16,384 x 768 x
// 2048: dh's product in 67 us, 76 with sixteen; 8,192 x 4096 x 11008 backward
// 2.77 ms, 2.86).  Sixteen finish one tile sooner, where no pair has another
// to go on with (2,000 x 256 x 688 backward in 35 us, 37 with eight).
template <int WARPS>
struct Gemm {
    static constexpr int kThreads = 64 + 32 * WARPS;
    static constexpr int kStages = WARPS == 16 ? 5 : 6;
    static constexpr int kSmem = kStages * kStageBytes + WARPS * kWarpTurn + 1024;
    static_assert(kSmem >= kAloneSmem, "two pairs could wait for each other's tensor memory");
};

struct GemmShared {
    uint64_t full[6], empty[6];
    uint64_t acc_full[2], acc_empty[2];
    uint64_t drain;
    uint32_t tmem;
    int abort;
    unsigned errors;
};

// bf16 operands (formats 1) of tc::instr_desc's f16 products.
__device__ __forceinline__ uint32_t bf16_desc(bool a_mn, bool b_mn)
{
    return tc::instr_desc(kFfnTile, kFfnTile, a_mn, b_mn) | (1u << 7) | (1u << 10);
}

// Where an item's tile lies: items are tiles, the slices of K of each one
// after another, in groups of 8 tile rows (all columns of a group before the
// next), so that the pairs at work share operands in L2.
struct Item {
    uint32_t job, row, col, begin, end, partial;    // k steps [begin, end) over all segments
};
template <int MODE>
__device__ __forceinline__ Item item_of(const FfnParams &p, uint32_t i)
{
    Item t;
    t.job = 0;
    while (MODE == kFfnPlain && t.job + 1 < p.jobs && i >= p.job[t.job + 1].first) ++t.job;
    const FfnJob &j = p.job[t.job];
    const uint32_t local = i - j.first, slice = local % j.slices, at = local / j.slices;
    const uint32_t span = 8 * j.tiles_n, group = at / span;
    const uint32_t height = min(8u, j.tiles_m - group * 8), in = at - group * span;
    t.row = (group * 8 + in % height) * kFfnTile;
    t.col = in / height * (MODE == kFfnGated ? kFfnTile / 2 : kFfnTile);
    const uint32_t steps = j.steps * j.segments;
    t.begin = (uint32_t)((uint64_t)steps * slice / j.slices);
    t.end = (uint32_t)((uint64_t)steps * (slice + 1) / j.slices);
    t.partial = j.partial + local;
    return t;
}

// How a warp's patch meets global memory: 16-byte pieces of a patch wholly
// inside the matrix, the same near an edge, or single entries.
enum Access : int { kWholePatch, kEdgePatch, kSingles };

// 32 x 32 fp32 of a warp go through shared memory, from one row a lane to a
// mapping that global memory likes, 8 values at a time (q = 0..3):
//   pieces:  row 8 q + lane / 4, columns 8 (lane % 4) on: 16-byte accesses,
//            64 bytes of a row side by side;
//   singles: column `lane` of rows 8 q on: 32 entries of a row side by side,
//            for rows that start off a 16-byte boundary.
// Row r keeps its 16-byte pieces exchanged by r % 8: no bank conflicts.
__device__ __forceinline__ uint32_t piece_at(uint32_t mem, uint32_t row, uint32_t piece)
{
    return mem + row * 128 + ((piece ^ (row & 7u)) * 16);
}
__device__ __forceinline__ void put_rows(uint32_t mem, const float x[32])
{
    const uint32_t lane = threadIdx.x & 31;
#pragma unroll
    for (uint32_t j = 0; j < 8; ++j)
        tc::st_shared(piece_at(mem, lane, j), make_uint4(__float_as_uint(x[4 * j]), __float_as_uint(x[4 * j + 1]),
                                                         __float_as_uint(x[4 * j + 2]), __float_as_uint(x[4 * j + 3])));
    __syncwarp();
}
template <int HOW>
__device__ __forceinline__ void get8(float v[8], uint32_t mem, uint32_t q)
{
    const uint32_t lane = threadIdx.x & 31;
    if (HOW != kSingles) {
#pragma unroll
        for (uint32_t j = 0; j < 2; ++j) {
            const uint4 w = tc::ld_shared(piece_at(mem, 8 * q + (lane >> 2), 2 * (lane & 3) + j));
            v[4 * j] = __uint_as_float(w.x);
            v[4 * j + 1] = __uint_as_float(w.y);
            v[4 * j + 2] = __uint_as_float(w.z);
            v[4 * j + 3] = __uint_as_float(w.w);
        }
    } else {
#pragma unroll
        for (uint32_t k = 0; k < 8; ++k)
            asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v[k]) : "r"(piece_at(mem, 8 * q + k, lane >> 2) + (lane & 3) * 4) : "memory");
    }
}

// 32 lanes x 32 fp32 columns of tensor memory, one row a lane.
__device__ __forceinline__ void tmem_load32(float v[32], uint32_t addr)
{
    uint32_t *r = reinterpret_cast<uint32_t *>(v);
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]),
          "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]),
          "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(addr)
        : "memory");
}

// The 32 x 32 that a warp stands before: its first entry, and how much of it
// lies inside the matrix.
struct Patch {
    uint64_t at;               // of entry (0, 0), in the matrix's entries
    uint64_t ld;
    uint32_t rows, cols;
};
// 8 values of the mapping above, as packed bf16; zeros outside the matrix.
template <int HOW>
__device__ __forceinline__ uint4 load8(const uint16_t *base, const Patch &p, uint32_t q)
{
    const uint32_t lane = threadIdx.x & 31;
    uint32_t w[8];
    if (HOW == kSingles) {
        const uint16_t *from = base + p.at + 8 * q * p.ld + lane;
#pragma unroll
        for (uint32_t k = 0; k < 8; ++k) w[k] = lane < p.cols && 8 * q + k < p.rows ? from[k * p.ld] : 0u;
    } else {
        const uint32_t r = 8 * q + (lane >> 2), c = (lane & 3) * 8;
        const uint16_t *from = base + p.at + r * p.ld + c;
        if (HOW == kWholePatch) return *reinterpret_cast<const uint4 *>(from);
        if (r >= p.rows || c >= p.cols) return make_uint4(0, 0, 0, 0);
        if (p.cols - c >= 8) return *reinterpret_cast<const uint4 *>(from);
#pragma unroll
        for (uint32_t k = 0; k < 8; ++k) w[k] = k < p.cols - c ? from[k] : 0u;
    }
    return make_uint4(w[0] | w[1] << 16, w[2] | w[3] << 16, w[4] | w[5] << 16, w[6] | w[7] << 16);
}
template <int HOW>
__device__ __forceinline__ void store8(uint16_t *base, const Patch &p, uint4 v, uint32_t q)
{
    const uint32_t lane = threadIdx.x & 31;
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    if (HOW == kSingles) {
        if (lane >= p.cols) return;
        uint16_t *to = base + p.at + 8 * q * p.ld + lane;
#pragma unroll
        for (uint32_t k = 0; k < 8; ++k)
            if (8 * q + k < p.rows) to[k * p.ld] = (uint16_t)(w[k / 2] >> (k & 1 ? 16 : 0));
    } else {
        const uint32_t r = 8 * q + (lane >> 2), c = (lane & 3) * 8;
        uint16_t *to = base + p.at + r * p.ld + c;
        if (HOW == kEdgePatch) {
            if (r >= p.rows || c >= p.cols) return;
            if (p.cols - c < 8) {
#pragma unroll
                for (uint32_t k = 0; k < 8; ++k)
                    if (k < p.cols - c) to[k] = (uint16_t)(w[k / 2] >> (k & 1 ? 16 : 0));
                return;
            }
        }
        *reinterpret_cast<uint4 *>(to) = v;
    }
}
__device__ __forceinline__ uint4 pack8(const float v[8])
{
    return make_uint4(ptx::pack2(v[0], v[1]), ptx::pack2(v[2], v[3]), ptx::pack2(v[4], v[5]), ptx::pack2(v[6], v[7]));
}

// Results that are bf16 already when they leave their row: 32 rows of 64
// bytes, in 2 KB.  Row r keeps its pieces exchanged by (r / 2) % 4.
__device__ __forceinline__ uint32_t narrow_at(uint32_t mem, uint32_t row, uint32_t piece)
{
    return mem + row * 64 + ((piece ^ ((row >> 1) & 3u)) * 16);
}
__device__ __forceinline__ void put_narrow(uint32_t mem, const float x[32])
{
    const uint32_t lane = threadIdx.x & 31;
#pragma unroll
    for (uint32_t j = 0; j < 4; ++j) tc::st_shared(narrow_at(mem, lane, j), pack8(x + 8 * j));
}
template <int HOW>
__device__ __forceinline__ uint4 get_narrow(uint32_t mem, uint32_t q)
{
    const uint32_t lane = threadIdx.x & 31;
    if (HOW != kSingles) return tc::ld_shared(narrow_at(mem, 8 * q + (lane >> 2), lane & 3));
    uint32_t w[8];
#pragma unroll
    for (uint32_t k = 0; k < 8; ++k) {
        uint16_t e;
        asm volatile("ld.shared.u16 %0, [%1];" : "=h"(e) : "r"(narrow_at(mem, 8 * q + k, lane >> 3) + (lane & 7) * 2) : "memory");
        w[k] = e;
    }
    return make_uint4(w[0] | w[1] << 16, w[2] | w[3] << 16, w[4] | w[5] << 16, w[6] | w[7] << 16);
}
template <int HOW>
__device__ __forceinline__ void write_narrow(uint16_t *base, const Patch &p, uint32_t mem)
{
#pragma unroll
    for (uint32_t q = 0; q < 4; ++q) store8<HOW>(base, p, get_narrow<HOW>(mem, q), q);
}

// Per pair: one thread of each block loads operands (TMA), one thread of the
// first issues the products, eight or sixteen warps of each block take its 128 rows of a
// finished tile out of one accumulator while the other fills.
template <int MODE, int WARPS>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(Gemm<WARPS>::kThreads, 1)
    zero1_ffn_gemm_kernel(const __grid_constant__ FfnParams p)
{
    constexpr int kStages = Gemm<WARPS>::kStages;
    extern __shared__ unsigned char raw[];
    __shared__ GemmShared sh;
    const uint32_t ring = (tc::smem_u32(raw) + 1023u) & ~1023u;
    const int warp = threadIdx.x >> 5;
    const uint32_t rank = tc::cluster_rank();
    unsigned *errors = p.errors ? p.errors : &sh.errors;
    volatile int *abort = &sh.abort;

    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) ptx::mbar_init(&sh.full[i], 1), ptx::mbar_init(&sh.empty[i], 1);
        for (int i = 0; i < 2; ++i) ptx::mbar_init(&sh.acc_full[i], 1), ptx::mbar_init(&sh.acc_empty[i], 2 * WARPS);
        ptx::mbar_init(&sh.drain, 1);
        sh.abort = 0;
        sh.errors = 0;
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
    ptx::grid_dependency_wait();   // what the launch before wrote, and what it still reads
    const uint32_t items = p.items, pairs = gridDim.x / 2, pair = blockIdx.x / 2;

    if (threadIdx.x == 0) {
        // ---- loads
        uint32_t issued = 0;
        bool ok = !p.stall;
        for (uint32_t i = pair; ok && i < items; i += pairs) {
            const Item t = item_of<MODE>(p, i);
            const FfnJob &j = p.job[t.job];
            const bool a_mn = MODE == kFfnPlain && j.a_mn, b_mn = MODE == kFfnGated || (MODE == kFfnPlain && j.b_mn);
            const int row = (int)(t.row + rank * 128);
            const int col = (int)(t.col + (MODE == kFfnGated ? 0 : rank * 128));
            for (uint32_t s = t.begin; s < t.end; ++s) {
                const uint32_t stage = issued % kStages;
                if (issued >= kStages) ok = tc::pair_wait(&sh.empty[stage], (issued / kStages - 1) & 1u, abort, errors);
                if (!ok) break;
                const uint32_t seg = s >= j.steps;
                const int k = (int)((s - seg * j.steps) * kFfnStep);
                const CUtensorMap *ma = &j.a[seg], *mb = &j.b[MODE == kFfnGated ? rank : seg];
                if (rank == 0) ptx::mbar_arrive_expect_tx(&sh.full[stage], 2 * kStageBytes);
                const uint32_t bar = tc::map_to(tc::smem_u32(&sh.full[stage]), 0), dst = ring + stage * kStageBytes;
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    const int r = row + 64 * b, c = col + 64 * b;
                    tc::tma_box_pair(dst + b * kBox, ma, a_mn ? r : k, a_mn ? k : r, 0, bar);
                    tc::tma_box_pair(dst + (2 + b) * kBox, mb, b_mn ? c : k, b_mn ? k : c, 0, bar);
                }
                ++issued;
            }
        }
        if (*abort && rank == 0) ptx::drain_loads<kStages>(sh.full, issued);
    } else if (threadIdx.x == 32 && rank == 0) {
        // ---- products
        uint32_t taken = 0, used = 0;   // stages, accumulators
        bool ok = true;
        for (uint32_t i = pair; ok && i < items; i += pairs, ++used) {
            const Item t = item_of<MODE>(p, i);
            const FfnJob &j = p.job[t.job];
            const bool a_mn = MODE == kFfnPlain && j.a_mn, b_mn = MODE == kFfnGated || (MODE == kFfnPlain && j.b_mn);
            const uint64_t a_step = tc::k16_step(a_mn), b_step = tc::k16_step(b_mn);
            const uint32_t idesc = bf16_desc(a_mn, b_mn);
            const uint32_t acc = used & 1, d = tmem + acc * kFfnTile;
            if (used >= 2) {
                if (!(ok = tc::pair_wait(&sh.acc_empty[acc], (used / 2 - 1) & 1u, abort, errors))) break;
                tc::fence_after_sync();
            }
            for (uint32_t s = t.begin; s < t.end; ++s) {
                const uint32_t stage = taken % kStages;
                if (!(ok = tc::pair_wait(&sh.full[stage], (taken / kStages) & 1u, abort, errors))) break;
                tc::fence_after_sync();
                const uint32_t src = ring + stage * kStageBytes;
                const uint64_t a = tc::smem_desc(src, a_mn), b = tc::smem_desc(src + 2 * kBox, b_mn);
#pragma unroll
                for (uint32_t q = 0; q < kFfnStep / 16; ++q)
                    tc::mma_f16(d, a + q * a_step, b + q * b_step, idesc, s > t.begin || q > 0);
                tc::mma_commit(&sh.empty[stage]);
                ++taken;
            }
            if (!ok) break;
            tc::mma_commit(&sh.acc_full[acc]);
        }
        if (!ok) {   // let the products in flight end before the operands and TMEM go
            tc::mma_commit(&sh.drain);
            const unsigned long long t0 = ptx::global_ns();
            while (!ptx::mbar_test(&sh.drain, 0) && ptx::global_ns() - t0 < ptx::kWaitLimitNs) {
            }
        }
    } else if (warp >= 2) {
        // ---- finished tiles: this block's 128 rows; each group of four warps its part of the columns
        const uint32_t group = (uint32_t)(warp - 2) >> 2, quarter = (uint32_t)warp & 3, lane = threadIdx.x & 31;
        const uint32_t mem = ring + kStages * kStageBytes + (uint32_t)(warp - 2) * kWarpTurn;
        constexpr uint32_t kCols = (MODE == kFfnGated ? 128 : 256) / (WARPS / 4);   // columns of a group
        const uint32_t at = tmem + (quarter << 21) + group * kCols;
        uint32_t used = 0;
        uint4 in[2][MODE == kFfnSlope ? 4 : 1];   // slope: gate and up of the 32 columns to come
        for (uint32_t i = pair; i < items; i += pairs, ++used) {
            const Item t = item_of<MODE>(p, i);
            const FfnJob &j = p.job[t.job];
            const uint32_t acc = used & 1, row = t.row + rank * 128 + quarter * 32, col = t.col + group * kCols;
            const bool vec = j.vec_out && (MODE != kFfnSlope || j.vec_in);
            const auto patch = [&](uint32_t c, uint64_t ld) {
                return Patch{(uint64_t)row * ld + col + c, ld, row < j.m ? min(32u, j.m - row) : 0,
                             col + c < j.n ? min(32u, j.n - col - c) : 0};
            };
            if (MODE == kFfnSlope && used == 0) {
                const Patch from = patch(0, j.ld_in);
#pragma unroll
                for (uint32_t q = 0; q < 4; ++q) {
                    in[0][q] = vec ? load8<kEdgePatch>(j.in[0], from, q) : load8<kSingles>(j.in[0], from, q);
                    in[1][q] = vec ? load8<kEdgePatch>(j.in[1], from, q) : load8<kSingles>(j.in[1], from, q);
                }
            }
            if (!__all_sync(~0u, tc::pair_wait(&sh.acc_full[acc], (used >> 1) & 1u, abort, errors))) break;
            tc::fence_after_sync();
#pragma unroll 1
            for (uint32_t c = 0; c < kCols; c += 32) {
                float x[32], y[MODE == kFfnGated ? 32 : 1];
                tmem_load32(x, at + acc * kFfnTile + c);
                if constexpr (MODE == kFfnGated) tmem_load32(y, at + acc * kFfnTile + 128 + c);
                if (c + 32 == kCols) {   // the accumulator may be written again
                    tc::fence_before_sync();
                    __syncwarp();
                    if (lane == 0) tc::arrive_cluster_relaxed(tc::map_to(tc::smem_u32(&sh.acc_empty[acc]), 0));
                }
                const Patch to = patch(c, j.ld_out);
                const int how = !vec ? kSingles : to.rows == 32 && to.cols == 32 ? kWholePatch : kEdgePatch;
                const auto by_access = [&](auto f) {
                    if (how == kWholePatch) f(ActOf<kWholePatch>{});
                    else if (how == kEdgePatch) f(ActOf<kEdgePatch>{});
                    else f(ActOf<kSingles>{});
                };
                if constexpr (MODE == kFfnPlain) {
                    if (j.slices > 1) {
                        put_rows(mem, x);
                        float *sums = p.partials + (uint64_t)t.partial * (kFfnTile * kFfnTile) + (row - t.row) * kFfnTile + (col - t.col) + c +
                                      (lane >> 2) * kFfnTile + (lane & 3) * 8;
#pragma unroll
                        for (uint32_t q = 0; q < 4; ++q) {
                            float v[8];
                            get8<kWholePatch>(v, mem, q);
                            *reinterpret_cast<float4 *>(sums + 8 * q * kFfnTile) = make_float4(v[0], v[1], v[2], v[3]);
                            *reinterpret_cast<float4 *>(sums + 8 * q * kFfnTile + 4) = make_float4(v[4], v[5], v[6], v[7]);
                        }
                    } else {
                        put_narrow(mem, x);
                        __syncwarp();
                        by_access([&](auto h) { write_narrow<decltype(h)::value>(j.out[0], to, mem); });
                    }
                } else if constexpr (MODE == kFfnGated) {
                    const uint32_t second = mem + kWarpTurn / 2;
                    if (j.out[1]) {
                        put_narrow(mem, x);
                        put_narrow(second, y);
                        __syncwarp();
                        by_access([&](auto h) {
                            write_narrow<decltype(h)::value>(j.out[1], to, mem);
                            write_narrow<decltype(h)::value>(j.out[2], to, second);
                        });
                        __syncwarp();
                    }
                    with_activation(p.act, [&](auto act) {
#pragma unroll
                        for (int k = 0; k < 32; ++k) {
                            float a, none;
                            activate<decltype(act)::value, false>(x[k], a, none);
                            x[k] = a * y[k];
                        }
                    });
                    put_narrow(mem, x);
                    __syncwarp();
                    by_access([&](auto h) { write_narrow<decltype(h)::value>(j.out[0], to, mem); });
                    if (j.copy) {   // of aligned rows
                        const Patch again = patch(c, j.ld_copy);
                        write_narrow<kEdgePatch>(j.copy, again, mem);
                    }
                } else {
                    // gate and up of the warp's next 32 columns are fetched as these are used
                    put_rows(mem, x);
                    Patch next = patch(c + 32, j.ld_in);
                    bool more = c + 32 < kCols;
                    if (!more && i + pairs < items) {
                        const Item then = item_of<MODE>(p, i + pairs);
                        const uint32_t r = then.row + rank * 128 + quarter * 32, cc = then.col + group * kCols;
                        next = Patch{(uint64_t)r * j.ld_in + cc, j.ld_in, r < j.m ? min(32u, j.m - r) : 0, cc < j.n ? min(32u, j.n - cc) : 0};
                        more = true;
                    }
                    const bool next_whole = next.rows == 32 && next.cols == 32;
                    by_access([&](auto h) {
                        constexpr int HOW = decltype(h)::value;
                        with_activation(p.act, [&](auto act) {
#pragma unroll
                            for (uint32_t q = 0; q < 4; ++q) {
                                float v[8], g[8], u[8];
                                get8<HOW>(v, mem, q);
                                ptx::set_widened(g, in[0][q]);
                                ptx::set_widened(u, in[1][q]);
                                if (more) {
                                    if (HOW != kSingles && next_whole) {
                                        in[0][q] = load8<kWholePatch>(j.in[0], next, q);
                                        in[1][q] = load8<kWholePatch>(j.in[1], next, q);
                                    } else {
                                        in[0][q] = load8<HOW == kSingles ? kSingles : kEdgePatch>(j.in[0], next, q);
                                        in[1][q] = load8<HOW == kSingles ? kSingles : kEdgePatch>(j.in[1], next, q);
                                    }
                                }
#pragma unroll
                                for (int k = 0; k < 8; ++k) {
                                    float a, slope;
                                    activate<decltype(act)::value, true>(g[k], a, slope);
                                    g[k] = v[k] * u[k] * slope;
                                    u[k] = v[k] * a;
                                }
                                store8<HOW>(j.out[0], to, pack8(g), q);
                                store8<HOW>(j.out[1], to, pack8(u), q);
                            }
                        });
                    });
                }
                __syncwarp();
            }
        }
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

// The slices' partial sums, added in order: one warp a row of a tile.
__global__ void __launch_bounds__(256) zero1_ffn_join_kernel(const __grid_constant__ FfnParams p)
{
    ptx::launch_dependents();
    ptx::grid_dependency_wait();
    const uint32_t tile = blockIdx.x / (kFfnTile / 8), lane = threadIdx.x & 31;
    uint32_t job = 0;   // the last that begins here and has something to join
    for (uint32_t k = 1; k < p.jobs; ++k)
        if (p.job[k].slices > 1 && (tile >= p.job[k].joins || p.job[job].slices == 1)) job = k;
    const FfnJob &j = p.job[job];
    const Item t = item_of<kFfnPlain>(p, j.first + (tile - j.joins) * j.slices);
    const uint32_t r = blockIdx.x % (kFfnTile / 8) * 8 + (threadIdx.x >> 5), row = t.row + r, col = t.col + lane * 8;
    if (row >= j.m || col >= j.n) return;
    float v[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = 0.f;
    const float *src = p.partials + (uint64_t)t.partial * (kFfnTile * kFfnTile) + r * kFfnTile + lane * 8;
#pragma unroll 4
    for (uint32_t s = 0; s < j.slices; ++s, src += kFfnTile * kFfnTile) {
        const float4 a = reinterpret_cast<const float4 *>(src)[0], b = reinterpret_cast<const float4 *>(src)[1];
        v[0] += a.x, v[1] += a.y, v[2] += a.z, v[3] += a.w, v[4] += b.x, v[5] += b.y, v[6] += b.z, v[7] += b.w;
    }
    uint16_t *to = j.out[0] + (uint64_t)row * j.ld_out + col;
    if (j.vec_out && j.n - col >= 8) {
        *reinterpret_cast<uint4 *>(to) =
            make_uint4(ptx::pack2(v[0], v[1]), ptx::pack2(v[2], v[3]), ptx::pack2(v[4], v[5]), ptx::pack2(v[6], v[7]));
    } else {
#pragma unroll
        for (uint32_t k = 0; k < 8; ++k)
            if (k < j.n - col) to[k] = __bfloat16_as_ushort(__float2bfloat16_rn(v[k]));
    }
}

template <int MODE, int WARPS>
cudaError_t gemm_t(const FfnParams &p, uint32_t pairs, cudaStream_t stream)
{
    using S = Gemm<WARPS>;
    const auto kernel = zero1_ffn_gemm_kernel<MODE, WARPS>;
    cudaError_t e = allow_dynamic_smem(reinterpret_cast<const void *>(kernel), S::kSmem);
    if (e != cudaSuccess) return e;
    const dim3 grid(2 * (p.items < pairs ? p.items : pairs));
    // after another kernel of the same call it may begin while that one ends
    e = p.follows ? launch_early(kernel, grid, S::kThreads, S::kSmem, stream, p)
                  : launch(kernel, grid, S::kThreads, S::kSmem, stream, p);
    if (e == cudaSuccess && p.joins)
        e = launch_early(zero1_ffn_join_kernel, dim3(p.joins * (kFfnTile / 8)), 256, 0, stream, p);
    return e;
}

template <int MODE>
cudaError_t gemm(const FfnParams &p, int sms, cudaStream_t stream)
{
    const uint32_t pairs = (uint32_t)sms / 2;
    return p.items <= pairs ? gemm_t<MODE, 16>(p, pairs, stream) : gemm_t<MODE, 8>(p, pairs, stream);
}

}  // namespace

cudaError_t launch_ffn_gated(const FfnParams &p, int sms, cudaStream_t stream) { return gemm<kFfnGated>(p, sms, stream); }

cudaError_t launch_ffn_slope(const FfnParams &p, int sms, cudaStream_t stream) { return gemm<kFfnSlope>(p, sms, stream); }

cudaError_t launch_ffn_plain(const FfnParams &p, int sms, cudaStream_t stream) { return gemm<kFfnPlain>(p, sms, stream); }

}  // namespace zero1
