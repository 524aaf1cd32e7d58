// zero1_ffn_thin.cu -- the gated feed-forward block's forward pass for at most
// 128 rows (tokens being generated, short prompts), which is bound by reading
// the weights once.
//
//   first:  h^T = act(Wg^T x^T) * (Wu^T x^T),   second: y^T = Wd^T h^T.
//
// The weights are the products' wide operand, 128 of their columns to a block,
// and the rows of x the narrow one (16, 32, 64 or 128).  A cluster of blocks
// shares 128 columns and splits K; sums meet in distributed shared memory and
// are added in block order.  Loads (TMA) keep 100 to 200 KB an SM in flight.
// The second launch begins while the first still runs, and fetches weights
// until it needs h.  Of 16 rows and fewer, h goes on as two bf16 parts, high
// and low, whose products are added: y then has no rounding of h in it.  (The
// narrow operand is free: one more product of the same weights.)
//
// Measured at 4096 x 11008 (271 MB of weights): one row 45 us (6.0 TB/s), 8 rows
// 47, 16 49, 32 57, 128 69 (the narrow operand is read again by every block);
// at 8192 x 28672 one row 215 us (6.5 TB/s).  768 x 2048: 10 us, all latency.
// Multiplying on the CUDA cores, weights from registers, took 69 us for one
// row and 169 for eight.
#include "zero1_ffn.h"
#include "zero1_ffn_device.cuh"
#include "zero1_internal.h"
#include "zero1_launch.h"
#include "zero1_tc.cuh"

namespace zero1 {
namespace {

constexpr uint32_t kBox = 8192;                // 64 x 64 bf16 of the weights
constexpr int kThinThreads = 192;              // loads, products, 4 warps that take sums out

constexpr uint32_t kMostStages = 10;

template <int N, bool GATED>
struct Thin {
    static constexpr uint32_t kParts = !GATED && N == 16 ? 2 : 1;         // of h
    static constexpr uint32_t kMats = GATED ? 2 : 1;
    static constexpr uint32_t kNarrow = N * 128;                          // bytes of one narrow box
    static constexpr uint32_t kStageBytes = kMats * 2 * kBox + kParts * kNarrow;   // 64 of K
    // 16 rows: two blocks an SM, one of which loads while the other begins or ends
    static constexpr uint32_t kFit = (N == 16 ? 104 : 200) * 1024 / kStageBytes;
    static constexpr uint32_t kStages = kFit < kMostStages ? kFit : kMostStages;
    static constexpr uint32_t kSums = GATED ? 2 * N : kParts * N;         // columns of fp32 sums
    static constexpr int kSmem = kStages * kStageBytes + 1024;
    static_assert(kSums * 128 * 4 <= kStages * kStageBytes, "sums lie where the operands were");
    static_assert(kSums >= 32 && (kSums & (kSums - 1)) == 0, "tensor memory is taken by powers of two");
};

struct ThinShared {
    uint64_t full[kMostStages], empty[kMostStages], done;
    uint32_t tmem;
    int abort;
    unsigned errors;
};

struct ThinParams {
    CUtensorMap wide[2], narrow;
    uint16_t *out[3];                          // h, gate, up (the last two may be null), or y
    uint16_t *part;                            // first: high parts of h, then `plane` entries further the low ones
    uint64_t ld_out, ld_part, plane;
    uint32_t rows, n, steps;                   // rows of x, columns of the result, 64s of K
    int act, stall, vec;                       // vec: rows of the outputs start at 8 bytes
    unsigned *errors;                          // may be null
};

// Box of a 3-D tensor map into this block's shared memory.
__device__ __forceinline__ void tma_box(uint32_t dst, const CUtensorMap *map, int x, int y, int z, uint64_t *bar)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(z), "r"(tc::smem_u32(bar))
        : "memory");
}

__device__ __forceinline__ float4 ld_cluster(uint32_t local, uint32_t rank)
{
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(tc::map_to(local, rank)));
    return v;
}
// The blocks' sums of four neighbouring columns, added in block order; their
// loads are in flight together.
__device__ __forceinline__ void sum_cluster(float out[4], uint32_t local, uint32_t ranks)
{
    float4 v[8];
#pragma unroll
    for (uint32_t i = 0; i < 8; ++i)
        if (i < ranks) v[i] = ld_cluster(local, i);
    out[0] = out[1] = out[2] = out[3] = 0.f;
#pragma unroll
    for (uint32_t i = 0; i < 8; ++i)
        if (i < ranks) out[0] += v[i].x, out[1] += v[i].y, out[2] += v[i].z, out[3] += v[i].w;
}
// Four neighbouring entries of a row, `left` of them inside the matrix.
__device__ __forceinline__ void store4(uint16_t *p, const float v[4], uint32_t left, bool vec)
{
    if (vec && left >= 4) {
        *reinterpret_cast<uint2 *>(p) = make_uint2(ptx::pack2(v[0], v[1]), ptx::pack2(v[2], v[3]));
    } else {
#pragma unroll
        for (uint32_t k = 0; k < 4; ++k)
            if (k < left) p[k] = __bfloat16_as_ushort(__float2bfloat16_rn(v[k]));
    }
}

template <int N, bool GATED>
__global__ void __launch_bounds__(kThinThreads) zero1_ffn_thin_kernel(const __grid_constant__ ThinParams p)
{
    using S = Thin<N, GATED>;
    extern __shared__ unsigned char raw[];
    __shared__ ThinShared sh;
    const uint32_t ring = (tc::smem_u32(raw) + 1023u) & ~1023u;
    const int warp = threadIdx.x >> 5;
    uint32_t ranks;
    asm volatile("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(ranks));
    const uint32_t rank = tc::cluster_rank();
    unsigned *errors = p.errors ? p.errors : &sh.errors;
    volatile int *abort = &sh.abort;
    ptx::launch_dependents();
    if (threadIdx.x == 0) {
        for (uint32_t i = 0; i < S::kStages; ++i) ptx::mbar_init(&sh.full[i], 1), ptx::mbar_init(&sh.empty[i], 1);
        ptx::mbar_init(&sh.done, 1);
        sh.abort = 0;
        sh.errors = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        tc::prefetch_map(&p.wide[0]);
        tc::prefetch_map(&p.narrow);
    }
    if (warp == 1) {
        __syncwarp();
        tc::tmem_alloc1(&sh.tmem, S::kSums);
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = sh.tmem, col0 = blockIdx.x / ranks * 128;
    const uint32_t begin = (uint32_t)((uint64_t)p.steps * rank / ranks), end = (uint32_t)((uint64_t)p.steps * (rank + 1) / ranks);

    if (threadIdx.x == 0 && p.stall) {
        ptx::grid_dependency_wait();   // a launch does not end before the one it began beside
    } else if (threadIdx.x == 0) {
        // ---- loads
        const auto wide = [&](uint32_t s, uint32_t stage) {
            ptx::mbar_arrive_expect_tx(&sh.full[stage], S::kStageBytes);
            const uint32_t dst = ring + stage * S::kStageBytes;
#pragma unroll
            for (uint32_t i = 0; i < 2 * S::kMats; ++i)
                tma_box(dst + i * kBox, &p.wide[i >> 1], (int)(col0 + 64 * (i & 1)), (int)(s * 64), 0, &sh.full[stage]);
        };
        const auto narrow = [&](uint32_t s, uint32_t stage) {
            const uint32_t dst = ring + stage * S::kStageBytes + 2 * S::kMats * kBox;
#pragma unroll
            for (uint32_t i = 0; i < S::kParts; ++i)
                tma_box(dst + i * S::kNarrow, &p.narrow, (int)(s * 64), 0, (int)i, &sh.full[stage]);
        };
        const uint32_t first = min(end, begin + S::kStages);
        for (uint32_t s = begin; s < first; ++s) wide(s, s - begin);
        if (!GATED) ptx::grid_dependency_wait();   // for h
        tc::fence_proxy_async_all();
        for (uint32_t s = begin; s < first; ++s) narrow(s, s - begin);
        for (uint32_t s = first; s < end; ++s) {
            const uint32_t i = s - begin, stage = i % S::kStages;
            if (!ptx::mbar_wait(&sh.empty[stage], (i / S::kStages - 1) & 1u, abort, errors)) break;
            wide(s, stage);
            narrow(s, stage);
        }
    } else if (threadIdx.x == 32) {
        // ---- products
        const uint32_t idesc = tc::instr_desc(128, N * S::kParts, true, false) | (1u << 7) | (1u << 10);   // bf16
        bool ok = true;
        for (uint32_t s = begin; s < end; ++s) {
            const uint32_t i = s - begin, stage = i % S::kStages;
            if (!(ok = ptx::mbar_wait(&sh.full[stage], (i / S::kStages) & 1u, abort, errors))) break;
            tc::fence_after_sync();
            const uint32_t src = ring + stage * S::kStageBytes;
            const uint64_t b = tc::smem_desc(src + 2 * S::kMats * kBox, false);
#pragma unroll
            for (uint32_t m = 0; m < S::kMats; ++m) {
                const uint64_t a = tc::smem_desc(src + m * 2 * kBox, true);
#pragma unroll
                for (uint32_t q = 0; q < 4; ++q)
                    tc::mma1_f16(tmem + m * N, a + q * (2048 >> 4), b + q * (32 >> 4), idesc, i > 0 || q > 0);
            }
            tc::mma1_commit(&sh.empty[stage]);
        }
        tc::mma1_commit(&sh.done);
        if (!ok) {   // let the products in flight end
            const unsigned long long t0 = ptx::global_ns();
            while (!ptx::mbar_test(&sh.done, 0) && ptx::global_ns() - t0 < ptx::kWaitLimitNs) {
            }
        }
    } else if (warp >= 2) {
        // ---- this block's sums, to shared memory: one row of it a column of the narrow operand
        if (__all_sync(~0u, ptx::mbar_wait(&sh.done, 0, abort, errors)) && !*abort) {
            tc::fence_after_sync();
            const uint32_t quarter = (uint32_t)warp & 3, lane = quarter * 32 + (threadIdx.x & 31);
#pragma unroll 2
            for (uint32_t c = 0; c < S::kSums; c += 16) {
                float v[16];
                tc::tmem_load16(v, tmem + (quarter << 21) + c);
#pragma unroll
                for (uint32_t j = 0; j < 16; ++j)
                    asm volatile("st.shared.f32 [%0], %1;" ::"r"(ring + ((c + j) * 128 + lane) * 4), "f"(v[j]) : "memory");
            }
            tc::fence_before_sync();
        }
    }
    if (*abort) {   // give copies that nothing above waits for 1 ms to land
        const unsigned long long t0 = ptx::global_ns();
        while (ptx::global_ns() - t0 < 1000000ull) {
        }
    }
    __syncwarp();
    __syncthreads();
    ptx::cluster_sync();
    tc::fence_after_sync();
    if (warp == 1) tc::tmem_free1(tmem, S::kSums);
    for (uint32_t o = threadIdx.x + kThinThreads * rank; o < p.rows * 32; o += kThinThreads * ranks) {
        const uint32_t r = o / 32, c = col0 + o % 32 * 4;
        if (c >= p.n) continue;
        const uint32_t left = p.n - c;
        float a[4], b[4];
        sum_cluster(a, ring + o * 16, ranks);
        if (GATED || S::kParts == 2) sum_cluster(b, ring + (N * 32 + o) * 16, ranks);
        const uint64_t at = (uint64_t)r * p.ld_out + c;
        if (GATED) {
            if (p.out[1]) {
                store4(p.out[1] + at, a, left, p.vec);
                store4(p.out[2] + at, b, left, p.vec);
            }
            float rest[4];
            with_activation(p.act, [&](auto act) {
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    float v, none;
                    activate<decltype(act)::value, false>(a[k], v, none);
                    a[k] = v * b[k];
                    rest[k] = a[k] - __bfloat162float(__float2bfloat16_rn(a[k]));
                    if (!isfinite(rest[k])) rest[k] = 0.f;   // an infinite h has no low part
                }
            });
            uint16_t *to = p.part + (uint64_t)r * p.ld_part + c;   // padded to 8 entries
            store4(to, a, left, true);
            if (N == 16) store4(to + p.plane, rest, left, true);
        } else if (S::kParts == 2) {
#pragma unroll
            for (int k = 0; k < 4; ++k) a[k] += b[k];
        }
        store4(p.out[0] + at, a, left, p.vec);
    }
    ptx::cluster_sync();   // no block's sums go while another reads them
}

// Blocks that share a tile's K: 1 to 8, each at least one stage, where the
// rounds that all blocks take together cost least: a round is the stages of
// one block and about `extra` stages' time of starting and joining.
uint32_t ranks_of(uint32_t tiles, uint32_t steps, uint32_t slots, uint32_t extra)
{
    uint32_t best = 1;
    uint64_t least = ~0ull;
    for (uint32_t c = 1; c <= 8 && c <= steps; ++c) {
        const uint64_t cost = (uint64_t)((tiles * c + slots - 1) / slots) * ((steps + c - 1) / c + extra);
        if (cost < least) least = cost, best = c;
    }
    return best;
}

// Whether a stream may use a part of the SMs only (zero1_sm_partition): then a
// cluster has to be asked for, which takes 2 us of a call that takes 10.
bool partitioned(cudaStream_t stream)
{
    typedef CUresult (*Fn)(CUstream, CUgreenCtx *);
    static const Fn fn = [] {
        void *f = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuStreamGetGreenCtx", &f, 12040, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            f = nullptr;
        return reinterpret_cast<Fn>(f);
    }();
    CUgreenCtx part = nullptr;
    return !fn || fn(reinterpret_cast<CUstream>(stream), &part) != CUDA_SUCCESS || part != nullptr;
}

template <int N, bool GATED>
cudaError_t thin_t(ThinParams &p, int sms, bool part, cudaStream_t stream)
{
    using S = Thin<N, GATED>;
    const auto kernel = zero1_ffn_thin_kernel<N, GATED>;
    cudaError_t e = allow_dynamic_smem(reinterpret_cast<const void *>(kernel), S::kSmem);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr[2]{};
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.blockDim = dim3(kThinThreads);
    cfg.dynamicSmemBytes = S::kSmem;
    cfg.stream = stream;
    cfg.attrs = attr;
    const uint32_t tiles = (p.n + 127) / 128;
    for (uint32_t ranks = ranks_of(tiles, p.steps, (uint32_t)sms * (N == 16 ? 2 : 1), 12 / S::kMats);; --ranks) {
        attr[0].val.clusterDim.x = ranks;
        cfg.gridDim = dim3(tiles * ranks);
        cfg.numAttrs = 1;
        if (ranks == 1 || !part) break;
        int fit = 0;   // an SM partition may hold no cluster of this size
        e = cudaOccupancyMaxActiveClusters(&fit, kernel, &cfg);
        if (e != cudaSuccess) return e;
        if (fit > 0) break;
    }
    cfg.numAttrs = GATED ? 1 : 2;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

template <bool GATED>
cudaError_t thin(ThinParams &p, int sms, bool part, cudaStream_t stream)
{
    if (p.rows <= 16) return thin_t<16, GATED>(p, sms, part, stream);
    if (p.rows <= 32) return thin_t<32, GATED>(p, sms, part, stream);
    if (p.rows <= 64) return thin_t<64, GATED>(p, sms, part, stream);
    return thin_t<128, GATED>(p, sms, part, stream);
}

}  // namespace

cudaError_t launch_ffn_thin(const FfnThin &f, int sms, cudaStream_t stream)
{
    ThinParams p{};
    p.wide[0] = f.w_gate;
    p.wide[1] = f.w_up;
    p.narrow = f.x;
    for (int i = 0; i < 3; ++i) p.out[i] = f.out[i];
    p.part = f.part;
    p.ld_out = f.ldh;
    p.ld_part = f.ld_part;
    p.plane = f.plane;
    p.rows = f.rows;
    p.n = f.hidden;
    p.steps = (f.width + 63) / 64;
    p.act = f.act;
    p.vec = f.vec[0];
    p.stall = f.stall;
    p.errors = f.errors;
    const bool part = partitioned(stream);
    cudaError_t e = thin<true>(p, sms, part, stream);
    if (e != cudaSuccess) return e;
    p.wide[0] = f.w_down;
    p.narrow = f.h;
    p.out[0] = f.y;
    p.ld_out = f.ldy;
    p.vec = f.vec[1];
    p.n = f.width;
    p.steps = (f.hidden + 63) / 64;
    return thin<false>(p, sms, part, stream);
}

}  // namespace zero1
