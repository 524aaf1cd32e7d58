// zero1_muon_small.cu -- the whole matrix step of small matrices in one
// launch: the smaller side at most 128, the larger at most 256 for one block
// or 192 for each block of a cluster of up to 8.
//
// The iteration is that of zero1_muon_kernels.cu (X <- P X with P = a I +
// b A + c A A, A = X X^T, every operand as f16 hi + lo), but X never leaves
// the block: it lies in shared memory with its smaller side as rows (128 of
// them, zeros below), transposed on the way in and out where the matrix is
// tall.  Each block of a cluster holds a slice of the columns.  Per
// iteration a block forms its slice's part of A on the tensor cores, the
// cluster adds the parts up (each block 128/C rows, in rank order, handed
// back to all), and every block forms P and its slice of P X itself.
//
// Bound by latency: three dependent products with an exchange between tensor
// memory, registers and shared memory after each.  What it saves is the
// trip of every product through L2 and a counter (a tiled product takes 13 us
// and more from one to the next, one here 1.7), and the separate kernels for
// momentum, norm, split and update.  A 64 x 64 step at W = 4 takes 29 us (by
// the tiled kernels 97), alone 27 us.
#include "zero1_internal.h"
#include "zero1_muon.h"
#include "zero1_muon_device.cuh"
#include "zero1_tc.cuh"

namespace zero1 {
namespace {

constexpr int kThreads = 256;
constexpr uint32_t kBox = 16384;              // 128 rows x 64 f16, 128-byte swizzle
constexpr uint32_t kGramBytes = 4 * kBox;     // 128 x 128: two boxes, high and low parts (or fp32)
constexpr uint32_t kGramTmem = 256, kSumTmem = 0;

template <int CAP>
struct SmallParams {
    const uint16_t *grads[CAP];
    uint16_t *params[CAP];
    MuonDev d;
    const uint32_t *list;      // matrices of this launch
    float *master, *momentum;  // a step, or
    const void *in;            // the orthogonalisation alone
    void *out;
    int in_bf16, out_bf16;
    int world;
    MuonScalars sc;
};

// Byte address of 16 bytes (8 f16 columns) of a row in boxes of 64 columns.
__device__ __forceinline__ uint32_t f16_piece(uint32_t base, uint32_t row, uint32_t piece)
{
    return base + (piece >> 3) * kBox + row * 128 + (((piece & 7) ^ (row & 7)) * 16);
}

// Byte address of 16 bytes (4 fp32 columns) of a row of `quads` such.
__device__ __forceinline__ uint32_t f32_piece(uint32_t base, uint32_t row, uint32_t quad, uint32_t quads)
{
    return base + (row * quads + (quad ^ (row & 7))) * 16;
}

__device__ __forceinline__ float4 ld_f4(uint32_t addr)
{
    const uint4 v = tc::ld_shared(addr);
    return make_float4(__uint_as_float(v.x), __uint_as_float(v.y), __uint_as_float(v.z), __uint_as_float(v.w));
}

__device__ __forceinline__ uint4 as_u4(float a, float b, float c, float d)
{
    return make_uint4(__float_as_uint(a), __float_as_uint(b), __float_as_uint(c), __float_as_uint(d));
}

// One product into TMEM columns at `d`: K from k0 in steps of 16, operands at
// a and b (K-major, or b MN-major), high parts first, low parts at +plane.
// The small products go first: the tensor cores cut additions off by the
// size of the sum so far.
__device__ __forceinline__ void product(uint32_t d, uint32_t a, uint32_t a_plane, uint32_t b, uint32_t b_plane, bool b_mn,
                                        uint32_t k0, uint32_t k1, uint32_t n)
{
    const uint32_t idesc = tc::instr_desc(128, n, false, b_mn);
    const auto at_k = [](uint32_t base, uint32_t k) { return base + (k >> 6) * kBox + (k & 63) * 2; };
    for (int big = 0; big < 2; ++big)
        for (uint32_t k = k0; k < k1; k += 16) {
            const uint64_t ah = tc::smem_desc(at_k(a, k), false, kBox);
            const uint64_t bh = tc::smem_desc(b_mn ? b + k * 128 : at_k(b, k), b_mn, kBox);
            if (big) {
                tc::mma1_f16(d, ah, bh, idesc, true);
            } else {
                tc::mma1_f16(d, ah, bh + (b_plane >> 4), idesc, k > k0);
                tc::mma1_f16(d, ah + (a_plane >> 4), bh, idesc, true);
            }
        }
}

template <int CAP>
__global__ void __launch_bounds__(kThreads, 1) muon_small_kernel(const __grid_constant__ SmallParams<CAP> p)
{
    extern __shared__ unsigned char raw[];
    __shared__ double norms[8], part[kThreads / 32];
    __shared__ uint64_t done;
    __shared__ uint32_t tmem_slot;
    __shared__ int abort_flag;
    const uint32_t tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    uint32_t blocks, rank;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(blocks));
    rank = tc::cluster_rank();
    const MuonMat &m = p.d.mats[p.list[blockIdx.x / blocks]];
    const uint32_t s = m.s, l = m.tall ? m.rows : m.cols;
    const uint32_t width = (((l + blocks - 1) / blocks) + 63) & ~63u;      // this launch's slice, 64 to 256 columns
    const uint32_t j0 = rank * width, cols = j0 < l ? min(width, l - j0) : 0;
    const uint32_t x = (tc::smem_u32(raw) + 1023u) & ~1023u;
    const uint32_t x_plane = (width >> 6) * kBox, quads = width >> 2;
    const uint32_t gram = x + 2 * x_plane, parts = gram + kGramBytes;
    volatile int *abort = &abort_flag;
    unsigned *errors = p.d.errors;

    if (tid == 0) {
        ptx::mbar_init(&done, 1);
        abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 0) tc::tmem_alloc1(&tmem_slot, 512);

    // ---- the update U, fp32 in the place of X, and its sum of squares.  A
    // thread takes 8 columns of a row of X at a time: neighbours of a row of
    // a wide matrix (threads along the row), of a column of a tall one
    // (threads across it).
    const uint32_t pieces = width >> 3, total = 128 * pieces;
    const auto place = [&](uint32_t id, uint32_t &i, uint32_t &j) {
        if (m.tall) i = id & 127, j = (id >> 7) * 8;
        else i = id / pieces, j = (id % pieces) * 8;
    };
    const auto flat = [&](uint32_t i, uint32_t j) {
        return m.tall ? m.offset + (uint64_t)(j0 + j) * m.ld + i : m.offset + (uint64_t)i * m.ld + j0 + j;
    };
    const bool vec = m.vec && !m.tall;
    SquareSum ss;
    for (uint32_t id = tid; id < total; id += kThreads) {
        uint32_t i, j;
        place(id, i, j);
        float u[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) u[e] = 0.f;
        if (i < s && j < cols) {
            const uint64_t f = flat(i, j), next = m.tall ? m.ld : 1;
            const uint32_t n = min(8u, cols - j);
            if (p.momentum) {
                float mom[8];
                if (vec) {
                    load8(u, p.grads[0] + f);
                    for (int r = 1; r < p.world; ++r) {
                        float g[8];
                        load8(g, p.grads[r] + f);
#pragma unroll
                        for (int e = 0; e < 8; ++e) u[e] += g[e];
                    }
                    load8(mom, p.momentum + f);
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e) mom[e] = e < n ? p.momentum[f + e * next] : 0.f;
                    for (int r = 0; r < p.world; ++r)
#pragma unroll
                        for (int e = 0; e < 8; ++e) u[e] += e < n ? load1(p.grads[r] + f + e * next) : 0.f;
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) u[e] = look_ahead(p.sc, u[e], mom[e]);
                if (vec) {
                    store8(p.momentum + f, mom);
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        if (e < n) p.momentum[f + e * next] = mom[e];
                }
            } else if (vec) {
                if (p.in_bf16) load8(u, static_cast<const uint16_t *>(p.in) + f);
                else load8(u, static_cast<const float *>(p.in) + f);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (e < n)
                        u[e] = p.in_bf16 ? load1(static_cast<const uint16_t *>(p.in) + f + e * next)
                                         : static_cast<const float *>(p.in)[f + e * next];
            }
            ss.add(u);
        }
        tc::st_shared(f32_piece(x, i, j >> 2, quads), as_u4(u[0], u[1], u[2], u[3]));
        tc::st_shared(f32_piece(x, i, (j >> 2) + 1, quads), as_u4(u[4], u[5], u[6], u[7]));
    }
    {
        double t = ss.total();
        for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(~0u, t, o);
        if (lane == 0) part[warp] = t;
    }
    tc::fence_before_sync();
    __syncthreads();
    ptx::cluster_sync();          // every block of the cluster runs: its shared memory may be written
    tc::fence_after_sync();
    const uint32_t tmem = tmem_slot;
    if (tid < blocks) {
        double t = 0.0;
        for (int i = 0; i < kThreads / 32; ++i) t += part[i];
        ptx::st_cluster_f64(&norms[rank], tid, t);
    }
    ptx::cluster_sync();
    double sum = 0.0;
    for (uint32_t i = 0; i < blocks; ++i) sum += norms[i];
    const float scale = (float)((double)kXScale / (sqrt(sum) + (double)p.sc.eps));

    // ---- X = U / (|U| + eps) in two f16 parts, in the place of U: all reads, then all writes
    {
        float u[16][8];
#pragma unroll
        for (int q = 0; q < 16; ++q) {
            const uint32_t id = tid + q * kThreads, i = id / pieces, j = id % pieces;
            if (id < total) {
                const float4 a = ld_f4(f32_piece(x, i, 2 * j, quads)), b = ld_f4(f32_piece(x, i, 2 * j + 1, quads));
                u[q][0] = a.x, u[q][1] = a.y, u[q][2] = a.z, u[q][3] = a.w;
                u[q][4] = b.x, u[q][5] = b.y, u[q][6] = b.z, u[q][7] = b.w;
            }
        }
        __syncthreads();
#pragma unroll
        for (int q = 0; q < 16; ++q) {
            const uint32_t id = tid + q * kThreads, i = id / pieces, j = id % pieces;
            if (id < total) {
                uint4 h, lo;
                split(u[q][0] * scale, u[q][1] * scale, h.x, lo.x);
                split(u[q][2] * scale, u[q][3] * scale, h.y, lo.y);
                split(u[q][4] * scale, u[q][5] * scale, h.z, lo.z);
                split(u[q][6] * scale, u[q][7] * scale, h.w, lo.w);
                tc::st_shared(f16_piece(x, i, j), h);
                tc::st_shared(f16_piece(x + x_plane, i, j), lo);
            }
        }
    }

    // This thread's row of a product, and its share of the columns: every
    // other 16.  Rows and columns past those that are computed (n) are left
    // as they are: they only ever reach each other.
    const uint32_t r = (warp & 3) * 32 + lane, half = warp >> 2;
    const uint32_t lanes = (warp & 3) << 21;
    const uint32_t n = (s + 15) & ~15u;        // rows of X the products take
    const bool active = (warp & 3) * 32 < n;   // this warp's rows
    const auto unit = [&](int q) { return (2 * q + half) * 16; };   // its q-th 16 columns
    constexpr float inv = 1.0f / kGramScale;
    uint32_t waits = 0;
    // Shared memory written by this block's threads is ready for the products.
    const auto ready = [&]() {
        ptx::fence_proxy_async_smem();
        tc::fence_before_sync();
        __syncthreads();
        tc::fence_after_sync();
    };
    // The products issued so far are done.  A wait that gives up is reported and the rest runs on without meaning.
    const auto finished = [&]() {
        if (tid == 0) tc::mma1_commit(&done);
        ptx::mbar_wait(&done, waits++ & 1u, abort, errors);
        __syncwarp();
        tc::fence_after_sync();
    };

    for (int iter = 0; iter < p.sc.steps; ++iter) {
        const float alpha = alpha_of(iter, p.sc.steps);
        const float linear = p.sc.b + 2.f * p.sc.c * alpha, constant = p.sc.a + alpha * (p.sc.b + alpha * p.sc.c);
        float w[64];

        // A, this slice's part: sums of 128 of K each
        ready();
        if (tid == 0)
            for (uint32_t k = 0; k < width; k += 128)
                product(tmem + kSumTmem + k, x, x_plane, x, x_plane, false, k, min(width, k + 128), n);
        finished();
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            if (active && unit(q) < n) {
                tc::tmem_load16(w + 16 * q, tmem + kSumTmem + lanes + unit(q));
                if (width > 128) {
                    float v[16];
                    tc::tmem_load16(v, tmem + kSumTmem + 128 + lanes + unit(q));
#pragma unroll
                    for (int e = 0; e < 16; ++e) w[16 * q + e] += v[e];
                }
            }
        }
        if (blocks > 1) {
            // to the block that adds up this row: its parts[rank][row % strip][128]
            const uint32_t strip = 128 / blocks, owner = r / strip, row = r % strip;
            const uint32_t there = tc::map_to(parts, owner);
#pragma unroll
            for (int q = 0; q < 4; ++q)
                if (active && unit(q) < n)
#pragma unroll
                    for (uint32_t e = 0; e < 4; ++e) {
                        const float *t = w + 16 * q + 4 * e;
                        tc::st_cluster(f32_piece(there, rank * strip + row, unit(q) / 4 + e, 32), as_u4(t[0], t[1], t[2], t[3]));
                    }
            ptx::cluster_sync();
            // and the sums to all blocks, in the place of the Gram matrix
            const uint32_t quads_n = n >> 2;
            for (uint32_t id = tid; id < strip * quads_n; id += kThreads) {
                const uint32_t row = id / quads_n, quad = id % quads_n;
                if (rank * strip + row >= n) continue;
                float4 t = ld_f4(f32_piece(parts, row, quad, 32));
                for (uint32_t b = 1; b < blocks; ++b) {
                    const float4 v = ld_f4(f32_piece(parts, b * strip + row, quad, 32));
                    t.x += v.x, t.y += v.y, t.z += v.z, t.w += v.w;
                }
                for (uint32_t b = 0; b < blocks; ++b)
                    tc::st_cluster(f32_piece(tc::map_to(gram, b), rank * strip + row, quad, 32), as_u4(t.x, t.y, t.z, t.w));
            }
            ptx::cluster_sync();
#pragma unroll
            for (int q = 0; q < 4; ++q)
                if (active && unit(q) < n)
#pragma unroll
                    for (uint32_t e = 0; e < 4; ++e) {
                        const float4 t = ld_f4(f32_piece(gram, r, unit(q) / 4 + e, 32));
                        w[16 * q + 4 * e] = t.x, w[16 * q + 4 * e + 1] = t.y, w[16 * q + 4 * e + 2] = t.z, w[16 * q + 4 * e + 3] = t.w;
                    }
            __syncthreads();
        }
        const auto put_gram = [&](int q) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float *v = w + 16 * q + 8 * e;
                uint4 h, lo;
                split(v[0], v[1], h.x, lo.x);
                split(v[2], v[3], h.y, lo.y);
                split(v[4], v[5], h.z, lo.z);
                split(v[6], v[7], h.w, lo.w);
                tc::st_shared(f16_piece(gram, r, unit(q) / 8 + e), h);
                tc::st_shared(f16_piece(gram + 2 * kBox, r, unit(q) / 8 + e), lo);
            }
        };
#pragma unroll
        for (int q = 0; q < 4; ++q)
            if (active && unit(q) < n) {
#pragma unroll
                for (uint32_t e = 0; e < 16; ++e) w[16 * q + e] = w[16 * q + e] * (kGramScale / (kXScale * kXScale)) - (unit(q) + e == r ? alpha * kGramScale : 0.f);
                put_gram(q);
            }

        // P = c A' A' + (b + 2 c alpha) A' + (a + b alpha + c alpha^2) I, about A' = A - alpha I
        ready();
        if (tid == 0) product(tmem + kGramTmem, gram, 2 * kBox, gram, 2 * kBox, false, 0, n, n);
        finished();
#pragma unroll
        for (int q = 0; q < 4; ++q)
            if (active && unit(q) < n) {
                float v[16];
                tc::tmem_load16(v, tmem + kGramTmem + lanes + unit(q));
#pragma unroll
                for (uint32_t e = 0; e < 16; ++e)
                    w[16 * q + e] = p.sc.c * inv * v[e] + linear * w[16 * q + e] + (unit(q) + e == r ? constant * kGramScale : 0.f);
                put_gram(q);
            }

        // X <- P X, or on the last iteration the result in fp32
        ready();
        if (tid == 0) product(tmem + kSumTmem, gram, 2 * kBox, x, x_plane, true, 0, n, width);
        finished();
        const bool last = iter + 1 == p.sc.steps;
        for (uint32_t c = half * 16; active && c < width; c += 32) {
            float v[16];
            tc::tmem_load16(v, tmem + kSumTmem + lanes + c);
            if (last) {
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    tc::st_shared(f32_piece(x, r, (c >> 2) + q, quads),
                                  as_u4(v[4 * q] * (inv / kXScale), v[4 * q + 1] * (inv / kXScale),
                                        v[4 * q + 2] * (inv / kXScale), v[4 * q + 3] * (inv / kXScale)));
            } else {
                uint4 h[2], lo[2];
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const float *y = v + 8 * q;
                    split(y[0] * inv, y[1] * inv, h[q].x, lo[q].x);
                    split(y[2] * inv, y[3] * inv, h[q].y, lo[q].y);
                    split(y[4] * inv, y[5] * inv, h[q].z, lo[q].z);
                    split(y[6] * inv, y[7] * inv, h[q].w, lo[q].w);
                    tc::st_shared(f16_piece(x, r, (c >> 3) + q), h[q]);
                    tc::st_shared(f16_piece(x + x_plane, r, (c >> 3) + q), lo[q]);
                }
            }
        }
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    if (warp == 0) tc::tmem_free1(tmem, 512);

    // ---- the update of the master and the replicas, or the result itself
    const float move = p.sc.lr * m.scale;
    for (uint32_t id = tid; id < total; id += kThreads) {
        uint32_t i, j;
        place(id, i, j);
        if (i >= s || j >= cols) continue;
        const float4 a = ld_f4(f32_piece(x, i, j >> 2, quads)), b = ld_f4(f32_piece(x, i, (j >> 2) + 1, quads));
        const float o[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
        const uint64_t f = flat(i, j), next = m.tall ? m.ld : 1;
        const uint32_t n_here = min(8u, cols - j);
        if (p.master) {
            if (vec) {
                float v[8];
                load8(v, p.master + f);
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = v[e] * p.sc.decay - move * o[e];
                store8(p.master + f, v);
                for (int q = 0; q < p.world; ++q) store8(p.params[q] + f, v);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (e < n_here) {
                        const float v = p.master[f + e * next] * p.sc.decay - move * o[e];
                        p.master[f + e * next] = v;
                        for (int q = 0; q < p.world; ++q) store1(p.params[q] + f + e * next, v);
                    }
            }
        } else if (vec) {
            if (p.out_bf16) store8(static_cast<uint16_t *>(p.out) + f, o);
            else store8(static_cast<float *>(p.out) + f, o);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (e < n_here) {
                    if (p.out_bf16) store1(static_cast<uint16_t *>(p.out) + f + e * next, o[e]);
                    else static_cast<float *>(p.out)[f + e * next] = o[e];
                }
        }
    }
    // no block leaves while another may still write to it
    ptx::cluster_sync();
}

// How the matrices of clusters of 2^i blocks are launched; `attr` has to outlive the configuration.
cudaLaunchConfig_t small_config(const MuonSmall &small, int i, cudaStream_t stream, cudaLaunchAttribute *attr)
{
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(small.count[i] << i);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = (size_t)small_smem(1 << i);
    cfg.stream = stream;
    attr->id = cudaLaunchAttributeClusterDimension;
    attr->val.clusterDim.x = 1u << i;
    attr->val.clusterDim.y = attr->val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cfg;
}

template <int CAP>
cudaError_t allow_small_smem()
{
    return allow_dynamic_smem(reinterpret_cast<const void *>(muon_small_kernel<CAP>),
                              small_smem(1) > small_smem(2) ? small_smem(1) : small_smem(2));
}

template <int CAP>
cudaError_t launch_small(const SmallParams<CAP> &base, const MuonSmall &small, cudaStream_t stream)
{
    cudaError_t e = allow_small_smem<CAP>();
    for (int i = 0; i < kSmallSizes && e == cudaSuccess; ++i) {
        if (small.count[i] == 0) continue;
        SmallParams<CAP> p = base;
        p.list = small.list + small.first[i];
        cudaLaunchAttribute attr{};
        const cudaLaunchConfig_t cfg = small_config(small, i, stream, &attr);
        e = cudaLaunchKernelEx(&cfg, muon_small_kernel<CAP>, p);
    }
    return e;
}

template <int CAP>
cudaError_t step_t(const MuonDev &d, const MuonSmall &small, const MuonScalars &sc, const void *const *grads,
                   void *const *params, int world, float *master, float *momentum, cudaStream_t stream)
{
    SmallParams<CAP> p{};
    for (int r = 0; r < world; ++r) {
        p.grads[r] = static_cast<const uint16_t *>(grads[r]);
        p.params[r] = static_cast<uint16_t *>(params[r]);
    }
    p.d = d;
    p.master = master;
    p.momentum = momentum;
    p.world = world;
    p.sc = sc;
    return launch_small<CAP>(p, small, stream);
}

}  // namespace

// 1 us a cluster size in use.  Shared memory decides, the same for every CAP.
cudaError_t muon_small_misfit(const MuonSmall &small, cudaStream_t stream, int *blocks)
{
    *blocks = 0;
    cudaError_t e = allow_small_smem<8>();
    for (int i = 1; i < kSmallSizes && e == cudaSuccess && *blocks == 0; ++i) {
        if (small.count[i] == 0) continue;
        cudaLaunchAttribute attr{};
        const cudaLaunchConfig_t cfg = small_config(small, i, stream, &attr);
        int fit = 0;
        e = cudaOccupancyMaxActiveClusters(&fit, muon_small_kernel<8>, &cfg);
        if (e == cudaSuccess && fit < 1) *blocks = 1 << i;
    }
    return e;
}

cudaError_t launch_muon_small_step(const MuonDev &d, const MuonSmall &small, const MuonScalars &sc,
                                   const void *const *grads, void *const *params, int world, float *master,
                                   float *momentum, cudaStream_t stream)
{
    if (world <= 8) return step_t<8>(d, small, sc, grads, params, world, master, momentum, stream);
    if (world <= 64) return step_t<64>(d, small, sc, grads, params, world, master, momentum, stream);
    return step_t<512>(d, small, sc, grads, params, world, master, momentum, stream);
}

cudaError_t launch_muon_small_orth(const MuonDev &d, const MuonSmall &small, const MuonScalars &sc, const void *in,
                                   bool in_bf16, void *out, bool out_bf16, cudaStream_t stream)
{
    SmallParams<8> p{};
    p.d = d;
    p.in = in;
    p.out = out;
    p.in_bf16 = in_bf16;
    p.out_bf16 = out_bf16;
    p.sc = sc;
    return launch_small<8>(p, small, stream);
}

}  // namespace zero1
