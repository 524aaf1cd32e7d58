// zero1_muon.cu -- C ABI of the matrix optimizer (include/zero1.h,
// zero1_muon_*): argument checks, the plan of tiles and elementwise blocks,
// the workspace and its tensor maps, and the launches.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <exception>
#include <memory>
#include <mutex>
#include <new>
#include <unordered_set>
#include <vector>

#include "zero1.h"
#include "zero1_internal.h"
#include "zero1_muon.h"

struct zero1_muon_ctx {
    uint64_t n = 0;
    int world = 0;
    zero1_muon_hparams hp{};
    int device = 0;
    int num_sms = 0;
    void *block = nullptr;        // one cudaMalloc holding the plan and the workspace
    uint64_t block_bytes = 0;
    uint64_t entries = 0;         // of all matrices
    zero1::MuonDev dev{};         // what the large matrices need: empty plan if there are none
    zero1::MuonSmall small{};
    bool any_small = false;
};

namespace {

using zero1::MuonMat;

std::mutex g_muon_mu;
std::unordered_set<zero1_muon_ctx *> g_muon_live;

int mfail(int code, const char *fmt, ...)
{
    char msg[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(msg, sizeof msg, fmt, ap);
    va_end(ap);
    zero1::set_error_message(msg);
    return code;
}

int mcuda(cudaError_t e, const char *what)
{
    cudaGetLastError();   // reported here, and not again by the caller's next launch
    return mfail(e == cudaErrorMemoryAllocation ? ZERO1_ENOMEM : ZERO1_ECUDA, "%s: %s", what, cudaGetErrorString(e));
}

bool muon_live(zero1_muon_ctx *h)
{
    std::lock_guard<std::mutex> lk(g_muon_mu);
    return h && g_muon_live.count(h);
}

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
uint64_t round_up(uint64_t x, uint64_t a) { return (x + a - 1) / a * a; }
uint64_t blocks(uint64_t n, uint64_t tile) { return zero1::tile_blocks(n, tile); }
bool finite_nonneg(double v) { return std::isfinite(v) && v >= 0.0; }

// Make the handle's device current for the duration of a call.
struct MuonDeviceGuard {
    int prev = -1;
    explicit MuonDeviceGuard(int dev)
    {
        if (cudaGetDevice(&prev) != cudaSuccess) prev = -1;
        if (prev != dev) cudaSetDevice(dev);
    }
    ~MuonDeviceGuard()
    {
        if (prev >= 0) cudaSetDevice(prev);
    }
};

int check_hparams(const zero1_muon_hparams *hp)
{
    if (!finite_nonneg(hp->lr)) return mfail(ZERO1_EINVAL, "lr must be finite and >= 0");
    if (!(hp->momentum >= 0.0 && hp->momentum < 1.0)) return mfail(ZERO1_EINVAL, "momentum must be in [0, 1)");
    if (!finite_nonneg(hp->weight_decay)) return mfail(ZERO1_EINVAL, "weight_decay must be finite and >= 0");
    // below 1e-15 an update whose fp32 squares vanish would leave f16's range
    if (!(std::isfinite(hp->eps) && hp->eps >= 1e-15)) return mfail(ZERO1_EINVAL, "eps must be finite and >= 1e-15");
    if (!finite_nonneg(hp->update_scale)) return mfail(ZERO1_EINVAL, "update_scale must be finite and >= 0");
    if (hp->inject_wait_timeout != 0 && hp->inject_wait_timeout != 1)
        return mfail(ZERO1_EINVAL, "inject_wait_timeout must be 0 or 1");
    if (hp->reserved != 0) return mfail(ZERO1_EINVAL, "reserved must be 0");
    if (hp->nesterov != 0 && hp->nesterov != 1) return mfail(ZERO1_EINVAL, "nesterov must be 0 or 1");
    if (hp->scale_rule != ZERO1_MUON_SCALE_RMS && hp->scale_rule != ZERO1_MUON_SCALE_SPECTRAL)
        return mfail(ZERO1_EINVAL, "unknown scale_rule %d", (int)hp->scale_rule);
    if (hp->ns_steps < 1 || hp->ns_steps > 32) return mfail(ZERO1_EINVAL, "ns_steps must be in [1, 32]");
    if (!std::isfinite(hp->ns_a) || !std::isfinite(hp->ns_b) || !std::isfinite(hp->ns_c) ||
        std::fabs(hp->ns_a) > 8.0 || std::fabs(hp->ns_b) > 8.0 || std::fabs(hp->ns_c) > 8.0)
        return mfail(ZERO1_EINVAL, "ns_a, ns_b and ns_c must be finite and at most 8 in magnitude");
    // A (A + (b/c) I) is what the tensor cores form: b/c has to fit beside A in f16
    if (std::fabs(hp->ns_b) > 8.0 * std::fabs(hp->ns_c) || hp->ns_c == 0.0)
        return mfail(ZERO1_EINVAL, "ns_c must not be 0, and |ns_b| at most 8 |ns_c|");
    return ZERO1_OK;
}

// Entries of the flat buffer from a matrix's first to one past its last.
uint64_t extent(const zero1_matrix &m) { return (uint64_t)(m.rows - 1) * m.ld + m.cols; }

// Whether two matrices of the same row stride share an entry: with the
// second's start d = q*ld + c entries after the first's, their columns meet
// at equal rows (q rows apart) when c < cols1, or one row later when the
// second's columns run past the stride into the first's next row.
bool same_stride_overlap(const zero1_matrix &a, const zero1_matrix &b)
{
    const uint64_t d = b.offset - a.offset, q = d / a.ld, c = d % a.ld;
    return (q < a.rows && c < a.cols) || (q + 1 < a.rows && c + b.cols > a.ld);
}

int check_matrices(uint64_t n, const zero1_matrix *mats, uint64_t count)
{
    for (uint64_t i = 0; i < count; ++i) {
        const zero1_matrix &m = mats[i];
        const unsigned long long k = i;
        if (m.rows == 0 || m.cols == 0 || m.rows > zero1::kMaxSide || m.cols > zero1::kMaxSide)
            return mfail(ZERO1_EINVAL, "matrix %llu: sides must be in [1, %u]", k, zero1::kMaxSide);
        if (m.ld < m.cols || m.ld > (uint64_t)1 << 40) return mfail(ZERO1_EINVAL, "matrix %llu: bad row stride", k);
        if (m.offset > n || extent(m) > n - m.offset)
            return mfail(ZERO1_EINVAL, "matrix %llu reaches past the buffer's %llu entries", k, (unsigned long long)n);
    }
    // No two matrices may share an entry (both would be written).
    std::vector<uint32_t> order(count);
    for (uint64_t i = 0; i < count; ++i) order[i] = (uint32_t)i;
    std::sort(order.begin(), order.end(), [&](uint32_t a, uint32_t b) {
        return mats[a].offset != mats[b].offset ? mats[a].offset < mats[b].offset : a < b;
    });
    for (uint64_t i = 0; i < count; ++i) {
        const zero1_matrix &a = mats[order[i]];
        for (uint64_t j = i + 1; j < count; ++j) {
            const zero1_matrix &b = mats[order[j]];
            if (b.offset >= a.offset + extent(a)) break;
            // interleaved matrices are taken where they have one row stride (column slices of one
            // larger matrix); of other strides only a single row can lie within another's extent
            if (a.ld != b.ld || same_stride_overlap(a, b))
                return mfail(ZERO1_EINVAL, "matrices %u and %u overlap or interleave with different row strides",
                             order[i], order[j]);
        }
    }
    return ZERO1_OK;
}

typedef CUresult (*EncodeFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                             const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                             CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// The tensor-map encoder, fetched from the driver through the runtime (the
// library does not link libcuda itself).
EncodeFn encoder()
{
    void *f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
        return nullptr;
    return reinterpret_cast<EncodeFn>(f);
}

// Two f16 planes of rows x cols, rows padded to ld: boxes of 64 x 64, 128-byte swizzle.
bool encode(EncodeFn fn, CUtensorMap *map, void *base, uint64_t rows, uint64_t cols, uint64_t ld, uint64_t plane)
{
    const cuuint64_t dims[3] = {cols, rows, 2}, strides[2] = {ld * 2, plane * 2};
    const cuuint32_t box[3] = {64, 64, 1}, unit[3] = {1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, base, dims, strides, box, unit, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// SMs of the current device; where there is none, creation fails later on.
int device_sms()
{
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return 0;
    return sms;
}

// A handle under construction: its memory goes with it.
struct FreeHandle {
    void operator()(zero1_muon_ctx *h) const
    {
        if (h->block) cudaFree(h->block);
        delete h;
    }
};

// Where each part of the one allocation lies.
struct Layout {
    uint64_t at = 0;
    uint64_t take(uint64_t bytes)
    {
        const uint64_t here = at;
        at = round_up(at + bytes, 256);
        return here;
    }
};

int create(uint64_t n, int world, const zero1_matrix *mats, uint64_t count, const zero1_muon_hparams *hp,
           zero1_muon_handle *out)
{
    if (!out) return mfail(ZERO1_EINVAL, "out is NULL");
    *out = nullptr;
    if (!hp || !mats) return mfail(ZERO1_EINVAL, "NULL pointer argument");
    if (hp->size != sizeof(zero1_muon_hparams))
        return mfail(ZERO1_EINVAL, "hp->size must be sizeof(zero1_muon_hparams)");
    if (n == 0 || n > (uint64_t)1 << 50) return mfail(ZERO1_EINVAL, "n must be in [1, 2^50]");
    if (world < 1 || world > ZERO1_MAX_WORLD)
        return mfail(ZERO1_EINVAL, "world must be in [1, %d], got %d", ZERO1_MAX_WORLD, world);
    if (count == 0 || count > 65536) return mfail(ZERO1_EINVAL, "count must be in [1, 65536]");
    int rc = check_hparams(hp);
    if (rc) return rc;
    if ((rc = check_matrices(n, mats, count))) return rc;

    // ---- the plan
    std::vector<MuonMat> plan(count);
    std::vector<uint2> work;
    std::vector<uint32_t> chunk_mat, large, small[zero1::kSmallSizes];
    std::vector<uint64_t> region0(count), region1(count), gram(count), poly(count), diag(count);
    uint64_t entries = 0, large_entries = 0, chunks = 0, tiles = 0;
    for (uint64_t i = 0; i < count; ++i) {
        const zero1_matrix &a = mats[i];
        MuonMat &m = plan[i];
        m.offset = a.offset;
        m.ld = a.ld;
        m.rows = a.rows;
        m.cols = a.cols;
        m.s = std::min(a.rows, a.cols);
        m.tall = a.rows > a.cols;
        m.ldx = (uint32_t)round_up(a.cols, 64);
        m.lds = (uint32_t)round_up(m.s, 64);
        m.xplane = (uint64_t)a.rows * m.ldx;
        m.splane = (uint64_t)m.s * m.lds;
        const uint64_t size = (uint64_t)a.rows * a.cols;
        m.vec = a.offset % 8 == 0 && a.ld % 8 == 0 && a.cols % 8 == 0;
        const double r = a.rows, k = a.cols;
        m.scale = (float)(hp->update_scale *
                          std::sqrt(hp->scale_rule == ZERO1_MUON_SCALE_RMS ? std::max(r, k) : std::max(1.0, r / k)));
        entries += size;
        const int blocks_log = zero1::small_blocks(m.s, std::max(a.rows, a.cols));
        if (blocks_log >= 0) {
            small[blocks_log].push_back((uint32_t)i);
            continue;
        }
        large.push_back((uint32_t)i);
        large_entries += size;
    }
    // Blocks of 16,384 entries, or of 2,048 and more so that small lists spread over the SMs too (each block of
    // the second kernel adds up all partial sums of its matrix: 4,096 at 67 million entries).
    uint32_t chunk = 2048;
    while (chunk < 16384 && large_entries / chunk > 2048) chunk *= 2;
    for (const uint32_t i : large) {
        MuonMat &m = plan[i];
        const uint64_t c = blocks((uint64_t)m.rows * m.cols, chunk);
        chunks += c;
        if (chunks > 0x7FFFFFFFull) return mfail(ZERO1_EINVAL, "the matrices are too large for one handle");
        m.chunk0 = (uint32_t)(chunks - c);
        m.chunks = (uint32_t)c;
    }
    const int sms_hint = device_sms();
    const auto sides = [&](size_t k, uint32_t &rows, uint32_t &cols) { rows = plan[large[k]].rows, cols = plan[large[k]].cols; };
    const uint32_t tile = zero1::tile_columns(large.size(), sides, sms_hint);
    for (const uint32_t i : large) {
        MuonMat &m = plan[i];
        const zero1::Tiles t = zero1::tiles_of(m.rows, m.cols, tile);
        tiles += 2 * t.gram + t.full;
        // tickets and per-matrix counts are 32-bit, over all steps
        if (tiles * 32 * zero1::kNsParts > 0x7FFFFFFFull)
            return mfail(ZERO1_EINVAL, "the matrices are too large for one handle");
        m.parts[0] = m.parts[1] = (uint32_t)(t.gram * zero1::kNsParts);
        m.parts[2] = (uint32_t)(t.full * zero1::kNsParts);
    }
    work.reserve(tiles);
    chunk_mat.reserve(chunks);
    const auto push = [&](uint32_t phase, uint64_t i, uint32_t r, uint32_t c) {
        work.push_back(make_uint2((uint32_t)i | phase << 30, r | c << 16));
    };
    const uint32_t per_row = zero1::kNsRows / tile;   // column tiles of a diagonal block
    for (uint32_t phase = 0; phase < 3; ++phase)
        for (const uint32_t i : large) {
            const MuonMat &m = plan[i];
            const uint32_t rb = (uint32_t)blocks(phase < 2 ? m.s : m.rows, zero1::kNsRows);
            const uint32_t cb = (uint32_t)blocks(phase < 2 ? m.s : m.cols, tile);
            if (phase < 2) {
                for (uint32_t r = 0; r < rb; ++r)
                    for (uint32_t c = per_row * r; c < cb; ++c) push(phase, i, r, c);
            } else {
                // the Gram-sized factor stays in L2 and X passes once: all of one block of X before the next
                for (uint32_t j = 0; j < (m.tall ? rb : cb); ++j)
                    for (uint32_t k = 0; k < (m.tall ? cb : rb); ++k) push(phase, i, m.tall ? j : k, m.tall ? k : j);
            }
        }
    for (const uint32_t i : large) chunk_mat.insert(chunk_mat.end(), plan[i].chunks, i);
    std::vector<uint32_t> small_list;
    for (const auto &v : small) small_list.insert(small_list.end(), v.begin(), v.end());

    // ---- the device
    int ndev = 0, dev = 0;
    cudaError_t e = cudaGetDeviceCount(&ndev);
    if (e != cudaSuccess || ndev == 0) return mfail(ZERO1_ENODEV, "no CUDA device (%s)", cudaGetErrorString(e));
    if ((e = cudaGetDevice(&dev)) != cudaSuccess) return mcuda(e, "cudaGetDevice");
    int major = 0, minor = 0, sms = 0;
    if ((e = cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev)) != cudaSuccess ||
        (e = cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev)) != cudaSuccess ||
        (e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess)
        return mcuda(e, "device query");
    if (major != 10 || minor != 3)
        return mfail(ZERO1_ENODEV, "device %d is sm_%d%d; this library is built for sm_103a", dev, major, minor);
    const EncodeFn fn = encoder();
    if (!fn) return mfail(ZERO1_ECUDA, "the driver has no tensor-map encoder");

    // ---- the workspace: plan | counters | per matrix: two regions, A, P, A's diagonal
    Layout l;
    const uint64_t at_mats = l.take(count * sizeof(MuonMat));
    const uint64_t at_maps = l.take(count * zero1::kMapsPerMat * sizeof(CUtensorMap));
    const uint64_t at_work = l.take(work.size() * sizeof(uint2));
    const uint64_t at_chunk = l.take(chunk_mat.size() * sizeof(uint32_t));
    const uint64_t at_small = l.take(small_list.size() * sizeof(uint32_t));
    const uint64_t at_part = l.take(chunk_mat.size() * sizeof(double));
    const uint64_t at_done = l.take(count * sizeof(unsigned));
    const uint64_t at_ticket = l.take(sizeof(unsigned)), at_errors = l.take(sizeof(unsigned));
    for (const uint32_t i : large) {
        region0[i] = l.take(plan[i].xplane * 4);
        region1[i] = l.take(plan[i].xplane * 4);
        gram[i] = l.take(plan[i].splane * 4);
        poly[i] = l.take(plan[i].splane * 4);
        diag[i] = l.take((uint64_t)plan[i].s * zero1::kNsRows * 4);
    }
    std::unique_ptr<zero1_muon_ctx, FreeHandle> h(new zero1_muon_ctx);
    h->n = n;
    h->world = world;
    h->hp = *hp;
    h->device = dev;
    h->num_sms = sms;
    h->entries = entries;
    h->block_bytes = l.at;
    if ((e = cudaMalloc(&h->block, h->block_bytes)) != cudaSuccess) {
        h->block = nullptr;
        return mcuda(e, "cudaMalloc of the matrix optimizer's workspace");
    }
    unsigned char *base = static_cast<unsigned char *>(h->block);
    std::vector<CUtensorMap> maps(count * zero1::kMapsPerMat);
    bool good = true;
    for (const uint32_t i : large) {
        if (!good) break;
        MuonMat &m = plan[i];
        m.region[0] = base + region0[i];
        m.region[1] = base + region1[i];
        m.gram = base + gram[i];
        m.poly = base + poly[i];
        m.diag = base + diag[i];
        CUtensorMap *t = &maps[(uint64_t)i * zero1::kMapsPerMat];
        good = encode(fn, t + zero1::kMapX0, m.region[0], m.rows, m.cols, m.ldx, m.xplane) &&
               encode(fn, t + zero1::kMapX1, m.region[1], m.rows, m.cols, m.ldx, m.xplane) &&
               encode(fn, t + zero1::kMapA, m.gram, m.s, m.s, m.lds, m.splane) &&
               encode(fn, t + zero1::kMapP, m.poly, m.s, m.s, m.lds, m.splane) &&
               encode(fn, t + zero1::kMapD, m.diag, m.s, std::min<uint64_t>(m.s, zero1::kNsRows), zero1::kNsRows,
                      (uint64_t)m.s * zero1::kNsRows);
    }
    e = good ? cudaMemset(h->block, 0, h->block_bytes) : cudaErrorInvalidValue;
    const auto put = [&](uint64_t at, const void *src, uint64_t bytes) {
        if (e == cudaSuccess && bytes) e = cudaMemcpy(base + at, src, bytes, cudaMemcpyHostToDevice);
    };
    put(at_mats, plan.data(), count * sizeof(MuonMat));
    put(at_maps, maps.data(), maps.size() * sizeof(CUtensorMap));
    put(at_work, work.data(), work.size() * sizeof(uint2));
    put(at_small, small_list.data(), small_list.size() * sizeof(uint32_t));
    put(at_chunk, chunk_mat.data(), chunk_mat.size() * sizeof(uint32_t));
    if (e == cudaSuccess) e = cudaDeviceSynchronize();
    if (e != cudaSuccess)
        return good ? mcuda(e, "filling the workspace") : mfail(ZERO1_ECUDA, "encoding a tensor map failed");
    zero1::MuonDev &d = h->dev;
    d.mats = reinterpret_cast<MuonMat *>(base + at_mats);
    d.maps = reinterpret_cast<CUtensorMap *>(base + at_maps);
    d.work = reinterpret_cast<uint2 *>(base + at_work);
    d.chunk_mat = reinterpret_cast<uint32_t *>(base + at_chunk);
    d.partials = reinterpret_cast<double *>(base + at_part);
    d.done = reinterpret_cast<unsigned *>(base + at_done);
    d.ticket = reinterpret_cast<unsigned *>(base + at_ticket);
    d.errors = reinterpret_cast<unsigned *>(base + at_errors);
    d.count = (uint32_t)count;
    d.nchunks = (uint32_t)chunk_mat.size();
    d.work_per_iter = (uint32_t)work.size();
    d.tile = tile;
    d.chunk = chunk;
    h->small.list = reinterpret_cast<uint32_t *>(base + at_small);
    for (int i = 0, at = 0; i < zero1::kSmallSizes; ++i) {
        h->small.first[i] = (uint32_t)at;
        h->small.count[i] = (uint32_t)small[i].size();
        at += (int)small[i].size();
    }
    h->any_small = !small_list.empty();
    {
        std::lock_guard<std::mutex> lk(g_muon_mu);
        g_muon_live.insert(h.get());
    }
    *out = h.release();
    return ZERO1_OK;
}

zero1::MuonScalars scalars(const zero1_muon_ctx *h)
{
    zero1::MuonScalars s{};
    s.inv_w = (float)(1.0 / h->world);
    s.momentum = (float)h->hp.momentum;
    s.one_minus_momentum = (float)(1.0 - h->hp.momentum);
    s.eps = (float)h->hp.eps;
    s.lr = (float)h->hp.lr;
    s.decay = (float)(1.0 - h->hp.lr * h->hp.weight_decay);
    s.a = (float)h->hp.ns_a;
    s.b = (float)h->hp.ns_b;
    s.c = (float)h->hp.ns_c;
    s.nesterov = h->hp.nesterov;
    s.steps = h->hp.ns_steps;
    s.stall = h->hp.inject_wait_timeout;
    return s;
}

// Before anything of a call runs: a cluster that the stream's SMs cannot hold would never start.
int check_clusters(const zero1_muon_ctx *h, cudaStream_t st)
{
    if (!h->any_small) return ZERO1_OK;
    int blocks = 0;
    const cudaError_t e = zero1::muon_small_misfit(h->small, st, &blocks);
    if (e != cudaSuccess) return mcuda(e, "cluster query");
    if (blocks)
        return mfail(ZERO1_EINVAL, "the stream's SMs hold no cluster of %d blocks, which a matrix of this handle needs", blocks);
    return ZERO1_OK;
}

}  // namespace

extern "C" {

int zero1_muon_create(uint64_t n, int world, const zero1_matrix *mats, uint64_t count, const zero1_muon_hparams *hp,
                      zero1_muon_handle *out)
{
    try {
        return create(n, world, mats, count, hp, out);
    } catch (const std::bad_alloc &) {
        return mfail(ZERO1_ENOMEM, "host allocation failed");
    } catch (const std::exception &x) {
        return mfail(ZERO1_EINVAL, "%s", x.what());
    }
}

int zero1_muon_destroy(zero1_muon_handle h)
{
    if (h == nullptr) return ZERO1_OK;
    {
        std::lock_guard<std::mutex> lk(g_muon_mu);
        if (!g_muon_live.erase(h)) return mfail(ZERO1_EINVAL, "unknown or already destroyed handle");
    }
    MuonDeviceGuard g(h->device);
    const cudaError_t e1 = cudaDeviceSynchronize(), e2 = cudaFree(h->block);
    delete h;
    if (e1 != cudaSuccess) return mcuda(e1, "cudaDeviceSynchronize in destroy");
    if (e2 != cudaSuccess) return mcuda(e2, "cudaFree");
    return ZERO1_OK;
}

int zero1_muon_step(zero1_muon_handle h, const void *const *grad_ptrs, void *const *param_ptrs, float *master,
                    float *momentum, void *stream)
{
    if (!muon_live(h)) return mfail(ZERO1_EINVAL, "invalid handle");
    if (!grad_ptrs || !param_ptrs) return mfail(ZERO1_EINVAL, "pointer array is NULL");
    if (!master || !momentum) return mfail(ZERO1_EINVAL, "master or momentum is NULL");
    for (int r = 0; r < h->world; ++r) {
        if (!grad_ptrs[r] || !param_ptrs[r]) return mfail(ZERO1_EINVAL, "rank %d buffer is NULL", r);
        if (!aligned16(grad_ptrs[r]) || !aligned16(param_ptrs[r]))
            return mfail(ZERO1_EALIGN, "rank %d buffer is not 16-byte aligned", r);
    }
    if (!aligned16(master) || !aligned16(momentum))
        return mfail(ZERO1_EALIGN, "master and momentum must be 16-byte aligned");
    MuonDeviceGuard g(h->device);
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (const int rc = check_clusters(h, st)) return rc;
    const zero1::MuonScalars sc = scalars(h);
    cudaError_t e = cudaSuccess;
    if (h->any_small)
        e = zero1::launch_muon_small_step(h->dev, h->small, sc, grad_ptrs, param_ptrs, h->world, master, momentum, st);
    if (h->dev.nchunks == 0) return e == cudaSuccess ? ZERO1_OK : mcuda(e, "kernel launch");
    if (e == cudaSuccess) e = zero1::launch_muon_momentum(h->dev, sc, grad_ptrs, h->world, momentum, st);
    if (e == cudaSuccess) e = zero1::launch_muon_split(h->dev, sc, nullptr, false, st);
    if (e == cudaSuccess) e = zero1::launch_muon_iterate(h->dev, sc, h->num_sms, st);
    if (e == cudaSuccess) e = zero1::launch_muon_apply(h->dev, sc, param_ptrs, h->world, master, st);
    return e == cudaSuccess ? ZERO1_OK : mcuda(e, "kernel launch");
}

int zero1_muon_orthogonalize(zero1_muon_handle h, const void *in, int in_dtype, void *out, int out_dtype, void *stream)
{
    if (!muon_live(h)) return mfail(ZERO1_EINVAL, "invalid handle");
    if (!in || !out) return mfail(ZERO1_EINVAL, "NULL buffer");
    if ((in_dtype != ZERO1_DTYPE_BF16 && in_dtype != ZERO1_DTYPE_F32) ||
        (out_dtype != ZERO1_DTYPE_BF16 && out_dtype != ZERO1_DTYPE_F32))
        return mfail(ZERO1_EINVAL, "bad dtype");
    // a block may write its matrix where another has yet to read its own
    if (in == out && in_dtype != out_dtype) return mfail(ZERO1_EINVAL, "out may be in only when their types are equal");
    if (!aligned16(in) || !aligned16(out)) return mfail(ZERO1_EALIGN, "buffers must be 16-byte aligned");
    MuonDeviceGuard g(h->device);
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (const int rc = check_clusters(h, st)) return rc;
    const zero1::MuonScalars sc = scalars(h);
    const bool bf = in_dtype == ZERO1_DTYPE_BF16;
    cudaError_t e = cudaSuccess;
    if (h->any_small)
        e = zero1::launch_muon_small_orth(h->dev, h->small, sc, in, bf, out, out_dtype == ZERO1_DTYPE_BF16, st);
    if (h->dev.nchunks == 0) return e == cudaSuccess ? ZERO1_OK : mcuda(e, "kernel launch");
    if (e == cudaSuccess) e = zero1::launch_muon_norm(h->dev, in, bf, st);
    if (e == cudaSuccess) e = zero1::launch_muon_split(h->dev, sc, in, bf, st);
    if (e == cudaSuccess) e = zero1::launch_muon_iterate(h->dev, sc, h->num_sms, st);
    if (e == cudaSuccess) e = zero1::launch_muon_out(h->dev, sc, out, out_dtype == ZERO1_DTYPE_BF16, st);
    return e == cudaSuccess ? ZERO1_OK : mcuda(e, "kernel launch");
}

int zero1_muon_set_lr(zero1_muon_handle h, double lr)
{
    if (!muon_live(h)) return mfail(ZERO1_EINVAL, "invalid handle");
    if (!finite_nonneg(lr)) return mfail(ZERO1_EINVAL, "lr must be finite and >= 0");
    h->hp.lr = lr;
    return ZERO1_OK;
}

int zero1_muon_status(zero1_muon_handle h, void *stream)
{
    if (!muon_live(h)) return mfail(ZERO1_EINVAL, "invalid handle");
    MuonDeviceGuard g(h->device);
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    unsigned errors = 0;
    cudaError_t e = cudaMemcpyAsync(&errors, h->dev.errors, sizeof errors, cudaMemcpyDeviceToHost, st);
    if (e == cudaSuccess) e = cudaStreamSynchronize(st);
    if (e != cudaSuccess) return mcuda(e, "reading the status");
    if (errors & zero1::kErrWaitTimeout)
        return mfail(ZERO1_ECUDA, "a kernel wait gave up after its 1 s limit; the results are not valid");
    return ZERO1_OK;
}

int zero1_muon_layout(zero1_muon_handle h, uint64_t *entries, uint64_t *device_bytes)
{
    if (!muon_live(h)) return mfail(ZERO1_EINVAL, "invalid handle");
    if (entries) *entries = h->entries;
    if (device_bytes) *device_bytes = h->block_bytes;
    return ZERO1_OK;
}

}  // extern "C"
