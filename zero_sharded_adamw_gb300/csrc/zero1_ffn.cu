// zero1_ffn.cu -- C ABI of the gated feed-forward block (include/zero1.h,
// zero1_ffn_*): argument checks, the workspace, copies of operands whose rows
// TMA cannot address, tensor maps and launches.
#include <cuda_runtime.h>

#include <cstdarg>
#include <cstdio>
#include <cstring>

#include "zero1.h"
#include "zero1_ffn.h"
#include "zero1_internal.h"
#include "zero1_launch.h"

namespace zero1 {
namespace {

constexpr uint64_t kMaxWidth = 65536, kMaxHidden = 1ull << 20;

int ffail(int code, const char *fmt, ...)
{
    char msg[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(msg, sizeof msg, fmt, ap);
    va_end(ap);
    set_error_message(msg);
    return code;
}

int fcuda(cudaError_t e, const char *what)
{
    cudaGetLastError();   // reported here, and not again by the caller's next launch
    return ffail(ZERO1_ECUDA, "%s: %s", what, cudaGetErrorString(e));
}

// A matrix of a call: bf16, rows `ld` entries apart.
struct Mat {
    const void *p;
    uint64_t rows, cols, ld;
    const char *name;
    bool written;
    bool aligned() const { return ld % 8 == 0 && reinterpret_cast<uintptr_t>(p) % 16 == 0; }
    uint64_t extent() const { return (rows - 1) * ld + cols; }   // entries from the first to one past the last
};

// The shape with its defaults put in.
int check_shape(const zero1_ffn_shape *in, zero1_ffn_shape &s)
{
    if (!in) return ffail(ZERO1_EINVAL, "shape is NULL");
    if (in->size != sizeof(zero1_ffn_shape)) return ffail(ZERO1_EINVAL, "shape size does not match");
    s = *in;
    if (s.activation < ZERO1_ACT_SILU || s.activation > ZERO1_ACT_RELU) return ffail(ZERO1_EINVAL, "unknown activation %d", (int)s.activation);
    if (s.unaligned != 0 && s.unaligned != 1) return ffail(ZERO1_EINVAL, "unaligned must be 0 or 1");
    if (s.inject_wait_timeout != 0 && s.inject_wait_timeout != 1) return ffail(ZERO1_EINVAL, "inject_wait_timeout must be 0 or 1");
    if (s.rows > 0x7FFFFFFFull) return ffail(ZERO1_EINVAL, "rows must be below 2^31");
    if (s.width < 1 || s.width > kMaxWidth) return ffail(ZERO1_EINVAL, "width must be in [1, 65536]");
    if (s.hidden < 1 || s.hidden > kMaxHidden) return ffail(ZERO1_EINVAL, "hidden must be in [1, 2^20]");
    const struct {
        uint64_t *ld, cols, rows;
        const char *name;
    } lds[6] = {{&s.ldx, s.width, s.rows, "ldx"},          {&s.ldy, s.width, s.rows, "ldy"},
                {&s.ldh, s.hidden, s.rows, "ldh"},         {&s.ld_gate, s.hidden, s.width, "ld_gate"},
                {&s.ld_up, s.hidden, s.width, "ld_up"},    {&s.ld_down, s.width, s.hidden, "ld_down"}};
    for (const auto &l : lds) {
        if (*l.ld == 0) *l.ld = l.cols;
        // strides whose last row is past 2^50 entries name no memory; a tensor map's are below 2^40 bytes
        if (*l.ld < l.cols || *l.ld >= (1ull << 38) || *l.ld > (1ull << 50) / (l.rows ? l.rows : 1))
            return ffail(ZERO1_EINVAL, "%s must be at least its matrix's columns, below 2^38, and times the rows at most 2^50", l.name);
    }
    // tiles of 256 x 256 (gated: of 128 columns) and their slices in one launch
    const uint64_t m = (s.rows + kFfnTile - 1) / kFfnTile, h = (s.hidden + 127) / 128, w = (s.width + kFfnTile - 1) / kFfnTile;
    if (m * h >= (1ull << 26) || m * w * ((s.hidden + 32767) / 32768) + 2 * w * h * ((s.rows + 65535) / 65536) >= (1ull << 26)) return ffail(ZERO1_EINVAL, "rows times hidden or width is too large");
    return ZERO1_OK;
}

// Whether two matrices share an entry.  With rows equally far apart, or a
// single row in one of them, it is exact (column slices of one matrix share
// none); else their extents decide.
bool share(Mat a, Mat b)
{
    if (reinterpret_cast<uintptr_t>(a.p) > reinterpret_cast<uintptr_t>(b.p)) {
        const Mat t = a;
        a = b;
        b = t;
    }
    const uint64_t bytes = reinterpret_cast<uintptr_t>(b.p) - reinterpret_cast<uintptr_t>(a.p);
    if (bytes >= 2 * a.extent()) return false;
    if (a.rows == 1) return true;    // no gaps: b's first entry is one of a's, over however many of b's rows a goes on
    if (b.rows == 1) b.ld = a.ld;    // as long as it may be: what counts is where it begins in a's rows
    if (a.ld != b.ld || bytes % 2) return true;
    const uint64_t d = bytes / 2, q = d / a.ld, c = d % a.ld;
    return (q < a.rows && c < a.cols) || (q + 1 < a.rows && c + b.cols > a.ld);
}

int check_mats(const zero1_ffn_shape &s, const Mat *m, int count)
{
    for (int i = 0; i < count; ++i) {
        if (!m[i].p) continue;
        const uintptr_t at = reinterpret_cast<uintptr_t>(m[i].p);
        if (at % 2 || (!s.unaligned && at % 16))
            return ffail(ZERO1_EALIGN, "%s is not %s", m[i].name,
                         at % 2 ? "aligned to its elements" : "16-byte aligned (set `unaligned` in the shape for such buffers)");
    }
    for (int i = 0; i < count; ++i)
        for (int j = i + 1; j < count; ++j)
            if (m[i].p && m[j].p && (m[i].written || m[j].written) && share(m[i], m[j]))
                return ffail(ZERO1_EINVAL, "%s and %s share memory", m[i].name, m[j].name);
    return ZERO1_OK;
}

// The error word shares no entry with a matrix.
int check_errors(const unsigned *errors, const Mat *m, int count)
{
    if (!errors) return ZERO1_OK;
    if (reinterpret_cast<uintptr_t>(errors) % 4) return ffail(ZERO1_EALIGN, "errors is not 4-byte aligned");
    const Mat word{errors, 1, 2, 2, "errors", true};
    for (int i = 0; i < count; ++i)
        if (m[i].p && share(word, m[i])) return ffail(ZERO1_EINVAL, "errors and %s share memory", m[i].name);
    return ZERO1_OK;
}

// ------------------------------------------------------------- workspace

uint64_t round_up(uint64_t x, uint64_t a) { return (x + a - 1) / a * a; }
uint64_t tiles_of(uint64_t m, uint64_t n) { return round_up(m, kFfnTile) / kFfnTile * (round_up(n, kFfnTile) / kFfnTile); }
uint64_t steps_of(uint64_t k) { return (k + kFfnStep - 1) / kFfnStep; }

// A matrix's copy in the workspace, rows padded to 16 bytes.
uint64_t copy_bytes(uint64_t rows, uint64_t cols) { return round_up(rows * round_up(cols, 8) * 2, 256); }

uint64_t partial_bytes(uint64_t tiles, uint32_t slices) { return slices > 1 ? tiles * slices * kFfnPartial : 0; }

// Tiles of the three weight gradients, which one launch takes.
uint64_t weight_tiles(const zero1_ffn_shape &s) { return 2 * tiles_of(s.width, s.hidden) + tiles_of(s.hidden, s.width); }

// The forward pass of few rows has kernels of its own.
bool thin_rows(const zero1_ffn_shape &s, bool backward)
{
    return !backward && s.rows <= kFfnThinRows && s.hidden <= kFfnThinHidden;
}

uint64_t workspace_of(const zero1_ffn_shape &s, bool backward)
{
    if (s.rows == 0) return 0;
    const auto copy = [&](uint64_t rows, uint64_t cols, uint64_t ld) {
        return s.unaligned || ld % 8 ? copy_bytes(rows, cols) : 0;
    };
    uint64_t b = copy(s.rows, s.width, s.ldx) + copy(s.width, s.hidden, s.ld_gate) + copy(s.width, s.hidden, s.ld_up) +
                 copy(s.hidden, s.width, s.ld_down);
    if (thin_rows(s, backward)) return b + 2 * copy_bytes(s.rows, s.hidden);   // h in two parts
    b += copy(s.rows, s.hidden, s.ldh);
    const uint64_t out_tiles = tiles_of(s.rows, s.width);
    if (!backward) return b + partial_bytes(out_tiles, ffn_slices(out_tiles, steps_of(s.hidden)).a);
    b += copy(s.rows, s.width, s.ldy) + 2 * copy_bytes(s.rows, s.hidden);
    const FfnSlices n = ffn_slices(weight_tiles(s), steps_of(s.rows), out_tiles, 2 * steps_of(s.hidden));
    const FfnSlices without = ffn_slices(weight_tiles(s), steps_of(s.rows));   // dx not wanted
    const uint64_t with_dx = partial_bytes(weight_tiles(s), n.a) + partial_bytes(out_tiles, n.b);
    const uint64_t only = partial_bytes(weight_tiles(s), without.a);
    return b + (with_dx > only ? with_dx : only);
}

// ---------------------------------------------------------------- copies

// Matrices whose rows start off a 16-byte boundary, copied to rows that start
// on one: all operands of a call in one launch, 8 entries a thread.
constexpr int kMostCopies = 6;
struct CopyParams {
    const uint16_t *src[kMostCopies];
    uint4 *dst[kMostCopies];
    uint64_t ld[kMostCopies], pieces[kMostCopies];   // pieces: of 8 entries, rows times those of a row
    uint32_t cols[kMostCopies], row_pieces[kMostCopies];
};
__global__ void __launch_bounds__(256) zero1_ffn_copy_kernel(const __grid_constant__ CopyParams p)
{
    const int m = blockIdx.y;
    const uint32_t per = p.row_pieces[m], cols = p.cols[m];
    for (uint64_t i = (uint64_t)blockIdx.x * 256 + threadIdx.x; i < p.pieces[m]; i += (uint64_t)gridDim.x * 256) {
        const uint64_t r = i / per;
        const uint32_t c = (uint32_t)(i - r * per) * 8;
        const uint16_t *src = p.src[m] + r * p.ld[m] + c;
        uint32_t w[8];
#pragma unroll
        for (uint32_t k = 0; k < 8; ++k) w[k] = c + k < cols ? src[k] : 0u;
        p.dst[m][i] = make_uint4(w[0] | w[1] << 16, w[2] | w[3] << 16, w[4] | w[5] << 16, w[6] | w[7] << 16);
    }
}

typedef CUresult (*EncodeFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *, const cuuint64_t *,
                             const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                             CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encoder()
{
    void *f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
        return nullptr;
    return reinterpret_cast<EncodeFn>(f);
}

// One call's state: the first error sticks, and nothing is launched after it.
struct Call {
    const zero1_ffn_shape &s;
    unsigned char *space;
    uint64_t at = 0;
    cudaStream_t stream;
    int sms = 0;
    unsigned *errors;
    EncodeFn fn = nullptr;
    int rc = ZERO1_OK;
    CopyParams copies{};
    int count = 0;           // of them
    uint64_t most = 0;       // pieces of the largest
    bool launched = false;   // a kernel of this call

    Call(const zero1_ffn_shape &shape, void *workspace, unsigned *err, void *st)
        : s(shape), space(static_cast<unsigned char *>(workspace)), stream(static_cast<cudaStream_t>(st)), errors(err)
    {
        static const EncodeFn found = encoder();
        fn = found;
        int dev = 0;
        cudaError_t e = cudaGetDevice(&dev);
        if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
        if (e != cudaSuccess) rc = fcuda(e, "device query");
        else if (!fn) rc = ffail(ZERO1_ECUDA, "the driver has no tensor-map encoder");
    }
    void check(cudaError_t e, const char *what)
    {
        if (rc == ZERO1_OK && e != cudaSuccess) rc = fcuda(e, what);
    }
    void *take(uint64_t bytes)
    {
        void *here = space + at;
        at += round_up(bytes, 256);
        return here;
    }
    // The matrix itself, or its copy that TMA can address (made by copy_all).
    Mat addressable(Mat m)
    {
        if (m.aligned()) return m;
        const uint64_t ld = round_up(m.cols, 8);
        void *to = take(copy_bytes(m.rows, m.cols));
        copies.src[count] = static_cast<const uint16_t *>(m.p);
        copies.dst[count] = static_cast<uint4 *>(to);
        copies.ld[count] = m.ld;
        copies.cols[count] = (uint32_t)m.cols;
        copies.row_pieces[count] = (uint32_t)(ld / 8);
        copies.pieces[count] = m.rows * (ld / 8);
        if (copies.pieces[count] > most) most = copies.pieces[count];
        ++count;
        m.p = to;
        m.ld = ld;
        return m;
    }
    void copy_all()
    {
        if (!count || rc != ZERO1_OK) return;
        const uint64_t need = (most + 255) / 256, cap = 16ull * (uint64_t)sms;
        check(launch(zero1_ffn_copy_kernel, dim3((unsigned)(need < cap ? need : cap), (unsigned)count), 256, 0, stream, copies),
              "kernel launch");
        launched = true;
    }
    // Boxes of 64 columns and `box_rows` rows; `planes` matrices `plane` entries apart.
    void map(CUtensorMap *to, const Mat &m, uint32_t box_rows = 64, uint64_t planes = 1, uint64_t plane = 0)
    {
        if (rc != ZERO1_OK) return;
        const cuuint64_t dims[3] = {m.cols, m.rows, planes}, strides[2] = {m.ld * 2, (planes > 1 ? plane : m.ld) * 2};
        const cuuint32_t box[3] = {64, box_rows, 1}, unit[3] = {1, 1, 1};
        if (fn(to, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(m.p), dims, strides, box, unit,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
            rc = ffail(ZERO1_ECUDA, "encoding the tensor map of %s failed", m.name);
    }
    void out(FfnJob &j, int i, const Mat &m)
    {
        j.out[i] = static_cast<uint16_t *>(const_cast<void *>(m.p));
        j.ld_out = m.ld;
        if (m.p) j.vec_out = (i == 0 || j.vec_out) && m.aligned();
    }
};

// The next job of a launch: out (m x n, in tiles of 256 x tile_n) over `segments` times k.
FfnJob &add_job(FfnParams &p, uint64_t m, uint64_t n, uint64_t tile_n, uint64_t k, uint32_t segments, uint32_t slices, bool a_mn,
                bool b_mn)
{
    FfnJob &j = p.job[p.jobs++];
    j.m = (uint32_t)m;
    j.n = (uint32_t)n;
    j.tiles_m = (uint32_t)((m + kFfnTile - 1) / kFfnTile);
    j.tiles_n = (uint32_t)((n + tile_n - 1) / tile_n);
    j.steps = (uint32_t)steps_of(k);
    j.segments = segments;
    j.slices = slices;
    j.a_mn = a_mn;
    j.b_mn = b_mn;
    j.first = p.items;
    j.joins = p.joins;
    const uint32_t tiles = j.tiles_m * j.tiles_n;
    p.items += tiles * slices;
    if (slices > 1) p.joins += tiles;
    return j;
}

// Where the partial tiles of the jobs that have some lie, one job's after another's.
void place_partials(FfnParams &p, void *partials)
{
    uint32_t at = 0;
    for (uint32_t i = 0; i < p.jobs; ++i) {
        FfnJob &j = p.job[i];
        j.partial = at;
        if (j.slices > 1) at += j.tiles_m * j.tiles_n * j.slices;
    }
    p.partials = static_cast<float *>(partials);
}

FfnParams params_of(const Call &c)
{
    FfnParams p;
    memset(&p, 0, sizeof p);
    p.act = c.s.activation;
    p.stall = c.s.inject_wait_timeout;
    p.errors = c.errors;
    return p;
}

// Launch a product of this call.
template <typename F>
void run(Call &c, FfnParams &p, F f)
{
    if (c.rc != ZERO1_OK) return;
    p.follows = c.launched;
    c.check(f(p), "kernel launch");
    c.launched = true;
}

int check_workspace(const zero1_ffn_shape &s, bool backward, const void *workspace, uint64_t bytes, const Mat *m, int count,
                    const unsigned *errors)
{
    const uint64_t need = workspace_of(s, backward);
    if (bytes < need) return ffail(ZERO1_EINVAL, "the workspace holds %llu bytes, the call needs %llu", (unsigned long long)bytes, (unsigned long long)need);
    if (need && !workspace) return ffail(ZERO1_EINVAL, "workspace is NULL");
    if (reinterpret_cast<uintptr_t>(workspace) % 256) return ffail(ZERO1_EALIGN, "the workspace is not 256-byte aligned");
    const uintptr_t from = reinterpret_cast<uintptr_t>(workspace);
    for (int i = 0; i < count; ++i) {
        const uintptr_t at = reinterpret_cast<uintptr_t>(m[i].p);
        if (need && m[i].p && at < from + need && from < at + 2 * m[i].extent())
            return ffail(ZERO1_EINVAL, "%s lies in the workspace", m[i].name);
    }
    const uintptr_t word = reinterpret_cast<uintptr_t>(errors);
    if (word && word < from + need && from < word + 4) return ffail(ZERO1_EINVAL, "errors lies in the workspace");
    return ZERO1_OK;
}

}  // namespace
}  // namespace zero1

extern "C" {

int zero1_ffn_workspace(const zero1_ffn_shape *shape, int backward, uint64_t *bytes)
{
    using namespace zero1;
    if (!bytes) return ffail(ZERO1_EINVAL, "bytes is NULL");
    zero1_ffn_shape s;
    if (const int rc = check_shape(shape, s)) return rc;
    *bytes = workspace_of(s, backward != 0);
    return ZERO1_OK;
}

int zero1_ffn_forward(const zero1_ffn_shape *shape, const void *x, const void *w_gate, const void *w_up, const void *w_down,
                      void *gate, void *up, void *h, void *y, void *workspace, uint64_t workspace_bytes, unsigned *errors,
                      void *stream)
{
    using namespace zero1;
    zero1_ffn_shape s;
    if (const int rc = check_shape(shape, s)) return rc;
    if (s.rows == 0) return ZERO1_OK;
    if (!x || !w_gate || !w_up || !w_down || !h || !y) return ffail(ZERO1_EINVAL, "NULL pointer argument");
    if ((gate == nullptr) != (up == nullptr)) return ffail(ZERO1_EINVAL, "gate and up are kept together, or neither");
    const Mat mats[8] = {{x, s.rows, s.width, s.ldx, "x", false},
                         {w_gate, s.width, s.hidden, s.ld_gate, "w_gate", false},
                         {w_up, s.width, s.hidden, s.ld_up, "w_up", false},
                         {w_down, s.hidden, s.width, s.ld_down, "w_down", false},
                         {h, s.rows, s.hidden, s.ldh, "h", true},
                         {y, s.rows, s.width, s.ldy, "y", true},
                         {gate, s.rows, s.hidden, s.ldh, "gate", true},
                         {up, s.rows, s.hidden, s.ldh, "up", true}};
    if (const int rc = check_mats(s, mats, 8)) return rc;
    if (const int rc = check_errors(errors, mats, 8)) return rc;
    if (const int rc = check_workspace(s, false, workspace, workspace_bytes, mats, 8, errors)) return rc;
    Call c(s, workspace, errors, stream);
    if (c.rc) return c.rc;

    const Mat ax = c.addressable(mats[0]), ag = c.addressable(mats[1]), au = c.addressable(mats[2]), ad = c.addressable(mats[3]);
    c.copy_all();
    if (thin_rows(s, false)) {
        const uint32_t box = ffn_thin_box(s.rows);
        const uint64_t plane = copy_bytes(s.rows, s.hidden) / 2;
        const Mat parts{c.take(4 * plane), s.rows, s.hidden, round_up(s.hidden, 8), "h", true};
        FfnThin f;
        memset(&f, 0, sizeof f);
        c.map(&f.x, ax, box);
        c.map(&f.w_gate, ag);
        c.map(&f.w_up, au);
        c.map(&f.w_down, ad);
        c.map(&f.h, parts, box, 2, plane);
        f.out[0] = static_cast<uint16_t *>(h);
        f.out[1] = static_cast<uint16_t *>(gate);
        f.out[2] = static_cast<uint16_t *>(up);
        f.y = static_cast<uint16_t *>(y);
        f.part = static_cast<uint16_t *>(const_cast<void *>(parts.p));
        f.ldh = s.ldh;
        f.ldy = s.ldy;
        f.ld_part = parts.ld;
        f.plane = plane;
        f.rows = (uint32_t)s.rows;
        f.width = (uint32_t)s.width;
        f.hidden = (uint32_t)s.hidden;
        f.act = s.activation;
        f.stall = s.inject_wait_timeout;
        f.vec[0] = mats[4].aligned() && (!gate || (mats[6].aligned() && mats[7].aligned()));
        f.vec[1] = mats[5].aligned();
        f.errors = errors;
        if (c.rc == ZERO1_OK) c.check(launch_ffn_thin(f, c.sms, c.stream), "kernel launch");
        return c.rc;
    }
    FfnParams p = params_of(c);
    FfnJob &first = add_job(p, s.rows, s.hidden, kFfnTile / 2, s.width, 1, 1, false, true);
    c.map(&first.a[0], ax);
    c.map(&first.b[0], ag);
    c.map(&first.b[1], au);
    c.out(first, 0, mats[4]);
    c.out(first, 1, mats[6]);
    c.out(first, 2, mats[7]);
    Mat ah = mats[4];
    if (!ah.aligned()) {   // written twice: TMA cannot address the caller's
        ah.ld = round_up(s.hidden, 8);
        ah.p = c.take(copy_bytes(s.rows, s.hidden));
        first.copy = static_cast<uint16_t *>(const_cast<void *>(ah.p));
        first.ld_copy = ah.ld;
    }
    run(c, p, [&](const FfnParams &x) { return launch_ffn_gated(x, c.sms, c.stream); });

    FfnParams q = params_of(c);
    FfnJob &second = add_job(q, s.rows, s.width, kFfnTile, s.hidden, 1, ffn_slices(tiles_of(s.rows, s.width), steps_of(s.hidden)).a,
                             false, true);
    c.map(&second.a[0], ah);
    c.map(&second.b[0], ad);
    c.out(second, 0, mats[5]);
    place_partials(q, c.space + c.at);
    run(c, q, [&](const FfnParams &x) { return launch_ffn_plain(x, c.sms, c.stream); });
    return c.rc;
}

int zero1_ffn_backward(const zero1_ffn_shape *shape, const void *dy, const void *x, const void *w_gate, const void *w_up,
                       const void *w_down, const void *gate, const void *up, const void *h, void *dx, void *dw_gate,
                       void *dw_up, void *dw_down, void *workspace, uint64_t workspace_bytes, unsigned *errors, void *stream)
{
    using namespace zero1;
    zero1_ffn_shape s;
    if (const int rc = check_shape(shape, s)) return rc;
    if (!dw_gate || !dw_up || !dw_down) return ffail(ZERO1_EINVAL, "NULL pointer argument");
    const Mat mats[12] = {{dw_gate, s.width, s.hidden, s.ld_gate, "dw_gate", true},
                          {dw_up, s.width, s.hidden, s.ld_up, "dw_up", true},
                          {dw_down, s.hidden, s.width, s.ld_down, "dw_down", true},
                          {dx, s.rows, s.width, s.ldx, "dx", true},
                          {dy, s.rows, s.width, s.ldy, "dy", false},
                          {x, s.rows, s.width, s.ldx, "x", false},
                          {gate, s.rows, s.hidden, s.ldh, "gate", false},
                          {up, s.rows, s.hidden, s.ldh, "up", false},
                          {h, s.rows, s.hidden, s.ldh, "h", false},
                          {w_gate, s.width, s.hidden, s.ld_gate, "w_gate", false},
                          {w_up, s.width, s.hidden, s.ld_up, "w_up", false},
                          {w_down, s.hidden, s.width, s.ld_down, "w_down", false}};
    if (s.rows == 0) {   // sums over no rows
        if (const int rc = check_mats(s, mats, 3)) return rc;
        for (int i = 0; i < 3; ++i) {
            const cudaError_t e = cudaMemset2DAsync(const_cast<void *>(mats[i].p), mats[i].ld * 2, 0, mats[i].cols * 2, mats[i].rows,
                                                    static_cast<cudaStream_t>(stream));
            if (e != cudaSuccess) return fcuda(e, "cudaMemset2DAsync");
        }
        return ZERO1_OK;
    }
    if (!dy || !x || !w_gate || !w_up || !w_down || !gate || !up || !h) return ffail(ZERO1_EINVAL, "NULL pointer argument");
    if (const int rc = check_mats(s, mats, 12)) return rc;
    if (const int rc = check_errors(errors, mats, 12)) return rc;
    if (const int rc = check_workspace(s, true, workspace, workspace_bytes, mats, 12, errors)) return rc;
    Call c(s, workspace, errors, stream);
    if (c.rc) return c.rc;

    const uint64_t ldw = round_up(s.hidden, 8);
    const Mat dgate{c.take(copy_bytes(s.rows, s.hidden)), s.rows, s.hidden, ldw, "dgate", true};
    const Mat dup{c.take(copy_bytes(s.rows, s.hidden)), s.rows, s.hidden, ldw, "dup", true};
    const Mat ady = c.addressable(mats[4]), ax = c.addressable(mats[5]), ah = c.addressable(mats[8]);
    const Mat ag = c.addressable(mats[9]), au = c.addressable(mats[10]), ad = c.addressable(mats[11]);
    c.copy_all();
    void *partials = c.space + c.at;

    FfnParams p = params_of(c);                      // dh, and from it dgate and dup
    FfnJob &first = add_job(p, s.rows, s.hidden, kFfnTile, s.width, 1, 1, false, false);
    c.map(&first.a[0], ady);
    c.map(&first.b[0], ad);
    c.out(first, 0, dgate);
    c.out(first, 1, dup);
    first.in[0] = static_cast<const uint16_t *>(gate);
    first.in[1] = static_cast<const uint16_t *>(up);
    first.ld_in = s.ldh;
    first.vec_in = mats[6].aligned() && mats[7].aligned();
    run(c, p, [&](const FfnParams &x) { return launch_ffn_slope(x, c.sms, c.stream); });

    // the gradients of the weights and of x, the longer sums first
    FfnParams w = params_of(c);
    const uint64_t out_tiles = tiles_of(s.rows, s.width), w_steps = steps_of(s.rows), x_steps = 2 * steps_of(s.hidden);
    const FfnSlices n = dx ? ffn_slices(weight_tiles(s), w_steps, out_tiles, x_steps) : ffn_slices(weight_tiles(s), w_steps);
    const auto weights = [&]() {
        const Mat a[3] = {ax, ax, ah}, b[3] = {dgate, dup, ady};
        for (int i = 0; i < 3; ++i) {
            FfnJob &j = add_job(w, mats[i].rows, mats[i].cols, kFfnTile, s.rows, 1, n.a, true, true);
            c.map(&j.a[0], a[i]);
            c.map(&j.b[0], b[i]);
            c.out(j, 0, mats[i]);
        }
    };
    const auto input = [&]() {
        if (!dx) return;
        FfnJob &j = add_job(w, s.rows, s.width, kFfnTile, s.hidden, 2, n.b, false, false);
        c.map(&j.a[0], dgate);
        c.map(&j.b[0], ag);
        c.map(&j.a[1], dup);
        c.map(&j.b[1], au);
        c.out(j, 0, mats[3]);
    };
    const bool input_first = x_steps / n.b > w_steps / n.a;
    if (input_first) input();
    weights();
    if (!input_first) input();
    place_partials(w, partials);
    run(c, w, [&](const FfnParams &x) { return launch_ffn_plain(x, c.sms, c.stream); });
    return c.rc;
}

}  // extern "C"
