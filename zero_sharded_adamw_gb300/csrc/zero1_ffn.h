// zero1_ffn.h -- what the gated feed-forward block's host code (zero1_ffn.cu)
// and its kernels share.
#pragma once

#include <cstdint>

#include <cuda.h>   // CUtensorMap
#include <cuda_runtime.h>

namespace zero1 {

// Tiles of 256 x 256 accumulators by pairs of blocks, 64 of K a step.
constexpr uint32_t kFfnTile = 256;
constexpr uint32_t kFfnStep = 64;
constexpr uint32_t kFfnJobs = 4;
constexpr uint32_t kFfnPairs = 76;            // pairs of SMs the rules below count on; results do not depend on it
constexpr uint64_t kFfnPartial = (uint64_t)kFfnTile * kFfnTile * sizeof(float);   // bytes of one tile's partial sums

// What a product does with its tiles.
enum FfnMode : int {
    kFfnGated = 0,   // columns 0..127 of a tile are x Wg, the others x Wu of the same 128 hidden columns
    kFfnPlain = 1,   // out = the sum of its segments' products
    kFfnSlope = 2,   // the product is dh: out are dgate and dup
};

// One product: out (m x n) = sum over segments of a[s] b[s].
struct FfnJob {
    CUtensorMap a[2], b[2];       // gated: b = gate's and up's weights; plain: one a segment
    uint16_t *out[3];             // gated: h, gate, up (the last two may be null); plain: out; slope: dgate, dup
    const uint16_t *in[2];        // slope: gate, up
    uint16_t *copy;               // gated: h once more, where TMA cannot address the caller's (or null)
    uint64_t ld_out, ld_in, ld_copy;
    uint32_t m, n;                // rows, columns of the result
    uint32_t tiles_m, tiles_n;
    uint32_t steps, segments;     // of 64 of K in a segment; segments
    uint32_t slices;              // parts of K that are summed apart
    uint32_t first;               // its first item (a tile's slice) in the launch
    uint32_t partial, joins;      // slices > 1: its first partial tile, and how many tiles earlier jobs have to join
    uint32_t a_mn, b_mn;          // plain: rows of the operand in memory are K, its columns the result's
    uint32_t vec_out, vec_in;     // 16-byte aligned rows
};

struct FfnParams {
    FfnJob job[kFfnJobs];
    uint32_t jobs, items, joins;
    int act, stall;
    int follows;                  // not the first launch of its call
    float *partials;              // of slices > 1
    unsigned *errors;             // may be null
};

// In how many slices the K of up to two kinds of tiles (`tiles` of `steps`
// each) is taken, so that few tiles still fill the pairs.  Where both kinds
// together do not: the shortest slices, of at least 8 steps (512 of K), that
// make no second round.  Where they do, items are dealt to the pairs in turn, so
// a kind that is fewer than the pairs by itself is cut to about one a pair (64
// x 4096 x 11008 backward, 16 long tiles beside 2,064 short ones: 138 us, 208
// uncut).  A long sum is taken in slices of 65,536 in any case: the
// tensor cores cut every addition of 16 products off below the sum's last
// place, so a sum of one sign falls short by 8e-8 of itself for each, 3.3e-4
// there, an eighth of a bf16 rounding.
struct FfnSlices {
    uint32_t a, b;
};
inline FfnSlices ffn_slices(uint64_t tiles_a, uint64_t steps_a, uint64_t tiles_b = 0, uint64_t steps_b = 1)
{
    const uint64_t least_a = (steps_a * kFfnStep + 65535) / 65536, least_b = (steps_b * kFfnStep + 65535) / 65536;
    FfnSlices s{(uint32_t)least_a, (uint32_t)least_b};
    if (tiles_a + tiles_b >= kFfnPairs) {
        const auto cut = [](uint64_t tiles, uint64_t steps, uint32_t &n) {
            if (tiles == 0 || tiles >= kFfnPairs) return;
            const uint64_t fill = kFfnPairs / tiles, most = steps / 8, wanted = fill < most ? fill : most;
            if (wanted > n) n = (uint32_t)wanted;
        };
        cut(tiles_a, steps_a, s.a);
        cut(tiles_b, steps_b, s.b);
        return s;
    }
    const uint64_t most = steps_a > steps_b ? steps_a : steps_b;
    for (uint64_t length = 8; length < most; length += 2) {
        const uint64_t a = (steps_a + length - 1) / length, b = (steps_b + length - 1) / length;
        if (tiles_a * a + tiles_b * b > kFfnPairs) continue;
        if (a > least_a) s.a = (uint32_t)a;
        if (b > least_b) s.b = (uint32_t)b;
        return s;
    }
    return s;
}

// The forward pass of at most kFfnThinRows rows (zero1_ffn_thin.cu; at 128
// rows, 4096 x 11008, 69 us to the tiles' 79), unless a sum over the hidden
// size has to be taken in slices (ffn_slices).
constexpr uint64_t kFfnThinRows = 128, kFfnThinHidden = 65536;

// Rows of x and of h that one box of the narrow operand holds.
inline uint32_t ffn_thin_box(uint64_t rows) { return rows <= 16 ? 16 : rows <= 32 ? 32 : rows <= 64 ? 64 : 128; }

struct FfnThin {
    CUtensorMap x, w_gate, w_up, w_down, h;   // h: the parts in the workspace
    uint16_t *out[3], *y, *part;              // h, gate, up (the last two may be null); high and low parts of h
    uint64_t ldh, ldy, ld_part, plane;
    uint32_t rows, width, hidden;
    int act, stall;
    bool vec[2];                              // aligned rows of h, gate and up; of y
    unsigned *errors;
};

cudaError_t launch_ffn_thin(const FfnThin &f, int sms, cudaStream_t stream);

cudaError_t launch_ffn_gated(const FfnParams &p, int sms, cudaStream_t stream);
cudaError_t launch_ffn_slope(const FfnParams &p, int sms, cudaStream_t stream);
cudaError_t launch_ffn_plain(const FfnParams &p, int sms, cudaStream_t stream);

}  // namespace zero1
