// zero1_muon_tiles.h -- how the matrix optimizer's matrices are cut up: which
// run as one small launch, and the tile width of those that do not.
// Host-only; shared by the C ABI (zero1_muon.cu) and its kernels' header.
// Not installed.
#pragma once

#include <algorithm>
#include <cstddef>
#include <cstdint>

namespace zero1 {

// Output tile of the matrix products: 256 rows, 128 in each block of a pair,
// by 256 or 128 columns (one choice for a handle).
constexpr uint32_t kNsRows = 256;

// Small matrices are stepped in one launch by clusters of 1, 2, 4 or 8 blocks.
constexpr int kSmallSizes = 4;
// Columns of the larger side a block holds, at most: X, two f16 parts of 128
// rows, beside the Gram matrix (64 KB) and, in a cluster, the parts of its
// sum (64 KB).
constexpr uint32_t small_width(int blocks) { return blocks == 1 ? 256 : 192; }

// log2 of the blocks that step a small matrix of sides s <= l in one launch,
// or -1.  An iteration takes one to eight blocks about 5 us, and the tiled
// products 38 us and more (13 for each of three).  One launch holds a smaller
// side up to 128 with a larger one up to 1,536.
inline int small_blocks(uint32_t s, uint32_t l)
{
    if (s > 128) return -1;
    for (int i = 0; i < kSmallSizes; ++i)
        if (l <= (small_width(1 << i) << i)) return i;
    return -1;
}

inline uint64_t tile_blocks(uint64_t n, uint64_t tile) { return (n + tile - 1) / tile; }

// Tiles of one product: of a Gram-sized matrix from its diagonal blocks on,
// and of X.
struct Tiles {
    uint64_t gram, full;
};

inline Tiles tiles_of(uint32_t rows, uint32_t cols, uint32_t tile)
{
    const uint32_t s = std::min(rows, cols);
    const uint64_t rb = tile_blocks(s, kNsRows), cb = tile_blocks(s, tile), per_row = kNsRows / tile;
    return Tiles{rb * cb - per_row * (rb * (rb - 1) / 2), tile_blocks(rows, kNsRows) * tile_blocks(cols, tile)};
}

// Microseconds of one iteration over a list of tiled matrices (`sides(i,
// rows, cols)` gives the i-th), in tiles of `tile` columns, on so many pairs
// of blocks: the time of all tiles over all pairs, or of the longest chain of
// three products with its hand-overs, whichever is longer, and a third of the
// other.  A step is 64 of K of one tile.  The constants are fitted to the
// iteration kernel's time on 45 lists, from three 768 x 768 to 4096 x 16384
// and from one matrix to 300: within 28% (128 columns) and 22% (256) of each,
// and the shorter of the two estimates is the shorter time in all of them.
// Some of those times, us an iteration at 128 | 256 columns: three 768 x 768
// 46 | 63, twelve 73 | 77, sixteen 92 | 87; 2048 x 2048 109 | 113, 2304 x 2304
// 187 | 152, 4096 x 16384 2267 | 1549; 40 of 300 x 517 64 | 70, 120 181 | 163;
// one GPT-2-small block 80 | 97, two 117 | 114, all twelve 682 | 462.  (A trace
// of three 768 x 768 at 128 columns gives each of three products 8 us for its
// 12 steps and 7.5 us to hand over; the fit spreads the same time otherwise.)
template <typename F>
double iteration_us(size_t count, F sides, uint32_t tile, double pairs)
{
    const bool wide = tile == 256;
    const double step = wide ? 0.88 : 0.66, per_tile = wide ? 2.2 : 1.9;         // of a full device
    const double chain_step = wide ? 0.66 : 0.69, hand_overs = wide ? 44.0 : 17.0;   // of a chain
    double steps = 0.0, tiles = 0.0, chain = 0.0;
    for (size_t i = 0; i < count; ++i) {
        uint32_t rows, cols;
        sides(i, rows, cols);
        const Tiles t = tiles_of(rows, cols, tile);
        const double gram = (double)tile_blocks(std::max(rows, cols), 64), rest = (double)tile_blocks(std::min(rows, cols), 64);
        steps += (double)t.gram * (gram + rest) + (double)t.full * rest;
        tiles += (double)(2 * t.gram + t.full);
        chain = std::max(chain, gram + 2 * rest);
    }
    const double all = (steps * step + tiles * per_tile) / pairs, longest = chain * chain_step + hand_overs;
    return std::max(all, longest) + 0.35 * std::min(all, longest);
}

// Columns of a tile for a list of tiled matrices on a device of so many SMs.
template <typename F>
uint32_t tile_columns(size_t count, F sides, int sms)
{
    const double pairs = std::max(1, sms / 2);
    return iteration_us(count, sides, 128, pairs) <= iteration_us(count, sides, 256, pairs) ? 128 : 256;
}

}  // namespace zero1
