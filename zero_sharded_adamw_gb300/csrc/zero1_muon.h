// zero1_muon.h -- declarations shared by the matrix optimizer's host code
// (zero1_muon.cu) and its kernels (zero1_muon_kernels.cu).  Not installed.
#pragma once

#include <cstdint>
#include <cuda.h>   // CUtensorMap
#include <cuda_runtime.h>

#include "zero1.h"
#include "zero1_muon_tiles.h"

namespace zero1 {

constexpr int kNsParts = 32;           // arrivals a finished tile makes: one by each warp that writes it
constexpr int kNsTileK = 64;           // K of one pipeline stage
constexpr uint32_t kMaxSide = 1u << 22;
// Powers of two the f16 operands are scaled by: singular values below 2 keep
// every iterate's entries below 2 and the Gram matrices' (and the linear
// term's beside them) below 14, so 2^14 and 2^12 keep them under f16's 65,504.
// An operand is held in a high and a low f16 part whose last places are 2^-24
// at the finest: an entry of X, whose norm starts at one, keeps 22 bits down
// to 2^-17 = 7.6e-6, and below that the absolute error 2^-25 / 2^14 = 1.8e-12;
// a Gram matrix's entries keep 22 bits down to 3.1e-5, and 7.3e-12 below.
constexpr float kXScale = 16384.0f;
constexpr float kGramScale = 4096.0f;

// One matrix of the plan, in device memory.  X (rows x cols) lives in one
// half of a two-region ping-pong; a region holds either two f16 planes (the
// high and the low part of S*X) or one fp32 array, each row padded to ldx.
struct MuonMat {
    uint64_t offset, ld;       // place in the flat buffers: entry (r, c) at offset + r*ld + c
    uint32_t rows, cols;
    uint32_t s;                // the smaller side: the Gram matrix is s x s
    uint32_t tall;             // rows > cols: Gram matrix X^T X, update X B
    uint32_t ldx, lds;         // padded row lengths of X and of the Gram matrices
    unsigned char *region[2];
    unsigned char *gram, *poly;   // A, and the polynomial X is multiplied by: two f16 planes each
    unsigned char *diag;       // diagonal 256 x 256 blocks of A + (b/c) I, one below the other: two f16 planes
    uint64_t xplane, splane;   // entries of one plane
    uint32_t parts[3];         // arrivals of the three products of one iteration: tiles x kNsParts
    uint32_t chunk0, chunks;   // elementwise blocks [chunk0, chunk0 + chunks)
    uint32_t vec;              // rows start and advance in multiples of 8 entries in the flat buffers
    float scale;               // update_scale times the side factor
};

// Tensor maps of one matrix: X in region 0 and 1, A, its diagonal blocks with
// the linear term, and the polynomial.
enum { kMapX0 = 0, kMapX1 = 1, kMapA = 2, kMapD = 3, kMapP = 4, kMapsPerMat = 5 };

// The plan and the workspace of one handle, in device memory.
struct MuonDev {
    const MuonMat *mats;
    const CUtensorMap *maps;
    const uint2 *work;         // one iteration's tiles: x = matrix | phase << 30, y = row tile | column tile << 16
    const uint32_t *chunk_mat; // matrix of each elementwise block
    double *partials;          // one sum of squares a block
    unsigned *done;            // arrivals of finished tiles, one counter a matrix
    unsigned *ticket;
    unsigned *errors;          // sticky: bit 0 = a wait gave up
    uint32_t count, nchunks, work_per_iter;
    uint32_t tile;             // columns of a tile
    uint32_t chunk;            // entries of one elementwise block
};

// Small matrices, whose whole step is one launch (zero1_muon_small.cu): lists
// of them by the number of blocks that share one, 1, 2, 4 or 8.
struct MuonSmall {
    const uint32_t *list;      // device memory: indices into MuonDev::mats
    uint32_t first[kSmallSizes], count[kSmallSizes];
};
constexpr int small_smem(int blocks) { return (int)(2 * 128 * 2 * small_width(blocks)) + (blocks == 1 ? 1 : 2) * 65536 + 1024; }

// Blocks of a cluster that take tensor memory have their SMs to themselves:
// with two such clusters on the same two SMs, each could hold the columns
// that the other's second block waits for.  Shared memory keeps them apart
// (228 KB an SM): 200 KB leave no room for another such block.
constexpr int kAloneSmem = 200 * 1024;
static_assert(small_smem(2) >= kAloneSmem, "two clusters could wait for each other's tensor memory");

struct MuonScalars {
    float inv_w, momentum, one_minus_momentum, eps;
    float lr, decay;           // decay = 1 - lr * weight_decay
    float a, b, c;
    int nesterov, steps;
    int stall;                 // failure test: no tiles are drawn
};

cudaError_t launch_muon_momentum(const MuonDev &d, const MuonScalars &sc, const void *const *grads, int world,
                                 float *momentum, cudaStream_t stream);
cudaError_t launch_muon_norm(const MuonDev &d, const void *in, bool bf16, cudaStream_t stream);
// `in` null: the fp32 update that launch_muon_momentum left in region 1.
cudaError_t launch_muon_split(const MuonDev &d, const MuonScalars &sc, const void *in, bool bf16, cudaStream_t stream);
cudaError_t launch_muon_iterate(const MuonDev &d, const MuonScalars &sc, int num_sms, cudaStream_t stream);
// The blocks of the smallest cluster in use that does not fit the stream's SMs
// (all blocks of a cluster run at once, on SMs of one processing cluster, and
// a stream of an SM partition may have too few of them), or 0 if all fit.
cudaError_t muon_small_misfit(const MuonSmall &small, cudaStream_t stream, int *blocks);
cudaError_t launch_muon_small_step(const MuonDev &d, const MuonSmall &small, const MuonScalars &sc,
                                   const void *const *grads, void *const *params, int world, float *master,
                                   float *momentum, cudaStream_t stream);
cudaError_t launch_muon_small_orth(const MuonDev &d, const MuonSmall &small, const MuonScalars &sc, const void *in,
                                   bool in_bf16, void *out, bool out_bf16, cudaStream_t stream);
cudaError_t launch_muon_apply(const MuonDev &d, const MuonScalars &sc, void *const *params, int world, float *master,
                              cudaStream_t stream);
cudaError_t launch_muon_out(const MuonDev &d, const MuonScalars &sc, void *out, bool bf16, cudaStream_t stream);

}  // namespace zero1
