// Internal interface of the cross entropy of unstored logits: what the host
// entry points (ar_cross_entropy_api.hip) hand to the kernels
// (ar_cross_entropy_kernels.hip).  Not installed; include/ar.h is the public
// ABI.
#pragma once

#include <hip/hip_runtime_api.h>

#include <algorithm>
#include <cstdint>

#include "ar.h"

namespace arimpl {

// Ranks of one launch: their pointers travel in the kernel's arguments.
constexpr int kCrossRanks = 32;

// Columns of a matrix product's operand are read 16 bytes at a time, so
// operands that do not start, or whose rows do not lie, on 16 bytes are copied
// first, each row with zeros up to a whole number of them.
constexpr int kOperandBytes = 16;
constexpr uint64_t padded_cols(uint64_t cols, uint64_t es) {
    return (cols * es + kOperandBytes - 1) / kOperandBytes * kOperandBytes / es;
}

// The vocabulary is worked off in pieces of whole tiles.  A piece's dz is
// written once and read twice; kPieceBytes of it in all keeps it in the 256 MB
// last-level cache, while a piece of kLeastPiece columns or more keeps the sum
// over it, and so the number of times that dx's sums are read and written,
// worth a launch.
constexpr uint64_t kVocabTile = 256;
constexpr uint64_t kPieceBytes = 256ull << 20, kLeastPiece = 2048;
inline uint64_t piece_of(uint64_t rows, uint64_t vocab, uint64_t es, int nranks) {
    const uint64_t tiles = (vocab + kVocabTile - 1) / kVocabTile;
    const uint64_t row_bytes = std::max<uint64_t>(1, rows) * nranks * es;
    const uint64_t most = std::max<uint64_t>(kLeastPiece, kPieceBytes / row_bytes) / kVocabTile;
    const uint64_t pieces = (tiles + most - 1) / most;
    return (tiles + pieces - 1) / pieces * kVocabTile;
}

// Large tiles need rows to fill them.
constexpr uint64_t kFewRows = 128;
constexpr uint64_t vocab_tile(uint64_t rows) { return rows <= kFewRows ? 128 : 256; }

// A rank's row of a launch, in the order of the rows that take part.
struct LiveRow {
    int64_t target;   // -1: none in the vocabulary (its g is NaN)
    float g, lse;
};

struct CrossArgs {
    // as given, or copies with aligned rows
    const char* x[kCrossRanks];
    const char* weight[kCrossRanks];
    const char* targets[kCrossRanks];
    const float* dloss[kCrossRanks];
    const float* lse_in[kCrossRanks];
    float* loss[kCrossRanks];
    float* lse[kCrossRanks];
    char* dx[kCrossRanks];
    char* dweight[kCrossRanks];
    uint64_t rows, vocab, cols;
    uint64_t x_stride, weight_stride, dx_stride, dweight_stride;   // elements
    int64_t ignore;
    float scale;
    int wide_index;
    // the piece of the vocabulary: its first column, its columns, their padded number
    uint64_t first, count, piece;
    // workspace, each part [rank of the launch][...]
    float* partials;      // forward: [tile of the vocabulary][row][2]: maximum, sum of exponentials
    float* target_logit;  // forward: [row]
    uint32_t tiles;       // of the vocabulary
    uint32_t* live_count; // backward: [1]
    uint32_t* place;      // backward: [row]: its place among the live rows, or ~0
    float* unscale;       // backward: [1]: undoes binary16's scaling
    LiveRow* live;        // backward: [row]
    char* x_live;         // backward: [row][padded cols]: the live rows of x
    char* dz;             // backward: [row][piece]
    float* sums;          // backward: [split][row][cols up to a multiple of 4]
    uint32_t splits;      // of the sum over a piece's vocabulary
};

inline uint64_t sum_cols(uint64_t cols) { return (cols + 3) / 4 * 4; }

// How many parts the sum over a piece is cut into so that few rows fill the
// GPU; at least 1,024 columns each.
inline uint32_t dx_splits(uint64_t rows, uint64_t cols, uint64_t piece, int nranks) {
    const uint64_t tiles = nranks * ((rows + 63) / 64) * ((cols + 127) / 128);
    const uint64_t wanted = tiles >= 256 ? 1 : 512 / std::max<uint64_t>(1, tiles);
    return static_cast<uint32_t>(std::max<uint64_t>(1, std::min(wanted, piece / 1024)));
}

// Copies of rows with zeros behind them: rows [first, first + count) of weight.
struct AlignArgs {
    const char* from[kCrossRanks];
    char* to;             // [rank][count][to_stride]
    uint64_t count, cols, from_stride, to_stride;
};
hipError_t launch_align(const AlignArgs& a, int nranks, ar_dtype_t dtype, hipStream_t stream);

// A piece's maxima and sums, then, after all pieces, the losses.
hipError_t launch_cross_stats(const CrossArgs& a, int nranks, ar_dtype_t dtype, hipStream_t stream);
hipError_t launch_cross_loss(const CrossArgs& a, int nranks, hipStream_t stream);
// The live rows, and their copies of x.
hipError_t launch_cross_live(const CrossArgs& a, int nranks, ar_dtype_t dtype, hipStream_t stream);
// A piece's dz, then its part of dx's sums and its rows of dweight.
hipError_t launch_cross_dz(const CrossArgs& a, int nranks, ar_dtype_t dtype, hipStream_t stream);
hipError_t launch_cross_dx(const CrossArgs& a, int nranks, bool add, ar_dtype_t dtype, hipStream_t stream);
hipError_t launch_cross_dweight(const CrossArgs& a, int nranks, ar_dtype_t dtype, hipStream_t stream);
hipError_t launch_cross_finish(const CrossArgs& a, int nranks, ar_dtype_t dtype, hipStream_t stream);

}  // namespace arimpl
