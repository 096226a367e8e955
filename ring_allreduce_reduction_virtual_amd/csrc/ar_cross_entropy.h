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
// first, each row with zeros up to a whole number of them; and so are those
// whose rows lie too far apart for 32-bit offsets.
constexpr int kOperandBytes = 16;
constexpr uint64_t kMostOperandStride = 1u << 23;
constexpr uint64_t padded_cols(uint64_t cols, uint64_t es) {
    return (cols * es + kOperandBytes - 1) / kOperandBytes * kOperandBytes / es;
}

// With few rows, reading the weight is the time, and its copy three times that:
// float32 operands are then read 4 bytes at a time where they lie.  Copied / in
// place, us: forward, 2 x 2 rows of 817 against 34,928 152 / 77, 55 of 490
// against 122,842 181 / 115, 59 of 3,110 against 1,611 65 / 70, 3 x 129 of 515
// against 5,003 56 / 55, 4 x 424 of 1,223 against 55,858 2,374 / 2,820;
// backward, whose one copy serves two products, the same 298 / 239, 397 / 371,
// 97 / 116, 131 / 154, 6,435 / 7,596.
constexpr uint64_t kWordRows = 64, kWordRowsBackward = 32;
constexpr bool in_words(uint64_t rows, uint64_t es, bool backward) {
    return es == 4 && rows <= (backward ? kWordRowsBackward : kWordRows);
}

constexpr uint64_t kVocabTile = 256;   // of the vocabulary's pieces: whole ones of any tile

// Tiles of the products, m x n: the large one keeps the matrix cores busiest,
// the smaller ones give few rows or columns more workgroups.
enum class CrossTile : int { kTiny = 0, kSmall, kMedium, kLarge };
constexpr uint64_t tile_m(CrossTile t) { return t == CrossTile::kLarge ? 256 : t == CrossTile::kTiny ? 64 : 128; }
constexpr uint64_t tile_n(CrossTile t) {
    return t == CrossTile::kLarge ? 256 : t == CrossTile::kMedium ? 128 : t == CrossTile::kSmall ? 64 : 32;
}
// The share of the large tile's rate that a tile reaches when it fills the GPU.
// Measured on MI355X, TFLOP/s, tiny / small / medium / large: bf16, 2 x 4,096
// rows of 4,096 against 65,536, forward 409 / 767 / 994 / 1,319, backward (6
// per logit and column) 346 / 702 / 970 / 1,269; float32, 2 x 4,096 rows of
// 2,048 against 32,768, forward 120 / 131 / 141 / 145, backward 117 / 130 / 139 /
// 143.  Where the large tile leaves compute units without work the others are
// ahead, us, forward and backward: bf16, 512 rows of 1,024 against 8,192 31 + 105 /
// 20 + 70 / 17 + 64 / 28 + 93 (picked: 17 + 65); 16 rows of 4,096 against 65,536
// 111 + 876 / 118 + 529 / 136 + 513 / 150 + 517 (picked: 110 + 447); float32, 3 x
// 129 rows of 515 against 5,003 56 + 132 / 62 + 167 / 61 + 158 / 154 + 337
// (picked: 56 + 132).
inline double tile_rate(CrossTile t, bool wide) {
    switch (t) {
        case CrossTile::kLarge: return 1.0;
        case CrossTile::kMedium: return wide ? 0.97 : 0.75;
        case CrossTile::kSmall: return wide ? 0.9 : 0.56;
        default: return wide ? 0.8 : 0.3;
    }
}
inline uint64_t tiles_in(uint64_t m, uint64_t n, CrossTile t) {
    return (m + tile_m(t) - 1) / tile_m(t) * ((n + tile_n(t) - 1) / tile_n(t));
}
constexpr uint64_t tile_threads(CrossTile t) { return t == CrossTile::kLarge || t == CrossTile::kMedium ? 512 : 256; }
// A launch's threads are counted with 32 bits: the workgroups that it has, whole
// eights of them (one for each XCD), and whether `batch` products of m x n fit.
constexpr uint64_t most_blocks(CrossTile t) { return 0xffffffffull / tile_threads(t) / 8 * 8; }
inline bool fits_launch(CrossTile t, uint64_t m, uint64_t n, uint64_t batch) {
    return tiles_in(m, n, t) * batch <= most_blocks(t);
}
constexpr uint64_t kUnits = 256;   // compute units
// Microseconds of `batch` products of m x n x depth: what the compute unit with
// the most tiles takes, at the large tile's 5.3 (float32: 0.56) TFLOP/s each.
inline double tile_time(CrossTile t, uint64_t m, uint64_t n, uint64_t depth, uint64_t batch, bool wide) {
    const uint64_t turns = (tiles_in(m, n, t) * batch + kUnits - 1) / kUnits;
    return 2e-6 * turns * tile_m(t) * tile_n(t) * depth / (tile_rate(t, wide) * (wide ? 0.56 : 5.3));
}
constexpr CrossTile kCrossTiles[] = {CrossTile::kLarge, CrossTile::kMedium, CrossTile::kSmall, CrossTile::kTiny};
inline CrossTile pick_tile(uint64_t m, uint64_t n, uint64_t batch, bool wide) {
    CrossTile best = CrossTile::kLarge;
    for (const CrossTile t : kCrossTiles) {
        if (tile_time(t, m, n, 1, batch, wide) < tile_time(best, m, n, 1, batch, wide)) best = t;
    }
    return best;
}
inline CrossTile forward_tile(uint64_t rows, uint64_t vocab, uint64_t es, int nranks) {
    return pick_tile(vocab, rows, nranks, es == 4);
}
// Columns of the vocabulary, whole tiles, that one forward launch has room for:
// at least one tile while the ranks of a launch have no more than kMostRows rows.
constexpr uint64_t kMostRows = 1ull << 28;
static_assert(kMostRows / tile_n(CrossTile::kTiny) <= most_blocks(CrossTile::kTiny) &&
                  kMostRows / tile_n(CrossTile::kMedium) <= most_blocks(CrossTile::kMedium),
              "a tile for every row: fewest rows a workgroup of 256 threads, and of 512");
inline uint64_t launch_vocab(CrossTile t, uint64_t rows, int nranks) {
    return most_blocks(t) / (tiles_in(1, rows, t) * nranks) * tile_m(t);
}

// The backward pass works the vocabulary off in pieces of whole tiles, so that
// what it keeps of dz is bounded whatever the vocabulary is: kPieceBytes in all,
// or kLeastPiece columns.  Every piece more reads and writes dx's float32 sums
// once more.  ms with 128 / 256 / 512 / 1,024 MiB, bf16: 2 x 4,096 rows of 4,096
// against 65,536 10.5 / 10.45 / 10.45 / 10.4, 8 x 2,048 rows of 768 against
// 50,257 4.41 / 4.34 / 4.27 / 4.05, 4 x 4,096 of 2,048 against 32,768 5.78 /
// 5.63 / 5.56 / 5.56.
constexpr uint64_t kPieceBytes = 512ull << 20, kLeastPiece = 2048;
// A weight that is copied is worked off in pieces in both passes: of kCopyBytes
// (the backward pass: kCopyBytesBackward) of all ranks, or as many rows as give
// each compute unit a tile (and the backward pass kLeastPiece).  us with 64 / 128 /
// 256 / 512 MiB, bf16, forward and backward: 16 rows of 4,095 against 65,536 340 /
// 293 / 311 / 333 and 790 / 735 / 698 / 755, 2 x 1,024 of 4,095 against 65,536
// 1,670 / 1,210 / 1,280 / 1,270 and 4,200 / 3,580 / 3,570 / 3,530, 2 x 4,096 of
// 4,095 against 65,536 3,590 / 3,560 / 3,610 / 3,590 and 11,640 / 11,170 / 11,080 /
// 11,090: what is copied comes back from the last-level cache.
constexpr uint64_t kCopyBytes = 128ull << 20, kCopyBytesBackward = 256ull << 20;
inline uint64_t even_pieces(uint64_t vocab, uint64_t most) {   // whole tiles
    const uint64_t tiles = (vocab + kVocabTile - 1) / kVocabTile, each = std::max<uint64_t>(1, most / kVocabTile);
    const uint64_t pieces = (tiles + each - 1) / each;
    return (tiles + pieces - 1) / pieces * kVocabTile;
}
// Rows of the weight that give each compute unit a tile.
inline uint64_t one_turn(uint64_t rows, uint64_t vocab, uint64_t es, int nranks) {
    const CrossTile t = pick_tile(vocab, rows, nranks, es == 4);
    const uint64_t beside = std::max<uint64_t>(1, tiles_in(1, rows, t) * nranks);
    return ((kUnits + beside - 1) / beside * tile_m(t) + kVocabTile - 1) / kVocabTile * kVocabTile;
}
// copy_bytes: of a copied row of the weight; 0: read where it lies.
inline uint64_t forward_piece(uint64_t rows, uint64_t vocab, uint64_t es, uint64_t copy_bytes, int nranks) {
    if (copy_bytes == 0) return even_pieces(vocab, vocab + kVocabTile);
    return even_pieces(vocab, std::max(one_turn(rows, vocab, es, nranks), kCopyBytes / (copy_bytes * nranks)));
}
inline uint64_t piece_of(uint64_t rows, uint64_t vocab, uint64_t es, uint64_t copy_bytes, int nranks) {
    const uint64_t row_bytes = std::max<uint64_t>(1, rows) * nranks * es;
    uint64_t most = std::min(std::max(kLeastPiece, kPieceBytes / row_bytes), kMostOperandStride / es);
    if (copy_bytes != 0)
        most = std::min(most, std::max({kLeastPiece, one_turn(rows, vocab, es, nranks),
                                        kCopyBytesBackward / (copy_bytes * nranks)}));
    return even_pieces(vocab, most);
}

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
    int whole;   // 0: float32 x (forward) and weight are read 4 bytes at a time
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
    float* unscale;       // backward: [1]: undoes the scaling of 16-bit dz
    LiveRow* live;        // backward: [row]
    char* x_live;         // backward: [row][padded cols]: the live rows of x
    char* dz;             // backward: [row][piece]
    float* sums;          // backward: [split][row][cols up to a multiple of 4]
    uint32_t splits;      // of the sum over a piece's vocabulary
};

inline uint64_t sum_cols(uint64_t cols) { return (cols + 3) / 4 * 4; }

// The tile of dx's sums, and how many parts the sum over a piece is cut into:
// few rows and columns make few tiles, and parts (at least 256 of the
// vocabulary each) more, at the cost of writing and reading their sums, 8 bytes
// each at 4 TB/s.
struct DxShape {
    CrossTile tile;
    uint32_t splits;
};
inline DxShape dx_shape(uint64_t rows, uint64_t cols, uint64_t piece, uint64_t es, int nranks) {
    DxShape best{CrossTile::kLarge, 1};
    double least = 0;
    for (const CrossTile t : kCrossTiles) {
        for (uint64_t s = 1; s <= piece / kVocabTile && s <= 64; s *= 2) {
            const double time = tile_time(t, cols, rows, (piece + s - 1) / s, s * nranks, es == 4) +
                                8e-6 / 4 * static_cast<double>(s * nranks * rows * cols);
            if (least == 0 || time < least) {
                least = time;
                best = {t, static_cast<uint32_t>(s)};
            }
        }
    }
    return best;
}

// Copies of rows with zeros behind them: rows [first, first + count) of weight.
struct AlignArgs {
    const char* from[kCrossRanks];
    char* to;             // [rank][count][to_stride]
    uint64_t count, cols, from_stride, to_stride;
};
hipError_t launch_align(const AlignArgs& a, int nranks, ar_dtype_t dtype, hipStream_t stream);

// A piece's maxima and sums, then, after all pieces, the losses.
hipError_t launch_cross_stats(const CrossArgs& a, int nranks, CrossTile tile, ar_dtype_t dtype, hipStream_t stream);
hipError_t launch_cross_loss(const CrossArgs& a, int nranks, hipStream_t stream);
// The live rows, and their copies of x.
hipError_t launch_cross_live(const CrossArgs& a, int nranks, ar_dtype_t dtype, hipStream_t stream);
// A piece's dz, then its part of dx's sums and its rows of dweight.
hipError_t launch_cross_dz(const CrossArgs& a, int nranks, ar_dtype_t dtype, hipStream_t stream);
hipError_t launch_cross_dx(const CrossArgs& a, int nranks, bool add, CrossTile tile, ar_dtype_t dtype,
                           hipStream_t stream);
hipError_t launch_cross_dweight(const CrossArgs& a, int nranks, ar_dtype_t dtype, hipStream_t stream);
hipError_t launch_cross_finish(const CrossArgs& a, int nranks, ar_dtype_t dtype, hipStream_t stream);

}  // namespace arimpl
