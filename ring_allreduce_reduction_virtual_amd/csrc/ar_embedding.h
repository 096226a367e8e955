// Internal interface of the embedding operators: what the host entry points
// (ar_embedding_api.hip) hand to the kernels (ar_embedding_kernels.hip).  Not
// installed; include/ar.h is the public ABI.
#pragma once

#include <hip/hip_runtime_api.h>

#include <algorithm>
#include <cstdint>

#include "ar.h"

namespace arimpl {

// Ranks of one launch: their pointers travel in the kernel's arguments.
constexpr int kEmbeddingRanks = 32;

struct EmbeddingArgs {
    const char* tokens[kEmbeddingRanks];
    const char* table[kEmbeddingRanks];
    char* out[kEmbeddingRanks];
    uint64_t rows, vocab, cols;
    uint64_t table_stride, out_stride;   // elements
    float scale;
    int wide_index;                      // tokens of 8 bytes, else 4
};

// The gradient sorts each rank's places by token (places of one token stay in
// their order), one digit of the token after the other from the lowest.
constexpr int kSortThreads = 1024;       // of the sort in one workgroup
constexpr int kSortEach = 8;             // places a thread
constexpr uint64_t kSortOne = static_cast<uint64_t>(kSortThreads) * kSortEach;
constexpr int kSortTileThreads = 256;    // of a tile of the sort over many workgroups
constexpr int kSortTileEach = 16;
constexpr uint64_t kSortTile = static_cast<uint64_t>(kSortTileThreads) * kSortTileEach;
constexpr int kDigitBits = 9;            // at most; 18 bits of token take two passes
constexpr int kDigits = 1 << kDigitBits;

// Places of the sorted order that one group of threads adds up (see the
// kernel): few, so that few tokens fill the GPU, or more, which leave fewer
// partial sums.  The choice goes by all ranks' places, so that the grouping of a
// token's sum does too.
constexpr uint64_t kFewPlaces = 16384;
inline uint64_t sum_chunk(uint64_t rows, int nranks) { return rows * nranks <= kFewPlaces ? 8 : 32; }

struct EmbeddingBackwardArgs {
    const char* dy[kEmbeddingRanks];
    const char* tokens[kEmbeddingRanks];
    char* dtable[kEmbeddingRanks];
    uint32_t* keys;       // [rank][2][rows]: the tokens in order (where `sorted` says), and the pass before's
    uint32_t* places;     // [rank][2][rows]: whose they are
    uint32_t* counts;     // [rank][digit][tile]
    float* partials;      // [rank][chunk][2][cols]
    uint64_t rows, vocab, cols;
    uint64_t dy_stride, dtable_stride;
    uint64_t tiles;       // of the sort
    uint64_t chunk;       // places of a chunk of the sum
    uint64_t chunks;
    int64_t padding;
    float scale;
    int wide_index, accumulate;
    int passes, digit_bits;
    int sorted;           // which of the two holds the result
};

inline int token_bits(uint64_t vocab) {   // of the values 0 to vocab (vocab: takes no part)
    int bits = 1;
    while (bits < 63 && (vocab >> bits) != 0) ++bits;
    return bits;
}
inline uint64_t sort_tiles(uint64_t rows) { return (rows + kSortTile - 1) / kSortTile; }
inline uint64_t sum_chunks(uint64_t rows, int nranks) {
    const uint64_t chunk = sum_chunk(rows, nranks);
    return (rows + chunk - 1) / chunk;
}

// 4-byte words of one rank's part of the workspace, in this order.
constexpr uint64_t sort_words(uint64_t rows) { return 2 * rows; }   // keys; places
inline uint64_t count_words(uint64_t rows) { return rows > kSortOne ? sort_tiles(rows) * kDigits : 0; }
inline uint64_t partial_words(uint64_t rows, uint64_t cols, int nranks) { return sum_chunks(rows, nranks) * 2 * cols; }

hipError_t launch_embedding(const EmbeddingArgs& a, int nranks, ar_dtype_t dtype, ar_dtype_t table, hipStream_t stream);
hipError_t launch_embedding_backward(const EmbeddingBackwardArgs& a, int nranks, ar_dtype_t dtype, ar_dtype_t table,
                                     hipStream_t stream);

}  // namespace arimpl
