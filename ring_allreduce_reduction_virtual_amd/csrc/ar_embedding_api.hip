// Host side of the embedding operators, declared in include/ar.h: validation,
// and the ranks' pointers handed to the kernels, up to kEmbeddingRanks ranks a
// launch.

#include <hip/hip_runtime.h>

#include <limits>

#include "ar_embedding.h"
#include "ar_rows.h"

using namespace arimpl;

namespace {

// Sorted places and tokens are 32-bit numbers; columns keep every grid within
// the device's limits.
constexpr uint64_t kMaxTokens = (1ull << 31) - 1, kMaxVocab = (1ull << 31) - 1, kMaxWidth = 1ull << 22;

ar_result_t check_embedding(size_t rows, size_t vocab, size_t cols, ar_index_t index, ar_dtype_t dtype,
                            ar_dtype_t table, double scale, int nranks) {
    ar_result_t rc = check_types(dtype, table, "table", nranks);
    if (rc != AR_SUCCESS || (rc = check_index(index)) != AR_SUCCESS) return rc;
    if (rows > kMaxTokens || vocab > kMaxVocab || cols > kMaxWidth)
        return fail_with(AR_ERR_INVALID_ARGUMENT, "%llu tokens of %llu, %llu columns wide, are too large",
                         static_cast<unsigned long long>(rows), static_cast<unsigned long long>(vocab),
                         static_cast<unsigned long long>(cols));
    const double most = std::numeric_limits<float>::max();
    if (!(scale >= -most && scale <= most))
        return fail_with(AR_ERR_INVALID_ARGUMENT, "scale %g is not a number in float32's range", scale);
    if (scale != 0 && static_cast<float>(scale) == 0.0f)
        return fail_with(AR_ERR_INVALID_ARGUMENT, "scale %g is 0 in float32", scale);
    return AR_SUCCESS;
}

struct Parts {   // of the workspace, in 4-byte words
    uint64_t keys, places, counts, partials;
    uint64_t all() const { return keys + places + counts + partials; }
};
Parts workspace_parts(uint64_t rows, uint64_t cols, int nranks) {
    const uint64_t n = static_cast<uint64_t>(nranks);
    return {n * sort_words(rows), n * sort_words(rows), n * count_words(rows), n * partial_words(rows, cols, nranks)};
}

}  // namespace

extern "C" {

ar_result_t ar_embedding(const void* const* tokens, const void* const* table, void* const* out, size_t rows,
                         size_t vocab, size_t cols, size_t table_stride, size_t out_stride, ar_index_t index_type,
                         ar_dtype_t dtype, ar_dtype_t table_dtype, double scale, int nranks, hipStream_t stream) {
    return guarded([&]() -> ar_result_t {
        ar_result_t rc = check_embedding(rows, vocab, cols, index_type, dtype, table_dtype, scale, nranks);
        if (rc != AR_SUCCESS || (rc = check_stride(table_stride, vocab, cols, "table_stride")) != AR_SUCCESS ||
            (rc = check_stride(out_stride, rows, cols, "out_stride")) != AR_SUCCESS)
            return rc;
        if (tokens == nullptr || table == nullptr || out == nullptr)
            return fail_with(AR_ERR_INVALID_ARGUMENT, "null pointer array");
        if (rows == 0 || cols == 0) return AR_SUCCESS;
        const size_t is = index_size(index_type), es = float_size(dtype), ts = float_size(table_dtype);
        std::vector<Range> v;
        v.reserve(3 * static_cast<size_t>(nranks));
        for (int r = 0; r < nranks; ++r) {
            if ((rc = add_range(v, tokens[r], rows * is, is, false, "tokens", r)) != AR_SUCCESS ||
                (rc = add_rows(v, table[r], vocab, cols, table_stride, ts, false, "table", r)) != AR_SUCCESS ||
                (rc = add_rows(v, out[r], rows, cols, out_stride, es, true, "out", r)) != AR_SUCCESS)
                return rc;
        }
        if ((rc = check_ranges(v)) != AR_SUCCESS) return rc;
        for (int first = 0; first < nranks; first += kEmbeddingRanks) {
            EmbeddingArgs a{};
            const int n = std::min(kEmbeddingRanks, nranks - first);
            for (int k = 0; k < n; ++k) {
                a.tokens[k] = static_cast<const char*>(tokens[first + k]);
                a.table[k] = static_cast<const char*>(table[first + k]);
                a.out[k] = static_cast<char*>(out[first + k]);
            }
            a.rows = rows;
            a.vocab = vocab;
            a.cols = cols;
            a.table_stride = table_stride;
            a.out_stride = out_stride;
            a.scale = static_cast<float>(scale);
            a.wide_index = index_type == AR_INDEX_INT64;
            rc = hip_result(launch_embedding(a, n, dtype, table_dtype, stream), "embedding launch");
            if (rc != AR_SUCCESS) return rc;
        }
        return AR_SUCCESS;
    });
}

size_t ar_embedding_workspace_bytes(size_t rows, size_t vocab, size_t cols, int nranks) {
    if (nranks < 1 || nranks > AR_MAX_RANKS || rows > kMaxTokens || vocab > kMaxVocab || cols > kMaxWidth)
        return static_cast<size_t>(-1);
    return cols == 0 ? 0 : workspace_parts(rows, cols, nranks).all() * 4;
}

ar_result_t ar_embedding_backward(const void* const* dy, const void* const* tokens, void* const* dtable, size_t rows,
                                  size_t vocab, size_t cols, size_t dy_stride, size_t dtable_stride,
                                  ar_index_t index_type, ar_dtype_t dtype, ar_dtype_t table_dtype, double scale,
                                  long long padding_index, int accumulate, int nranks, void* workspace,
                                  size_t workspace_bytes, hipStream_t stream) {
    return guarded([&]() -> ar_result_t {
        ar_result_t rc = check_embedding(rows, vocab, cols, index_type, dtype, table_dtype, scale, nranks);
        if (rc != AR_SUCCESS || (rc = check_stride(dy_stride, rows, cols, "dy_stride")) != AR_SUCCESS ||
            (rc = check_stride(dtable_stride, vocab, cols, "dtable_stride")) != AR_SUCCESS)
            return rc;
        if (dy == nullptr || tokens == nullptr || dtable == nullptr)
            return fail_with(AR_ERR_INVALID_ARGUMENT, "null pointer array");
        if (vocab == 0 || cols == 0) return AR_SUCCESS;
        const size_t is = index_size(index_type), es = float_size(dtype), ts = float_size(table_dtype);
        std::vector<Range> v;
        v.reserve(3 * static_cast<size_t>(nranks) + 1);
        for (int r = 0; r < nranks; ++r) {
            if ((rc = add_rows(v, dy[r], rows, cols, dy_stride, es, false, "dy", r)) != AR_SUCCESS ||
                (rc = add_range(v, tokens[r], rows * is, is, false, "tokens", r)) != AR_SUCCESS ||
                (rc = add_rows(v, dtable[r], vocab, cols, dtable_stride, ts, true, "dtable", r)) != AR_SUCCESS)
                return rc;
        }
        const Parts parts = workspace_parts(rows, cols, nranks);
        if ((rc = add_scratch(v, workspace, workspace_bytes, parts.all() * 4, 4)) != AR_SUCCESS) return rc;
        if ((rc = check_ranges(v)) != AR_SUCCESS) return rc;
        uint32_t* const words = static_cast<uint32_t*>(workspace);
        for (int first = 0; first < nranks; first += kEmbeddingRanks) {
            EmbeddingBackwardArgs a{};
            const int n = std::min(kEmbeddingRanks, nranks - first);
            for (int k = 0; k < n; ++k) {
                a.dy[k] = static_cast<const char*>(dy[first + k]);
                a.tokens[k] = static_cast<const char*>(tokens[first + k]);
                a.dtable[k] = static_cast<char*>(dtable[first + k]);
            }
            if (rows > 0) {
                const uint64_t f = static_cast<uint64_t>(first);
                a.keys = words + f * sort_words(rows);
                a.places = words + parts.keys + f * sort_words(rows);
                a.counts = words + parts.keys + parts.places + f * count_words(rows);
                a.partials = reinterpret_cast<float*>(words + parts.keys + parts.places + parts.counts +
                                                      f * partial_words(rows, cols, nranks));
            }
            a.rows = rows;
            a.vocab = vocab;
            a.cols = cols;
            a.dy_stride = dy_stride;
            a.dtable_stride = dtable_stride;
            a.tiles = sort_tiles(rows);
            a.chunk = sum_chunk(rows, nranks);
            a.chunks = sum_chunks(rows, nranks);
            a.padding = padding_index;
            a.scale = static_cast<float>(scale);
            a.wide_index = index_type == AR_INDEX_INT64;
            a.accumulate = accumulate != 0;
            const int bits = token_bits(vocab);
            a.passes = (bits + kDigitBits - 1) / kDigitBits;
            a.digit_bits = (bits + a.passes - 1) / a.passes;
            a.sorted = rows > kSortOne ? (a.passes - 1) & 1 : 0;
            rc = hip_result(launch_embedding_backward(a, n, dtype, table_dtype, stream), "embedding_backward launch");
            if (rc != AR_SUCCESS) return rc;
        }
        return AR_SUCCESS;
    });
}

}  // extern "C"
