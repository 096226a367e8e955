// Host side of the cross entropy of unstored logits, declared in include/ar.h:
// validation, the parts of the workspace, and the launches piece by piece of
// the vocabulary, up to kCrossRanks ranks a launch.

#include <hip/hip_runtime.h>

#include <limits>

#include "ar_cross_entropy.h"
#include "ar_rows.h"

using namespace arimpl;

namespace {

constexpr uint64_t kMaxTokens = (1ull << 31) - 1, kMaxVocab = (1ull << 31) - 1, kMaxWidth = 1ull << 20;
// Rows of a launch's ranks, those of each rounded up to whole tiles.
bool rows_fit(uint64_t rows, int nranks) {
    return tiles_in(1, rows, CrossTile::kLarge) * nranks * tile_n(CrossTile::kLarge) <= kMostRows;
}

ar_result_t check_sizes(size_t rows, size_t vocab, size_t cols, ar_dtype_t dtype, int nranks, bool backward) {
    const ar_result_t rc = check_types(dtype, dtype, "same", nranks);
    if (rc != AR_SUCCESS) return rc;
    if (vocab == 0) return fail_with(AR_ERR_INVALID_ARGUMENT, "a vocabulary of 0");
    const int n = std::min(nranks, kCrossRanks);
    bool fits = rows <= kMaxTokens && vocab <= kMaxVocab && cols <= kMaxWidth && rows_fit(rows, n);
    if (fits && backward) {   // its launches, with the weight as it lies and copied; the forward pass's are cut to fit
        const uint64_t es = float_size(dtype);
        const bool wide = es == 4;
        for (uint64_t piece = piece_of(rows, vocab, es, 0, n), checked = 0; fits && piece != checked;
             checked = piece, piece = piece_of(rows, vocab, es, padded_cols(cols, es) * es, n)) {
            const DxShape dx = dx_shape(rows, cols, piece, es, n);
            fits = fits_launch(pick_tile(piece, rows, n, wide), piece, rows, n) &&
                   fits_launch(dx.tile, cols, rows, static_cast<uint64_t>(n) * dx.splits) &&
                   fits_launch(pick_tile(cols, piece, n, wide), cols, piece, n) &&
                   fits_launch(pick_tile(cols, vocab % piece, n, wide), cols, vocab % piece, n);
        }
    }
    if (!fits)
        return fail_with(AR_ERR_INVALID_ARGUMENT, "%llu rows of %llu columns against a vocabulary of %llu are too large",
                         static_cast<unsigned long long>(rows), static_cast<unsigned long long>(cols),
                         static_cast<unsigned long long>(vocab));
    return AR_SUCCESS;
}

// The parts of the workspace, in bytes from its start.  `aligned`: no operand
// needs a copy.
struct Layout {
    uint64_t piece = 0, padded = 0, all = 0;
    uint64_t x = 0, weight = 0;                                                    // aligned copies, or live rows
    uint64_t partials = 0, target_logit = 0;                                       // forward
    uint64_t live_count = 0, place = 0, unscale = 0, live = 0, dz = 0, sums = 0;   // backward
    DxShape dx{};
    CrossTile tile{};
    uint64_t tiles = 0;   // forward, of the vocabulary

    uint64_t take(uint64_t bytes) {
        const uint64_t at = all;
        all += (bytes + 255) / 256 * 256;
        return at;
    }
    Layout(uint64_t rows, uint64_t vocab, uint64_t cols, ar_dtype_t dtype, int nranks, bool backward, bool aligned) {
        const uint64_t n = static_cast<uint64_t>(std::min(nranks, kCrossRanks)), es = float_size(dtype);
        padded = padded_cols(cols, es);
        const bool copies = !aligned && !in_words(rows, es, backward);
        const uint64_t copy_bytes = copies ? padded * es : 0;
        piece = backward ? piece_of(rows, vocab, es, copy_bytes, static_cast<int>(n))
                         : forward_piece(rows, vocab, es, copy_bytes, static_cast<int>(n));
        if (backward || copies) x = take(n * rows * padded * es);
        if (copies) weight = take(n * std::min(piece, vocab) * padded * es);
        if (backward) {
            dx = dx_shape(rows, cols, piece, es, static_cast<int>(n));
            live_count = take(n * 4);
            unscale = take(n * 4);
            place = take(n * rows * 4);
            live = take(n * rows * sizeof(LiveRow));
            dz = take(n * rows * piece * es);
            sums = take(n * dx.splits * rows * sum_cols(cols) * 4);
        } else {
            tile = forward_tile(rows, vocab, es, static_cast<int>(n));
            tiles = (vocab + tile_m(tile) - 1) / tile_m(tile);
            partials = take(n * tiles * rows * 8);
            target_logit = take(n * rows * 4);
        }
    }
};

// Whether an operand's rows can be read 16 bytes at a time, with nothing but
// the row's own elements in the last ones.
bool aligned(const void* const* p, int n, uint64_t stride, uint64_t cols, uint64_t es) {
    if (stride * es % kOperandBytes != 0 || cols * es % kOperandBytes != 0 || stride * es > kMostOperandStride)
        return false;
    for (int r = 0; r < n; ++r) {
        if (reinterpret_cast<uintptr_t>(p[r]) % kOperandBytes != 0) return false;
    }
    return true;
}

// Rows [first, first + count) of n operands, copied with aligned rows.
ar_result_t align(const void* const* from, int n, uint64_t first, uint64_t count, uint64_t cols, uint64_t stride,
                  uint64_t padded, ar_dtype_t dtype, char* to, const char** copies, hipStream_t stream) {
    const uint64_t es = float_size(dtype);
    AlignArgs c{};
    for (int k = 0; k < n; ++k) {
        c.from[k] = static_cast<const char*>(from[k]) + first * stride * es;
        copies[k] = to + static_cast<uint64_t>(k) * count * padded * es;
    }
    c.to = to;
    c.count = count;
    c.cols = cols;
    c.from_stride = stride;
    c.to_stride = padded;
    return hip_result(launch_align(c, n, dtype, stream), "aligned copy launch");
}

// One piece's rows of the weight in a.weight, copied where they have to be.
ar_result_t set_piece(CrossArgs& a, const Layout& at, char* ws, const void* const* weight, int n, uint64_t first,
                      uint64_t count, uint64_t stride, bool as_is, ar_dtype_t dtype, hipStream_t stream) {
    a.first = first;
    a.count = count;
    if (!as_is) {
        a.weight_stride = at.padded;
        return align(weight, n, first, count, a.cols, stride, at.padded, dtype, ws + at.weight, a.weight, stream);
    }
    a.weight_stride = stride;
    for (int k = 0; k < n; ++k) a.weight[k] = static_cast<const char*>(weight[k]) + first * stride * float_size(dtype);
    return AR_SUCCESS;
}

}  // namespace

extern "C" {

size_t ar_cross_entropy_workspace_bytes(size_t rows, size_t vocab, size_t cols, ar_dtype_t dtype, int nranks,
                                        int backward) {
    set_error_detail("");
    if (check_sizes(rows, vocab, cols, dtype, nranks, backward != 0) != AR_SUCCESS) return static_cast<size_t>(-1);
    // smaller pieces can need less than none to copy
    return std::max(Layout(rows, vocab, cols, dtype, nranks, backward != 0, false).all,
                    Layout(rows, vocab, cols, dtype, nranks, backward != 0, true).all);
}

size_t ar_cross_entropy_aligned_workspace_bytes(size_t rows, size_t vocab, size_t cols, ar_dtype_t dtype, int nranks,
                                                int backward) {
    set_error_detail("");
    if (check_sizes(rows, vocab, cols, dtype, nranks, backward != 0) != AR_SUCCESS) return static_cast<size_t>(-1);
    if (cols * float_size(dtype) % kOperandBytes != 0)   // they cannot be
        return ar_cross_entropy_workspace_bytes(rows, vocab, cols, dtype, nranks, backward);
    return Layout(rows, vocab, cols, dtype, nranks, backward != 0, true).all;
}

ar_result_t ar_cross_entropy(const void* const* x, const void* const* weight, const void* const* targets,
                             float* const* loss, float* const* lse, size_t rows, size_t vocab, size_t cols,
                             size_t x_stride, size_t weight_stride, ar_index_t index_type, long long ignore_index,
                             ar_dtype_t dtype, int nranks, void* workspace, size_t workspace_bytes,
                             hipStream_t stream) {
    return guarded([&]() -> ar_result_t {
        ar_result_t rc = check_sizes(rows, vocab, cols, dtype, nranks, false);
        if (rc != AR_SUCCESS || (rc = check_index(index_type)) != AR_SUCCESS ||
            (rc = check_stride(x_stride, rows, cols, "x_stride")) != AR_SUCCESS ||
            (rc = check_stride(weight_stride, vocab, cols, "weight_stride")) != AR_SUCCESS)
            return rc;
        if (x == nullptr || weight == nullptr || targets == nullptr || loss == nullptr || lse == nullptr)
            return fail_with(AR_ERR_INVALID_ARGUMENT, "null pointer array");
        if (rows == 0) return AR_SUCCESS;
        const size_t is = index_size(index_type), es = float_size(dtype);
        std::vector<Range> v;
        v.reserve(5 * static_cast<size_t>(nranks) + 1);
        for (int r = 0; r < nranks; ++r) {
            if ((rc = add_rows(v, x[r], rows, cols, x_stride, es, false, "x", r)) != AR_SUCCESS ||
                (rc = add_rows(v, weight[r], vocab, cols, weight_stride, es, false, "weight", r)) != AR_SUCCESS ||
                (rc = add_range(v, targets[r], rows * is, is, false, "targets", r)) != AR_SUCCESS ||
                (rc = add_range(v, loss[r], rows * 4, 4, true, "loss", r)) != AR_SUCCESS ||
                (rc = add_range(v, lse[r], rows * 4, 4, true, "lse", r)) != AR_SUCCESS)
                return rc;
        }
        const bool all_aligned = aligned(x, nranks, x_stride, cols, es) && aligned(weight, nranks, weight_stride, cols, es);
        const Layout at(rows, vocab, cols, dtype, nranks, false, all_aligned);
        if ((rc = add_scratch(v, workspace, workspace_bytes, at.all, 16)) != AR_SUCCESS) return rc;
        if ((rc = check_ranges(v)) != AR_SUCCESS) return rc;
        char* const ws = static_cast<char*>(workspace);
        for (int g = 0; g < nranks; g += kCrossRanks) {
            CrossArgs a{};
            const int n = std::min(kCrossRanks, nranks - g);
            a.rows = rows;
            a.vocab = vocab;
            a.cols = cols;
            a.ignore = ignore_index;
            a.wide_index = index_type == AR_INDEX_INT64;
            a.partials = reinterpret_cast<float*>(ws + at.partials);
            a.target_logit = reinterpret_cast<float*>(ws + at.target_logit);
            a.tiles = static_cast<uint32_t>(at.tiles);
            for (int k = 0; k < n; ++k) {
                a.x[k] = static_cast<const char*>(x[g + k]);
                a.targets[k] = static_cast<const char*>(targets[g + k]);
                a.loss[k] = loss[g + k];
                a.lse[k] = lse[g + k];
            }
            a.x_stride = x_stride;
            const bool x_aligned = aligned(x + g, n, x_stride, cols, es);
            const bool weight_aligned = aligned(weight + g, n, weight_stride, cols, es);
            const bool words = in_words(rows, es, false) && !(x_aligned && weight_aligned);
            a.whole = !words;
            if (!x_aligned && !words) {
                a.x_stride = at.padded;
                rc = align(x + g, n, 0, rows, cols, x_stride, at.padded, dtype, ws + at.x, a.x, stream);
                if (rc != AR_SUCCESS) return rc;
            }
            // a weight that needs no copy is one piece, as far as one launch goes
            const bool as_is = weight_aligned || words;
            const uint64_t most = launch_vocab(at.tile, rows, n);
            for (uint64_t first = 0; first < vocab;) {
                const uint64_t count = std::min<uint64_t>(vocab - first, as_is ? most : std::min(most, at.piece));
                rc = set_piece(a, at, ws, weight + g, n, first, count, weight_stride, as_is, dtype, stream);
                if (rc == AR_SUCCESS)
                    rc = hip_result(launch_cross_stats(a, n, at.tile, dtype, stream), "cross_entropy launch");
                if (rc != AR_SUCCESS) return rc;
                first += count;
            }
            if ((rc = hip_result(launch_cross_loss(a, n, stream), "cross_entropy launch")) != AR_SUCCESS) return rc;
        }
        return AR_SUCCESS;
    });
}

ar_result_t ar_cross_entropy_backward(const float* const* dloss, const void* const* x, const void* const* weight,
                                      const void* const* targets, const float* const* lse, void* const* dx,
                                      void* const* dweight, size_t rows, size_t vocab, size_t cols, size_t x_stride,
                                      size_t weight_stride, size_t dx_stride, size_t dweight_stride,
                                      ar_index_t index_type, long long ignore_index, ar_dtype_t dtype, double scale,
                                      int nranks, void* workspace, size_t workspace_bytes, hipStream_t stream) {
    return guarded([&]() -> ar_result_t {
        ar_result_t rc = check_sizes(rows, vocab, cols, dtype, nranks, true);
        if (rc != AR_SUCCESS || (rc = check_index(index_type)) != AR_SUCCESS ||
            (rc = check_stride(x_stride, rows, cols, "x_stride")) != AR_SUCCESS ||
            (rc = check_stride(weight_stride, vocab, cols, "weight_stride")) != AR_SUCCESS ||
            (dx != nullptr && (rc = check_stride(dx_stride, rows, cols, "dx_stride")) != AR_SUCCESS) ||
            (dweight != nullptr && (rc = check_stride(dweight_stride, vocab, cols, "dweight_stride")) != AR_SUCCESS))
            return rc;
        const double most = std::numeric_limits<float>::max();
        if (!(scale >= -most && scale <= most))
            return fail_with(AR_ERR_INVALID_ARGUMENT, "scale %g is not a number in float32's range", scale);
        if (scale != 0 && static_cast<float>(scale) == 0.0f)
            return fail_with(AR_ERR_INVALID_ARGUMENT, "scale %g is 0 in float32", scale);
        if (x == nullptr || weight == nullptr || targets == nullptr || lse == nullptr)
            return fail_with(AR_ERR_INVALID_ARGUMENT, "null pointer array");
        const size_t is = index_size(index_type), es = float_size(dtype);
        std::vector<Range> v;
        v.reserve(7 * static_cast<size_t>(nranks) + 1);
        for (int r = 0; r < nranks; ++r) {
            const bool in_place = dx != nullptr && dx[r] == x[r] && dx_stride == x_stride;
            if ((!in_place && (rc = add_rows(v, x[r], rows, cols, x_stride, es, false, "x", r)) != AR_SUCCESS) ||
                (rc = add_rows(v, weight[r], vocab, cols, weight_stride, es, false, "weight", r)) != AR_SUCCESS ||
                (rc = add_range(v, targets[r], rows * is, is, false, "targets", r)) != AR_SUCCESS ||
                (rc = add_range(v, lse[r], rows * 4, 4, false, "lse", r)) != AR_SUCCESS ||
                (dloss != nullptr &&
                 (rc = add_range(v, dloss[r], rows * 4, 4, false, "dloss", r)) != AR_SUCCESS) ||
                (dx != nullptr &&
                 (rc = add_rows(v, dx[r], rows, cols, dx_stride, es, true, "dx", r)) != AR_SUCCESS) ||
                (dweight != nullptr &&
                 (rc = add_rows(v, dweight[r], vocab, cols, dweight_stride, es, true, "dweight", r)) != AR_SUCCESS))
                return rc;
        }
        const Layout at(rows, vocab, cols, dtype, nranks, true, aligned(weight, nranks, weight_stride, cols, es));
        if ((rc = add_scratch(v, workspace, workspace_bytes, at.all, 16)) != AR_SUCCESS) return rc;
        if ((rc = check_ranges(v)) != AR_SUCCESS) return rc;
        if (cols == 0 || (dx == nullptr && dweight == nullptr) || (rows == 0 && dweight == nullptr)) return AR_SUCCESS;
        char* const ws = static_cast<char*>(workspace);
        for (int g = 0; g < nranks; g += kCrossRanks) {
            CrossArgs a{};
            const int n = std::min(kCrossRanks, nranks - g);
            a.rows = rows;
            a.vocab = vocab;
            a.cols = cols;
            a.x_stride = x_stride;
            a.dx_stride = dx_stride;
            a.dweight_stride = dweight_stride;
            a.ignore = ignore_index;
            a.scale = static_cast<float>(scale);
            a.wide_index = index_type == AR_INDEX_INT64;
            a.piece = at.piece;
            a.splits = at.dx.splits;
            a.live_count = reinterpret_cast<uint32_t*>(ws + at.live_count);
            a.place = reinterpret_cast<uint32_t*>(ws + at.place);
            a.unscale = reinterpret_cast<float*>(ws + at.unscale);
            a.live = reinterpret_cast<LiveRow*>(ws + at.live);
            a.x_live = ws + at.x;
            a.dz = ws + at.dz;
            a.sums = reinterpret_cast<float*>(ws + at.sums);
            for (int k = 0; k < n; ++k) {
                a.x[k] = static_cast<const char*>(x[g + k]);
                a.targets[k] = static_cast<const char*>(targets[g + k]);
                a.dloss[k] = dloss == nullptr ? nullptr : dloss[g + k];
                a.lse_in[k] = lse[g + k];
                a.dx[k] = dx == nullptr ? nullptr : static_cast<char*>(dx[g + k]);
                a.dweight[k] = dweight == nullptr ? nullptr : static_cast<char*>(dweight[g + k]);
            }
            const char* const what = "cross_entropy_backward launch";
            if ((rc = hip_result(launch_cross_live(a, n, dtype, stream), what)) != AR_SUCCESS) return rc;
            const bool weight_aligned = aligned(weight + g, n, weight_stride, cols, es);
            a.whole = weight_aligned || !in_words(rows, es, true);
            const bool as_is = weight_aligned || !a.whole;
            for (uint64_t first = 0; first < vocab; first += at.piece) {
                const uint64_t count = std::min<uint64_t>(vocab - first, at.piece);
                rc = set_piece(a, at, ws, weight + g, n, first, count, weight_stride, as_is, dtype, stream);
                if (rc == AR_SUCCESS && rows > 0) rc = hip_result(launch_cross_dz(a, n, dtype, stream), what);
                if (rc == AR_SUCCESS && rows > 0 && dx != nullptr)
                    rc = hip_result(launch_cross_dx(a, n, first > 0, at.dx.tile, dtype, stream), what);
                if (rc == AR_SUCCESS && dweight != nullptr)
                    rc = hip_result(launch_cross_dweight(a, n, dtype, stream), what);
                if (rc != AR_SUCCESS) return rc;
            }
            if (rows > 0 && dx != nullptr &&
                (rc = hip_result(launch_cross_finish(a, n, dtype, stream), what)) != AR_SUCCESS)
                return rc;
        }
        return AR_SUCCESS;
    });
}

}  // extern "C"
