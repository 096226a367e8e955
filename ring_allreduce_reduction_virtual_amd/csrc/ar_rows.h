// Host-side checks shared by the entry points over every rank's rows of
// activations, tokens and weights (ar_embedding_api.hip, ar_activations_api.hip,
// ar_cross_entropy_api.hip).  Everything is inline in an unnamed namespace.
#pragma once

#include "ar_host.h"

namespace arimpl {
namespace {

inline size_t float_size(ar_dtype_t dt) { return dt == AR_FLOAT32 ? 4 : 2; }
inline size_t index_size(ar_index_t index) { return index == AR_INDEX_INT64 ? 8 : 4; }

// Keeps every product of sizes within 64 bits.
constexpr uint64_t kMaxStride = 1ull << 40;
constexpr uint64_t kMaxSpan = 1ull << 48;   // elements from a buffer's first row to its last

inline ar_result_t check_types(ar_dtype_t dtype, ar_dtype_t other, const char* what, int nranks) {
    if (!float_type(dtype) || (other != dtype && other != AR_FLOAT32))
        return fail_with(AR_ERR_INVALID_ARGUMENT, "unsupported dtype %d with %s dtype %d", static_cast<int>(dtype), what,
                         static_cast<int>(other));
    if (nranks < 1 || nranks > AR_MAX_RANKS)
        return fail_with(AR_ERR_INVALID_ARGUMENT, "nranks %d outside [1, %d]", nranks, AR_MAX_RANKS);
    return AR_SUCCESS;
}

inline ar_result_t check_index(ar_index_t index) {
    if (index != AR_INDEX_INT32 && index != AR_INDEX_INT64)
        return fail_with(AR_ERR_INVALID_ARGUMENT, "unsupported index type %d", static_cast<int>(index));
    return AR_SUCCESS;
}

inline ar_result_t check_stride(size_t stride, size_t rows, size_t cols, const char* what) {
    if (stride < cols || stride > kMaxStride)
        return fail_with(AR_ERR_INVALID_ARGUMENT, "%s %llu is below the row's %llu elements, or too large", what,
                         static_cast<unsigned long long>(stride), static_cast<unsigned long long>(cols));
    if (rows > 1 && stride > 0 && rows - 1 > kMaxSpan / stride)
        return fail_with(AR_ERR_INVALID_ARGUMENT, "%s %llu with %llu rows is too large", what,
                         static_cast<unsigned long long>(stride), static_cast<unsigned long long>(rows));
    return AR_SUCCESS;
}

inline ar_result_t add_rows(std::vector<Range>& v, const void* p, size_t rows, size_t cols, size_t stride, size_t es,
                            bool writable, const char* what, int r) {
    if (rows == 0 || cols == 0) return AR_SUCCESS;
    return add_range(v, p, ((rows - 1) * stride + cols) * es, es, writable, what, r, cols * es, stride * es);
}

inline ar_result_t add_scratch(std::vector<Range>& v, void* ws, size_t have, uint64_t need, size_t align) {
    if (need == 0) return AR_SUCCESS;
    if (ws == nullptr || have < need)
        return fail_with(AR_ERR_INVALID_ARGUMENT, "this call needs a workspace of %llu bytes",
                         static_cast<unsigned long long>(need));
    return add_range(v, ws, need, align, true, "workspace", 0);
}

}  // namespace
}  // namespace arimpl
