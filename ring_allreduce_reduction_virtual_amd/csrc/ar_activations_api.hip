// Host side of activations in 8 bits, declared in include/ar.h: validation,
// and the ranks' pointers handed to the kernels, up to kActivationRanks ranks
// a launch.  (Layer norm's backward pass from them is in ar_layer_norm_api.hip.)

#include <hip/hip_runtime.h>

#include "ar_activations.h"
#include "ar_rows.h"

using namespace arimpl;

namespace {

constexpr uint64_t kMaxRows = 1ull << 40, kMaxCols = 1ull << 26;

ar_result_t check_shape(size_t rows, size_t cols, ar_dtype_t dtype, int nranks) {
    const ar_result_t rc = check_types(dtype, dtype, "same", nranks);
    if (rc != AR_SUCCESS) return rc;
    if (rows > kMaxRows || cols > kMaxCols || (rows > 0 && cols > kMaxSpan / rows))
        return fail_with(AR_ERR_INVALID_ARGUMENT, "%llu rows of %llu elements are too large",
                         static_cast<unsigned long long>(rows), static_cast<unsigned long long>(cols));
    return AR_SUCCESS;
}

// One rank's codes and scales.
ar_result_t add_packed(std::vector<Range>& v, const void* codes, const void* scales, size_t rows, size_t cols,
                       bool writable, int r) {
    const uint64_t blocks = (cols + AR_ACTIVATION_BLOCK - 1) / AR_ACTIVATION_BLOCK;
    const ar_result_t rc = add_range(v, codes, rows * cols, 1, writable, "codes", r);
    return rc != AR_SUCCESS ? rc : add_range(v, scales, rows * blocks, 1, writable, "scales", r);
}

}  // namespace

extern "C" {

ar_result_t ar_pack_activations(const void* const* x, void* const* codes, void* const* scales, size_t rows,
                                size_t cols, size_t x_stride, ar_dtype_t dtype, int nranks, hipStream_t stream) {
    return guarded([&]() -> ar_result_t {
        ar_result_t rc = check_shape(rows, cols, dtype, nranks);
        if (rc != AR_SUCCESS || (rc = check_stride(x_stride, rows, cols, "x_stride")) != AR_SUCCESS) return rc;
        if (x == nullptr || codes == nullptr || scales == nullptr)
            return fail_with(AR_ERR_INVALID_ARGUMENT, "null pointer array");
        if (rows == 0 || cols == 0) return AR_SUCCESS;
        std::vector<Range> v;
        v.reserve(3 * static_cast<size_t>(nranks));
        for (int r = 0; r < nranks; ++r) {
            if ((rc = add_rows(v, x[r], rows, cols, x_stride, float_size(dtype), false, "x", r)) != AR_SUCCESS ||
                (rc = add_packed(v, codes[r], scales[r], rows, cols, true, r)) != AR_SUCCESS)
                return rc;
        }
        if ((rc = check_ranges(v)) != AR_SUCCESS) return rc;
        for (int first = 0; first < nranks; first += kActivationRanks) {
            PackArgs a{};
            const int n = std::min(kActivationRanks, nranks - first);
            for (int k = 0; k < n; ++k) {
                a.x[k] = static_cast<const char*>(x[first + k]);
                a.codes[k] = static_cast<uint8_t*>(codes[first + k]);
                a.scales[k] = static_cast<uint8_t*>(scales[first + k]);
            }
            a.rows = rows;
            a.cols = cols;
            a.x_stride = x_stride;
            rc = hip_result(launch_pack(a, n, dtype, stream), "pack_activations launch");
            if (rc != AR_SUCCESS) return rc;
        }
        return AR_SUCCESS;
    });
}

ar_result_t ar_unpack_activations(const void* const* codes, const void* const* scales, void* const* x, size_t rows,
                                  size_t cols, size_t x_stride, ar_dtype_t dtype, int nranks, hipStream_t stream) {
    return guarded([&]() -> ar_result_t {
        ar_result_t rc = check_shape(rows, cols, dtype, nranks);
        if (rc != AR_SUCCESS || (rc = check_stride(x_stride, rows, cols, "x_stride")) != AR_SUCCESS) return rc;
        if (x == nullptr || codes == nullptr || scales == nullptr)
            return fail_with(AR_ERR_INVALID_ARGUMENT, "null pointer array");
        if (rows == 0 || cols == 0) return AR_SUCCESS;
        std::vector<Range> v;
        v.reserve(3 * static_cast<size_t>(nranks));
        for (int r = 0; r < nranks; ++r) {
            if ((rc = add_packed(v, codes[r], scales[r], rows, cols, false, r)) != AR_SUCCESS ||
                (rc = add_rows(v, x[r], rows, cols, x_stride, float_size(dtype), true, "x", r)) != AR_SUCCESS)
                return rc;
        }
        if ((rc = check_ranges(v)) != AR_SUCCESS) return rc;
        for (int first = 0; first < nranks; first += kActivationRanks) {
            UnpackArgs a{};
            const int n = std::min(kActivationRanks, nranks - first);
            for (int k = 0; k < n; ++k) {
                a.codes[k] = static_cast<const uint8_t*>(codes[first + k]);
                a.scales[k] = static_cast<const uint8_t*>(scales[first + k]);
                a.x[k] = static_cast<char*>(x[first + k]);
            }
            a.rows = rows;
            a.cols = cols;
            a.x_stride = x_stride;
            rc = hip_result(launch_unpack(a, n, dtype, stream), "unpack_activations launch");
            if (rc != AR_SUCCESS) return rc;
        }
        return AR_SUCCESS;
    });
}

}  // extern "C"
