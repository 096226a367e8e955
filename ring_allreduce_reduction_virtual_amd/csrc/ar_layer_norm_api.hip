// Host side of layer norm, declared in include/ar.h: validation, and the
// ranks' pointers handed to the kernels, up to kNormRanks ranks a launch.

#include <hip/hip_runtime.h>

#include "ar_host.h"
#include "ar_layer_norm.h"

using namespace arimpl;

namespace {

size_t esize(ar_dtype_t dt) { return dt == AR_FLOAT32 ? 4 : 2; }

// Keeps every product of sizes below within 64 bits, and every launch's grid
// within the device's limits.
constexpr uint64_t kMaxRows = 1ull << 40, kMaxCols = 1ull << 26, kMaxStride = 1ull << 40;
constexpr uint64_t kMaxSpan = 1ull << 48;   // elements from a buffer's first row to its last

ar_result_t check_shape(size_t rows, size_t cols, ar_dtype_t dtype, ar_dtype_t weight, int nranks) {
    if (!float_type(dtype) || (weight != dtype && weight != AR_FLOAT32))
        return fail_with(AR_ERR_INVALID_ARGUMENT, "unsupported dtype %d with weight dtype %d", static_cast<int>(dtype),
                         static_cast<int>(weight));
    if (nranks < 1 || nranks > AR_MAX_RANKS)
        return fail_with(AR_ERR_INVALID_ARGUMENT, "nranks %d outside [1, %d]", nranks, AR_MAX_RANKS);
    if (rows > kMaxRows || cols > kMaxCols)
        return fail_with(AR_ERR_INVALID_ARGUMENT, "%llu rows of %llu elements are too large",
                         static_cast<unsigned long long>(rows), static_cast<unsigned long long>(cols));
    return AR_SUCCESS;
}

ar_result_t check_stride(size_t stride, size_t rows, size_t cols, const char* what) {
    if (stride < cols || stride > kMaxStride)
        return fail_with(AR_ERR_INVALID_ARGUMENT, "%s %llu is below the row's %llu elements, or too large", what,
                         static_cast<unsigned long long>(stride), static_cast<unsigned long long>(cols));
    if (rows > 1 && stride > 0 && rows - 1 > kMaxSpan / stride)
        return fail_with(AR_ERR_INVALID_ARGUMENT, "%s %llu with %llu rows is too large", what,
                         static_cast<unsigned long long>(stride), static_cast<unsigned long long>(rows));
    return AR_SUCCESS;
}

ar_result_t add_rows(std::vector<Range>& v, const void* p, size_t rows, size_t cols, size_t stride, size_t es,
                     bool writable, const char* what, int r) {
    if (rows == 0 || cols == 0) return AR_SUCCESS;
    return add_range(v, p, ((rows - 1) * stride + cols) * es, es, writable, what, r, cols * es, stride * es);
}

// One rank's codes and scales of x.
ar_result_t add_packed(std::vector<Range>& v, const void* codes, const void* scales, size_t rows, size_t cols, int r) {
    const uint64_t blocks = (cols + AR_ACTIVATION_BLOCK - 1) / AR_ACTIVATION_BLOCK;
    const ar_result_t rc = add_range(v, codes, rows * cols, 1, false, "codes", r);
    return rc != AR_SUCCESS ? rc : add_range(v, scales, rows * blocks, 1, false, "scales", r);
}

// Both backward passes: `scales` null, x as it was, else its codes.
ar_result_t backward(const void* const* dy, const void* const* x, const void* const* scales, const void* const* gamma,
                     const float* const* mean, const float* const* rstd, void* const* dx, void* const* dgamma,
                     void* const* dbeta, size_t rows, size_t cols, size_t dy_stride, size_t x_stride, size_t dx_stride,
                     ar_dtype_t dtype, ar_dtype_t weight_dtype, int nranks, void* workspace, size_t workspace_bytes,
                     hipStream_t stream) {
    const bool packed = scales != nullptr;
    ar_result_t rc = check_shape(rows, cols, dtype, weight_dtype, nranks);
    if (rc != AR_SUCCESS || (rc = check_stride(dy_stride, rows, cols, "dy_stride")) != AR_SUCCESS ||
        (rc = check_stride(x_stride, rows, cols, "x_stride")) != AR_SUCCESS ||
        (rc = check_stride(dx_stride, rows, cols, "dx_stride")) != AR_SUCCESS)
        return rc;
    if (dy == nullptr || x == nullptr || mean == nullptr || rstd == nullptr || dx == nullptr)
        return fail_with(AR_ERR_INVALID_ARGUMENT, "null pointer array");
    if (cols == 0) return AR_SUCCESS;
    const bool weights = dgamma != nullptr || dbeta != nullptr;
    const size_t es = esize(dtype), ws = esize(weight_dtype);
    std::vector<Range> v;
    v.reserve(9 * static_cast<size_t>(nranks) + 1);
    for (int r = 0; r < nranks; ++r) {
        const bool in_place = dy[r] == dx[r] && dy_stride == dx_stride;
        if ((!in_place && (rc = add_rows(v, dy[r], rows, cols, dy_stride, es, false, "dy", r)) != AR_SUCCESS) ||
            (rc = packed ? add_packed(v, x[r], scales[r], rows, cols, r)
                         : add_rows(v, x[r], rows, cols, x_stride, es, false, "x", r)) != AR_SUCCESS ||
            (rc = add_rows(v, dx[r], rows, cols, dx_stride, es, true, "dx", r)) != AR_SUCCESS ||
            (rc = add_range(v, mean[r], rows * 4, 4, false, "mean", r)) != AR_SUCCESS ||
            (rc = add_range(v, rstd[r], rows * 4, 4, false, "rstd", r)) != AR_SUCCESS)
            return rc;
        if ((gamma != nullptr &&
             (rc = add_range(v, gamma[r], cols * ws, ws, false, "gamma", r)) != AR_SUCCESS) ||
            (dgamma != nullptr &&
             (rc = add_range(v, dgamma[r], cols * ws, ws, true, "dgamma", r)) != AR_SUCCESS) ||
            (dbeta != nullptr && (rc = add_range(v, dbeta[r], cols * ws, ws, true, "dbeta", r)) != AR_SUCCESS))
            return rc;
    }
    const uint32_t blocks = backward_blocks(rows, cols, nranks, 16 / static_cast<int>(es));
    if (weights) {
        const uint64_t need = ar_layer_norm_workspace_bytes(rows, cols, nranks);
        if (need > 0 && (workspace == nullptr || workspace_bytes < need))
            return fail_with(AR_ERR_INVALID_ARGUMENT, "this call needs a workspace of %llu bytes",
                             static_cast<unsigned long long>(need));
        if ((rc = add_range(v, workspace, need, 4, true, "workspace", 0)) != AR_SUCCESS) return rc;
    }
    if ((rc = check_ranges(v)) != AR_SUCCESS) return rc;
    if (rows == 0 && !weights) return AR_SUCCESS;
    for (int first = 0; first < nranks; first += kNormRanks) {
        NormBackwardArgs a{};
        const int n = std::min(kNormRanks, nranks - first);
        for (int k = 0; k < n; ++k) {
            a.dy[k] = static_cast<const char*>(dy[first + k]);
            a.x[k] = static_cast<const char*>(x[first + k]);
            a.scales[k] = packed ? static_cast<const uint8_t*>(scales[first + k]) : nullptr;
            a.gamma[k] = gamma == nullptr ? nullptr : static_cast<const char*>(gamma[first + k]);
            a.mean[k] = mean[first + k];
            a.rstd[k] = rstd[first + k];
            a.dx[k] = static_cast<char*>(dx[first + k]);
            a.dgamma[k] = dgamma == nullptr ? nullptr : static_cast<char*>(dgamma[first + k]);
            a.dbeta[k] = dbeta == nullptr ? nullptr : static_cast<char*>(dbeta[first + k]);
        }
        a.partials = weights && rows > 0
                         ? static_cast<float*>(workspace) + static_cast<uint64_t>(first) * blocks * 2 * cols
                         : nullptr;
        a.rows = rows;
        a.cols = cols;
        a.dy_stride = dy_stride;
        a.x_stride = x_stride;
        a.dx_stride = dx_stride;
        a.blocks = blocks;
        rc = hip_result(packed ? launch_norm_backward_packed(a, n, weights, dtype, weight_dtype, stream)
                               : launch_norm_backward(a, n, weights, dtype, weight_dtype, stream),
                        "layer_norm_backward launch");
        if (rc != AR_SUCCESS) return rc;
    }
    return AR_SUCCESS;
}

}  // namespace

extern "C" {

ar_result_t ar_layer_norm(const void* const* x, const void* const* gamma, const void* const* beta, void* const* y,
                          float* const* mean, float* const* rstd, size_t rows, size_t cols, size_t x_stride,
                          size_t y_stride, ar_dtype_t dtype, ar_dtype_t weight_dtype, double eps, int nranks,
                          hipStream_t stream) {
    return guarded([&]() -> ar_result_t {
        ar_result_t rc = check_shape(rows, cols, dtype, weight_dtype, nranks);
        if (rc != AR_SUCCESS || (rc = check_stride(x_stride, rows, cols, "x_stride")) != AR_SUCCESS ||
            (rc = check_stride(y_stride, rows, cols, "y_stride")) != AR_SUCCESS)
            return rc;
        if (!(eps >= 0 && eps < 1e30)) return fail_with(AR_ERR_INVALID_ARGUMENT, "eps %g is not a finite number >= 0", eps);
        if (rounds_to_zero(eps)) return fail_with(AR_ERR_INVALID_ARGUMENT, "eps %g is 0 in float32", eps);
        if (x == nullptr || y == nullptr) return fail_with(AR_ERR_INVALID_ARGUMENT, "null pointer array");
        if ((mean == nullptr) != (rstd == nullptr))
            return fail_with(AR_ERR_INVALID_ARGUMENT, "mean and rstd are wanted together or not at all");
        if (rows == 0 || cols == 0) return AR_SUCCESS;
        const size_t es = esize(dtype), ws = esize(weight_dtype);
        std::vector<Range> v;
        v.reserve(6 * static_cast<size_t>(nranks));
        for (int r = 0; r < nranks; ++r) {
            const bool in_place = x[r] == y[r] && x_stride == y_stride;
            if ((!in_place && (rc = add_rows(v, x[r], rows, cols, x_stride, es, false, "x", r)) != AR_SUCCESS) ||
                (rc = add_rows(v, y[r], rows, cols, y_stride, es, true, "y", r)) != AR_SUCCESS)
                return rc;
            if ((gamma != nullptr &&
                 (rc = add_range(v, gamma[r], cols * ws, ws, false, "gamma", r)) != AR_SUCCESS) ||
                (beta != nullptr && (rc = add_range(v, beta[r], cols * ws, ws, false, "beta", r)) != AR_SUCCESS))
                return rc;
            if (mean != nullptr && ((rc = add_range(v, mean[r], rows * 4, 4, true, "mean", r)) != AR_SUCCESS ||
                                    (rc = add_range(v, rstd[r], rows * 4, 4, true, "rstd", r)) != AR_SUCCESS))
                return rc;
        }
        if ((rc = check_ranges(v)) != AR_SUCCESS) return rc;
        for (int first = 0; first < nranks; first += kNormRanks) {
            NormForwardArgs a{};
            const int n = std::min(kNormRanks, nranks - first);
            for (int k = 0; k < n; ++k) {
                a.x[k] = static_cast<const char*>(x[first + k]);
                a.y[k] = static_cast<char*>(y[first + k]);
                a.gamma[k] = gamma == nullptr ? nullptr : static_cast<const char*>(gamma[first + k]);
                a.beta[k] = beta == nullptr ? nullptr : static_cast<const char*>(beta[first + k]);
                a.mean[k] = mean == nullptr ? nullptr : mean[first + k];
                a.rstd[k] = rstd == nullptr ? nullptr : rstd[first + k];
            }
            a.rows = rows;
            a.cols = cols;
            a.x_stride = x_stride;
            a.y_stride = y_stride;
            a.eps = static_cast<float>(eps);
            rc = hip_result(launch_norm_forward(a, n, dtype, weight_dtype, stream), "layer_norm launch");
            if (rc != AR_SUCCESS) return rc;
        }
        return AR_SUCCESS;
    });
}

size_t ar_layer_norm_workspace_bytes(size_t rows, size_t cols, int nranks) {
    if (nranks < 1 || nranks > AR_MAX_RANKS || rows > kMaxRows || cols > kMaxCols) return static_cast<size_t>(-1);
    const uint32_t blocks = std::max(backward_blocks(rows, cols, nranks, 4), backward_blocks(rows, cols, nranks, 8));
    return static_cast<size_t>(nranks) * blocks * 2 * cols * sizeof(float);
}

ar_result_t ar_layer_norm_backward(const void* const* dy, const void* const* x, const void* const* gamma,
                                   const float* const* mean, const float* const* rstd, void* const* dx,
                                   void* const* dgamma, void* const* dbeta, size_t rows, size_t cols,
                                   size_t dy_stride, size_t x_stride, size_t dx_stride, ar_dtype_t dtype,
                                   ar_dtype_t weight_dtype, int nranks, void* workspace, size_t workspace_bytes,
                                   hipStream_t stream) {
    return guarded([&]() -> ar_result_t {
        return backward(dy, x, nullptr, gamma, mean, rstd, dx, dgamma, dbeta, rows, cols, dy_stride, x_stride,
                        dx_stride, dtype, weight_dtype, nranks, workspace, workspace_bytes, stream);
    });
}

ar_result_t ar_layer_norm_backward_packed(const void* const* dy, const void* const* codes, const void* const* scales,
                                          const void* const* gamma, const float* const* mean,
                                          const float* const* rstd, void* const* dx, void* const* dgamma,
                                          void* const* dbeta, size_t rows, size_t cols, size_t dy_stride,
                                          size_t dx_stride, ar_dtype_t dtype, ar_dtype_t weight_dtype, int nranks,
                                          void* workspace, size_t workspace_bytes, hipStream_t stream) {
    return guarded([&]() -> ar_result_t {
        if (scales == nullptr) return fail_with(AR_ERR_INVALID_ARGUMENT, "null pointer array");
        return backward(dy, codes, scales, gamma, mean, rstd, dx, dgamma, dbeta, rows, cols, dy_stride, cols,
                        dx_stride, dtype, weight_dtype, nranks, workspace, workspace_bytes, stream);
    });
}

}  // extern "C"
