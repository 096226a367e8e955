// Internal interface of layer norm: what the host entry points
// (ar_layer_norm_api.hip) hand to the kernels (ar_layer_norm_kernels.hip, the
// forward pass, and ar_layer_norm_backward_kernels.hip).  Not installed;
// include/ar.h is the public ABI.
#pragma once

#include <hip/hip_runtime_api.h>

#include <algorithm>
#include <cstdint>

#include "ar.h"

namespace arimpl {

// Ranks of one launch: their pointers travel in the kernel's arguments.
constexpr int kNormRanks = 32;

struct NormForwardArgs {
    const char* x[kNormRanks];
    const char* gamma[kNormRanks];   // null: 1
    const char* beta[kNormRanks];    // null: 0
    char* y[kNormRanks];
    float* mean[kNormRanks];         // null, with rstd: not wanted
    float* rstd[kNormRanks];
    uint64_t rows, cols;
    uint64_t x_stride, y_stride;     // elements
    float eps;
};

struct NormBackwardArgs {
    const char* dy[kNormRanks];
    const char* x[kNormRanks];
    const char* gamma[kNormRanks];
    const float* mean[kNormRanks];
    const float* rstd[kNormRanks];
    char* dx[kNormRanks];
    char* dgamma[kNormRanks];        // null: not wanted
    char* dbeta[kNormRanks];
    float* partials;                 // [rank of the launch][block][2][cols]
    uint64_t rows, cols;
    uint64_t dy_stride, x_stride, dx_stride;
    uint32_t blocks;                 // partial sums per rank
};

// How a row lies over threads: `threads` threads a row, each holding `each` of
// its elements in registers; each == 0: the row does not fit and is read again
// for every pass (the wide form).  The narrowest form that holds the row: lanes
// without elements would idle, and more elements per thread mean fewer lanes
// to combine.
struct RowShape {
    int threads, each;
};
constexpr uint64_t kWidestRow = 16384;   // elements held in registers at most
inline RowShape row_shape(uint64_t cols) {
    if (cols <= 128) return {16, 8};
    if (cols <= 512) return {64, 8};
    if (cols <= 1024) return {64, 16};
    if (cols <= 2048) return {64, 32};
    if (cols <= 4096) return {256, 16};
    if (cols <= 8192) return {256, 32};
    if (cols <= kWidestRow) return {1024, 16};
    return {1024, 0};
}
// Rows that one workgroup works on at a time (256 threads, or one row).
constexpr int rows_at_once(int threads_per_row) { return threads_per_row < 256 ? 256 / threads_per_row : 1; }

// Partial sums of dgamma and dbeta that a rank's backward pass leaves: one a
// workgroup.  Together the ranks start about kBackwardBlocks workgroups.
constexpr uint32_t kBackwardBlocks = 512;
inline uint32_t backward_blocks(uint64_t rows, uint64_t cols, int nranks) {
    const uint64_t all = (rows + rows_at_once(row_shape(cols).threads) - 1) / rows_at_once(row_shape(cols).threads);
    return static_cast<uint32_t>(std::min<uint64_t>(all, std::max(1, static_cast<int>(kBackwardBlocks) / nranks)));
}

hipError_t launch_norm_forward(const NormForwardArgs& a, int nranks, ar_dtype_t dtype, ar_dtype_t weight,
                               hipStream_t stream);
// dx, and the partial sums when `weights`; then the sums.
hipError_t launch_norm_backward(const NormBackwardArgs& a, int nranks, bool weights, ar_dtype_t dtype,
                                ar_dtype_t weight, hipStream_t stream);

}  // namespace arimpl
