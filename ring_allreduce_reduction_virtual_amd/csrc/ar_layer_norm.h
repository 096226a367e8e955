// Internal interface of layer norm: what the host entry points
// (ar_layer_norm_api.hip) hand to the kernels (ar_layer_norm_kernels.hip, the
// forward pass, and ar_layer_norm_backward_device.h).  Not installed;
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
    const char* x[kNormRanks];       // packed: the codes
    const uint8_t* scales[kNormRanks];
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

// How a row lies over threads: `threads` threads a row, each holding `vectors`
// 16-byte vectors of it in registers; vectors == 0: the row does not fit and is
// read again for every pass (the wide form).
struct RowShape {
    int threads, vectors;
};

// Threads of a workgroup, and the rows that it works on at a time: four
// wavefronts of short rows, or one long row.
constexpr int block_threads(int threads_per_row) { return threads_per_row <= 64 ? 256 : threads_per_row; }
constexpr int rows_at_once(int threads_per_row) { return block_threads(threads_per_row) / threads_per_row; }

// The forward pass: as few threads as hold the row, so that short rows leave no
// lanes idle and rows of up to a wavefront's registers need no barrier.
// Measured on MI355X, 2^26 bf16 elements on 8 ranks (45.5 us at 5.9 TB/s), us:
// 64 columns 8x1 51, 16x1 90; 256 32x1 52, 64x1 75; 1,024 64x2 51.6, 128x1
// 50.2, 256x1 72; 2,048 64x4 48.0, 256x1 48.9, 512x1 72; 4,096 128x4 47.4,
// 256x2 49.8, 1024x1 80; 8,192 256x4 48.5, 512x2 49.6, wide 77; 16,384 1024x2
// 53.9, 512x4 59.
// float32, 2^25 elements: 1,024 64x4 45.7; 4,096 256x4 47.4; 8,192 1024x2 47.7,
// 512x4 48.9; 16,384 1024x4 50.2, wide 72.
inline RowShape forward_shape(uint64_t cols, int vector_elements) {
    const uint64_t need = (cols + vector_elements - 1) / vector_elements;
    if (need <= 8) return {8, 1};
    if (need <= 16) return {16, 1};
    if (need <= 32) return {32, 1};
    if (need <= 64) return {64, 1};
    if (need <= 128) return {64, 2};
    if (need <= 256) return {64, 4};
    if (need <= 512) return {128, 4};
    if (need <= 1024) return {256, 4};
    if (need <= 2048) return {1024, 2};
    if (need <= 4096 && vector_elements == 4) return {1024, 4};
    return {1024, 0};
}

// The backward pass holds each column's two sums besides the row: fewer
// vectors a thread.  Same sizes (68.4 us at 5.9 TB/s), bf16, us: 64 columns 8x1
// 74, 16x1 107; 256 32x1 76, 64x1 90; 1,024 128x1 78, 64x2 82, 256x1 88; 2,048
// 256x1 79, 128x2 91, 64x4 94; 4,096 256x2 80, 512x1 80, 128x4 85, 1024x1 103;
// 8,192 512x2 89, 1024x1 91, 256x4 102, wide 158; float32: 1,024 256x1 78,
// 128x2 75; 4,096 512x2 80; 8,192 512x4 87, wide 143 (all with 512 workgroups;
// with 256, as below, 8,192 86 in bf16, 81 in float32, and 16,384 bf16 100).
inline RowShape backward_shape(uint64_t cols, int vector_elements) {
    const uint64_t need = (cols + vector_elements - 1) / vector_elements;
    if (need <= 8) return {8, 1};
    if (need <= 16) return {16, 1};
    if (need <= 32) return {32, 1};
    if (need <= 64) return {64, 1};
    if (need <= 128) return {128, 1};
    if (need <= 256) return {256, 1};
    if (need <= 512) return {256, 2};
    if (need <= 1024) return {512, 2};
    if (need <= 2048) return {512, 4};
    if (need <= 4096 && vector_elements == 4) return {512, 8};
    return {1024, 0};
}

// Workgroups of a rank's backward pass; each leaves one partial sum of dgamma
// and dbeta per column.  All ranks together: enough to fill the GPU, more when
// every one still has 64 rows, over which its partial sums' traffic is small.
// Rows over 512 threads fill it with half as many (us, 512 / 256 workgroups:
// 4 x 1,024 x 8,192 bf16 56 / 49, 2 x 512 x 16,384 bf16 47 / 37, 4 x 512 x
// 16,384 float32 103 / 93).  Rows over 128 threads leave it half full, so up
// to twice as many while every one has 8 rows (us, 512 / 1,024 workgroups: 4 x
// 4,096 x 768 bf16 34 / 24, 8 x 1,024 x 768 20 / 16, 2 x 8,192 x 512 float32 30 /
// 26, but 4,096 rows of 1,024 bf16 15.9 / 17.3).
//
// Wide rows: their sums are made by stretches of kColumnThreads vectors, and
// kColumnBlocks of these fill the GPU (us with about 4,000 / 2,000 / 1,000 /
// 500 workgroups: 2 x 512 x 40,000 bf16 148 / 121 / 105 / 102; 1,024 x 50,257
// bf16 168 / 158 / 165 for 3,200 / 1,600 / 800).
constexpr uint64_t kBackwardBlocks = 512, kBackwardLongBlocks = 256, kBackwardMostBlocks = 4096;
constexpr uint64_t kBackwardRows = 64, kBackwardFewRows = 8;
constexpr int kColumnThreads = 256;
constexpr uint64_t kColumnBlocks = 1024;
inline uint64_t column_stretches(uint64_t cols, int vector_elements) {
    const uint64_t per = static_cast<uint64_t>(kColumnThreads) * vector_elements;
    return (cols + per - 1) / per;
}
inline uint32_t backward_blocks(uint64_t rows, uint64_t cols, int nranks, int vector_elements) {
    const RowShape shape = backward_shape(cols, vector_elements);
    const int at_once = rows_at_once(shape.threads);
    uint64_t wanted;
    if (shape.vectors == 0) {
        wanted = kColumnBlocks / column_stretches(cols, vector_elements);
    } else {
        const uint64_t total = rows * nranks;
        uint64_t least = shape.threads > 256 ? kBackwardLongBlocks : kBackwardBlocks;
        if (shape.threads == 128) least = std::min(2 * least, std::max(least, total / kBackwardFewRows));
        wanted = std::min(kBackwardMostBlocks, std::max(least, total / kBackwardRows));
    }
    wanted = std::max<uint64_t>(1, wanted / nranks);
    return static_cast<uint32_t>(std::min<uint64_t>((rows + at_once - 1) / at_once, wanted));
}

hipError_t launch_norm_forward(const NormForwardArgs& a, int nranks, ar_dtype_t dtype, ar_dtype_t weight,
                               hipStream_t stream);
// dx, and the partial sums when `weights`; then the sums.
hipError_t launch_norm_backward(const NormBackwardArgs& a, int nranks, bool weights, ar_dtype_t dtype,
                                ar_dtype_t weight, hipStream_t stream);
// The same from x's codes and scales.
hipError_t launch_norm_backward_packed(const NormBackwardArgs& a, int nranks, bool weights, ar_dtype_t dtype,
                                       ar_dtype_t weight, hipStream_t stream);

}  // namespace arimpl
