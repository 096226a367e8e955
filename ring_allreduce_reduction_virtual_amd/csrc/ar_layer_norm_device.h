// Device-side building blocks of the layer norm kernels.  Inline device code
// in an unnamed namespace, so each kernel source gets its own copy.
#pragma once

#include "ar_layer_norm.h"
#include "ar_step_device.h"

namespace arimpl {
namespace {

// Elements of a row in one 16-byte vector.
template <int DT>
constexpr int kRowVec = 16 / elem_size<DT>();

// Sums over the THREADS threads of a row, in every one of them, always in the
// same order.  Rows of up to 64 threads stay within a wavefront; wider ones
// meet in `part`, one row of it for each sum of a loop's turn: a turn's sums
// use different rows, each followed by a barrier, so a row's next writer comes
// after all its readers.
template <int THREADS, int N>
__device__ __forceinline__ void sum_over_row(float (&x)[N], float (*part)[N]) {
#pragma unroll
    for (int k = 0; k < N; ++k) x[k] = sum_over_lanes<(THREADS < 64 ? THREADS : 64)>(x[k]);
    if constexpr (THREADS > 64) {
        if ((threadIdx.x & 63) == 0) {
#pragma unroll
            for (int k = 0; k < N; ++k) part[threadIdx.x >> 6][k] = x[k];
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < N; ++k) {
            float s = 0;
#pragma unroll
            for (int w = 0; w < THREADS / 64; ++w) s += part[w][k];
            x[k] = s;
        }
    }
}

}  // namespace
}  // namespace arimpl
