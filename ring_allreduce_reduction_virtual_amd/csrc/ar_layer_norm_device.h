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

// A thread's vectors of a row and the elements in them that are its own.  Rows
// of at least a vector (THREADS > 8) are read without a branch: a vector that
// would cross the row's end is moved back to end there, and its first `skip`
// elements belong to the thread before (all of them, when the whole vector
// lies past the end).  Shorter rows are read up to their end.
template <int THREADS, int V>
struct RowPart {
    int at, skip;   // first element, elements that are another thread's
    __device__ __forceinline__ RowPart(int u, int cols) {
        at = (u * THREADS + static_cast<int>(threadIdx.x % THREADS)) * V;
        skip = 0;
        if constexpr (THREADS > 8) {
            const int last = cols - V;
            skip = at > last ? at - last : 0;
            at = at > last ? last : at;
        }
    }
    // whether element j of the vector is this thread's
    __device__ __forceinline__ bool mine(int j, int cols) const {
        if constexpr (THREADS > 8) return j >= skip;
        return at + j < cols;
    }
    // makes the other threads' elements 0
    template <int DT>
    __device__ __forceinline__ void clear(Raw<DT, V>& r) const {
        if constexpr (THREADS > 8) {
            constexpr int kPer = 4 / elem_size<DT>();   // elements in a word
#pragma unroll
            for (int k = 0; k < Raw<DT, V>::kWords; ++k) {
                const int gone = skip - k * kPer;       // of this word's elements
                const uint32_t keep = gone <= 0 ? 0xffffffffu : (gone >= kPer ? 0u : 0xffff0000u);
                r.w[k] &= keep;
            }
        }
    }
    template <bool NT, int DT>
    __device__ __forceinline__ void load(Raw<DT, V>& r, const char* row, int cols) const {
        if constexpr (THREADS > 8) {
            r.template load<NT>(row + static_cast<uint32_t>(at * elem_size<DT>()));
        } else {
            load_at<false, NT>(r, row, at, cols);
        }
    }
    template <int DT>
    __device__ __forceinline__ void store(const Raw<DT, V>& r, char* row, int cols) const {
        if constexpr (THREADS > 8) {
            char* const p = row + static_cast<uint32_t>(at * elem_size<DT>());
            if (skip == 0) {
                r.template store<true>(p);
            } else if (skip < V) {   // one thread of a row that is no whole number of vectors
                r.store_from(p, skip);
            }
        } else {
            store_at<false, true>(r, row, at, cols);
        }
    }
};

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

// A value's sum over the rows that a wavefront holds, THREADS < 64 lanes each.
template <int THREADS>
__device__ __forceinline__ float sum_over_rows(float x) {
    const auto add = [](uint32_t p, uint32_t q) { return as_u(as_f(p) + as_f(q)); };
    uint32_t u = as_u(x);
    if constexpr (THREADS <= 8) u = add(u, dpp<kDppRotate8>(u));
    if constexpr (THREADS <= 16) u = across16(u, add);
    u = across32(u, add);
    return as_f(u);
}

// The row of the workgroup's first turn that this thread works on.  Up to a
// wavefront's width and above, the same in all the wavefront's lanes.
template <int THREADS>
__device__ __forceinline__ uint64_t first_row() {
    uint32_t r = threadIdx.x / THREADS;
    if constexpr (THREADS >= 64) r = __builtin_amdgcn_readfirstlane(r);
    return static_cast<uint64_t>(blockIdx.x) * rows_at_once(THREADS) + r;
}

}  // namespace
}  // namespace arimpl
