// The kernels of layer norm's backward pass (include/ar.h states the formulas),
// with the forward pass's input as it was (ar_layer_norm_backward_kernels.hip)
// or kept in 8 bits (ar_layer_norm_packed_kernels.hip).  Inline device code in
// an unnamed namespace, so each kernel source gets its own copy.
//
// One pass over dy and x makes dx, and each thread adds its columns' parts of
// dgamma and dbeta over all the rows that its workgroup takes: a thread keeps
// the same columns from row to row, so these sums stay in registers.  Each
// workgroup leaves one partial sum per column; a second launch adds them in
// the order of the workgroups, so that the result does not depend on which
// one finishes first.  The activations' two reads and one write bound it: 8
// ranks x 4,096 x 4,096 bf16 150-153 us (825 MB with the partial sums, 5.4-5.5
// TB/s) and 4.8 us for the second launch.  Without partial sums dx takes 142 us; more
// workgroups would bring it to 135 and cost more than that in partial sums.

#pragma once

#include <hip/hip_runtime.h>

#include "ar_activations_device.h"
#include "ar_layer_norm_device.h"

namespace arimpl {
namespace {

template <int N>
__device__ __forceinline__ void store_floats(float* to, const float* x) {
#pragma unroll
    for (int j = 0; j < N; j += 4) {
        const u32x4 v = {as_u(x[j]), as_u(x[j + 1]), as_u(x[j + 2]), as_u(x[j + 3])};
        store_as<false, u32x4_a4>(reinterpret_cast<char*>(to + j), v);
    }
}

// How the forward pass's input is kept: as it was; in 8 bits, rows of whole
// vectors (which lie within blocks); in 8 bits, rows of any width, whose last
// vector is moved back to end with the row and may cross a block's end.
enum Kept { kAsItWas, kPackedWhole, kPackedAny };

// V elements of it.
template <int DT, int V, int KEPT>
struct Input : Raw<DT, V> {
    __device__ __forceinline__ void ready() {}
};

template <int V, int KEPT>
struct PackedInput {
    static constexpr int kWords = V / 4;
    uint32_t w[kWords];
    // the scale of the block that the first element is in and of the last one's,
    // bytes until ready(), which comes when they are needed: a use waits for the
    // load; and how many elements are in the first block
    uint32_t e[2];
    float scale[2];
    int edge;
    __device__ __forceinline__ void ready() {
        scale[0] = activation_scale_value(e[0]);
        if constexpr (KEPT == kPackedAny) scale[1] = activation_scale_value(e[1]);
    }
    __device__ __forceinline__ float get(int j) const {
        return activation_value(w[j / 4], j % 4, KEPT == kPackedWhole || j < edge ? scale[0] : scale[1]);
    }
    // from element `at` of a row; WHOLE: all V elements are in it
    template <bool WHOLE>
    __device__ __forceinline__ void load(const uint8_t* codes, const uint8_t* scales, uint64_t at, uint64_t cols) {
#pragma unroll
        for (int k = 0; k < kWords; ++k) w[k] = 0;
        e[0] = e[1] = 0;
        edge = AR_ACTIVATION_BLOCK - static_cast<int>(at % AR_ACTIVATION_BLOCK);
        if (!WHOLE && at >= cols) return;
        const uint64_t last = (WHOLE || at + V <= cols ? at + V : cols) - 1;
        e[0] = scales[at / AR_ACTIVATION_BLOCK];
        if constexpr (KEPT == kPackedAny) e[1] = scales[last / AR_ACTIVATION_BLOCK];
        const char* const p = reinterpret_cast<const char*>(codes + at);
        if (WHOLE || at + V <= cols) {
            if constexpr (kWords == 2) {
                const u32x2 v = load_as<true, u32x2_a1>(p);
                w[0] = v.x;
                w[1] = v.y;
            } else {
                typedef uint32_t u32_a1 __attribute__((aligned(1)));
                w[0] = load_as<true, u32_a1>(p);
            }
        } else {
#pragma unroll
            for (int j = 0; j < V; ++j) {
                if (at + j < cols) w[j / 4] |= static_cast<uint32_t>(codes[at + j]) << (8 * (j % 4));
            }
        }
    }
};
template <int DT, int V>
struct Input<DT, V, kPackedWhole> : PackedInput<V, kPackedWhole> {};
template <int DT, int V>
struct Input<DT, V, kPackedAny> : PackedInput<V, kPackedAny> {};

// A row of the forward pass's input.
template <int DT, int KEPT>
struct InputRow {
    const char* x;
    const uint8_t* scales;   // of a packed row
    __device__ __forceinline__ InputRow(const NormBackwardArgs& a, int rank, uint64_t row) {
        if constexpr (KEPT != kAsItWas) {
            x = a.x[rank] + row * a.cols;
            scales = a.scales[rank] + row * ((a.cols + AR_ACTIVATION_BLOCK - 1) / AR_ACTIVATION_BLOCK);
        } else {
            x = a.x[rank] + row * a.x_stride * elem_size<DT>();
            scales = nullptr;
        }
    }
    // a thread's vector of a row in registers
    template <int THREADS, int V>
    __device__ __forceinline__ void load(Input<DT, V, KEPT>& r, const RowPart<THREADS, V>& at, int cols) const {
        if constexpr (KEPT != kAsItWas) {
            r.template load<(THREADS > 8)>(reinterpret_cast<const uint8_t*>(x), scales, at.at, cols);
        } else {
            at.template load<true, DT>(r, x, cols);
        }
    }
    // V elements at c, or up to the row's end
    template <int V>
    __device__ __forceinline__ void load(Input<DT, V, KEPT>& r, uint64_t c, uint64_t cols) const {
        if constexpr (KEPT != kAsItWas) {
            r.template load<false>(reinterpret_cast<const uint8_t*>(x), scales, c, cols);
        } else {
            load_at<false, false, DT, V>(r, x, c, cols);
        }
    }
};

template <int DT, int WDT, int KEPT, int THREADS, int NV>
__global__ void __launch_bounds__(block_threads(THREADS)) k_layer_norm_backward(NormBackwardArgs a, int weights) {
    constexpr int V = kRowVec<DT>;
    constexpr int EACH = NV * V;
    // rows in registers: the longer the row, the fewer fill the memory's queues
    constexpr int DEPTH = THREADS * NV >= 2048 ? 1 : (THREADS * NV >= 1024 ? 2 : 3);
    constexpr int kRows = rows_at_once(THREADS);
    __shared__ float part[2][THREADS / 64 + 1][2];
    const int rank = blockIdx.y;
    const int cols = static_cast<int>(a.cols);
    const char* const gamma = a.gamma[rank];
    const float over = static_cast<float>(cols);
    const uint64_t step = static_cast<uint64_t>(gridDim.x) * kRows;
    uint64_t row = first_row<THREADS>();
    const char* const dy0 = a.dy[rank];
    char* const dx0 = a.dx[rank];
    const float *const mean0 = a.mean[rank], *const rstd0 = a.rstd[rank];
    // DEPTH rows on their way: the one worked on and those whose loads run beside it
    Raw<DT, V> rd[DEPTH][NV];
    Input<DT, V, KEPT> rx[DEPTH][NV];
    float mean[DEPTH], rstd[DEPTH];
    // The ranks start at different rows: their buffers often lie a power of two
    // apart, and equal rows would meet in the same memory channels (8 ranks x
    // 4,096 x 4,096 bf16, dx alone: 152 us from row 0 on every rank, 142 so, 138
    // with all rows on one rank).
    const uint64_t turned = a.rows * rank / gridDim.y;
    const auto real_row = [&](uint64_t r) { return r + turned < a.rows ? r + turned : r + turned - a.rows; };
    const auto fetch = [&](int k, uint64_t r) {
        r = real_row(r);
        const char* const dy = dy0 + r * a.dy_stride * elem_size<DT>();
        const InputRow<DT, KEPT> x(a, rank, r);
#pragma unroll
        for (int u = 0; u < NV; ++u) {
            RowPart<THREADS, V>(u, cols).template load<true>(rd[k][u], dy, cols);
            x.load(rx[k][u], RowPart<THREADS, V>(u, cols), cols);
        }
        mean[k] = mean0[r];
        rstd[k] = rstd0[r];
    };
#pragma unroll
    for (int k = 0; k < DEPTH; ++k) {
        if (row + k * step < a.rows) fetch(k, row + k * step);
    }
    Raw<WDT, V> g[NV] = {};
    float dg[EACH], db[EACH];
#pragma unroll
    for (int u = 0; u < NV; ++u) {
        if (gamma != nullptr) RowPart<THREADS, V>(u, cols).template load<false>(g[u], gamma, cols);
    }
    // an infinite weight times a cleared dy would be NaN: a moved-back vector has
    // one of each, also where a whole number of vectors leaves threads without any
#pragma unroll
    for (int u = 0; u < NV; ++u) RowPart<THREADS, V>(u, cols).clear(g[u]);
#pragma unroll
    for (int k = 0; k < EACH; ++k) dg[k] = db[k] = 0;
    int turn = 0;
    while (row < a.rows) {
#pragma unroll
        for (int k = 0; k < DEPTH; ++k) {
            if (row >= a.rows) break;
            float s[2] = {0, 0};
#pragma unroll
            for (int u = 0; u < NV; ++u) {
                // no gradient, no part in any sum: only dy is cleared
                RowPart<THREADS, V>(u, cols).clear(rd[k][u]);
                rx[k][u].ready();
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    const float d = rd[k][u].get(j);
                    const float h = (rx[k][u].get(j) - mean[k]) * rstd[k];
                    const float w = gamma != nullptr ? d * g[u].get(j) : d;
                    s[0] += w;
                    s[1] = __builtin_fmaf(w, h, s[1]);
                    dg[u * V + j] = __builtin_fmaf(d, h, dg[u * V + j]);
                    db[u * V + j] += d;
                }
            }
            sum_over_row<THREADS>(s, part[turn]);
            turn ^= 1;
            const float a0 = s[0] / over, a1 = s[1] / over;
            if constexpr (EACH >= 32) {
                // work the elements out again from their vectors below: kept as floats,
                // they and the sums would not fit the registers
#pragma unroll
                for (int u = 0; u < NV; ++u) {
#pragma unroll
                    for (int w = 0; w < Raw<DT, V>::kWords; ++w) asm volatile("" : "+v"(rd[k][u].w[w]));
#pragma unroll
                    for (int w = 0; w < Input<DT, V, KEPT>::kWords; ++w) asm volatile("" : "+v"(rx[k][u].w[w]));
#pragma unroll
                    for (int w = 0; w < Raw<WDT, V>::kWords; ++w) asm volatile("" : "+v"(g[u].w[w]));
                }
            }
            char* const dx = dx0 + real_row(row) * a.dx_stride * elem_size<DT>();
#pragma unroll
            for (int u = 0; u < NV; ++u) {
                float out[V];
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    const float d = rd[k][u].get(j);
                    const float h = (rx[k][u].get(j) - mean[k]) * rstd[k];
                    const float w = gamma != nullptr ? d * g[u].get(j) : d;
                    out[j] = rstd[k] * __builtin_fmaf(-h, a1, w - a0);
                }
                Raw<DT, V> o;
                o.set_all(out);
                RowPart<THREADS, V>(u, cols).store(o, dx, cols);
            }
            if (row + DEPTH * step < a.rows) fetch(k, row + DEPTH * step);
            row += step;
        }
    }
    if (!weights) return;
    float* const to = a.partials + (static_cast<uint64_t>(rank) * a.blocks + blockIdx.x) * 2 * a.cols;
    if constexpr (THREADS > 64) {
#pragma unroll
        for (int u = 0; u < NV; ++u) {
            const RowPart<THREADS, V> at(u, cols);
            if (at.skip == 0) {
                store_floats<V>(to + at.at, dg + u * V);
                store_floats<V>(to + cols + at.at, db + u * V);
            } else {
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    if (j >= at.skip) {
                        to[at.at + j] = dg[u * V + j];
                        to[cols + at.at + j] = db[u * V + j];
                    }
                }
            }
        }
    } else {
        // the workgroup's rows together: first the rows of a wavefront, where there
        // are several, then one wavefront after the other
        if constexpr (THREADS < 64) {
#pragma unroll
            for (int k = 0; k < EACH; ++k) {
                dg[k] = sum_over_rows<THREADS>(dg[k]);
                db[k] = sum_over_rows<THREADS>(db[k]);
            }
        }
        __shared__ float all[2][THREADS * EACH];
        for (int w = 0; w < 4; ++w) {
            if (threadIdx.x / 64 == w && threadIdx.x % 64 < THREADS) {
#pragma unroll
                for (int u = 0; u < NV; ++u) {
                    const RowPart<THREADS, V> at(u, cols);
#pragma unroll
                    for (int j = 0; j < V; ++j) {
                        if (at.mine(j, cols)) {
                            const int c = at.at + j, k = u * V + j;
                            all[0][c] = w == 0 ? dg[k] : all[0][c] + dg[k];
                            all[1][c] = w == 0 ? db[k] : all[1][c] + db[k];
                        }
                    }
                }
            }
            __syncthreads();
        }
        for (int c = threadIdx.x; c < cols; c += 256) {
            to[c] = all[0][c];
            to[cols + c] = all[1][c];
        }
    }
}

// Rows past what registers hold: dx alone, in two passes over the row; with the
// columns' sums below, 2^26 bf16 elements take 149 us (rows of 16,640) where rows
// in registers take 100 (16,384).
template <int DT, int WDT, int KEPT>
__global__ void __launch_bounds__(1024) k_layer_norm_backward_wide(NormBackwardArgs a) {
    constexpr int V = kRowVec<DT>;
    constexpr uint64_t kStep = 1024 * V;
    __shared__ float part[2][16][2];
    const int rank = blockIdx.y;
    const char* const gamma = a.gamma[rank];
    int turn = 0;
    for (uint64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const char* const dy = a.dy[rank] + row * a.dy_stride * elem_size<DT>();
        const InputRow<DT, KEPT> x(a, rank, row);
        char* const dx = a.dx[rank] + row * a.dx_stride * elem_size<DT>();
        const float mean = a.mean[rank][row], rstd = a.rstd[rank][row];
        float s[2] = {0, 0};
        for (uint64_t c = threadIdx.x * V; c < a.cols; c += kStep) {
            Raw<DT, V> rd;
            Input<DT, V, KEPT> rx;
            Raw<WDT, V> g;
            load_at<false, false>(rd, dy, c, a.cols);
            x.load(rx, c, a.cols);
            rx.ready();
            if (gamma != nullptr) load_at<false, false>(g, gamma, c, a.cols);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float d = rd.get(j);
                const float w = gamma != nullptr ? d * g.get(j) : d;
                const float h = c + j < a.cols ? (rx.get(j) - mean) * rstd : 0.0f;
                s[0] += w;
                s[1] += w * h;
            }
        }
        sum_over_row<1024>(s, part[turn]);
        turn ^= 1;
        const float a0 = s[0] / static_cast<float>(a.cols), a1 = s[1] / static_cast<float>(a.cols);
        for (uint64_t c = threadIdx.x * V; c < a.cols; c += kStep) {
            Raw<DT, V> rd;
            Input<DT, V, KEPT> rx;
            Raw<WDT, V> g;
            load_at<false, false>(rd, dy, c, a.cols);
            x.load(rx, c, a.cols);
            rx.ready();
            if (gamma != nullptr) load_at<false, false>(g, gamma, c, a.cols);
            float out[V];
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float d = rd.get(j);
                const float w = gamma != nullptr ? d * g.get(j) : d;
                out[j] = rstd * (w - a0 - (rx.get(j) - mean) * rstd * a1);
            }
            rd.set_all(out);
            store_at<false, true>(rd, dx, c, a.cols);
        }
    }
}

// The partial sums of such rows, before dx is written (dx may be dy): a
// workgroup takes one vector of columns a thread and every a.blocks-th row.
template <int DT, int KEPT>
__global__ void __launch_bounds__(kColumnThreads) k_layer_norm_columns(NormBackwardArgs a) {
    constexpr int V = kRowVec<DT>;
    const int rank = blockIdx.z;
    const uint64_t c = (static_cast<uint64_t>(blockIdx.x) * kColumnThreads + threadIdx.x) * V;
    if (c >= a.cols) return;
    float dg[V], db[V];
#pragma unroll
    for (int j = 0; j < V; ++j) dg[j] = db[j] = 0;
    for (uint64_t row = blockIdx.y; row < a.rows; row += a.blocks) {
        Raw<DT, V> rd;
        Input<DT, V, KEPT> rx;
        load_at<false, false>(rd, a.dy[rank] + row * a.dy_stride * elem_size<DT>(), c, a.cols);
        InputRow<DT, KEPT>(a, rank, row).load(rx, c, a.cols);
        rx.ready();
        const float mean = a.mean[rank][row], rstd = a.rstd[rank][row];
#pragma unroll
        for (int j = 0; j < V; ++j) {
            dg[j] += rd.get(j) * ((rx.get(j) - mean) * rstd);
            db[j] += rd.get(j);
        }
    }
    float* const to = a.partials + (static_cast<uint64_t>(rank) * a.blocks + blockIdx.y) * 2 * a.cols;
#pragma unroll
    for (int j = 0; j < V; ++j) {
        if (c + j < a.cols) {
            to[c + j] = dg[j];
            to[a.cols + c + j] = db[j];
        }
    }
}

// dgamma and dbeta from the partial sums: 64 columns a workgroup, 16 threads a
// column, each adding every 16th partial sum; then the 16 in order.
template <int WDT>
__global__ void __launch_bounds__(1024) k_layer_norm_weight_sums(NormBackwardArgs a) {
    const int rank = blockIdx.z;
    char* const out = blockIdx.y == 0 ? a.dgamma[rank] : a.dbeta[rank];
    if (out == nullptr) return;
    const int col = threadIdx.x % 64, group = threadIdx.x / 64;
    const uint64_t c = static_cast<uint64_t>(blockIdx.x) * 64 + col;
    __shared__ float sums[16][64];
    float s = 0;
    if (c < a.cols) {
        const float* from = a.partials + static_cast<uint64_t>(rank) * a.blocks * 2 * a.cols + blockIdx.y * a.cols + c;
#pragma unroll 4
        for (uint32_t b = group; b < a.blocks; b += 16) s += from[static_cast<uint64_t>(b) * 2 * a.cols];
    }
    sums[group][col] = s;
    __syncthreads();
    if (group == 0 && c < a.cols) {
        float t = 0;
#pragma unroll
        for (int k = 0; k < 16; ++k) t += sums[k][col];
        store_elem<elem_size<WDT>(), false>(out + c * elem_size<WDT>(), narrow<WDT>(t));
    }
}

constexpr uint64_t kMostBlocks = 1u << 18;

template <int DT, int WDT, int KEPT, int THREADS, int NV>
hipError_t start(const NormBackwardArgs& a, int nranks, bool weights, hipStream_t s) {
    const dim3 block(block_threads(THREADS));
    if constexpr (NV == 0) {
        if (weights) {
            const dim3 columns(static_cast<unsigned>(column_stretches(a.cols, kRowVec<DT>)), a.blocks, nranks);
            hipLaunchKernelGGL((k_layer_norm_columns<DT, KEPT>), columns, dim3(kColumnThreads), 0, s, a);
            const hipError_t e = hipGetLastError();
            if (e != hipSuccess) return e;
        }
        const dim3 grid(static_cast<unsigned>(std::min<uint64_t>(a.rows, kMostBlocks)), nranks);
        hipLaunchKernelGGL((k_layer_norm_backward_wide<DT, WDT, KEPT>), grid, block, 0, s, a);
    } else {
        const dim3 grid(a.blocks, nranks);
        hipLaunchKernelGGL((k_layer_norm_backward<DT, WDT, KEPT, THREADS, NV>), grid, block, 0, s, a, weights ? 1 : 0);
    }
    return hipGetLastError();
}

template <int DT, int WDT, int KEPT>
hipError_t rows_by_shape(const NormBackwardArgs& a, int nranks, bool weights, hipStream_t s) {
    const RowShape w = backward_shape(a.cols, kRowVec<DT>);
    switch (w.threads * 16 + w.vectors) {
        case 8 * 16 + 1: return start<DT, WDT, KEPT, 8, 1>(a, nranks, weights, s);
        case 16 * 16 + 1: return start<DT, WDT, KEPT, 16, 1>(a, nranks, weights, s);
        case 32 * 16 + 1: return start<DT, WDT, KEPT, 32, 1>(a, nranks, weights, s);
        case 64 * 16 + 1: return start<DT, WDT, KEPT, 64, 1>(a, nranks, weights, s);
        case 128 * 16 + 1: return start<DT, WDT, KEPT, 128, 1>(a, nranks, weights, s);
        case 256 * 16 + 1: return start<DT, WDT, KEPT, 256, 1>(a, nranks, weights, s);
        case 256 * 16 + 2: return start<DT, WDT, KEPT, 256, 2>(a, nranks, weights, s);
        case 512 * 16 + 2: return start<DT, WDT, KEPT, 512, 2>(a, nranks, weights, s);
        case 512 * 16 + 4: return start<DT, WDT, KEPT, 512, 4>(a, nranks, weights, s);
        case 512 * 16 + 8:
            if constexpr (DT == AR_FLOAT32) return start<DT, WDT, KEPT, 512, 8>(a, nranks, weights, s);
            return hipErrorInvalidValue;
        case 1024 * 16: return start<DT, WDT, KEPT, 1024, 0>(a, nranks, weights, s);
        default: return hipErrorInvalidValue;
    }
}

template <int DT, int WDT, int KEPT>
hipError_t by_shape(const NormBackwardArgs& a, int nranks, bool weights, hipStream_t s) {
    if (a.rows > 0) {   // else nothing but zeros to write below
        const hipError_t e = rows_by_shape<DT, WDT, KEPT>(a, nranks, weights, s);
        if (e != hipSuccess) return e;
    }
    if (!weights) return hipSuccess;
    const dim3 sums(static_cast<unsigned>((a.cols + 63) / 64), 2, nranks);
    hipLaunchKernelGGL((k_layer_norm_weight_sums<WDT>), sums, dim3(1024), 0, s, a);
    return hipGetLastError();
}

template <int KEPT>
hipError_t launch_backward(const NormBackwardArgs& a, int nranks, bool weights, ar_dtype_t dtype, ar_dtype_t weight,
                           hipStream_t s) {
    switch (dtype) {
        case AR_FLOAT32: return by_shape<AR_FLOAT32, AR_FLOAT32, KEPT>(a, nranks, weights, s);
        case AR_BFLOAT16:
            return weight == AR_FLOAT32 ? by_shape<AR_BFLOAT16, AR_FLOAT32, KEPT>(a, nranks, weights, s)
                                        : by_shape<AR_BFLOAT16, AR_BFLOAT16, KEPT>(a, nranks, weights, s);
        case AR_FLOAT16:
            return weight == AR_FLOAT32 ? by_shape<AR_FLOAT16, AR_FLOAT32, KEPT>(a, nranks, weights, s)
                                        : by_shape<AR_FLOAT16, AR_FLOAT16, KEPT>(a, nranks, weights, s);
        default: return hipErrorInvalidValue;
    }
}

}  // namespace
}  // namespace arimpl
