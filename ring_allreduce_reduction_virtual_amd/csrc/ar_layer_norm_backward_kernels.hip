// HIP kernels of layer norm's backward pass (include/ar.h states the
// formulas).
//
// One pass over dy and x makes dx, and each thread adds its columns' parts of
// dgamma and dbeta over all the rows that its workgroup takes: a thread keeps
// the same columns from row to row, so these sums stay in registers.  Each
// workgroup leaves one partial sum per column; a second launch adds them in
// the order of the workgroups, so that the result does not depend on which
// one finishes first.  The activations' two reads and one write bound it.

#include <hip/hip_runtime.h>

#include "ar_layer_norm_device.h"

namespace arimpl {
namespace {

template <int DT, int WDT, int THREADS, int EACH>
__global__ void __launch_bounds__(THREADS < 256 ? 256 : THREADS) k_layer_norm_backward(NormBackwardArgs a,
                                                                                      int weights) {
    constexpr int V = kRowVec<DT>;
    constexpr int NV = EACH / V;
    constexpr int kRows = rows_at_once(THREADS);
    __shared__ float part[2][THREADS / 64 + 1][2];
    const int rank = blockIdx.y;
    const int lane = threadIdx.x % THREADS;
    const int cols = static_cast<int>(a.cols);
    const char* const gamma = a.gamma[rank];
    const float over = static_cast<float>(cols);
    Raw<WDT, V> g[NV];
    float dg[EACH], db[EACH];
#pragma unroll
    for (int u = 0; u < NV; ++u) {
        if (gamma != nullptr) load_at<false, false>(g[u], gamma, (u * THREADS + lane) * V, cols);
    }
#pragma unroll
    for (int k = 0; k < EACH; ++k) dg[k] = db[k] = 0;
    int turn = 0;
    for (uint64_t row = static_cast<uint64_t>(blockIdx.x) * kRows + threadIdx.x / THREADS; row < a.rows;
         row += static_cast<uint64_t>(gridDim.x) * kRows) {
        const char* const dy = a.dy[rank] + row * a.dy_stride * elem_size<DT>();
        const char* const x = a.x[rank] + row * a.x_stride * elem_size<DT>();
        Raw<DT, V> rd[NV], rx[NV];
#pragma unroll
        for (int u = 0; u < NV; ++u) {
            load_at<false, true>(rd[u], dy, (u * THREADS + lane) * V, cols);
            load_at<false, true>(rx[u], x, (u * THREADS + lane) * V, cols);
        }
        const float mean = a.mean[rank][row], rstd = a.rstd[rank][row];
        float s[2] = {0, 0};
#pragma unroll
        for (int u = 0; u < NV; ++u) {
            const int left = cols - (u * THREADS + lane) * V;
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float d = rd[u].get(j);   // 0 beyond the end
                const float h = j < left ? (rx[u].get(j) - mean) * rstd : 0.0f;
                const float w = gamma != nullptr ? d * g[u].get(j) : d;
                s[0] += w;
                s[1] += w * h;
                dg[u * V + j] += d * h;
                db[u * V + j] += d;
            }
        }
        sum_over_row<THREADS>(s, part[turn]);
        turn ^= 1;
        const float a0 = s[0] / over, a1 = s[1] / over;
        char* const dx = a.dx[rank] + row * a.dx_stride * elem_size<DT>();
#pragma unroll
        for (int u = 0; u < NV; ++u) {
            float out[V];
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float d = rd[u].get(j);
                const float w = gamma != nullptr ? d * g[u].get(j) : d;
                out[j] = rstd * (w - a0 - (rx[u].get(j) - mean) * rstd * a1);
            }
            rx[u].set_all(out);
            store_at<false, true>(rx[u], dx, (u * THREADS + lane) * V, cols);
        }
    }
    if (!weights) return;
    float* const to = a.partials + (static_cast<uint64_t>(rank) * a.blocks + blockIdx.x) * 2 * a.cols;
    if constexpr (THREADS >= 256) {
#pragma unroll
        for (int k = 0; k < EACH; ++k) {
            const int c = ((k / V) * THREADS + lane) * V + k % V;
            if (c < cols) {
                to[c] = dg[k];
                to[cols + c] = db[k];
            }
        }
    } else {
        // the workgroup's rows together: first the four rows of a wavefront, where
        // there are four, then one wavefront after the other
        if constexpr (THREADS == 16) {
            const auto add = [](uint32_t p, uint32_t q) { return as_u(as_f(p) + as_f(q)); };
#pragma unroll
            for (int k = 0; k < EACH; ++k) {
                dg[k] = as_f(across32(across16(as_u(dg[k]), add), add));
                db[k] = as_f(across32(across16(as_u(db[k]), add), add));
            }
        }
        __shared__ float all[2][THREADS * EACH];
        for (int w = 0; w < 4; ++w) {
            if (threadIdx.x / 64 == w && threadIdx.x % 64 < THREADS) {
#pragma unroll
                for (int k = 0; k < EACH; ++k) {
                    const int c = ((k / V) * THREADS + lane) * V + k % V;
                    all[0][c] = w == 0 ? dg[k] : all[0][c] + dg[k];
                    all[1][c] = w == 0 ? db[k] : all[1][c] + db[k];
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

// Rows past what registers hold: dx alone, in two passes over the row.
template <int DT, int WDT>
__global__ void __launch_bounds__(1024) k_layer_norm_backward_wide(NormBackwardArgs a) {
    constexpr int V = kRowVec<DT>;
    constexpr uint64_t kStep = 1024 * V;
    __shared__ float part[2][16][2];
    const int rank = blockIdx.y;
    const char* const gamma = a.gamma[rank];
    int turn = 0;
    for (uint64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const char* const dy = a.dy[rank] + row * a.dy_stride * elem_size<DT>();
        const char* const x = a.x[rank] + row * a.x_stride * elem_size<DT>();
        char* const dx = a.dx[rank] + row * a.dx_stride * elem_size<DT>();
        const float mean = a.mean[rank][row], rstd = a.rstd[rank][row];
        float s[2] = {0, 0};
        for (uint64_t c = threadIdx.x * V; c < a.cols; c += kStep) {
            Raw<DT, V> rd, rx;
            Raw<WDT, V> g;
            load_at<false, false>(rd, dy, c, a.cols);
            load_at<false, false>(rx, x, c, a.cols);
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
            Raw<DT, V> rd, rx;
            Raw<WDT, V> g;
            load_at<false, false>(rd, dy, c, a.cols);
            load_at<false, false>(rx, x, c, a.cols);
            if (gamma != nullptr) load_at<false, false>(g, gamma, c, a.cols);
            float out[V];
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float d = rd.get(j);
                const float w = gamma != nullptr ? d * g.get(j) : d;
                out[j] = rstd * (w - a0 - (rx.get(j) - mean) * rstd * a1);
            }
            rx.set_all(out);
            store_at<false, true>(rx, dx, c, a.cols);
        }
    }
}

// The partial sums of such rows, before dx is written (dx may be dy): a
// workgroup takes 256 vectors of columns and every a.blocks-th row.
template <int DT>
__global__ void __launch_bounds__(256) k_layer_norm_columns(NormBackwardArgs a) {
    constexpr int V = kRowVec<DT>;
    const int rank = blockIdx.z;
    const uint64_t c = (static_cast<uint64_t>(blockIdx.x) * 256 + threadIdx.x) * V;
    if (c >= a.cols) return;
    float dg[V], db[V];
#pragma unroll
    for (int j = 0; j < V; ++j) dg[j] = db[j] = 0;
    for (uint64_t row = blockIdx.y; row < a.rows; row += a.blocks) {
        Raw<DT, V> rd, rx;
        load_at<false, false>(rd, a.dy[rank] + row * a.dy_stride * elem_size<DT>(), c, a.cols);
        load_at<false, false>(rx, a.x[rank] + row * a.x_stride * elem_size<DT>(), c, a.cols);
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

template <int DT, int WDT>
hipError_t by_shape(const NormBackwardArgs& a, int nranks, bool weights, hipStream_t s) {
    const RowShape w = row_shape(a.cols);
    const dim3 block(w.threads < 256 ? 256 : w.threads);
    dim3 grid(a.blocks, nranks);
    const int wg = weights ? 1 : 0;
    hipError_t e = hipSuccess;
    if (a.rows == 0) {
        // nothing but zeros to write below
    } else if (w.each == 0) {
        if (weights) {
            constexpr uint64_t per = 256 * kRowVec<DT>;
            const dim3 columns(static_cast<unsigned>((a.cols + per - 1) / per), a.blocks, nranks);
            hipLaunchKernelGGL((k_layer_norm_columns<DT>), columns, dim3(256), 0, s, a);
            if ((e = hipGetLastError()) != hipSuccess) return e;
        }
        grid.x = static_cast<unsigned>(std::min<uint64_t>(a.rows, kMostBlocks));
        hipLaunchKernelGGL((k_layer_norm_backward_wide<DT, WDT>), grid, block, 0, s, a);
    } else if (w.threads == 16) {
        hipLaunchKernelGGL((k_layer_norm_backward<DT, WDT, 16, 8>), grid, block, 0, s, a, wg);
    } else if (w.threads == 64) {
        if (w.each == 8) {
            hipLaunchKernelGGL((k_layer_norm_backward<DT, WDT, 64, 8>), grid, block, 0, s, a, wg);
        } else if (w.each == 16) {
            hipLaunchKernelGGL((k_layer_norm_backward<DT, WDT, 64, 16>), grid, block, 0, s, a, wg);
        } else {
            hipLaunchKernelGGL((k_layer_norm_backward<DT, WDT, 64, 32>), grid, block, 0, s, a, wg);
        }
    } else if (w.threads == 256) {
        if (w.each == 16) {
            hipLaunchKernelGGL((k_layer_norm_backward<DT, WDT, 256, 16>), grid, block, 0, s, a, wg);
        } else {
            hipLaunchKernelGGL((k_layer_norm_backward<DT, WDT, 256, 32>), grid, block, 0, s, a, wg);
        }
    } else {
        hipLaunchKernelGGL((k_layer_norm_backward<DT, WDT, 1024, 16>), grid, block, 0, s, a, wg);
    }
    if ((e = hipGetLastError()) != hipSuccess || !weights) return e;
    const dim3 sums(static_cast<unsigned>((a.cols + 63) / 64), 2, nranks);
    hipLaunchKernelGGL((k_layer_norm_weight_sums<WDT>), sums, dim3(1024), 0, s, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_norm_backward(const NormBackwardArgs& a, int nranks, bool weights, ar_dtype_t dtype,
                                ar_dtype_t weight, hipStream_t s) {
    switch (dtype) {
        case AR_FLOAT32: return by_shape<AR_FLOAT32, AR_FLOAT32>(a, nranks, weights, s);
        case AR_BFLOAT16:
            return weight == AR_FLOAT32 ? by_shape<AR_BFLOAT16, AR_FLOAT32>(a, nranks, weights, s)
                                        : by_shape<AR_BFLOAT16, AR_BFLOAT16>(a, nranks, weights, s);
        case AR_FLOAT16:
            return weight == AR_FLOAT32 ? by_shape<AR_FLOAT16, AR_FLOAT32>(a, nranks, weights, s)
                                        : by_shape<AR_FLOAT16, AR_FLOAT16>(a, nranks, weights, s);
        default: return hipErrorInvalidValue;
    }
}

}  // namespace arimpl
