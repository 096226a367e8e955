// HIP kernels of layer norm's forward pass (include/ar.h states the formulas).
//
// A row is read once into registers: its mean, then the sum of squares around
// that mean (not the difference of two large sums), then the normalised row
// come from there.  The activations' read and write bound it.

#include <hip/hip_runtime.h>

#include "ar_layer_norm_device.h"

namespace arimpl {
namespace {

template <int DT, int WDT, int THREADS, int EACH>
__global__ void __launch_bounds__(THREADS < 256 ? 256 : THREADS) k_layer_norm(NormForwardArgs a) {
    constexpr int V = kRowVec<DT>;
    constexpr int NV = EACH / V;
    constexpr int kRows = rows_at_once(THREADS);
    __shared__ float part[2][THREADS / 64 + 1][1];
    const int rank = blockIdx.y;
    const int lane = threadIdx.x % THREADS;
    const int cols = static_cast<int>(a.cols);
    const char* const gamma = a.gamma[rank];
    const char* const beta = a.beta[rank];
    for (uint64_t row = static_cast<uint64_t>(blockIdx.x) * kRows + threadIdx.x / THREADS; row < a.rows;
         row += static_cast<uint64_t>(gridDim.x) * kRows) {
        const char* const x = a.x[rank] + row * a.x_stride * elem_size<DT>();
        Raw<DT, V> r[NV];
        Raw<WDT, V> g[NV], b[NV];
#pragma unroll
        for (int u = 0; u < NV; ++u) load_at<false, true>(r[u], x, (u * THREADS + lane) * V, cols);
#pragma unroll
        for (int u = 0; u < NV; ++u) {
            if (gamma != nullptr) load_at<false, false>(g[u], gamma, (u * THREADS + lane) * V, cols);
            if (beta != nullptr) load_at<false, false>(b[u], beta, (u * THREADS + lane) * V, cols);
        }
        float sum[1] = {0};
#pragma unroll
        for (int u = 0; u < NV; ++u) {
#pragma unroll
            for (int j = 0; j < V; ++j) sum[0] += r[u].get(j);   // 0 beyond the end
        }
        sum_over_row<THREADS>(sum, part[0]);
        const float mean = sum[0] / static_cast<float>(cols);
        float sq[1] = {0};
#pragma unroll
        for (int u = 0; u < NV; ++u) {
            const int left = cols - (u * THREADS + lane) * V;
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float d = j < left ? r[u].get(j) - mean : 0.0f;
                sq[0] += d * d;
            }
        }
        sum_over_row<THREADS>(sq, part[1]);
        const float rstd = 1.0f / sqrtf(sq[0] / static_cast<float>(cols) + a.eps);
        char* const y = a.y[rank] + row * a.y_stride * elem_size<DT>();
#pragma unroll
        for (int u = 0; u < NV; ++u) {
            float out[V];
#pragma unroll
            for (int j = 0; j < V; ++j) {
                out[j] = (r[u].get(j) - mean) * rstd;
                if (gamma != nullptr) out[j] *= g[u].get(j);
                if (beta != nullptr) out[j] += b[u].get(j);
            }
            r[u].set_all(out);
            store_at<false, true>(r[u], y, (u * THREADS + lane) * V, cols);
        }
        if (lane == 0 && a.mean[rank] != nullptr) {
            a.mean[rank][row] = mean;
            a.rstd[rank][row] = rstd;
        }
    }
}

// Rows past what registers hold: three passes over the row, the second and
// third served by the caches.
template <int DT, int WDT>
__global__ void __launch_bounds__(1024) k_layer_norm_wide(NormForwardArgs a) {
    constexpr int V = kRowVec<DT>;
    constexpr uint64_t kStep = 1024 * V;
    __shared__ float part[2][16][1];
    const int rank = blockIdx.y;
    const char* const gamma = a.gamma[rank];
    const char* const beta = a.beta[rank];
    for (uint64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const char* const x = a.x[rank] + row * a.x_stride * elem_size<DT>();
        char* const y = a.y[rank] + row * a.y_stride * elem_size<DT>();
        float sum[1] = {0}, sq[1] = {0};
        for (uint64_t c = threadIdx.x * V; c < a.cols; c += kStep) {
            Raw<DT, V> r;
            load_at<false, false>(r, x, c, a.cols);
#pragma unroll
            for (int j = 0; j < V; ++j) sum[0] += r.get(j);
        }
        sum_over_row<1024>(sum, part[0]);
        const float mean = sum[0] / static_cast<float>(a.cols);
        for (uint64_t c = threadIdx.x * V; c < a.cols; c += kStep) {
            Raw<DT, V> r;
            load_at<false, false>(r, x, c, a.cols);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float d = c + j < a.cols ? r.get(j) - mean : 0.0f;
                sq[0] += d * d;
            }
        }
        sum_over_row<1024>(sq, part[1]);
        const float rstd = 1.0f / sqrtf(sq[0] / static_cast<float>(a.cols) + a.eps);
        for (uint64_t c = threadIdx.x * V; c < a.cols; c += kStep) {
            Raw<DT, V> r;
            Raw<WDT, V> g, b;
            load_at<false, false>(r, x, c, a.cols);
            if (gamma != nullptr) load_at<false, false>(g, gamma, c, a.cols);
            if (beta != nullptr) load_at<false, false>(b, beta, c, a.cols);
            float out[V];
#pragma unroll
            for (int j = 0; j < V; ++j) {
                out[j] = (r.get(j) - mean) * rstd;
                if (gamma != nullptr) out[j] *= g.get(j);
                if (beta != nullptr) out[j] += b.get(j);
            }
            r.set_all(out);
            store_at<false, true>(r, y, c, a.cols);
        }
        if (threadIdx.x == 0 && a.mean[rank] != nullptr) {
            a.mean[rank][row] = mean;
            a.rstd[rank][row] = rstd;
        }
    }
}

// Workgroups a rank at most; each then takes further rows in turn.
constexpr uint64_t kMostBlocks = 1u << 18;

template <int DT, int WDT>
hipError_t by_shape(const NormForwardArgs& a, int nranks, hipStream_t s) {
    const RowShape w = row_shape(a.cols);
    const uint64_t at_once = rows_at_once(w.threads);
    const dim3 grid(static_cast<unsigned>(std::min<uint64_t>((a.rows + at_once - 1) / at_once, kMostBlocks)), nranks);
    const dim3 block(w.threads < 256 ? 256 : w.threads);
    if (w.each == 0) {
        hipLaunchKernelGGL((k_layer_norm_wide<DT, WDT>), grid, block, 0, s, a);
    } else if (w.threads == 16) {
        hipLaunchKernelGGL((k_layer_norm<DT, WDT, 16, 8>), grid, block, 0, s, a);
    } else if (w.threads == 64) {
        if (w.each == 8) {
            hipLaunchKernelGGL((k_layer_norm<DT, WDT, 64, 8>), grid, block, 0, s, a);
        } else if (w.each == 16) {
            hipLaunchKernelGGL((k_layer_norm<DT, WDT, 64, 16>), grid, block, 0, s, a);
        } else {
            hipLaunchKernelGGL((k_layer_norm<DT, WDT, 64, 32>), grid, block, 0, s, a);
        }
    } else if (w.threads == 256) {
        if (w.each == 16) {
            hipLaunchKernelGGL((k_layer_norm<DT, WDT, 256, 16>), grid, block, 0, s, a);
        } else {
            hipLaunchKernelGGL((k_layer_norm<DT, WDT, 256, 32>), grid, block, 0, s, a);
        }
    } else {
        hipLaunchKernelGGL((k_layer_norm<DT, WDT, 1024, 16>), grid, block, 0, s, a);
    }
    return hipGetLastError();
}

}  // namespace

hipError_t launch_norm_forward(const NormForwardArgs& a, int nranks, ar_dtype_t dtype, ar_dtype_t weight,
                               hipStream_t s) {
    switch (dtype) {
        case AR_FLOAT32: return by_shape<AR_FLOAT32, AR_FLOAT32>(a, nranks, s);
        case AR_BFLOAT16:
            return weight == AR_FLOAT32 ? by_shape<AR_BFLOAT16, AR_FLOAT32>(a, nranks, s)
                                        : by_shape<AR_BFLOAT16, AR_BFLOAT16>(a, nranks, s);
        case AR_FLOAT16:
            return weight == AR_FLOAT32 ? by_shape<AR_FLOAT16, AR_FLOAT32>(a, nranks, s)
                                        : by_shape<AR_FLOAT16, AR_FLOAT16>(a, nranks, s);
        default: return hipErrorInvalidValue;
    }
}

}  // namespace arimpl
