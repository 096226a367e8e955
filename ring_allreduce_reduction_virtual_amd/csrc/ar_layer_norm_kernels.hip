// HIP kernels of layer norm's forward pass (include/ar.h states the formulas).
//
// A row is read once into registers: its mean, then the sum of squares around
// that mean (not the difference of two large sums), then the normalised row
// come from there.  A workgroup keeps the weights in registers over the rows
// that it takes, and the next row's loads run beside this row's sums.  The
// activations' read and write bound it: 8 ranks x 4,096 x 4,096 bf16 91.6 us,
// 5.9 TB/s.

#include <hip/hip_runtime.h>

#include "ar_layer_norm_device.h"

namespace arimpl {
namespace {

template <int DT, int WDT, int THREADS, int NV>
__global__ void __launch_bounds__(block_threads(THREADS)) k_layer_norm(NormForwardArgs a) {
    constexpr int V = kRowVec<DT>;
    constexpr int kRows = rows_at_once(THREADS);
    __shared__ float part[2][THREADS / 64 + 1][1];
    const int rank = blockIdx.y;
    const int cols = static_cast<int>(a.cols);
    const char* const gamma = a.gamma[rank];
    const char* const beta = a.beta[rank];
    const uint64_t step = static_cast<uint64_t>(gridDim.x) * kRows;
    uint64_t row = first_row<THREADS>();
    if (row >= a.rows) return;   // whole rows of threads: no barrier is missed
    Raw<DT, V> next[NV];
#pragma unroll
    for (int u = 0; u < NV; ++u)
        RowPart<THREADS, V>(u, cols).template load<true>(next[u], a.x[rank] + row * a.x_stride * elem_size<DT>(), cols);
    Raw<WDT, V> g[NV], b[NV];
#pragma unroll
    for (int u = 0; u < NV; ++u) {
        if (gamma != nullptr) RowPart<THREADS, V>(u, cols).template load<false>(g[u], gamma, cols);
        if (beta != nullptr) RowPart<THREADS, V>(u, cols).template load<false>(b[u], beta, cols);
    }
    for (; row < a.rows; row += step) {
        Raw<DT, V> r[NV];
#pragma unroll
        for (int u = 0; u < NV; ++u) r[u] = next[u];
        if (row + step < a.rows) {   // the next row's loads run beside this row's sums
#pragma unroll
            for (int u = 0; u < NV; ++u)
                RowPart<THREADS, V>(u, cols).template load<true>(
                    next[u], a.x[rank] + (row + step) * a.x_stride * elem_size<DT>(), cols);
        }
        float sum[1] = {0};
#pragma unroll
        for (int u = 0; u < NV; ++u) {
            const RowPart<THREADS, V> at(u, cols);
#pragma unroll
            for (int j = 0; j < V; ++j) sum[0] += at.mine(j, cols) ? r[u].get(j) : 0.0f;
        }
        sum_over_row<THREADS>(sum, part[0]);
        const float mean = sum[0] / static_cast<float>(cols);
        float sq[1] = {0};
#pragma unroll
        for (int u = 0; u < NV; ++u) {
            const RowPart<THREADS, V> at(u, cols);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float d = at.mine(j, cols) ? r[u].get(j) - mean : 0.0f;
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
            RowPart<THREADS, V>(u, cols).store(r[u], y, cols);
        }
        if (threadIdx.x % THREADS == 0 && a.mean[rank] != nullptr) {
            a.mean[rank][row] = mean;
            a.rstd[rank][row] = rstd;
        }
    }
}

// Rows past what registers hold: three passes over the row, the second and
// third served by the caches (2^26 bf16 elements in rows of 16,384: 73-77 us,
// where a row in registers takes 54).
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

// Wavefronts in all that are started at most, about twice what the GPU holds at
// once; each takes rows in turn and keeps the weights.  A half as many: 2,048
// columns of bf16 51.5 us against 48.0, 4,096 55.0 against 52.4.
constexpr uint64_t kForwardWaves = 16384;

template <int DT, int WDT, int THREADS, int NV>
hipError_t start(const NormForwardArgs& a, int nranks, hipStream_t s) {
    constexpr int kBlock = block_threads(THREADS), kRows = rows_at_once(THREADS);
    const uint64_t most = std::max<uint64_t>(1, kForwardWaves * 64 / kBlock / nranks);
    const dim3 grid(static_cast<unsigned>(std::min<uint64_t>((a.rows + kRows - 1) / kRows, most)), nranks);
    if constexpr (NV == 0) {
        hipLaunchKernelGGL((k_layer_norm_wide<DT, WDT>), grid, dim3(kBlock), 0, s, a);
    } else {
        hipLaunchKernelGGL((k_layer_norm<DT, WDT, THREADS, NV>), grid, dim3(kBlock), 0, s, a);
    }
    return hipGetLastError();
}

template <int DT, int WDT>
hipError_t by_shape(const NormForwardArgs& a, int nranks, hipStream_t s) {
    const RowShape w = forward_shape(a.cols, kRowVec<DT>);
    switch (w.threads * 16 + w.vectors) {
        case 8 * 16 + 1: return start<DT, WDT, 8, 1>(a, nranks, s);
        case 16 * 16 + 1: return start<DT, WDT, 16, 1>(a, nranks, s);
        case 32 * 16 + 1: return start<DT, WDT, 32, 1>(a, nranks, s);
        case 64 * 16 + 1: return start<DT, WDT, 64, 1>(a, nranks, s);
        case 64 * 16 + 2: return start<DT, WDT, 64, 2>(a, nranks, s);
        case 64 * 16 + 4: return start<DT, WDT, 64, 4>(a, nranks, s);
        case 128 * 16 + 4: return start<DT, WDT, 128, 4>(a, nranks, s);
        case 256 * 16 + 4: return start<DT, WDT, 256, 4>(a, nranks, s);
        case 1024 * 16 + 2: return start<DT, WDT, 1024, 2>(a, nranks, s);
        case 1024 * 16 + 4:
            if constexpr (DT == AR_FLOAT32) return start<DT, WDT, 1024, 4>(a, nranks, s);
            return hipErrorInvalidValue;
        case 1024 * 16: return start<DT, WDT, 1024, 0>(a, nranks, s);
        default: return hipErrorInvalidValue;
    }
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
