// HIP kernels of activations in 8 bits (include/ar.h states the format).
//
// One pass: a thread holds 8 neighbouring elements of a row, 4 threads a
// block.  Packing takes the block's largest magnitude over their lanes, and
// power-of-two scales make the quotient exact, so the only rounding is the one
// to the nearest code.  Reading and writing bound both directions.

#include <hip/hip_runtime.h>

#include "ar_activations.h"
#include "ar_activations_device.h"

namespace arimpl {
namespace {

constexpr int kPackVec = 8;                                          // elements a thread
constexpr int kBlockLanes = AR_ACTIVATION_BLOCK / kPackVec;          // threads a block
static_assert(kBlockLanes == 4, "a block is a quad of lanes");

// TPR threads a row, 256 / TPR rows a workgroup.
template <int TPR>
constexpr int kRowsAtOnce = 256 / TPR;

__device__ __forceinline__ uint64_t blocks_of(uint64_t cols) {
    return (cols + AR_ACTIVATION_BLOCK - 1) / AR_ACTIVATION_BLOCK;
}

template <int DT, int TPR>
__global__ void __launch_bounds__(256) k_pack(PackArgs a) {
    const int rank = blockIdx.y;
    const uint64_t blocks = blocks_of(a.cols);
    const uint64_t step = static_cast<uint64_t>(gridDim.x) * kRowsAtOnce<TPR>;
    for (uint64_t row = static_cast<uint64_t>(blockIdx.x) * kRowsAtOnce<TPR> + threadIdx.x / TPR; row < a.rows;
         row += step) {
        const char* const from = a.x[rank] + row * a.x_stride * elem_size<DT>();
        uint8_t* const codes = a.codes[rank] + row * a.cols;
        uint8_t* const scales = a.scales[rank] + row * blocks;
        // whole blocks of lanes, so that a quad's lanes all take part
        for (uint64_t u = threadIdx.x % TPR; u < blocks * kBlockLanes; u += TPR) {
            const uint64_t c = u * kPackVec;
            Raw<DT, kPackVec> r;
            load_at<false, true>(r, from, c, a.cols);
            uint32_t top = 0;
#pragma unroll
            for (int j = 0; j < kPackVec; ++j) top = std::max(top, as_u(r.get(j)) & 0x7fffffffu);
            const auto most = [](uint32_t p, uint32_t q) { return p > q ? p : q; };
            top = most(top, dpp<kDppXor1>(top));
            top = most(top, dpp<kDppXor2>(top));
            const uint32_t e = activation_scale(top);
            uint32_t w[2] = {0, 0};
#pragma unroll
            for (int j = 0; j < kPackVec; ++j) w[j / 4] |= activation_code(r.get(j), e) << (8 * (j % 4));
            if (e == 255) w[0] = w[1] = 0;
            if (c + kPackVec <= a.cols) {
                const u32x2 v = {w[0], w[1]};
                store_as<true, u32x2_a1>(reinterpret_cast<char*>(codes + c), v);
            } else {
#pragma unroll
                for (int j = 0; j < kPackVec; ++j) {
                    if (c + j < a.cols) codes[c + j] = static_cast<uint8_t>(w[j / 4] >> (8 * (j % 4)));
                }
            }
            if (u % kBlockLanes == 0) scales[u / kBlockLanes] = static_cast<uint8_t>(e);
        }
    }
}

template <int DT, int TPR>
__global__ void __launch_bounds__(256) k_unpack_activations(UnpackArgs a) {
    const int rank = blockIdx.y;
    const uint64_t blocks = blocks_of(a.cols);
    const uint64_t step = static_cast<uint64_t>(gridDim.x) * kRowsAtOnce<TPR>;
    for (uint64_t row = static_cast<uint64_t>(blockIdx.x) * kRowsAtOnce<TPR> + threadIdx.x / TPR; row < a.rows;
         row += step) {
        const uint8_t* const codes = a.codes[rank] + row * a.cols;
        const uint8_t* const scales = a.scales[rank] + row * blocks;
        char* const to = a.x[rank] + row * a.x_stride * elem_size<DT>();
        for (uint64_t c = (threadIdx.x % TPR) * kPackVec; c < a.cols; c += TPR * kPackVec) {
            const float scale = activation_scale_value(scales[c / AR_ACTIVATION_BLOCK]);
            uint32_t w[2] = {0, 0};
            if (c + kPackVec <= a.cols) {
                const u32x2 v = load_as<true, u32x2_a1>(reinterpret_cast<const char*>(codes + c));
                w[0] = v.x;
                w[1] = v.y;
            } else {
#pragma unroll
                for (int j = 0; j < kPackVec; ++j) {
                    if (c + j < a.cols) w[j / 4] |= static_cast<uint32_t>(codes[c + j]) << (8 * (j % 4));
                }
            }
            float x[kPackVec];
#pragma unroll
            for (int j = 0; j < kPackVec; ++j) x[j] = activation_value(w[j / 4], j % 4, scale);
            Raw<DT, kPackVec> o;
            o.set_all(x);
            store_at<false, true>(o, to, c, a.cols);
        }
    }
}

int row_threads(uint64_t cols) {
    const uint64_t need = (cols + AR_ACTIVATION_BLOCK - 1) / AR_ACTIVATION_BLOCK * kBlockLanes;
    return need <= 16 ? 16 : need <= 64 ? 64 : 256;
}

constexpr uint64_t kMostBlocks = 1u << 16;

template <int TPR>
dim3 grid_of(uint64_t rows, int nranks) {
    const uint64_t need = (rows + kRowsAtOnce<TPR> - 1) / kRowsAtOnce<TPR>;
    return dim3(static_cast<unsigned>(std::min(need, kMostBlocks)), nranks);
}

template <int DT>
hipError_t start_pack(const PackArgs& a, int nranks, hipStream_t s) {
    switch (row_threads(a.cols)) {
        case 16: hipLaunchKernelGGL((k_pack<DT, 16>), grid_of<16>(a.rows, nranks), dim3(256), 0, s, a); break;
        case 64: hipLaunchKernelGGL((k_pack<DT, 64>), grid_of<64>(a.rows, nranks), dim3(256), 0, s, a); break;
        default: hipLaunchKernelGGL((k_pack<DT, 256>), grid_of<256>(a.rows, nranks), dim3(256), 0, s, a); break;
    }
    return hipGetLastError();
}

template <int DT>
hipError_t start_unpack(const UnpackArgs& a, int nranks, hipStream_t s) {
    const dim3 block(256);
    switch (row_threads(a.cols)) {
        case 16: hipLaunchKernelGGL((k_unpack_activations<DT, 16>), grid_of<16>(a.rows, nranks), block, 0, s, a); break;
        case 64: hipLaunchKernelGGL((k_unpack_activations<DT, 64>), grid_of<64>(a.rows, nranks), block, 0, s, a); break;
        default: hipLaunchKernelGGL((k_unpack_activations<DT, 256>), grid_of<256>(a.rows, nranks), block, 0, s, a); break;
    }
    return hipGetLastError();
}

}  // namespace

hipError_t launch_pack(const PackArgs& a, int nranks, ar_dtype_t dtype, hipStream_t s) {
    switch (dtype) {
        case AR_FLOAT32: return start_pack<AR_FLOAT32>(a, nranks, s);
        case AR_BFLOAT16: return start_pack<AR_BFLOAT16>(a, nranks, s);
        case AR_FLOAT16: return start_pack<AR_FLOAT16>(a, nranks, s);
        default: return hipErrorInvalidValue;
    }
}

hipError_t launch_unpack(const UnpackArgs& a, int nranks, ar_dtype_t dtype, hipStream_t s) {
    switch (dtype) {
        case AR_FLOAT32: return start_unpack<AR_FLOAT32>(a, nranks, s);
        case AR_BFLOAT16: return start_unpack<AR_BFLOAT16>(a, nranks, s);
        case AR_FLOAT16: return start_unpack<AR_FLOAT16>(a, nranks, s);
        default: return hipErrorInvalidValue;
    }
}

}  // namespace arimpl
