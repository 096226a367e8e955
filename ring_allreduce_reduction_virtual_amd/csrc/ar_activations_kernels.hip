// HIP kernels of activations in 8 bits (include/ar.h states the format).
//
// One pass: a thread holds 16 bytes of a row's neighbouring elements, 4 threads
// (float32: 8) a block.  Packing takes the block's largest magnitude over their
// lanes, and power-of-two scales make the quotient exact, so the only rounding
// is the one to the nearest code.  Reading and writing bound both directions: 8
// ranks x 4,096 x 4,096 bf16 68 us to pack (407 MB, 6.0 TB/s), 65 to unpack.

#include <hip/hip_runtime.h>

#include "ar_activations.h"
#include "ar_activations_device.h"

namespace arimpl {
namespace {

template <int DT>
constexpr int kPackVec = 16 / elem_size<DT>();                     // elements a thread
template <int DT>
constexpr int kBlockLanes = AR_ACTIVATION_BLOCK / kPackVec<DT>;    // threads a block

// TPR threads a row, 256 / TPR rows a workgroup.
template <int TPR>
constexpr int kRowsAtOnce = 256 / TPR;

__device__ __forceinline__ uint64_t blocks_of(uint64_t cols) {
    return (cols + AR_ACTIVATION_BLOCK - 1) / AR_ACTIVATION_BLOCK;
}

// The codes of V elements, in one store where all of them are in the row.
template <int V>
__device__ __forceinline__ void store_codes(uint8_t* p, const uint32_t (&w)[V / 4], int left) {
    if (left >= V) {
        if constexpr (V == 8) {
            const u32x2 v = {w[0], w[1]};
            store_as<true, u32x2_a1>(reinterpret_cast<char*>(p), v);
        } else {
            typedef uint32_t u32_a1 __attribute__((aligned(1)));
            store_as<true, u32_a1>(reinterpret_cast<char*>(p), w[0]);
        }
    } else {
#pragma unroll
        for (int j = 0; j < V; ++j) {
            if (j < left) p[j] = static_cast<uint8_t>(w[j / 4] >> (8 * (j % 4)));
        }
    }
}
template <int V>
__device__ __forceinline__ void load_codes(uint32_t (&w)[V / 4], const uint8_t* p, int left) {
    if (left >= V) {
        if constexpr (V == 8) {
            const u32x2 v = load_as<true, u32x2_a1>(reinterpret_cast<const char*>(p));
            w[0] = v.x;
            w[1] = v.y;
        } else {
            typedef uint32_t u32_a1 __attribute__((aligned(1)));
            w[0] = load_as<true, u32_a1>(reinterpret_cast<const char*>(p));
        }
    } else {
#pragma unroll
        for (int k = 0; k < V / 4; ++k) w[k] = 0;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            if (j < left) w[j / 4] |= static_cast<uint32_t>(p[j]) << (8 * (j % 4));
        }
    }
}

template <int DT, int TPR>
__global__ void __launch_bounds__(256) k_pack(PackArgs a) {
    constexpr int V = kPackVec<DT>, kLanes = kBlockLanes<DT>;
    const int rank = blockIdx.y;
    const uint64_t blocks = blocks_of(a.cols);
    const uint64_t step = static_cast<uint64_t>(gridDim.x) * kRowsAtOnce<TPR>;
    for (uint64_t row = static_cast<uint64_t>(blockIdx.x) * kRowsAtOnce<TPR> + threadIdx.x / TPR; row < a.rows;
         row += step) {
        const char* const from = a.x[rank] + row * a.x_stride * elem_size<DT>();
        uint8_t* const codes = a.codes[rank] + row * a.cols;
        uint8_t* const scales = a.scales[rank] + row * blocks;
        // whole blocks of lanes, so that all of a block's lanes take part
        for (uint64_t u = threadIdx.x % TPR; u < blocks * kLanes; u += TPR) {
            const uint64_t c = u * V;
            Raw<DT, V> r;
            load_at<false, true>(r, from, c, a.cols);
            uint32_t top = 0;
#pragma unroll
            for (int j = 0; j < V; ++j) top = std::max(top, as_u(r.get(j)) & 0x7fffffffu);
            const auto most = [](uint32_t p, uint32_t q) { return p > q ? p : q; };
            top = most(top, dpp<kDppXor1>(top));
            top = most(top, dpp<kDppXor2>(top));
            if constexpr (kLanes == 8) top = most(top, dpp<kDppHalfMirror>(top));
            const uint32_t e = activation_scale(top);
            uint32_t w[V / 4] = {};
#pragma unroll
            for (int j = 0; j < V; ++j) w[j / 4] |= activation_code(r.get(j), e) << (8 * (j % 4));
            if (e == 255) {
#pragma unroll
                for (int k = 0; k < V / 4; ++k) w[k] = 0;
            }
            if (c < a.cols) store_codes<V>(codes + c, w, static_cast<int>(std::min<uint64_t>(V, a.cols - c)));
            if (u % kLanes == 0) scales[u / kLanes] = static_cast<uint8_t>(e);
        }
    }
}

template <int DT, int TPR>
__global__ void __launch_bounds__(256) k_unpack_activations(UnpackArgs a) {
    constexpr int V = kPackVec<DT>;
    const int rank = blockIdx.y;
    const uint64_t blocks = blocks_of(a.cols);
    const uint64_t step = static_cast<uint64_t>(gridDim.x) * kRowsAtOnce<TPR>;
    for (uint64_t row = static_cast<uint64_t>(blockIdx.x) * kRowsAtOnce<TPR> + threadIdx.x / TPR; row < a.rows;
         row += step) {
        const uint8_t* const codes = a.codes[rank] + row * a.cols;
        const uint8_t* const scales = a.scales[rank] + row * blocks;
        char* const to = a.x[rank] + row * a.x_stride * elem_size<DT>();
        for (uint64_t c = (threadIdx.x % TPR) * V; c < a.cols; c += TPR * V) {
            const uint32_t e = scales[c / AR_ACTIVATION_BLOCK];
            uint32_t w[V / 4];
            load_codes<V>(w, codes + c, static_cast<int>(std::min<uint64_t>(V, a.cols - c)));
            const float scale = activation_scale_value(e);
            float x[V];
#pragma unroll
            for (int j = 0; j < V; ++j) x[j] = activation_value(w[j / 4], j % 4, scale);
            Raw<DT, V> o;
            o.set_all(x);
            store_at<false, true>(o, to, c, a.cols);
        }
    }
}

int row_threads(uint64_t cols, int block_lanes) {
    const uint64_t need = (cols + AR_ACTIVATION_BLOCK - 1) / AR_ACTIVATION_BLOCK * block_lanes;
    return need <= 16 ? 16 : need <= 64 ? 64 : need <= 128 ? 128 : 256;
}

constexpr uint64_t kMostBlocks = 1u << 16;

template <int TPR>
dim3 grid_of(uint64_t rows, int nranks) {
    const uint64_t need = (rows + kRowsAtOnce<TPR> - 1) / kRowsAtOnce<TPR>;
    return dim3(static_cast<unsigned>(std::min(need, kMostBlocks)), nranks);
}

template <int DT>
hipError_t start_pack(const PackArgs& a, int nranks, hipStream_t s) {
    switch (row_threads(a.cols, kBlockLanes<DT>)) {
        case 16: hipLaunchKernelGGL((k_pack<DT, 16>), grid_of<16>(a.rows, nranks), dim3(256), 0, s, a); break;
        case 64: hipLaunchKernelGGL((k_pack<DT, 64>), grid_of<64>(a.rows, nranks), dim3(256), 0, s, a); break;
        case 128: hipLaunchKernelGGL((k_pack<DT, 128>), grid_of<128>(a.rows, nranks), dim3(256), 0, s, a); break;
        default: hipLaunchKernelGGL((k_pack<DT, 256>), grid_of<256>(a.rows, nranks), dim3(256), 0, s, a); break;
    }
    return hipGetLastError();
}

template <int DT>
hipError_t start_unpack(const UnpackArgs& a, int nranks, hipStream_t s) {
    const dim3 block(256);
    switch (row_threads(a.cols, kBlockLanes<DT>)) {
        case 16: hipLaunchKernelGGL((k_unpack_activations<DT, 16>), grid_of<16>(a.rows, nranks), block, 0, s, a); break;
        case 64: hipLaunchKernelGGL((k_unpack_activations<DT, 64>), grid_of<64>(a.rows, nranks), block, 0, s, a); break;
        case 128: hipLaunchKernelGGL((k_unpack_activations<DT, 128>), grid_of<128>(a.rows, nranks), block, 0, s, a); break;
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
