// Internal interface of the 8-bit activations: what the host entry points
// (ar_activations_api.hip) hand to the kernels (ar_activations_kernels.hip).
// Not installed; include/ar.h is the public ABI.
#pragma once

#include <hip/hip_runtime_api.h>

#include <algorithm>
#include <cstdint>

#include "ar.h"

namespace arimpl {

// Ranks of one launch: their pointers travel in the kernel's arguments.
constexpr int kActivationRanks = 32;

struct PackArgs {
    const char* x[kActivationRanks];
    uint8_t* codes[kActivationRanks];
    uint8_t* scales[kActivationRanks];
    uint64_t rows, cols, x_stride;   // elements
};
struct UnpackArgs {
    const uint8_t* codes[kActivationRanks];
    const uint8_t* scales[kActivationRanks];
    char* x[kActivationRanks];
    uint64_t rows, cols, x_stride;
};

hipError_t launch_pack(const PackArgs& a, int nranks, ar_dtype_t dtype, hipStream_t stream);
hipError_t launch_unpack(const UnpackArgs& a, int nranks, ar_dtype_t dtype, hipStream_t stream);

}  // namespace arimpl
