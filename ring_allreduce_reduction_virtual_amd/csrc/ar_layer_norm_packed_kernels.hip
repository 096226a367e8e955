// Layer norm's backward pass from the forward pass's input kept in 8 bits
// (ar_layer_norm_backward_device.h has the kernels).  HBM bounds it: 8 x 4,096
// rows of 4,096, dy and dx in bf16, 128 us for 407 MB read and 285 written (5.4
// TB/s); from bf16 activations 150.

#include "ar_layer_norm_backward_device.h"

namespace arimpl {

hipError_t launch_norm_backward_packed(const NormBackwardArgs& a, int nranks, bool weights, ar_dtype_t dtype,
                                       ar_dtype_t weight, hipStream_t s) {
    // whole vectors: 16 bytes of dy and dx
    return a.cols % (dtype == AR_FLOAT32 ? 4 : 8) == 0
               ? launch_backward<kPackedWhole>(a, nranks, weights, dtype, weight, s)
               : launch_backward<kPackedAny>(a, nranks, weights, dtype, weight, s);
}

}  // namespace arimpl
