// Layer norm's backward pass from the forward pass's input as it was
// (ar_layer_norm_backward_device.h has the kernels).

#include "ar_layer_norm_backward_device.h"

namespace arimpl {

hipError_t launch_norm_backward(const NormBackwardArgs& a, int nranks, bool weights, ar_dtype_t dtype,
                                ar_dtype_t weight, hipStream_t s) {
    return launch_backward<kAsItWas>(a, nranks, weights, dtype, weight, s);
}

}  // namespace arimpl
