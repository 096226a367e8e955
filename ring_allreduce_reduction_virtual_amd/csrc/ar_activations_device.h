// Device-side building blocks of activations in 8 bits (include/ar.h states
// the format).  Inline device code in an unnamed namespace, so each kernel
// source gets its own copy.
#pragma once

#include "ar_step_device.h"

namespace arimpl {
namespace {

// A scale byte e is worth 2^(e - kActivationShift).
constexpr int kActivationShift = 133;

// The scale byte of a block whose largest magnitude has these bits, NaN and
// infinity among them (255): adding just under the distance from 127/64 to 2
// carries into the exponent when the mantissa is above 127/64.
__device__ __forceinline__ uint32_t activation_scale(uint32_t top_bits) {
    const uint32_t e = (top_bits + 0x0001ffffu) >> 23;
    return e == 0 ? 1 : (e > 255 ? 255 : e);
}

// x (at most 127 scales) as a code: scaled exactly, then rounded to the nearest
// integer, ties to even.
__device__ __forceinline__ uint32_t activation_code(float x, uint32_t e) {
    const float y = __builtin_rintf(__builtin_amdgcn_ldexpf(x, kActivationShift - static_cast<int>(e)));
    return static_cast<uint32_t>(static_cast<int>(y)) & 0xffu;
}

// What a scale byte is worth, NaN for 255 and 1's worth for 0: subnormal for
// the smallest scales, which float32's arithmetic keeps.
__device__ __forceinline__ float activation_scale_value(uint32_t e) {
    const float s = __builtin_amdgcn_ldexpf(1.0f, static_cast<int>(e == 0 ? 1 : e) - kActivationShift);
    return e == 255 ? as_f(0x7fc00000u) : s;
}

// Code j of four in a word; the product is exact in float32 for every scale.
__device__ __forceinline__ float activation_value(uint32_t word, int j, float scale) {
    return static_cast<float>(static_cast<int>(word << (24 - 8 * j)) >> 24) * scale;
}

}  // namespace
}  // namespace arimpl
