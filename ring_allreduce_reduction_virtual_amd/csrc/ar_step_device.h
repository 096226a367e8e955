// Device-side building blocks of the training-step kernels: vectors of
// elements moved between memory and float32 registers at any element
// alignment, sums over lanes, and the packed states' codes.  Inline device
// code in an unnamed namespace, so each kernel source gets its own copy.
#pragma once

#include "ar_device.h"

namespace arimpl {
namespace {

// Vector types with the element's alignment: a global load or store of 4, 8
// or 16 bytes needs no more on gfx950, so tensors that start anywhere (slices
// of a bucket, rows of odd width) take the same path as aligned ones.
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef u32x4 u32x4_a2 __attribute__((aligned(2)));
typedef u32x2 u32x2_a2 __attribute__((aligned(2)));
typedef u32x4 u32x4_a4 __attribute__((aligned(4)));
typedef u32x2 u32x2_a1 __attribute__((aligned(1)));

template <bool NT, class T>
__device__ __forceinline__ auto load_as(const char* p) {
    const T* q = reinterpret_cast<const T*>(p);
    if constexpr (NT) {
        return __builtin_nontemporal_load(q);
    } else {
        return *q;
    }
}
template <bool NT, class T, class U>
__device__ __forceinline__ void store_as(char* p, U v) {
    T* q = reinterpret_cast<T*>(p);
    if constexpr (NT) {
        __builtin_nontemporal_store(v, q);
    } else {
        *q = v;
    }
}

template <int DT>
__device__ __forceinline__ float widen(uint32_t h) {
    if constexpr (DT == AR_FLOAT32) {
        return as_f(h);
    } else if constexpr (DT == AR_FLOAT16) {
        return f16_widen(h & 0xffffu);
    } else {
        return bf16_widen(h & 0xffffu);
    }
}
template <int DT>
__device__ __forceinline__ uint32_t narrow(float x) {
    if constexpr (DT == AR_FLOAT32) {
        return as_u(x);
    } else if constexpr (DT == AR_FLOAT16) {
        return f16_round(x);
    } else {
        return bf16_round(x);
    }
}
template <int DT>
__device__ __forceinline__ uint32_t narrow2(float lo, float hi) {
    if constexpr (DT == AR_FLOAT16) {
        return f16_round(lo) | (f16_round(hi) << 16);
    } else {
        return bf16_round2(lo, hi);
    }
}

// V elements at p, 4 or 8 of them, as they are in memory.
template <int DT, int V>
struct Raw {
    static constexpr int kWords = V * elem_size<DT>() / 4;
    uint32_t w[kWords];

    template <bool NT>
    __device__ __forceinline__ void load(const char* p) {
        if constexpr (kWords == 2) {
            const u32x2 v = load_as<NT, u32x2_a2>(p);
            w[0] = v.x;
            w[1] = v.y;
        } else {
            typedef typename std::conditional<elem_size<DT>() == 2, u32x4_a2, u32x4_a4>::type vec;
#pragma unroll
            for (int k = 0; k < kWords; k += 4) {
                const u32x4 v = load_as<NT, vec>(p + 4 * k);
                w[k] = v.x;
                w[k + 1] = v.y;
                w[k + 2] = v.z;
                w[k + 3] = v.w;
            }
        }
    }
    template <bool NT>
    __device__ __forceinline__ void store(char* p) const {
        if constexpr (kWords == 2) {
            const u32x2 v = {w[0], w[1]};
            store_as<NT, u32x2_a2>(p, v);
        } else {
            typedef typename std::conditional<elem_size<DT>() == 2, u32x4_a2, u32x4_a4>::type vec;
#pragma unroll
            for (int k = 0; k < kWords; k += 4) {
                const u32x4 v = {w[k], w[k + 1], w[k + 2], w[k + 3]};
                store_as<NT, vec>(p + 4 * k, v);
            }
        }
    }
    // the first `left` < V elements only; the others read as 0
    __device__ __forceinline__ void load_some(const char* p, int left) {
#pragma unroll
        for (int k = 0; k < kWords; ++k) w[k] = 0;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            if (j < left) {
                const uint32_t h = load_elem<elem_size<DT>()>(p + j * elem_size<DT>());
                if constexpr (elem_size<DT>() == 4) {
                    w[j] = h;
                } else {
                    w[j / 2] |= h << (16 * (j % 2));
                }
            }
        }
    }
    __device__ __forceinline__ void store_some(char* p, int left) const {
#pragma unroll
        for (int j = 0; j < V; ++j) {
            if (j < left) {
                const uint32_t h = elem_size<DT>() == 4 ? w[j * elem_size<DT>() / 4] : w[j / 2] >> (16 * (j % 2));
                store_elem<elem_size<DT>(), false>(p + j * elem_size<DT>(), h);
            }
        }
    }
    // all but the first `skip`
    __device__ __forceinline__ void store_from(char* p, int skip) const {
#pragma unroll
        for (int j = 0; j < V; ++j) {
            if (j >= skip) {
                const uint32_t h = elem_size<DT>() == 4 ? w[j * elem_size<DT>() / 4] : w[j / 2] >> (16 * (j % 2));
                store_elem<elem_size<DT>(), false>(p + j * elem_size<DT>(), h);
            }
        }
    }
    __device__ __forceinline__ float get(int j) const {
        if constexpr (elem_size<DT>() == 4) {
            return as_f(w[j]);
        } else {
            return widen<DT>(w[j / 2] >> (16 * (j % 2)));
        }
    }
    __device__ __forceinline__ void set_all(const float (&x)[V]) {
        if constexpr (elem_size<DT>() == 4) {
#pragma unroll
            for (int j = 0; j < V; ++j) w[j] = as_u(x[j]);
        } else {
#pragma unroll
            for (int j = 0; j < V; j += 2) w[j / 2] = narrow2<DT>(x[j], x[j + 1]);
        }
    }
};

// V elements at element index i of a tensor of n, whole or up to its end.
template <bool FULL, bool NT, int DT, int V>
__device__ __forceinline__ void load_at(Raw<DT, V>& r, const char* base, uint64_t i, uint64_t n) {
    const char* p = base + i * elem_size<DT>();
    if (FULL || i + V <= n) {
        r.template load<NT>(p);
    } else {
        r.load_some(p, i < n ? static_cast<int>(n - i) : 0);
    }
}
template <bool FULL, bool NT, int DT, int V>
__device__ __forceinline__ void store_at(const Raw<DT, V>& r, char* base, uint64_t i, uint64_t n) {
    char* p = base + i * elem_size<DT>();
    if (FULL || i + V <= n) {
        r.template store<NT>(p);
    } else if (i < n) {
        r.store_some(p, static_cast<int>(n - i));
    }
}

// ---------------------------------------------------------------------------
// over lanes
// ---------------------------------------------------------------------------

template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t x) {
    return static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(x), CTRL, 0xf, 0xf, false));
}
constexpr int kDppXor1 = 0xB1, kDppXor2 = 0x4E;             // quad permutations 1,0,3,2 and 2,3,0,1
constexpr int kDppHalfMirror = 0x141, kDppMirror = 0x140;   // lanes of 8 and of 16 reversed
constexpr int kDppRotate8 = 0x128;                          // 16 lanes turned by 8

// The same lane's value in the other 16 (other 32) lanes, given that f combines
// a pair regardless of its order.
template <class F>
__device__ __forceinline__ uint32_t across16(uint32_t x, F f) {
    const auto s = __builtin_amdgcn_permlane16_swap(x, x, false, false);
    return f(s[0], s[1]);
}
template <class F>
__device__ __forceinline__ uint32_t across32(uint32_t x, F f) {
    const auto s = __builtin_amdgcn_permlane32_swap(x, x, false, false);
    return f(s[0], s[1]);
}

// f over each group of LANES (8, 16, 32 or 64) neighbouring lanes, in every lane.
// After two exchanges the four lanes of a quad agree, so a mirrored half row
// brings the other quad's value, and a mirrored row the other half's.
template <int LANES, class F>
__device__ __forceinline__ uint32_t over_lanes(uint32_t x, F f) {
    x = f(x, dpp<kDppXor1>(x));
    x = f(x, dpp<kDppXor2>(x));
    x = f(x, dpp<kDppHalfMirror>(x));
    if constexpr (LANES >= 16) x = f(x, dpp<kDppMirror>(x));
    if constexpr (LANES >= 32) x = across16(x, f);
    if constexpr (LANES >= 64) x = across32(x, f);
    return x;
}

template <int LANES>
__device__ __forceinline__ uint32_t max_over_lanes(uint32_t x) {
    return over_lanes<LANES>(x, [](uint32_t a, uint32_t b) { return a > b ? a : b; });
}
template <int LANES>
__device__ __forceinline__ float sum_over_lanes(float x) {
    return as_f(over_lanes<LANES>(as_u(x), [](uint32_t a, uint32_t b) { return as_u(as_f(a) + as_f(b)); }));
}

// ---------------------------------------------------------------------------
// packed states
// ---------------------------------------------------------------------------

// A code's exponent and mantissa bits, put at bits 20 and up of a float32,
// read as 2^(E-127) (1 + F/8) or, for E = 0, the subnormal F/8 2^-126: one
// exact shift of the exponent (v_ldexp_f32, which keeps subnormals) gives the
// code's value times its scale for every E alike; the same in reverse rounds.
// SIGNED is exp_avg's form (4 exponent bits), else exp_avg_sq's (5).
template <bool SIGNED>
constexpr int kCodeShift = SIGNED ? 15 : 31;

// The scale byte of a block whose largest magnitude, finite or infinite, has
// these bits: adding just under an eighth of the exponent's step carries when
// the mantissa is above 1.875.
__device__ __forceinline__ uint32_t scale_for(uint32_t top_bits) {
    const uint32_t e = (top_bits + 0x000fffffu) >> 23;
    return e == 0 ? 1 : (e > 255 ? 255 : e);
}

// Code j of four in a word, with scale byte `e`.  A block whose scale is 255
// (NaN) is its caller's to mark.
template <bool SIGNED>
__device__ __forceinline__ float decode(uint32_t word, int j, uint32_t e) {
    const int shift = static_cast<int>(e > 0 ? e : 1) - kCodeShift<SIGNED>;
    if constexpr (SIGNED) {
        // to the top byte, then back by four with the sign's copies cut off
        const int top = static_cast<int>(word << (24 - 8 * j)) >> 4;
        return __builtin_amdgcn_ldexpf(as_f(static_cast<uint32_t>(top) & 0x87f00000u), shift);
    } else {
        const uint32_t body = j < 3 ? word << (20 - 8 * j) : word >> 4;
        return __builtin_amdgcn_ldexpf(as_f(body & 0x0ff00000u), shift);
    }
}

// x (at most 1.875 scales) to one of its two neighbours, the code in the
// result's top byte: `noise`, a multiple of 16 below 2^20, plus 8 is added
// below the code's last bit; the bits under the top byte are not the code's.
template <bool SIGNED>
__device__ __forceinline__ uint32_t encode(float x, uint32_t e, uint32_t noise) {
    const int shift = kCodeShift<SIGNED> - static_cast<int>(e);
    const uint32_t y = as_u(__builtin_amdgcn_ldexpf(__builtin_fabsf(x), shift)) + noise + 8;
    if constexpr (SIGNED) return (as_u(x) & 0x80000000u) | ((y << 4) & 0x7fffffffu);
    return y << 4;
}

// The top bytes of four words as one.
__device__ __forceinline__ uint32_t top_bytes(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    const uint32_t lo = __builtin_amdgcn_perm(b, a, 0x0c0c0703u), hi = __builtin_amdgcn_perm(d, c, 0x0c0c0703u);
    return __builtin_amdgcn_perm(hi, lo, 0x05040100u);
}

__device__ __forceinline__ uint32_t mix32(uint32_t x) {
    x ^= x >> 16;
    x *= 0x7feb352du;
    x ^= x >> 15;
    x *= 0x846ca68bu;
    x ^= x >> 16;
    return x;
}

}  // namespace
}  // namespace arimpl
