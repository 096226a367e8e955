// HIP kernels of the training step around the gradient reduction: the global
// gradient norm, the AdamW step over many tensors (states in float32, or in 8
// bits), and the packed states' values.  include/ar.h states the formulas.
//
// All of them stream their tensors once, and HBM's rate on the bytes that the
// formulas name bounds them once there are a few million elements; below, the
// launch does.  One launch covers many tensors: a tile is a stretch of one
// tensor, and a workgroup finds the tensor of its tile in a table (in the
// arguments, or in device memory for a plan).  The times in the comments are
// kernel times on MI355X.

#include "ar_step.h"
#include "ar_step_device.h"

namespace arimpl {
namespace {

template <class Entry>
__device__ __forceinline__ const Entry& find(const InlineTable<Entry>& t, uint32_t tile) {
    int lo = 0, hi = t.n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (t.e[mid].first_tile <= tile) {
            lo = mid;
        } else {
            hi = mid;
        }
    }
    return t.e[lo];
}
template <class Entry>
__device__ __forceinline__ const Entry& find(const DeviceTable<Entry>& t, uint32_t tile) {
    return t.e[__builtin_amdgcn_readfirstlane(t.tile_entry[tile])];
}

// ---------------------------------------------------------------------------
// gradient norm
// ---------------------------------------------------------------------------

// The sum of a value over the block, valid in thread 0.
__device__ __forceinline__ double block_sum(double x) {
    __shared__ double part[kStepThreads / 64];
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) x += __shfl_down(x, d, 64);
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = x;
    __syncthreads();
    double s = 0;
    if (threadIdx.x == 0) {
        for (int w = 0; w < kStepThreads / 64; ++w) s += part[w];
    }
    return s;
}

// Sum of squares in float64: the square of a float32 is exact there and can
// neither overflow nor vanish, and the float64 units keep up with HBM.
// Workgroup b takes tiles b, b + gridDim.x, ... and leaves one partial sum, or
// the norm itself when it is the only one.  2^27 float32 in 8 tensors: 79 us
// (6.8 TB/s, reads only), and 4.8 us for the sum of the partial sums; 9.7 million
// bf16 in 97 tensors back to back 6.9 and 2.1 us.
//
// With a counter (of a plan's workspace, 0 between calls) the workgroup that
// finishes last adds the partial sums, in their order, and no second launch
// follows: 4.7 us against 6.7 for 3 workgroups, 5.1 against 6.6 for 70.  Each
// workgroup has to write its XCD's cache back before it counts itself: 256 took
// 9.2 us against 6.7, and 1,024 took 25-45 us more than the second launch.
template <int DT, class Table>
__global__ void __launch_bounds__(kStepThreads) k_grad_norm(Table t, uint32_t tiles, double* partials, float* norm,
                                                            uint32_t* counter) {
    constexpr int V = 16 / elem_size<DT>();
    constexpr int U = kNormTile / (kStepThreads * V);
    double acc[4] = {0, 0, 0, 0};
    for (uint32_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
        const auto& e = find(t, tile);
        const char* const g = e.g;
        const uint64_t n = e.n;
        const uint64_t at = static_cast<uint64_t>(tile - e.first_tile) * kNormTile + threadIdx.x * V;
        Raw<DT, V> r[U];
        if (at - threadIdx.x * V + kNormTile <= n) {
#pragma unroll
            for (int u = 0; u < U; ++u) load_at<true, true>(r[u], g, at + u * kStepThreads * V, n);
        } else {
#pragma unroll
            for (int u = 0; u < U; ++u) load_at<false, false>(r[u], g, at + u * kStepThreads * V, n);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const double x = r[u].get(j);
                acc[j % 4] = __builtin_fma(x, x, acc[j % 4]);
            }
        }
    }
    const double s = block_sum((acc[0] + acc[1]) + (acc[2] + acc[3]));
    if (gridDim.x == 1 && norm != nullptr) {
        if (threadIdx.x == 0) *norm = static_cast<float>(sqrt(s));
        return;
    }
    if (threadIdx.x == 0) partials[blockIdx.x] = s;
    if (counter == nullptr) return;
    __shared__ bool last;
    if (threadIdx.x == 0) {
        // releases this partial sum, and acquires the others' when it is the last
        last = __hip_atomic_fetch_add(counter, 1u, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) == gridDim.x - 1;
    }
    __syncthreads();
    if (!last) return;
    const double all = block_sum(threadIdx.x < gridDim.x ? partials[threadIdx.x] : 0.0);
    if (threadIdx.x == 0) {
        *norm = static_cast<float>(sqrt(all));
        *counter = 0;
    }
}
static_assert(kNormJoinBlocks <= kStepThreads, "one thread per partial sum");

__global__ void __launch_bounds__(kStepThreads) k_grad_norm_final(const double* partials, uint32_t n, float* norm) {
    double acc = 0;
    for (uint32_t i = threadIdx.x; i < n; i += kStepThreads) acc += partials[i];
    const double s = block_sum(acc);
    if (threadIdx.x == 0) *norm = static_cast<float>(sqrt(s));
}

// ---------------------------------------------------------------------------
// AdamW
// ---------------------------------------------------------------------------

// Four streams in, three or four out, about 40 instructions an element (the root
// and the quotient rounded correctly): HBM bounds it.  2^27 float32 elements
// 636 us, 5.9 TB/s on 28 bytes an element, as fast as plain streams of the same
// mix (6.1); 25 million elements of 149 tensors back to back, with bf16
// gradients and copies, 132 us, 5.3 TB/s: tensors that start anywhere share
// cache lines with their neighbours.

// The gradient's factor, and whether the step is skipped.
struct Gate {
    float factor;
    bool skip;
};
__device__ __forceinline__ Gate gate(const AdamwScalars& s) {
    Gate r{s.grad_scale, false};
    if (s.grad_norm != nullptr) {
        const float norm = *s.grad_norm;
        r.skip = s.skip_nonfinite != 0 && (as_u(norm) & 0x7f800000u) == 0x7f800000u;
        if (s.max_norm > 0.0f) {
            // a NaN norm makes the factor NaN, as min() in the formula does not
            const float f = s.max_norm / (norm * s.grad_scale + 1e-6f);
            r.factor = s.grad_scale * (f > 1.0f ? 1.0f : f);
        }
    }
    return r;
}

// One element: the new states and parameter from the old ones.
__device__ __forceinline__ void adamw_update(const AdamwScalars& s, float factor, float g, float& p, float& m,
                                             float& v) {
    const float gs = factor * g;
    m = m * s.beta1 + gs * s.one_minus_beta1;
    v = v * s.beta2 + (gs * gs) * s.one_minus_beta2;
    const float d = sqrtf(v) * s.rsqrt_correction2 + s.eps;
    p = p * s.decay - (m / d) * s.step_size;
}

// V new parameters rounded to the copies' type.
template <bool FULL, int V>
__device__ __forceinline__ void store_copy(char* copy, const AdamwScalars& s, uint64_t at, uint64_t n,
                                           const float (&p)[V]) {
    if (s.copy_f16) {
        Raw<AR_FLOAT16, V> c;
        c.set_all(p);
        store_at<FULL, true>(c, copy, at, n);
    } else {
        Raw<AR_BFLOAT16, V> c;
        c.set_all(p);
        store_at<FULL, true>(c, copy, at, n);
    }
}

template <int PD, int GD, bool LARGE, bool FULL>
__device__ __forceinline__ void adamw_tile(const AdamwEntry& e, const AdamwScalars& s, uint64_t at, uint64_t n) {
    constexpr int V = 4;
    constexpr int U = adamw_vectors(LARGE, PD == AR_FLOAT32 && GD == AR_FLOAT32);
    constexpr int kStep = kStepThreads * V;
    Raw<PD, V> p[U];
    Raw<GD, V> g[U];
    Raw<AR_FLOAT32, V> m[U], v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        load_at<FULL, LARGE>(g[u], e.g, at + u * kStep, n);
        load_at<FULL, LARGE>(p[u], e.p, at + u * kStep, n);
        load_at<FULL, LARGE>(m[u], e.m, at + u * kStep, n);
        load_at<FULL, LARGE>(v[u], e.v, at + u * kStep, n);
    }
    const Gate gt = gate(s);
#pragma unroll
    for (int u = 0; u < U; ++u) {
        float pn[V], mn[V], vn[V];
#pragma unroll
        for (int j = 0; j < V; ++j) {
            pn[j] = p[u].get(j);
            mn[j] = m[u].get(j);
            vn[j] = v[u].get(j);
        }
        if (!gt.skip) {
#pragma unroll
            for (int j = 0; j < V; ++j) adamw_update(s, gt.factor, g[u].get(j), pn[j], mn[j], vn[j]);
        }
        p[u].set_all(pn);
        m[u].set_all(mn);
        v[u].set_all(vn);
        store_at<FULL, true>(p[u], e.p_out, at + u * kStep, n);
        store_at<FULL, true>(m[u], e.m_out, at + u * kStep, n);
        store_at<FULL, true>(v[u], e.v_out, at + u * kStep, n);
        if (PD == AR_FLOAT32 && e.copy != nullptr) store_copy<FULL>(e.copy, s, at + u * kStep, n, pn);
    }
}

template <int PD, int GD, bool LARGE, class Table>
__global__ void __launch_bounds__(kStepThreads) k_adamw(Table t, AdamwScalars s) {
    constexpr uint32_t kTile = kAdamwTile * adamw_vectors(LARGE, PD == AR_FLOAT32 && GD == AR_FLOAT32);
    const AdamwEntry e = find(t, blockIdx.x);
    const uint64_t tile = static_cast<uint64_t>(blockIdx.x - e.first_tile) * kTile;
    if (tile + kTile <= e.n) {
        adamw_tile<PD, GD, LARGE, true>(e, s, tile + threadIdx.x * 4, e.n);
    } else {
        adamw_tile<PD, GD, LARGE, false>(e, s, tile + threadIdx.x * 4, e.n);
    }
}

// ---------------------------------------------------------------------------
// AdamW, states in 8 bits
// ---------------------------------------------------------------------------

// 8 codes at p, whole or up to the tensor's end.
template <bool FULL, bool NT>
__device__ __forceinline__ u32x2 load_codes(const uint8_t* base, uint64_t i, uint64_t n) {
    if (FULL || i + 8 <= n) return load_as<NT, u32x2_a1>(reinterpret_cast<const char*>(base + i));
    u32x2 r = {0, 0};
    for (int j = 0; j < 8; ++j) {
        if (i + j < n) r[j / 4] |= static_cast<uint32_t>(base[i + j]) << (8 * (j % 4));
    }
    return r;
}
template <bool FULL>
__device__ __forceinline__ void store_codes(uint8_t* base, uint64_t i, uint64_t n, u32x2 c) {
    if (FULL || i + 8 <= n) {
        store_as<true, u32x2_a1>(reinterpret_cast<char*>(base + i), c);
        return;
    }
    for (int j = 0; j < 8; ++j) {
        if (i + j < n) base[i + j] = static_cast<uint8_t>(c[j / 4] >> (8 * (j % 4)));
    }
}

// A thread's 8 parameters and codes, and a block's scale bytes.
template <bool FULL, int PD>
__device__ __forceinline__ void store_packed(const PackedEntry& e, uint64_t at, uint64_t n, const Raw<PD, 8>& p,
                                             u32x2 m, u32x2 v, uint32_t mscale, uint32_t vscale) {
    store_at<FULL, true>(p, e.p_out, at, n);
    store_codes<FULL>(e.m_out, at, n, m);
    store_codes<FULL>(e.v_out, at, n, v);
    if (threadIdx.x % 32 == 0 && (FULL || at < n)) {
        e.ms_out[at / AR_STATE_BLOCK] = static_cast<uint8_t>(mscale);
        e.vs_out[at / AR_STATE_BLOCK] = static_cast<uint8_t>(vscale);
    }
}

// One element of the packed step.  The states that are kept are the formula's
// bit for bit, and so are float32 parameters (EXACT).  The quotient of 16-bit
// parameters takes the hardware's root and reciprocal (within 1.6 half-ulps
// each, measured): their own rounding is 2^13 times coarser or more, and rounding
// the quotient correctly as well takes 2^27 bf16 elements from 226 us to 272.
// (What it costs float32 parameters: 2^26 elements 187 us against 185, with bf16
// gradients 173 against 166, 12 tensors of 87,382 8.1 against 7.7.)  The root
// takes a subnormal for 0, which only a tiny eps leaves visible: EXACT there too.
template <bool EXACT>
__device__ __forceinline__ void packed_update(const AdamwScalars& s, float correction2, float factor, float g, float& p,
                                              float& m, float& v) {
    const float gs = factor * g;
    m = m * s.beta1 + gs * s.one_minus_beta1;
    v = v * s.beta2 + (gs * gs) * s.one_minus_beta2;
    if constexpr (EXACT) {
        const float d = sqrtf(v) * correction2 + s.eps;
        p = p * s.decay - (m / d) * s.step_size;
    } else {
        const float d = __builtin_amdgcn_sqrtf(v) * correction2 + s.eps;
        p = p * s.decay - (m * __builtin_amdgcn_rcpf(d)) * s.step_size;
    }
}

// A thread has 8 neighbouring elements, half a wavefront a state block of 256:
// the block's largest magnitude is a maximum over 32 lanes, with no LDS.  About
// 60 instructions an element, of which a quarter is the hash, against 10 bytes
// (bf16): both HBM and the vector units are near their limit.  2^27 bf16
// elements 224-235 us, 5.8 TB/s; with the codes taken apart by multiplications
// and the quotient rounded correctly, 100 instructions, it took 304.
template <int PD, int GD, bool LARGE, bool EXACT, bool FULL>
__device__ __forceinline__ void packed_tile(const PackedEntry& e, const AdamwScalars& s, uint64_t at, uint64_t n) {
    constexpr int V = 8;
    const uint64_t block = at / AR_STATE_BLOCK;
    const bool live = FULL || block * AR_STATE_BLOCK < n;
    Raw<PD, V> p;
    Raw<GD, V> g;
    load_at<FULL, LARGE>(g, e.g, at, n);
    load_at<FULL, LARGE>(p, e.p, at, n);
    const u32x2 mc = load_codes<FULL, LARGE>(e.m, at, n), vc = load_codes<FULL, LARGE>(e.v, at, n);
    const uint32_t me = live ? e.ms[block] : 0, ve = live ? e.vs[block] : 0;
    const Gate gt = gate(s);
    if (gt.skip) {
        if (PD == AR_FLOAT32 && e.copy != nullptr) {
            float same[V];
#pragma unroll
            for (int j = 0; j < V; ++j) same[j] = p.get(j);
            store_copy<FULL>(e.copy, s, at, n, same);
        }
        store_packed<FULL>(e, at, n, p, mc, vc, me, ve);
        return;
    }
    // a block of NaN stays one, and takes its parameters along
    const bool mbad = me == 255, vbad = ve == 255;
    const float correction2 = mbad || vbad ? as_f(0x7fc00000u) : s.rsqrt_correction2;
    float pn[V], mn[V], vn[V];
    float mtop = 0;
    uint32_t vtop = 0;
#pragma unroll
    for (int j = 0; j < V; ++j) {
        pn[j] = p.get(j);
        mn[j] = decode<true>(mc[j / 4], j % 4, me);
        vn[j] = decode<false>(vc[j / 4], j % 4, ve);
        packed_update<EXACT>(s, correction2, gt.factor, g.get(j), pn[j], mn[j], vn[j]);
        // beyond the end there is nothing
        if (!FULL && at + j >= n) mn[j] = vn[j] = 0.0f;
        mtop = __builtin_fmaxf(mtop, __builtin_fabsf(mn[j]));
        vtop = as_u(vn[j]) > vtop ? as_u(vn[j]) : vtop;   // v is never negative
    }
    // The maximum of m passes over NaN.  One comes only with the gradient's, and
    // that makes v, whose bits compare as integers, a NaN too, of the gradient's
    // sign: no magnitude that scale_for could take.
    vtop = max_over_lanes<32>(vtop);
    const bool nan = vtop > 0x7f800000u;
    const uint32_t me_new = mbad || nan ? 255 : scale_for(max_over_lanes<32>(as_u(mtop)));
    const uint32_t ve_new = vbad || nan ? 255 : scale_for(vtop);
    const uint32_t key = mix32(s.seed + 0x9e3779b9u * (e.index + 1)) + 0x9e3779b9u * static_cast<uint32_t>(at);
    uint32_t mo[V], vo[V], least = 0xffffffffu;
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const uint32_t r = mix32(key + 0x9e3779b9u * j);
        mo[j] = encode<true>(mn[j], me_new, (r << 4) & 0xffff0u);
        vo[j] = encode<false>(vn[j], ve_new, (r >> 12) & 0xffff0u);
        least = vo[j] < least ? vo[j] : least;
    }
    // a positive second moment is never rounded to 0: rare, so looked for first
    if (__builtin_expect(__ballot(least < (1u << 24)) != 0, 0)) {
#pragma unroll
        for (int j = 0; j < V; ++j) {
            if (vo[j] < (1u << 24) && vn[j] > 0.0f) vo[j] = 1u << 24;
        }
    }
    u32x2 mw = {top_bytes(mo[0], mo[1], mo[2], mo[3]), top_bytes(mo[4], mo[5], mo[6], mo[7])};
    u32x2 vw = {top_bytes(vo[0], vo[1], vo[2], vo[3]), top_bytes(vo[4], vo[5], vo[6], vo[7])};
    if (me_new == 255) mw = u32x2{0, 0};
    if (ve_new == 255) vw = u32x2{0, 0};
    p.set_all(pn);
    if (PD == AR_FLOAT32 && e.copy != nullptr) store_copy<FULL>(e.copy, s, at, n, pn);
    store_packed<FULL>(e, at, n, p, mw, vw, me_new, ve_new);
}

template <int PD, int GD, bool LARGE, bool EXACT, class Table>
__global__ void __launch_bounds__(kStepThreads) k_adamw_packed(Table t, AdamwScalars s) {
    constexpr uint32_t kTile = kPackedTile * packed_vectors(LARGE);
    const PackedEntry e = find(t, blockIdx.x);
    const uint64_t tile = static_cast<uint64_t>(blockIdx.x - e.first_tile) * kTile;
    const bool full = tile + kTile <= e.n;
#pragma unroll
    for (uint32_t u = 0; u < kTile; u += kPackedTile) {
        if (full) {
            packed_tile<PD, GD, LARGE, EXACT, true>(e, s, tile + u + threadIdx.x * 8, e.n);
        } else {
            packed_tile<PD, GD, LARGE, EXACT, false>(e, s, tile + u + threadIdx.x * 8, e.n);
        }
    }
}

// One byte in, an element out.  2^27 elements to bf16: 80 us, 5.1 TB/s.
template <int DT, bool SIGNED>
__global__ void __launch_bounds__(kStepThreads) k_unpack(InlineTable<UnpackEntry> t) {
    static_assert(kUnpackTile == kStepThreads * 8, "one vector per thread");
    const UnpackEntry& e = find(t, blockIdx.x);
    const uint64_t at = static_cast<uint64_t>(blockIdx.x - e.first_tile) * kUnpackTile + threadIdx.x * 8;
    if (at >= e.n) return;
    const u32x2 c = load_codes<false, true>(e.codes, at, e.n);
    const uint32_t scale = e.scales[at / AR_STATE_BLOCK];
    float x[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        x[j] = decode<SIGNED>(c[j / 4], j % 4, scale);
        if (scale == 255) x[j] = as_f(0x7fc00000u);
    }
    Raw<DT, 8> r;
    r.set_all(x);
    store_at<false, true>(r, e.out, at, e.n);
}

}  // namespace

// ---------------------------------------------------------------------------
// launches
// ---------------------------------------------------------------------------

template <class Table>
hipError_t launch_norm(const Table& t, uint32_t tiles, uint32_t blocks, ar_dtype_t dtype, double* partials,
                       float* norm, uint32_t* counter, hipStream_t stream) {
    const dim3 grid(blocks), block(kStepThreads);
    switch (dtype) {
        case AR_FLOAT32:
            hipLaunchKernelGGL((k_grad_norm<AR_FLOAT32, Table>), grid, block, 0, stream, t, tiles, partials, norm,
                               counter);
            break;
        case AR_BFLOAT16:
            hipLaunchKernelGGL((k_grad_norm<AR_BFLOAT16, Table>), grid, block, 0, stream, t, tiles, partials, norm,
                               counter);
            break;
        case AR_FLOAT16:
            hipLaunchKernelGGL((k_grad_norm<AR_FLOAT16, Table>), grid, block, 0, stream, t, tiles, partials, norm,
                               counter);
            break;
        default: return hipErrorInvalidValue;
    }
    return hipGetLastError();
}

hipError_t launch_norm_final(const double* partials, uint32_t n, float* norm, hipStream_t stream) {
    hipLaunchKernelGGL(k_grad_norm_final, dim3(1), dim3(kStepThreads), 0, stream, partials, n, norm);
    return hipGetLastError();
}

namespace {

template <int PD, int GD, class Table>
void adamw_by_form(const Table& t, uint32_t tiles, const AdamwScalars& s, bool large, hipStream_t stream) {
    const dim3 grid(tiles), block(kStepThreads);
    if (large) {
        hipLaunchKernelGGL((k_adamw<PD, GD, true, Table>), grid, block, 0, stream, t, s);
    } else {
        hipLaunchKernelGGL((k_adamw<PD, GD, false, Table>), grid, block, 0, stream, t, s);
    }
}

template <int PD, class Table>
hipError_t adamw_by_grad(const Table& t, uint32_t tiles, const AdamwScalars& s, const StepForm& f, hipStream_t stream) {
    switch (f.grad) {
        case AR_FLOAT32: adamw_by_form<PD, AR_FLOAT32>(t, tiles, s, f.large, stream); break;
        case AR_BFLOAT16: adamw_by_form<PD, AR_BFLOAT16>(t, tiles, s, f.large, stream); break;
        case AR_FLOAT16: adamw_by_form<PD, AR_FLOAT16>(t, tiles, s, f.large, stream); break;
        default: return hipErrorInvalidValue;
    }
    return hipGetLastError();
}

template <int PD, int GD, bool LARGE, class Table>
void packed_by_root(const Table& t, uint32_t tiles, const AdamwScalars& s, hipStream_t stream) {
    const dim3 grid(tiles), block(kStepThreads);
    if constexpr (PD != AR_FLOAT32) {
        // The hardware's root takes v below 2^-126 for 0, which moves the denominator
        // by up to 2^-63 times the correction: at most half an ulp of this eps.
        if (s.eps >= 0x1p-38f * s.rsqrt_correction2) {
            hipLaunchKernelGGL((k_adamw_packed<PD, GD, LARGE, false, Table>), grid, block, 0, stream, t, s);
            return;
        }
    }
    hipLaunchKernelGGL((k_adamw_packed<PD, GD, LARGE, true, Table>), grid, block, 0, stream, t, s);
}

template <int PD, int GD, class Table>
void packed_by_form(const Table& t, uint32_t tiles, const AdamwScalars& s, bool large, hipStream_t stream) {
    if constexpr (elem_size<PD>() == 2 && elem_size<GD>() == 2) {
        if (large) {
            packed_by_root<PD, GD, true>(t, tiles, s, stream);
            return;
        }
    }
    packed_by_root<PD, GD, false>(t, tiles, s, stream);
}

template <int PD, class Table>
hipError_t packed_by_grad(const Table& t, uint32_t tiles, const AdamwScalars& s, const StepForm& f,
                          hipStream_t stream) {
    switch (f.grad) {
        case AR_FLOAT32: packed_by_form<PD, AR_FLOAT32>(t, tiles, s, f.large, stream); break;
        case AR_BFLOAT16: packed_by_form<PD, AR_BFLOAT16>(t, tiles, s, f.large, stream); break;
        case AR_FLOAT16: packed_by_form<PD, AR_FLOAT16>(t, tiles, s, f.large, stream); break;
        default: return hipErrorInvalidValue;
    }
    return hipGetLastError();
}

template <int DT>
hipError_t unpack_by_state(const InlineTable<UnpackEntry>& t, uint32_t tiles, ar_state_t state, hipStream_t stream) {
    const dim3 grid(tiles), block(kStepThreads);
    if (state == AR_STATE_EXP_AVG) {
        hipLaunchKernelGGL((k_unpack<DT, true>), grid, block, 0, stream, t);
    } else {
        hipLaunchKernelGGL((k_unpack<DT, false>), grid, block, 0, stream, t);
    }
    return hipGetLastError();
}

}  // namespace

template <class Table>
hipError_t launch_adamw(const Table& t, uint32_t tiles, const AdamwScalars& s, const StepForm& f, hipStream_t stream) {
    switch (f.param) {
        case AR_FLOAT32: return adamw_by_grad<AR_FLOAT32>(t, tiles, s, f, stream);
        case AR_BFLOAT16: return adamw_by_grad<AR_BFLOAT16>(t, tiles, s, f, stream);
        case AR_FLOAT16: return adamw_by_grad<AR_FLOAT16>(t, tiles, s, f, stream);
        default: return hipErrorInvalidValue;
    }
}

template <class Table>
hipError_t launch_packed(const Table& t, uint32_t tiles, const AdamwScalars& s, const StepForm& f, hipStream_t stream) {
    switch (f.param) {
        case AR_FLOAT32: return packed_by_grad<AR_FLOAT32>(t, tiles, s, f, stream);
        case AR_BFLOAT16: return packed_by_grad<AR_BFLOAT16>(t, tiles, s, f, stream);
        case AR_FLOAT16: return packed_by_grad<AR_FLOAT16>(t, tiles, s, f, stream);
        default: return hipErrorInvalidValue;
    }
}

hipError_t launch_unpack(const InlineTable<UnpackEntry>& t, uint32_t tiles, ar_state_t state, ar_dtype_t dtype,
                         hipStream_t stream) {
    switch (dtype) {
        case AR_FLOAT32: return unpack_by_state<AR_FLOAT32>(t, tiles, state, stream);
        case AR_BFLOAT16: return unpack_by_state<AR_BFLOAT16>(t, tiles, state, stream);
        case AR_FLOAT16: return unpack_by_state<AR_FLOAT16>(t, tiles, state, stream);
        default: return hipErrorInvalidValue;
    }
}

template hipError_t launch_norm(const InlineTable<NormEntry>&, uint32_t, uint32_t, ar_dtype_t, double*, float*,
                                uint32_t*, hipStream_t);
template hipError_t launch_norm(const DeviceTable<NormEntry>&, uint32_t, uint32_t, ar_dtype_t, double*, float*,
                                uint32_t*, hipStream_t);
template hipError_t launch_adamw(const InlineTable<AdamwEntry>&, uint32_t, const AdamwScalars&, const StepForm&,
                                 hipStream_t);
template hipError_t launch_adamw(const DeviceTable<AdamwEntry>&, uint32_t, const AdamwScalars&, const StepForm&,
                                 hipStream_t);
template hipError_t launch_packed(const InlineTable<PackedEntry>&, uint32_t, const AdamwScalars&, const StepForm&,
                                  hipStream_t);
template hipError_t launch_packed(const DeviceTable<PackedEntry>&, uint32_t, const AdamwScalars&, const StepForm&,
                                  hipStream_t);

}  // namespace arimpl
