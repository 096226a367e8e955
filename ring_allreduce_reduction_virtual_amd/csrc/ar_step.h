// Internal interface of the training-step operators (gradient norm, AdamW,
// packed states): what the host entry points (ar_step_api.hip) hand to the
// kernels (ar_step_kernels.hip).  Not installed; include/ar.h is the public
// ABI.
#pragma once

#include <hip/hip_runtime_api.h>

#include <cstdint>

#include "ar.h"

namespace arimpl {

constexpr int kStepThreads = 256;   // threads per block: four 64-wide wavefronts

// Elements per tile (one workgroup's share of one tensor).  The AdamW steps'
// threads take vectors of 4 (packed: 8) elements, one in the small form, two
// or four in the large one.
constexpr uint32_t kNormTile = 8192;
constexpr uint32_t kAdamwTile = kStepThreads * 4;
constexpr uint32_t kPackedTile = kStepThreads * 8;
constexpr uint32_t kUnpackTile = 2048;
static_assert(kPackedTile % AR_STATE_BLOCK == 0 && kUnpackTile % AR_STATE_BLOCK == 0, "whole state blocks per tile");

// The AdamW steps' two forms.  The small one reads with cache-allocating loads
// and a vector per thread: more workgroups, and what the reduction, the norm
// or the last step left in the 256 MB last-level cache is found there.  The
// large one streams past the cache (nontemporal loads), with more vectors per
// thread in flight.
//
// Float32 states: large above kAdamwLargeBytes read and written; two vectors,
// or four when parameters and gradients are both float32.  Measured on MI355X,
// us, small / two / four vectors: float32 29 MB 6.7 / 6.6 / 6.7, 117 MB 19.0 /
// 21.5 / 21.3, 235 MB 43.2 / 41.5 / 41.3, 1.9 GB 346 / 313 / 314, 8 tensors of
// 470 MB 681 / 655 / 631; float32 with bf16 gradients and copies 117 MB 20.7 /
// 25.2 / 26.5, 235 MB 44.3 / 46.8 / 49.1, 1.9 GB 357 / 342 / 358; bf16 92 MB
// 17.1 / 18.6 / 20.6, 184 MB 32.6 / 33.4 / 35.9, 1.5 GB 250 / 234 / 243.
//
// Packed states: two vectors from kPackedLargeElements when parameters and
// gradients both have 16 bits; 32-bit ones fill a thread's loads with one.  us,
// small / two vectors: bf16 2^22 elements 12.7 / 15.4, 2^23 18.9 / 19.5, 2^24
// 37.2 / 35.5, 2^27 247 / 227; 2^26 float32 192 / 207, float32 with bf16
// gradients 179 / 177, with copies too 192 / 203.
constexpr uint64_t kAdamwLargeBytes = 128ull << 20;
constexpr uint64_t kPackedLargeElements = 1ull << 24;
constexpr int adamw_vectors(bool large, bool all_f32) { return large ? (all_f32 ? 4 : 2) : 1; }
constexpr int packed_vectors(bool large) { return large ? 2 : 1; }

// Most partial sums one launch of the gradient norm leaves (its workgroups).
constexpr uint32_t kNormBlocks = 1024;
// Up to this many, a plan's last workgroup adds them itself.
constexpr uint32_t kNormJoinBlocks = 128;

// One tensor's line in a table.  first_tile counts the tiles of the lines
// before it in the same table; index is the tensor's number in the call.
struct NormEntry {
    const char* g;
    uint64_t n;
    uint32_t first_tile;
    uint32_t index;
};

struct AdamwEntry {
    const char* p;
    const char* g;
    const char* m;
    const char* v;
    char* p_out;
    char* m_out;
    char* v_out;
    char* copy;
    uint64_t n;
    uint32_t first_tile;
    uint32_t index;
};

struct PackedEntry {
    const char* p;
    const char* g;
    const uint8_t* m;
    const uint8_t* v;
    const uint8_t* ms;
    const uint8_t* vs;
    char* p_out;
    uint8_t* m_out;
    uint8_t* v_out;
    uint8_t* ms_out;
    uint8_t* vs_out;
    char* copy;
    uint64_t n;
    uint32_t first_tile;
    uint32_t index;
};

struct UnpackEntry {
    const uint8_t* codes;
    const uint8_t* scales;
    char* out;
    uint64_t n;
    uint32_t first_tile;
    uint32_t index;
};

// A table that travels in the kernel's arguments (one-shot calls): as many
// lines as stay, with the other arguments, under 4 KiB.  A workgroup finds its
// line by bisection over first_tile.
template <class Entry>
struct InlineTable {
    static constexpr int kMax = static_cast<int>((4096 - 256) / sizeof(Entry));
    Entry e[kMax];
    int n;
};

// A table in device memory (plans): any number of lines, and each tile's line
// number, so that a workgroup finds its line with one load.
template <class Entry>
struct DeviceTable {
    const Entry* e;
    const uint32_t* tile_entry;
};

// An AdamW step's scalars, rounded once on the host.
struct AdamwScalars {
    const float* grad_norm;   // device memory, or null
    float beta1, one_minus_beta1;
    float beta2, one_minus_beta2;
    float eps;
    float decay;              // 1 - lr * weight_decay
    float step_size;          // lr / (1 - beta1^t)
    float rsqrt_correction2;  // 1 / sqrt(1 - beta2^t)
    float max_norm;           // 0: no clipping
    float grad_scale;
    int skip_nonfinite;
    uint32_t seed;
    int copy_f16;             // copies are binary16, else bf16
};

// Each enqueues one kernel over `tiles` tiles of the table; dtypes were
// validated by the caller.
template <class Table>
hipError_t launch_norm(const Table& t, uint32_t tiles, uint32_t blocks, ar_dtype_t dtype, double* partials,
                       float* norm, uint32_t* counter, hipStream_t stream);
// What the steps' kernels are chosen by.
struct StepForm {
    ar_dtype_t param, grad;
    bool large;
};
template <class Table>
hipError_t launch_adamw(const Table& t, uint32_t tiles, const AdamwScalars& s, const StepForm& f, hipStream_t stream);
template <class Table>
hipError_t launch_packed(const Table& t, uint32_t tiles, const AdamwScalars& s, const StepForm& f, hipStream_t stream);
hipError_t launch_unpack(const InlineTable<UnpackEntry>& t, uint32_t tiles, ar_state_t state, ar_dtype_t dtype,
                         hipStream_t stream);
// *norm = sqrt(sum of `n` partial sums), in a fixed order.
hipError_t launch_norm_final(const double* partials, uint32_t n, float* norm, hipStream_t stream);

}  // namespace arimpl
