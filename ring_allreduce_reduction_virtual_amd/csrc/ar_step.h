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

// Elements per tile (one workgroup's share of one tensor).
constexpr uint32_t kNormTile = 8192;
constexpr uint32_t kAdamwTile = 4096;
constexpr uint32_t kPackedTile = 2048;
constexpr uint32_t kUnpackTile = 2048;
static_assert(kPackedTile % AR_STATE_BLOCK == 0 && kUnpackTile % AR_STATE_BLOCK == 0, "whole state blocks per tile");

// Most partial sums one launch of the gradient norm leaves (its workgroups).
constexpr uint32_t kNormBlocks = 1024;

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
                       float* norm, hipStream_t stream);
template <class Table>
hipError_t launch_adamw(const Table& t, uint32_t tiles, const AdamwScalars& s, ar_dtype_t param, ar_dtype_t grad,
                        hipStream_t stream);
template <class Table>
hipError_t launch_packed(const Table& t, uint32_t tiles, const AdamwScalars& s, ar_dtype_t param, ar_dtype_t grad,
                         hipStream_t stream);
hipError_t launch_unpack(const InlineTable<UnpackEntry>& t, uint32_t tiles, ar_state_t state, ar_dtype_t dtype,
                         hipStream_t stream);
// *norm = sqrt(sum of `n` partial sums), in a fixed order.
hipError_t launch_norm_final(const double* partials, uint32_t n, float* norm, hipStream_t stream);

}  // namespace arimpl
