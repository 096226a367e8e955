// Host side of the training-step operators declared in include/ar.h: the
// global gradient norm, the AdamW step with float32 or packed states, the
// packed states' values, and their persistent forms.  Every entry point
// validates first, then cuts the tensors into tiles, one line of a table per
// tensor, and enqueues the kernels of ar_step_kernels.hip: one-shot calls
// with the table in the kernel's arguments, as many launches as it takes;
// plans with the table in the caller's workspace, in one launch.

#include <hip/hip_runtime.h>

#include <cmath>
#include <cstring>
#include <limits>
#include <utility>

#include "ar_host.h"
#include "ar_step.h"

using namespace arimpl;

namespace {

size_t esize(ar_dtype_t dt) { return dt == AR_FLOAT32 ? 4 : 2; }

// Far above any tensor that a GPU holds, far below where tile counts overflow.
constexpr uint64_t kMaxCount = 1ull << 48;
// One workgroup per tile; a launch has fewer than 2^32 threads in all.
constexpr uint64_t kMaxTiles = 0xffffffffull / kStepThreads;

ar_result_t check_counts(const size_t* counts, int n) {
    if (n < 0 || n > AR_MAX_TENSORS)
        return fail_with(AR_ERR_INVALID_ARGUMENT, "ntensors %d outside [0, %d]", n, AR_MAX_TENSORS);
    if (n > 0 && counts == nullptr) return fail_with(AR_ERR_INVALID_ARGUMENT, "null counts array");
    for (int t = 0; t < n; ++t) {
        if (counts[t] > kMaxCount)
            return fail_with(AR_ERR_INVALID_ARGUMENT, "counts[%d] = %llu is too large", t,
                             static_cast<unsigned long long>(counts[t]));
    }
    return AR_SUCCESS;
}

uint64_t tiles_of(uint64_t count, uint32_t tile) { return (count + tile - 1) / tile; }

ar_result_t check_tiles(const size_t* counts, int n, uint32_t tile) {
    uint64_t all = 0;
    for (int t = 0; t < n; ++t) {
        all += tiles_of(counts[t], tile);
        if (all > kMaxTiles) return fail_with(AR_ERR_INVALID_ARGUMENT, "the tensors hold too many elements for one call");
    }
    return AR_SUCCESS;
}

uint64_t state_blocks(uint64_t count) { return (count + AR_STATE_BLOCK - 1) / AR_STATE_BLOCK; }

// ---------------------------------------------------------------------------
// tables
// ---------------------------------------------------------------------------

// The lines of a call's tensors that hold anything, first_tile unset.
template <class Entry>
struct Lines {
    std::vector<Entry> e;
    uint32_t tile;   // elements per tile
};

// One launch after another, each over as many lines as fit its arguments:
// launch(table, tiles, number of the launch).
template <class Entry, class Launch>
ar_result_t in_launches(const Lines<Entry>& lines, const char* what, Launch launch) {
    InlineTable<Entry> t;
    size_t at = 0;
    for (uint32_t k = 0; at < lines.e.size(); ++k) {
        t.n = 0;
        uint64_t tiles = 0;
        while (at < lines.e.size() && t.n < InlineTable<Entry>::kMax) {
            t.e[t.n] = lines.e[at];
            t.e[t.n].first_tile = static_cast<uint32_t>(tiles);
            tiles += tiles_of(lines.e[at].n, lines.tile);
            ++t.n;
            ++at;
        }
        const ar_result_t rc = hip_result(launch(t, static_cast<uint32_t>(tiles), k), what);
        if (rc != AR_SUCCESS) return rc;
    }
    return AR_SUCCESS;
}

uint64_t launches_of(uint64_t lines, int per_launch) {
    return (lines + static_cast<uint64_t>(per_launch) - 1) / static_cast<uint64_t>(per_launch);
}

// A plan's table in the workspace: the lines, then each tile's line number.
template <class Entry>
uint64_t table_bytes(uint64_t lines, uint64_t tiles) {
    return (lines * sizeof(Entry) + tiles * sizeof(uint32_t) + 7) / 8 * 8;
}

// Copies the table to `at`, after `zeros` bytes of zero.
template <class Entry>
ar_result_t upload(Lines<Entry>& lines, char* at, size_t zeros, hipStream_t stream, DeviceTable<Entry>* out,
                   uint32_t* out_tiles) {
    uint64_t tiles = 0;
    for (Entry& e : lines.e) {
        e.first_tile = static_cast<uint32_t>(tiles);
        tiles += tiles_of(e.n, lines.tile);
    }
    *out = {reinterpret_cast<const Entry*>(at + zeros),
            reinterpret_cast<const uint32_t*>(at + zeros + lines.e.size() * sizeof(Entry))};
    *out_tiles = static_cast<uint32_t>(tiles);
    if (tiles == 0) return AR_SUCCESS;
    std::vector<char> host(zeros + lines.e.size() * sizeof(Entry) + tiles * sizeof(uint32_t));
    std::memcpy(host.data() + zeros, lines.e.data(), lines.e.size() * sizeof(Entry));
    char* to = host.data() + zeros + lines.e.size() * sizeof(Entry);
    for (uint32_t k = 0; k < lines.e.size(); ++k) {
        for (uint64_t j = tiles_of(lines.e[k].n, lines.tile); j > 0; --j, to += sizeof(uint32_t))
            std::memcpy(to, &k, sizeof(uint32_t));
    }
    ar_result_t rc = hip_result(hipMemcpyAsync(at, host.data(), host.size(), hipMemcpyHostToDevice, stream),
                                "copying the plan's table");
    if (rc == AR_SUCCESS) rc = hip_result(hipStreamSynchronize(stream), "copying the plan's table");
    return rc;
}

ar_result_t refuse_capture(hipStream_t stream) {
    hipStreamCaptureStatus status = hipStreamCaptureStatusNone;
    const ar_result_t rc = hip_result(hipStreamIsCapturing(stream, &status), "hipStreamIsCapturing");
    if (rc != AR_SUCCESS) return rc;
    if (status != hipStreamCaptureStatusNone)
        return fail_with(AR_ERR_UNSUPPORTED, "a plan cannot be made while its stream is being captured");
    return AR_SUCCESS;
}

ar_result_t add_workspace(std::vector<Range>& v, void* ws, size_t have, uint64_t need) {
    if (need == 0) return AR_SUCCESS;
    if (ws == nullptr || have < need)
        return fail_with(AR_ERR_INVALID_ARGUMENT, "this call needs a workspace of %llu bytes",
                         static_cast<unsigned long long>(need));
    return add_range(v, ws, need, 8, true, "workspace", 0);
}

// ---------------------------------------------------------------------------
// gradient norm
// ---------------------------------------------------------------------------

// Workgroups of one launch: enough to fill the GPU; more would only leave more
// partial sums.
uint32_t norm_blocks(uint64_t tiles) { return static_cast<uint32_t>(std::min<uint64_t>(tiles, kNormBlocks)); }

// A plan's counter of finished workgroups stands between its partial sums and
// its table.
constexpr size_t kCounterBytes = 8;

// Partial sums of a one-shot call (at most kNormBlocks a launch) or a plan.
uint64_t norm_workspace(const size_t* counts, int n) {
    uint64_t lines = 0, tiles = 0;
    for (int t = 0; t < n; ++t) {
        lines += counts[t] > 0 ? 1 : 0;
        tiles += tiles_of(counts[t], kNormTile);
    }
    const uint64_t partials = launches_of(lines, InlineTable<NormEntry>::kMax) * kNormBlocks * sizeof(double);
    return lines == 0 ? 0 : partials + kCounterBytes + table_bytes<NormEntry>(lines, tiles);
}

ar_result_t norm_lines(const void* const* grads, const size_t* counts, int n, ar_dtype_t dtype, float* norm, void* ws,
                       size_t ws_bytes, Lines<NormEntry>& lines, std::vector<Range>& ranges) {
    if (!float_type(dtype)) return fail_with(AR_ERR_INVALID_ARGUMENT, "unsupported dtype %d", static_cast<int>(dtype));
    ar_result_t rc = check_counts(counts, n);
    if (rc != AR_SUCCESS || (rc = check_tiles(counts, n, kNormTile)) != AR_SUCCESS) return rc;
    if (n > 0 && grads == nullptr) return fail_with(AR_ERR_INVALID_ARGUMENT, "null pointer array");
    lines.tile = kNormTile;
    for (int t = 0; t < n; ++t) {
        if ((rc = add_range(ranges, grads[t], counts[t] * esize(dtype), esize(dtype), false, "grads", t)) != AR_SUCCESS)
            return rc;
        if (counts[t] > 0)
            lines.e.push_back({static_cast<const char*>(grads[t]), counts[t], 0, static_cast<uint32_t>(t)});
    }
    if ((rc = add_range(ranges, norm, sizeof(float), alignof(float), true, "norm", 0)) != AR_SUCCESS) return rc;
    if ((rc = add_workspace(ranges, ws, ws_bytes, norm_workspace(counts, n))) != AR_SUCCESS) return rc;
    return check_ranges(ranges);
}

// ---------------------------------------------------------------------------
// AdamW
// ---------------------------------------------------------------------------

ar_result_t scalars(const ar_adamw_config_t* c, const float* grad_norm, ar_dtype_t copy_dtype, AdamwScalars* out) {
    if (c == nullptr) return fail_with(AR_ERR_INVALID_ARGUMENT, "null config");
    const auto range = [](double x, double lo, double hi) { return x >= lo && x <= hi; };   // false for NaN
    const double most = std::numeric_limits<float>::max();
    if (!range(c->lr, 0, most)) return fail_with(AR_ERR_INVALID_ARGUMENT, "lr %g is not a finite number >= 0", c->lr);
    if (!(c->beta1 >= 0 && c->beta1 < 1) || !(c->beta2 >= 0 && c->beta2 < 1))
        return fail_with(AR_ERR_INVALID_ARGUMENT, "betas %g, %g outside [0, 1)", c->beta1, c->beta2);
    if (!range(c->eps, 0, most)) return fail_with(AR_ERR_INVALID_ARGUMENT, "eps %g is not a finite number >= 0", c->eps);
    if (!range(c->weight_decay, 0, most))
        return fail_with(AR_ERR_INVALID_ARGUMENT, "weight_decay %g is not a finite number >= 0", c->weight_decay);
    if (!range(c->max_norm, 0, most))
        return fail_with(AR_ERR_INVALID_ARGUMENT, "max_norm %g is not a finite number >= 0", c->max_norm);
    if (!(c->grad_scale > 0 && c->grad_scale <= most))
        return fail_with(AR_ERR_INVALID_ARGUMENT, "grad_scale %g is not a finite number > 0", c->grad_scale);
    if (c->step < 1) return fail_with(AR_ERR_INVALID_ARGUMENT, "step counts from 1");
    if (grad_norm == nullptr && (c->max_norm > 0 || c->skip_nonfinite))
        return fail_with(AR_ERR_INVALID_ARGUMENT, "max_norm and skip_nonfinite need grad_norm");
    if (reinterpret_cast<uintptr_t>(grad_norm) % alignof(float) != 0)
        return fail_with(AR_ERR_INVALID_ARGUMENT, "grad_norm not aligned to its 4-byte element");
    // what the kernels get is float32: a setting that is on must not round to off
    for (const auto& [x, name] : {std::pair<double, const char*>{c->eps, "eps"},
                                  {c->max_norm, "max_norm"},
                                  {c->grad_scale, "grad_scale"}}) {
        if (rounds_to_zero(x)) return fail_with(AR_ERR_INVALID_ARGUMENT, "%s %g is 0 in float32", name, x);
    }
    const double t = static_cast<double>(c->step);
    const double step_size = c->lr / (1 - std::pow(c->beta1, t)), decay = 1 - c->lr * c->weight_decay;
    if (!(step_size <= most))
        return fail_with(AR_ERR_INVALID_ARGUMENT, "lr %g / (1 - beta1^step) is past float32's range", c->lr);
    if (!(decay >= -most))
        return fail_with(AR_ERR_INVALID_ARGUMENT, "lr %g * weight_decay %g is past float32's range", c->lr,
                         c->weight_decay);
    AdamwScalars s{};
    s.grad_norm = grad_norm;
    s.beta1 = static_cast<float>(c->beta1);
    s.one_minus_beta1 = static_cast<float>(1 - c->beta1);
    s.beta2 = static_cast<float>(c->beta2);
    s.one_minus_beta2 = static_cast<float>(1 - c->beta2);
    s.eps = static_cast<float>(c->eps);
    s.decay = static_cast<float>(decay);
    s.step_size = static_cast<float>(step_size);
    s.rsqrt_correction2 = static_cast<float>(1 / std::sqrt(1 - std::pow(c->beta2, t)));
    s.max_norm = static_cast<float>(c->max_norm);
    s.grad_scale = static_cast<float>(c->grad_scale);
    s.skip_nonfinite = c->skip_nonfinite != 0;
    s.seed = c->seed;
    s.copy_f16 = copy_dtype == AR_FLOAT16;
    *out = s;
    return AR_SUCCESS;
}

// An input and where its new values go: one writable range in place, else one
// of each.
ar_result_t add_pair(std::vector<Range>& v, const void* const* in, void* const* out, int t, uint64_t bytes, size_t align,
                     const char* what, const char* out_what, const void** from, void** to) {
    *from = in[t];
    *to = out == nullptr ? const_cast<void*>(in[t]) : out[t];
    if (*to == *from) return add_range(v, *from, bytes, align, true, what, t);
    const ar_result_t rc = add_range(v, *from, bytes, align, false, what, t);
    return rc != AR_SUCCESS ? rc : add_range(v, *to, bytes, align, true, out_what, t);
}

template <bool PACKED>
using EntryOf = typename std::conditional<PACKED, PackedEntry, AdamwEntry>::type;
template <bool PACKED>
constexpr uint32_t kTileOf = PACKED ? kPackedTile : kAdamwTile;

// Which form the call's kernels take (the measurements stand at the bounds).
template <bool PACKED>
bool large_step(const ar_adamw_tensors_t* a) {
    uint64_t n = 0;
    for (int t = 0; t < a->ntensors; ++t) n += a->counts[t];
    if (PACKED) return a->param_dtype != AR_FLOAT32 && a->grad_dtype != AR_FLOAT32 && n >= kPackedLargeElements;
    const uint64_t per = 2 * esize(a->param_dtype) + esize(a->grad_dtype) + (a->copies != nullptr ? 2 : 0) + 16;
    return n * per > kAdamwLargeBytes;
}

template <bool PACKED>
ar_result_t adamw_lines(const ar_adamw_tensors_t* a, Lines<EntryOf<PACKED>>& lines, std::vector<Range>& ranges,
                        StepForm& form) {
    if (a == nullptr) return fail_with(AR_ERR_INVALID_ARGUMENT, "null tensors");
    if (!float_type(a->param_dtype) || !float_type(a->grad_dtype))
        return fail_with(AR_ERR_INVALID_ARGUMENT, "unsupported param dtype %d or grad dtype %d",
                         static_cast<int>(a->param_dtype), static_cast<int>(a->grad_dtype));
    if (a->copies != nullptr) {
        if (a->param_dtype != AR_FLOAT32)
            return fail_with(AR_ERR_INVALID_ARGUMENT, "copies are kept of float32 parameters only");
        if (a->copy_dtype != AR_BFLOAT16 && a->copy_dtype != AR_FLOAT16)
            return fail_with(AR_ERR_INVALID_ARGUMENT, "unsupported copy dtype %d", static_cast<int>(a->copy_dtype));
    }
    ar_result_t rc = check_counts(a->counts, a->ntensors);
    if (rc != AR_SUCCESS || (rc = check_tiles(a->counts, a->ntensors, kTileOf<PACKED>)) != AR_SUCCESS) return rc;
    if (a->ntensors > 0) {
        if (a->params == nullptr || a->grads == nullptr || a->exp_avgs == nullptr || a->exp_avg_sqs == nullptr)
            return fail_with(AR_ERR_INVALID_ARGUMENT, "null pointer array");
        if (PACKED && (a->exp_avg_scales == nullptr || a->exp_avg_sq_scales == nullptr))
            return fail_with(AR_ERR_INVALID_ARGUMENT, "null pointer array of scales");
    }
    if (!PACKED && (a->exp_avg_scales != nullptr || a->exp_avg_sq_scales != nullptr ||
                    a->exp_avg_scales_out != nullptr || a->exp_avg_sq_scales_out != nullptr))
        return fail_with(AR_ERR_INVALID_ARGUMENT, "float32 states have no scales");
    form = {a->param_dtype, a->grad_dtype, large_step<PACKED>(a)};
    const bool all_f32 = form.param == AR_FLOAT32 && form.grad == AR_FLOAT32;
    lines.tile = kTileOf<PACKED> * static_cast<uint32_t>(PACKED ? packed_vectors(form.large) : adamw_vectors(form.large, all_f32));
    const size_t ps = esize(a->param_dtype), gs = esize(a->grad_dtype), ss = PACKED ? 1 : 4;
    for (int t = 0; t < a->ntensors; ++t) {
        const uint64_t n = a->counts[t];
        if (n == 0) continue;
        const void *p, *m, *v, *ms = nullptr, *vs = nullptr;
        void *po, *mo, *vo, *mso = nullptr, *vso = nullptr, *copy = nullptr;
        if ((rc = add_range(ranges, a->grads[t], n * gs, gs, false, "grads", t)) != AR_SUCCESS ||
            (rc = add_pair(ranges, a->params, a->params_out, t, n * ps, ps, "params", "params_out", &p, &po)) !=
                AR_SUCCESS ||
            (rc = add_pair(ranges, a->exp_avgs, a->exp_avgs_out, t, n * ss, ss, "exp_avgs", "exp_avgs_out", &m, &mo)) !=
                AR_SUCCESS ||
            (rc = add_pair(ranges, a->exp_avg_sqs, a->exp_avg_sqs_out, t, n * ss, ss, "exp_avg_sqs", "exp_avg_sqs_out",
                           &v, &vo)) != AR_SUCCESS)
            return rc;
        if (a->copies != nullptr) {
            copy = a->copies[t];
            if ((rc = add_range(ranges, copy, n * 2, 2, true, "copies", t)) != AR_SUCCESS) return rc;
        }
        if constexpr (PACKED) {
            const uint64_t b = state_blocks(n);
            if ((rc = add_pair(ranges, a->exp_avg_scales, a->exp_avg_scales_out, t, b, 1, "exp_avg_scales",
                               "exp_avg_scales_out", &ms, &mso)) != AR_SUCCESS ||
                (rc = add_pair(ranges, a->exp_avg_sq_scales, a->exp_avg_sq_scales_out, t, b, 1, "exp_avg_sq_scales",
                               "exp_avg_sq_scales_out", &vs, &vso)) != AR_SUCCESS)
                return rc;
            lines.e.push_back({static_cast<const char*>(p), static_cast<const char*>(a->grads[t]),
                               static_cast<const uint8_t*>(m), static_cast<const uint8_t*>(v),
                               static_cast<const uint8_t*>(ms), static_cast<const uint8_t*>(vs),
                               static_cast<char*>(po), static_cast<uint8_t*>(mo), static_cast<uint8_t*>(vo),
                               static_cast<uint8_t*>(mso), static_cast<uint8_t*>(vso), static_cast<char*>(copy), n, 0,
                               static_cast<uint32_t>(t)});
        } else {
            lines.e.push_back({static_cast<const char*>(p), static_cast<const char*>(a->grads[t]),
                               static_cast<const char*>(m), static_cast<const char*>(v), static_cast<char*>(po),
                               static_cast<char*>(mo), static_cast<char*>(vo), static_cast<char*>(copy), n, 0,
                               static_cast<uint32_t>(t)});
        }
    }
    return AR_SUCCESS;
}

template <bool PACKED, class Table>
hipError_t launch_step(const Table& t, uint32_t tiles, const AdamwScalars& s, const StepForm& f, hipStream_t stream) {
    if constexpr (PACKED) {
        return launch_packed(t, tiles, s, f, stream);
    } else {
        return launch_adamw(t, tiles, s, f, stream);
    }
}

template <bool PACKED>
ar_result_t adamw_now(const ar_adamw_tensors_t* a, const ar_adamw_config_t* config, const float* grad_norm,
                      hipStream_t stream) {
    Lines<EntryOf<PACKED>> lines;
    std::vector<Range> ranges;
    AdamwScalars s;
    StepForm form;
    ar_result_t rc = adamw_lines<PACKED>(a, lines, ranges, form);
    if (rc != AR_SUCCESS || (rc = scalars(config, grad_norm, a->copy_dtype, &s)) != AR_SUCCESS) return rc;
    if (grad_norm != nullptr &&
        (rc = add_range(ranges, grad_norm, sizeof(float), alignof(float), false, "grad_norm", 0)) != AR_SUCCESS)
        return rc;
    if ((rc = check_ranges(ranges)) != AR_SUCCESS) return rc;
    return in_launches(lines, PACKED ? "adamw_packed launch" : "adamw launch",
                       [&](const InlineTable<EntryOf<PACKED>>& t, uint32_t tiles, uint32_t) {
                           return launch_step<PACKED>(t, tiles, s, form, stream);
                       });
}

// Room for a plan's table in either form: the small one has more tiles.
template <bool PACKED>
uint64_t adamw_workspace(const size_t* counts, int n) {
    uint64_t lines = 0, tiles = 0;
    for (int t = 0; t < n; ++t) {
        lines += counts[t] > 0 ? 1 : 0;
        tiles += tiles_of(counts[t], kTileOf<PACKED>);
    }
    return table_bytes<EntryOf<PACKED>>(lines, tiles);
}

}  // namespace

// A persistent norm or step: its table on the device, and what the launch needs.
struct ar_update_s {
    ar_update_kind_t kind;
    uint32_t tiles = 0;
    StepForm form{AR_FLOAT32, AR_FLOAT32, false};   // a norm: the gradients' type only
    ar_dtype_t copy = AR_BFLOAT16;
    float* norm = nullptr;
    double* partials = nullptr;
    DeviceTable<NormEntry> norm_table{};
    DeviceTable<AdamwEntry> adamw_table{};
    DeviceTable<PackedEntry> packed_table{};
};

namespace {

// Launches of a norm of so many workgroups: one when one of them can finish
// the sum, else a second that adds the partial sums (and writes 0 where there
// is nothing to add).
int norm_launches(uint32_t blocks) { return blocks <= kNormJoinBlocks ? 1 : 2; }

ar_result_t start_norm(const ar_update_s& u, hipStream_t stream) {
    const uint32_t blocks = norm_blocks(u.tiles);
    if (blocks > 0) {
        const bool join = norm_launches(blocks) == 1;
        uint32_t* const counter = reinterpret_cast<uint32_t*>(u.partials + kNormBlocks);
        const ar_result_t rc =
            hip_result(launch_norm(u.norm_table, u.tiles, blocks, u.form.grad, u.partials, join ? u.norm : nullptr,
                                   join ? counter : nullptr, stream),
                       "grad_norm launch");
        if (rc != AR_SUCCESS || join) return rc;
    }
    return hip_result(launch_norm_final(u.partials, blocks, u.norm, stream), "grad_norm launch");
}

// Makes an update: build(update) validates and uploads.
template <class Build>
ar_result_t make_update(ar_update_t* out, ar_update_kind_t kind, Build build) {
    if (out == nullptr) return fail_with(AR_ERR_INVALID_ARGUMENT, "null update pointer");
    *out = nullptr;
    ar_update_s u{};
    u.kind = kind;
    const ar_result_t rc = build(u);
    if (rc != AR_SUCCESS) return rc;
    *out = new ar_update_s(u);
    return AR_SUCCESS;
}

template <bool PACKED>
ar_result_t init_adamw(const ar_adamw_tensors_t* a, void* ws, size_t ws_bytes, hipStream_t stream, ar_update_s& u) {
    Lines<EntryOf<PACKED>> lines;
    std::vector<Range> ranges;
    ar_result_t rc = adamw_lines<PACKED>(a, lines, ranges, u.form);
    if (rc != AR_SUCCESS ||
        (rc = add_workspace(ranges, ws, ws_bytes, adamw_workspace<PACKED>(a->counts, a->ntensors))) != AR_SUCCESS ||
        (rc = check_ranges(ranges)) != AR_SUCCESS)
        return rc;
    u.copy = a->copy_dtype;
    if (lines.e.empty()) return AR_SUCCESS;   // nothing to place: no device is asked
    if ((rc = refuse_capture(stream)) != AR_SUCCESS || (rc = check_device_memory(ranges)) != AR_SUCCESS) return rc;
    if constexpr (PACKED) {
        return upload(lines, static_cast<char*>(ws), 0, stream, &u.packed_table, &u.tiles);
    } else {
        return upload(lines, static_cast<char*>(ws), 0, stream, &u.adamw_table, &u.tiles);
    }
}

}  // namespace

extern "C" {

ar_result_t ar_grad_norm(const void* const* grads, const size_t* counts, int ntensors, ar_dtype_t dtype, float* norm,
                         void* workspace, size_t workspace_bytes, hipStream_t stream) {
    return guarded([&]() -> ar_result_t {
        Lines<NormEntry> lines;
        std::vector<Range> ranges;
        ar_result_t rc = norm_lines(grads, counts, ntensors, dtype, norm, workspace, workspace_bytes, lines, ranges);
        if (rc != AR_SUCCESS) return rc;
        const bool single = lines.e.size() == 1 && lines.e[0].n <= kNormTile;
        double* partials = static_cast<double*>(workspace);
        uint32_t written = 0;
        rc = in_launches(lines, "grad_norm launch", [&](const InlineTable<NormEntry>& t, uint32_t tiles, uint32_t) {
            const uint32_t blocks = norm_blocks(tiles);
            const hipError_t e =
                launch_norm(t, tiles, blocks, dtype, partials + written, single ? norm : nullptr, nullptr, stream);
            written += blocks;
            return e;
        });
        if (rc != AR_SUCCESS || single) return rc;
        return hip_result(launch_norm_final(partials, written, norm, stream), "grad_norm launch");
    });
}

ar_result_t ar_adamw(const ar_adamw_tensors_t* tensors, const ar_adamw_config_t* config, const float* grad_norm,
                     hipStream_t stream) {
    return guarded([&] { return adamw_now<false>(tensors, config, grad_norm, stream); });
}

ar_result_t ar_adamw_packed(const ar_adamw_tensors_t* tensors, const ar_adamw_config_t* config, const float* grad_norm,
                            hipStream_t stream) {
    return guarded([&] { return adamw_now<true>(tensors, config, grad_norm, stream); });
}

ar_result_t ar_unpack_states(const void* const* codes, const void* const* scales, void* const* outs,
                             const size_t* counts, int ntensors, ar_state_t state, ar_dtype_t dtype,
                             hipStream_t stream) {
    return guarded([&]() -> ar_result_t {
        if (!float_type(dtype))
            return fail_with(AR_ERR_INVALID_ARGUMENT, "unsupported dtype %d", static_cast<int>(dtype));
        if (state != AR_STATE_EXP_AVG && state != AR_STATE_EXP_AVG_SQ)
            return fail_with(AR_ERR_INVALID_ARGUMENT, "unknown state %d", static_cast<int>(state));
        ar_result_t rc = check_counts(counts, ntensors);
        if (rc != AR_SUCCESS || (rc = check_tiles(counts, ntensors, kUnpackTile)) != AR_SUCCESS) return rc;
        if (ntensors > 0 && (codes == nullptr || scales == nullptr || outs == nullptr))
            return fail_with(AR_ERR_INVALID_ARGUMENT, "null pointer array");
        Lines<UnpackEntry> lines;
        lines.tile = kUnpackTile;
        std::vector<Range> ranges;
        for (int t = 0; t < ntensors; ++t) {
            const uint64_t n = counts[t];
            if (n == 0) continue;
            if ((rc = add_range(ranges, codes[t], n, 1, false, "codes", t)) != AR_SUCCESS ||
                (rc = add_range(ranges, scales[t], state_blocks(n), 1, false, "scales", t)) != AR_SUCCESS ||
                (rc = add_range(ranges, outs[t], n * esize(dtype), esize(dtype), true, "outs", t)) != AR_SUCCESS)
                return rc;
            lines.e.push_back({static_cast<const uint8_t*>(codes[t]), static_cast<const uint8_t*>(scales[t]),
                               static_cast<char*>(outs[t]), n, 0, static_cast<uint32_t>(t)});
        }
        if ((rc = check_ranges(ranges)) != AR_SUCCESS) return rc;
        return in_launches(lines, "unpack_states launch",
                           [&](const InlineTable<UnpackEntry>& t, uint32_t tiles, uint32_t) {
                               return launch_unpack(t, tiles, state, dtype, stream);
                           });
    });
}

size_t ar_update_workspace_bytes(ar_update_kind_t kind, const size_t* counts, int ntensors) {
    if (ntensors < 0 || ntensors > AR_MAX_TENSORS || (ntensors > 0 && counts == nullptr)) return static_cast<size_t>(-1);
    for (int t = 0; t < ntensors; ++t)
        if (counts[t] > kMaxCount) return static_cast<size_t>(-1);
    switch (kind) {
        case AR_UPDATE_GRAD_NORM: return norm_workspace(counts, ntensors);
        case AR_UPDATE_ADAMW: return adamw_workspace<false>(counts, ntensors);
        case AR_UPDATE_ADAMW_PACKED: return adamw_workspace<true>(counts, ntensors);
    }
    return static_cast<size_t>(-1);
}

ar_result_t ar_grad_norm_init(const void* const* grads, const size_t* counts, int ntensors, ar_dtype_t dtype,
                              float* norm, void* workspace, size_t workspace_bytes, hipStream_t stream,
                              ar_update_t* update) {
    return guarded([&] {
        return make_update(update, AR_UPDATE_GRAD_NORM, [&](ar_update_s& u) -> ar_result_t {
            Lines<NormEntry> lines;
            std::vector<Range> ranges;
            ar_result_t rc =
                norm_lines(grads, counts, ntensors, dtype, norm, workspace, workspace_bytes, lines, ranges);
            if (rc != AR_SUCCESS || (rc = refuse_capture(stream)) != AR_SUCCESS ||
                (rc = check_device_memory(ranges)) != AR_SUCCESS)
                return rc;
            u.form.grad = dtype;
            u.norm = norm;
            u.partials = static_cast<double*>(workspace);
            return upload(lines, static_cast<char*>(workspace) + kNormBlocks * sizeof(double), kCounterBytes, stream,
                          &u.norm_table, &u.tiles);
        });
    });
}

ar_result_t ar_adamw_init(const ar_adamw_tensors_t* tensors, void* workspace, size_t workspace_bytes,
                          hipStream_t stream, ar_update_t* update) {
    return guarded([&] {
        return make_update(update, AR_UPDATE_ADAMW, [&](ar_update_s& u) {
            return init_adamw<false>(tensors, workspace, workspace_bytes, stream, u);
        });
    });
}

ar_result_t ar_adamw_packed_init(const ar_adamw_tensors_t* tensors, void* workspace, size_t workspace_bytes,
                                 hipStream_t stream, ar_update_t* update) {
    return guarded([&] {
        return make_update(update, AR_UPDATE_ADAMW_PACKED, [&](ar_update_s& u) {
            return init_adamw<true>(tensors, workspace, workspace_bytes, stream, u);
        });
    });
}

ar_result_t ar_grad_norm_start(ar_update_t update, hipStream_t stream) {
    return guarded([&]() -> ar_result_t {
        if (update == nullptr) return fail_with(AR_ERR_INVALID_ARGUMENT, "null update");
        if (update->kind != AR_UPDATE_GRAD_NORM)
            return fail_with(AR_ERR_INVALID_ARGUMENT, "not a plan of ar_grad_norm_init");
        return start_norm(*update, stream);
    });
}

ar_result_t ar_adamw_start(ar_update_t update, const ar_adamw_config_t* config, const float* grad_norm,
                           hipStream_t stream) {
    return guarded([&]() -> ar_result_t {
        if (update == nullptr) return fail_with(AR_ERR_INVALID_ARGUMENT, "null update");
        if (update->kind == AR_UPDATE_GRAD_NORM)
            return fail_with(AR_ERR_INVALID_ARGUMENT, "not a plan of ar_adamw_init or ar_adamw_packed_init");
        AdamwScalars s;
        const ar_result_t rc = scalars(config, grad_norm, update->copy, &s);
        if (rc != AR_SUCCESS || update->tiles == 0) return rc;
        const ar_update_s& u = *update;
        return hip_result(u.kind == AR_UPDATE_ADAMW_PACKED
                              ? launch_packed(u.packed_table, u.tiles, s, u.form, stream)
                              : launch_adamw(u.adamw_table, u.tiles, s, u.form, stream),
                          "adamw launch");
    });
}

int ar_update_num_launches(ar_update_t update) {
    if (update == nullptr) return -1;
    if (update->kind == AR_UPDATE_GRAD_NORM) return norm_launches(norm_blocks(update->tiles));
    return update->tiles > 0 ? 1 : 0;
}

ar_result_t ar_update_free(ar_update_t update) {
    delete update;
    return AR_SUCCESS;
}

}  // extern "C"
