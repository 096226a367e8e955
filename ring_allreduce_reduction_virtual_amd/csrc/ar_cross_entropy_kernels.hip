// HIP kernels of the cross entropy of logits that are never stored
// (include/ar.h states the formulas).
//
// Every product has the vocabulary or the columns on its m side and tokens (or
// for dweight the vocabulary) on its n side: a lane then holds one token's
// logits of a tile in its registers, so that a tile's maximum and sum of
// exponentials are almost all registers' work, and what a lane stores is
// contiguous.
//
// Forward: one product over the whole vocabulary; a tile leaves each token's
// maximum and sum of exponentials, which a small launch joins in order.
//
// Backward: the logits cost a second product; stored since the forward pass they
// would hold 2 or 4 bytes each until here.  Piece by piece of the vocabulary: dz =
// g (p - onehot) from the logits' product's registers, rounded to the operands'
// type; dx's sums gain dz W of the piece (the order of pieces is fixed); the
// piece's rows of dweight = dz^T x are complete.  The rows that take part are
// gathered first, so that ignored rows cost nothing and reach nothing.
//
// 16-bit dz is the one value that is held in fewer than 32 bits: the matrix
// instructions take both operands in one type, and W and x are 16-bit.  It costs
// a rounding beside the results' own where the rows' g differ: 4,096 rows of 4,096
// against 65,536 in bf16, error of dx and dweight against float64 relative to
// their 2-norm, 0.0022 with g of 0.5 to 1 and 0.0017 with one g, which is what
// rounding the exact results gives.  dz in two 16-bit parts would undo it and make
// both products twice as long (10.3 ms of 2 x 4,096 rows to some 17).
//
// The matrix cores bound the large sizes: 2 x 4,096 rows of 4,096 against
// 65,536 in bf16 take 3.3 ms forward (1,340 TFLOP/s; operands of zeros, which
// draw less power, 1,615) and 10.3 backward (1,280), each of the three products
// the same 1.75 ms for half of the vocabulary; float32, 2 x 4,096 of 2,048 against
// 32,768, 7.6 ms (146) and 23.1.  With few rows reading the weight does: 16 rows
// of 4,096 against 65,536 112 us (4.8 TB/s).

#include <hip/hip_runtime.h>

#include "ar_cross_entropy.h"
#include "ar_product_device.h"

namespace arimpl {
namespace {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

__device__ __forceinline__ int64_t index_at(const char* p, uint64_t i, int wide) {
    return wide ? reinterpret_cast<const int64_t*>(p)[i] : reinterpret_cast<const int32_t*>(p)[i];
}

// The tiles that pick_tile chooses from.  The smallest one waits for memory most:
// 16 bits have twice the k a step (16 rows of 1,024 against 8,192 10.5 -> 9.2 us,
// 32 of 768 against 50,257, backward, 84 -> 81, the same elsewhere); float32 has
// three short steps, so that four workgroups share a compute unit (3 x 129 rows
// of 515 against 5,003, backward, 143 us with four -> 134; two cost 16 rows of
// 4,096 against 65,536 832 -> 978).
typedef TileOf<256, 256, 2, 4, 128, 2> LargeTile;
typedef TileOf<128, 128, 4, 2, 128, 2> MediumTile;
typedef TileOf<128, 64, 4, 1, 128, 3> SmallTile;
template <int DT>
using TinyTile = TileOf<64, 32, 2, 2, DT == AR_FLOAT32 ? 128 : 256, 3>;

// ---------------------------------------------------------------------------
// forward
// ---------------------------------------------------------------------------

template <int DT, class Tile, bool WHOLE>
__global__ void __launch_bounds__(Tile::kThreads) k_cross_stats(CrossArgs a, uint32_t tiles_m, uint32_t tiles_n,
                                                                uint32_t ranks) {
    __shared__ __attribute__((aligned(1024))) char buffers[Tile::kShared];
    __shared__ float most[Tile::WM][Tile::EN], total[Tile::WM][Tile::EN];
    const TilePlace tile(blockIdx.x, tiles_m, tiles_n, ranks);
    if (!tile.valid) return;
    constexpr int kEs = elem_size<DT>();
    const uint64_t m0 = static_cast<uint64_t>(tile.m) * Tile::EM, n0 = static_cast<uint64_t>(tile.n) * Tile::EN;
    f32x4 sum[Tile::TM][Tile::TN];
    product<DT, Tile, WHOLE, true, true>(buffers, a.weight[tile.rank], a.weight_stride * kEs, m0, a.count, a.x[tile.rank],
                                  a.x_stride * kEs, n0, a.rows, a.cols, sum);
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const int wm = wave / Tile::WN, wn = wave % Tile::WN;
    const uint64_t first = m0 + wm * Tile::TM * kSquare + 4 * (lane >> 4);   // this lane's first row of the piece
    if (m0 + Tile::EM > a.count) {
#pragma unroll
        for (int i = 0; i < Tile::TM; ++i) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if (first + i * kSquare + k >= a.count) {
#pragma unroll
                    for (int j = 0; j < Tile::TN; ++j) sum[i][j][k] = -INFINITY;
                }
            }
        }
    }
#pragma unroll
    for (int j = 0; j < Tile::TN; ++j) {
        const int n = (wn * Tile::TN + j) * kSquare + (lane & 15);
        float top = -INFINITY;
#pragma unroll
        for (int i = 0; i < Tile::TM; ++i) {
#pragma unroll
            for (int k = 0; k < 4; ++k) top = fmaxf(top, sum[i][j][k]);
        }
        const auto higher = [](uint32_t p, uint32_t q) { return as_u(fmaxf(as_f(p), as_f(q))); };
        top = as_f(across32(across16(as_u(top), higher), higher));
        // a tile of -infinities (a stretch past the vocabulary) adds 0
        const float from = top == -INFINITY ? 0.0f : top;
        float s = 0;
#pragma unroll
        for (int i = 0; i < Tile::TM; ++i) {
#pragma unroll
            for (int k = 0; k < 4; ++k) s += __builtin_amdgcn_exp2f((sum[i][j][k] - from) * kLog2e);
        }
        const auto both = [](uint32_t p, uint32_t q) { return as_u(as_f(p) + as_f(q)); };
        s = as_f(across32(across16(as_u(s), both), both));
        if (lane < 16) {
            most[wm][n] = top;
            total[wm][n] = s;
        }
        if (n0 + n < a.rows) {
            const int64_t t = index_at(a.targets[tile.rank], n0 + n, a.wide_index);
            const int64_t in = t - static_cast<int64_t>(a.first + first);   // this lane's rows: i * kSquare + k
            if (in >= 0 && in < Tile::TM * kSquare && t < static_cast<int64_t>(a.vocab)) {
                float z = 0;
                bool mine = false;
#pragma unroll
                for (int i = 0; i < Tile::TM; ++i) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        if (in == i * kSquare + k) {
                            z = sum[i][j][k];
                            mine = true;
                        }
                    }
                }
                if (mine) a.target_logit[tile.rank * a.rows + n0 + n] = z;
            }
        }
    }
    __syncthreads();
    for (int n = threadIdx.x; n < Tile::EN; n += Tile::kThreads) {
        if (n0 + n >= a.rows) continue;
        float top = most[0][n];
#pragma unroll
        for (int w = 1; w < Tile::WM; ++w) top = fmaxf(top, most[w][n]);
        const float from = top == -INFINITY ? 0.0f : top;
        float s = 0;
#pragma unroll
        for (int w = 0; w < Tile::WM; ++w) s += total[w][n] * __builtin_amdgcn_exp2f((most[w][n] - from) * kLog2e);
        const uint64_t stretch = a.first / Tile::EM + tile.m;
        float* const to = a.partials + ((tile.rank * a.tiles + stretch) * a.rows + n0 + n) * 2;
        to[0] = top;
        to[1] = s;
    }
}

// lse and loss of 16 rows a workgroup at a time: 16 threads a row, each over
// every 16th tile of the vocabulary, then the 16 in order.
__global__ void __launch_bounds__(256) k_cross_loss(CrossArgs a) {
    __shared__ float most[16][17], total[16][17];
    const int rank = blockIdx.y, r = threadIdx.x % 16, part = threadIdx.x / 16;
    for (uint64_t first = blockIdx.x * 16ull; first < a.rows; first += gridDim.x * 16ull) {
        const uint64_t row = first + r;
        float top = -INFINITY, s = 0;
        if (row < a.rows) {
            const float* const from = a.partials + (static_cast<uint64_t>(rank) * a.tiles * a.rows + row) * 2;
#pragma unroll 8
            for (uint32_t t = part; t < a.tiles; t += 16) {
                const float2 each = *reinterpret_cast<const float2*>(from + t * a.rows * 2);
                const float x = each.x, y = each.y;
                const float higher = fmaxf(top, x), base = higher == -INFINITY ? 0.0f : higher;
                s = s * __builtin_amdgcn_exp2f((top - base) * kLog2e) + y * __builtin_amdgcn_exp2f((x - base) * kLog2e);
                top = higher;
            }
        }
        most[part][r] = top;
        total[part][r] = s;
        __syncthreads();
        if (part == 0 && row < a.rows) {
            for (int p = 1; p < 16; ++p) top = fmaxf(top, most[p][r]);
            const float base = top == -INFINITY ? 0.0f : top;
            s = 0;
            for (int p = 0; p < 16; ++p) s += total[p][r] * __builtin_amdgcn_exp2f((most[p][r] - base) * kLog2e);
            const float rest = __builtin_amdgcn_logf(s) * kLn2;
            a.lse[rank][row] = base + rest;
            const int64_t t = index_at(a.targets[rank], row, a.wide_index);
            float loss = as_f(0x7fc00000u);
            if (t == a.ignore) {
                loss = 0;
            } else if (t >= 0 && static_cast<uint64_t>(t) < a.vocab) {
                // not lse - z: where the logits are large, lse has rounded a small loss away
                loss = (base - a.target_logit[rank * a.rows + row]) + rest;
            }
            a.loss[rank][row] = loss;
        }
        __syncthreads();   // the next rows' maxima go to the same place
    }
}

// ---------------------------------------------------------------------------
// aligned copies
// ---------------------------------------------------------------------------

// Rows with zeros behind them, a vector of 16 bytes of the copy a thread: 3 x
// 5,003 rows of 515 float32, 11 us (5.6 TB/s).
template <int DT>
__global__ void __launch_bounds__(256) k_align(AlignArgs a) {
    constexpr int V = kOperandBytes / elem_size<DT>();
    const uint64_t each = a.to_stride / V, all = a.count * each;
    char* const to = a.to + static_cast<uint64_t>(blockIdx.y) * a.count * a.to_stride * elem_size<DT>();
    for (uint64_t i = blockIdx.x * 256ull + threadIdx.x; i < all; i += gridDim.x * 256ull) {
        // 32-bit division where it will do: it takes a fraction of the 64-bit one
        const uint64_t row = all >> 32 ? i / each : static_cast<uint32_t>(i) / static_cast<uint32_t>(each);
        const uint64_t c = (i - row * each) * V;
        Raw<DT, V> r;
        load_at<false, false>(r, a.from[blockIdx.y] + row * a.from_stride * elem_size<DT>(), c, a.cols);
        r.template store<false>(to + (row * a.to_stride + c) * elem_size<DT>());
    }
}

// ---------------------------------------------------------------------------
// backward
// ---------------------------------------------------------------------------

// The rows that take part, in order, with their g: one workgroup a rank.
__global__ void __launch_bounds__(1024) k_cross_live(CrossArgs a, float span) {
    __shared__ uint32_t counts[2][16];
    __shared__ float tops[16];
    const int rank = blockIdx.x, wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const auto weight = [&](uint64_t row) {
        return a.dloss[rank] != nullptr ? a.scale * a.dloss[rank][row] : a.scale;
    };
    // The g of a 16-bit dz are relative to the largest finite |g|, which becomes
    // `span`: rows that count alike lose nothing by g's own rounding, and binary16
    // keeps small ones.  span 0 (float32): g as it is.
    float largest = 1.0f;
    if (span > 0) {
        float top = 0;
        for (uint64_t row = threadIdx.x; row < a.rows; row += 1024) {
            const float g = fabsf(weight(row));
            if (g < INFINITY && index_at(a.targets[rank], row, a.wide_index) != a.ignore) top = fmaxf(top, g);
        }
        top = as_f(max_over_lanes<64>(as_u(top)));   // not negative: ordered as integers are
        if (lane == 0) tops[wave] = top;
        __syncthreads();
        for (int w = 0; w < 16; ++w) top = fmaxf(top, tops[w]);
        if (top > 0) largest = top;
    }
    if (threadIdx.x == 0) a.unscale[rank] = span > 0 ? largest / span : 1.0f;
    uint32_t before = 0;
    int turn = 0;
    for (uint64_t first = 0; first < a.rows; first += 1024) {
        const uint64_t row = first + threadIdx.x;
        LiveRow r{};
        bool live = false;
        if (row < a.rows) {
            const int64_t t = index_at(a.targets[rank], row, a.wide_index);
            r.g = weight(row);
            live = t != a.ignore && r.g != 0;
            const bool known = t >= 0 && static_cast<uint64_t>(t) < a.vocab;
            r.target = known ? t : -1;
            if (span > 0) r.g = r.g / largest * span;
            if (!known) r.g = as_f(0x7fc00000u);
            r.lse = a.lse_in[rank][row];
        }
        const uint64_t mask = __ballot(live);
        if (lane == 0) counts[turn][wave] = __popcll(mask);
        __syncthreads();
        uint32_t at = before + __popcll(mask & ((1ull << lane) - 1));
        for (int w = 0; w < 16; ++w) {
            if (w < wave) at += counts[turn][w];
            before += counts[turn][w];
        }
        turn ^= 1;   // the next turn's counts go elsewhere: one barrier a turn
        if (live) a.live[rank * a.rows + at] = r;
        if (row < a.rows) a.place[rank * a.rows + row] = live ? at : ~0u;
    }
    if (threadIdx.x == 0) a.live_count[rank] = before;
}

// The live rows of x, one after another with zeros behind each: a copy, 24 us
// for 2 x 4,096 rows of 4,096 bf16 (5.3 TB/s).
template <int DT>
__global__ void __launch_bounds__(256) k_cross_gather(CrossArgs a, uint64_t padded) {
    constexpr int V = kOperandBytes / elem_size<DT>();
    const int rank = blockIdx.y;
    for (uint64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const uint32_t place = a.place[rank * a.rows + row];
        if (place == ~0u) continue;
        const char* const from = a.x[rank] + row * a.x_stride * elem_size<DT>();
        char* const to = a.x_live + (rank * a.rows + place) * padded * elem_size<DT>();
        for (uint64_t c = threadIdx.x * V; c < padded; c += 256 * V) {
            Raw<DT, V> r;
            load_at<false, false>(r, from, c, a.cols);
            r.template store<false>(to + c * elem_size<DT>());
        }
    }
}

// dz of a piece's columns: [live row][piece], zeros behind the vocabulary's end.
template <int DT, class Tile, bool WHOLE>
__global__ void __launch_bounds__(Tile::kThreads) k_cross_dz(CrossArgs a, uint64_t padded, uint32_t tiles_m,
                                                             uint32_t ranks) {
    __shared__ __attribute__((aligned(1024))) char buffers[Tile::kShared];
    const TilePlace tile(blockIdx.x, tiles_m, a.live_count, Tile::EN, 1, ranks);
    if (!tile.valid) return;
    constexpr int kEs = elem_size<DT>();
    const uint64_t live = a.live_count[tile.rank];
    const uint64_t m0 = static_cast<uint64_t>(tile.m) * Tile::EM, n0 = static_cast<uint64_t>(tile.n) * Tile::EN;
    f32x4 sum[Tile::TM][Tile::TN];
    // a tile past the vocabulary's end (the piece is padded) has its last row for all
    product<DT, Tile, WHOLE, true, true>(buffers, a.weight[tile.rank], a.weight_stride * kEs, m0, a.count,
                                  a.x_live + tile.rank * a.rows * padded * kEs, padded * kEs, n0, live, a.cols, sum);
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const uint64_t first = m0 + (wave / Tile::WN) * Tile::TM * kSquare + 4 * (lane >> 4);
#pragma unroll
    for (int j = 0; j < Tile::TN; ++j) {
        const uint64_t n = n0 + ((wave % Tile::WN) * Tile::TN + j) * kSquare + (lane & 15);
        if (n >= live) continue;
        const LiveRow row = a.live[tile.rank * a.rows + n];
        const int64_t target = row.target - static_cast<int64_t>(a.first + first);
        char* const to = a.dz + ((tile.rank * a.rows + n) * a.piece + first) * kEs;
#pragma unroll
        for (int i = 0; i < Tile::TM; ++i) {
            float d[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int m = i * kSquare + k;
                float p = __builtin_amdgcn_exp2f((sum[i][j][k] - row.lse) * kLog2e);
                if (target == m) p -= 1.0f;
                d[k] = first + m < a.count ? row.g * p : 0.0f;
            }
            Raw<DT, 4> r;
            r.set_all(d);
            r.template store<false>(to + i * kSquare * kEs);
        }
    }
}

// A piece's part of dx's sums: [split][live row][column].
template <int DT, class Tile, bool WHOLE>
__global__ void __launch_bounds__(Tile::kThreads) k_cross_dx(CrossArgs a, int add, uint32_t tiles_m, uint32_t ranks) {
    __shared__ __attribute__((aligned(1024))) char buffers[Tile::kShared];
    const TilePlace tile(blockIdx.x, tiles_m, a.live_count, Tile::EN, a.splits, ranks);
    if (!tile.valid) return;
    constexpr int kEs = elem_size<DT>();
    const uint32_t rank = tile.rank, split = tile.part;
    const uint64_t live = a.live_count[rank];
    const uint64_t m0 = static_cast<uint64_t>(tile.m) * Tile::EM, n0 = static_cast<uint64_t>(tile.n) * Tile::EN;
    // this split's columns of the piece, whole tiles of the vocabulary
    const uint64_t blocks = a.piece / kVocabTile;
    const uint64_t from = blocks * split / a.splits * kVocabTile;
    const uint64_t end = std::min(a.count, blocks * (split + 1) / a.splits * kVocabTile);
    const uint64_t depth = end > from ? end - from : 0;
    f32x4 sum[Tile::TM][Tile::TN];
    product<DT, Tile, WHOLE, false, true>(buffers, a.weight[rank] + from * a.weight_stride * kEs, a.weight_stride * kEs, m0,
                                   a.cols, a.dz + (rank * a.rows * a.piece + from) * kEs, a.piece * kEs, n0, live, depth,
                                   sum);
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const uint64_t first = m0 + (wave / Tile::WN) * Tile::TM * kSquare + 4 * (lane >> 4);
    const uint64_t width = (a.cols + 3) / 4 * 4;
#pragma unroll
    for (int j = 0; j < Tile::TN; ++j) {
        const uint64_t n = n0 + ((wave % Tile::WN) * Tile::TN + j) * kSquare + (lane & 15);
        if (n >= live) continue;
        float* const to = a.sums + ((static_cast<uint64_t>(rank) * a.splits + split) * a.rows + n) * width + first;
#pragma unroll
        for (int i = 0; i < Tile::TM; ++i) {
            if (first + i * kSquare >= a.cols) continue;
            f32x4* const p = reinterpret_cast<f32x4*>(to + i * kSquare);
            *p = add ? sum[i][j] + *p : sum[i][j];
        }
    }
}

// A piece's rows of dweight.
template <int DT, class Tile>
__global__ void __launch_bounds__(Tile::kThreads) k_cross_dweight(CrossArgs a, uint64_t padded, uint32_t tiles_m,
                                                                  uint32_t tiles_n, uint32_t ranks) {
    __shared__ __attribute__((aligned(1024))) char buffers[Tile::kShared];
    const TilePlace tile(blockIdx.x, tiles_m, tiles_n, ranks);
    if (!tile.valid) return;
    constexpr int kEs = elem_size<DT>();
    const uint64_t m0 = static_cast<uint64_t>(tile.m) * Tile::EM, n0 = static_cast<uint64_t>(tile.n) * Tile::EN;
    f32x4 sum[Tile::TM][Tile::TN];
    product<DT, Tile, true, false, false>(buffers, a.x_live + tile.rank * a.rows * padded * kEs, padded * kEs, m0, a.cols,
                                    a.dz + tile.rank * a.rows * a.piece * kEs, a.piece * kEs, n0, a.count,
                                    a.live_count[tile.rank], sum);
    const float unscale = a.unscale[tile.rank];
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const uint64_t first = m0 + (wave / Tile::WN) * Tile::TM * kSquare + 4 * (lane >> 4);
#pragma unroll
    for (int j = 0; j < Tile::TN; ++j) {
        const uint64_t n = n0 + ((wave % Tile::WN) * Tile::TN + j) * kSquare + (lane & 15);
        if (n >= a.count) continue;
        char* const to = a.dweight[tile.rank] + (a.first + n) * a.dweight_stride * kEs;
#pragma unroll
        for (int i = 0; i < Tile::TM; ++i) {
            float d[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) d[k] = sum[i][j][k] * unscale;
            Raw<DT, 4> r;
            r.set_all(d);
            store_at<false, false>(r, to, first + i * kSquare, a.cols);
        }
    }
}

// dx from its sums; 0 for the rows that take no part.
template <int DT>
__global__ void __launch_bounds__(256) k_cross_finish(CrossArgs a) {
    const int rank = blockIdx.y;
    const uint64_t width = (a.cols + 3) / 4 * 4;
    const float unscale = a.unscale[rank];
    for (uint64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const uint32_t place = a.place[rank * a.rows + row];
        char* const to = a.dx[rank] + row * a.dx_stride * elem_size<DT>();
        for (uint64_t c = threadIdx.x * 4; c < a.cols; c += 1024) {
            f32x4 v = {0, 0, 0, 0};
            if (place != ~0u) {
                for (uint32_t s = 0; s < a.splits; ++s)
                    v += *reinterpret_cast<const f32x4*>(
                        a.sums + ((static_cast<uint64_t>(rank) * a.splits + s) * a.rows + place) * width + c);
            }
            const float d[4] = {v.x * unscale, v.y * unscale, v.z * unscale, v.w * unscale};
            Raw<DT, 4> r;
            r.set_all(d);
            store_at<false, true>(r, to, c, a.cols);
        }
    }
}

// ---------------------------------------------------------------------------
// launches
// ---------------------------------------------------------------------------

constexpr uint64_t kMostBlocks = 1u << 16;

uint32_t tiles_of(uint64_t n, int tile) { return static_cast<uint32_t>((n + tile - 1) / tile); }

template <class Tile>
constexpr bool is_tile(CrossTile t) {
    return static_cast<uint64_t>(Tile::EM) == tile_m(t) && static_cast<uint64_t>(Tile::EN) == tile_n(t) &&
           static_cast<uint64_t>(Tile::kThreads) == tile_threads(t);
}
// Workgroups of one launch, which the host keeps to.
template <class Tile>
constexpr uint64_t kMostTiles = 0xffffffffull / Tile::kThreads;
static_assert(kMostStride == kMostOperandStride && kCrossRanks <= 64, "the host's operands");
static_assert(is_tile<LargeTile>(CrossTile::kLarge) && is_tile<MediumTile>(CrossTile::kMedium) &&
                  is_tile<SmallTile>(CrossTile::kSmall) && is_tile<TinyTile<AR_FLOAT32>>(CrossTile::kTiny),
              "the host's tiles");

// f(WHOLE), and what the launch says.  Few rows (in_words) never get a tile wider
// than they are: one that is costs more in any number of tiles.
template <int DT, class Tile, class F>
hipError_t by_rows(const CrossArgs& a, const F& f) {
    constexpr bool kWords = DT == AR_FLOAT32 && Tile::EN <= static_cast<int>(kWordRows);
    if constexpr (kWords) {
        if (!a.whole) {
            f(std::false_type{});
            return hipGetLastError();
        }
    }
    if (!a.whole) return hipErrorInvalidValue;
    f(std::true_type{});
    return hipGetLastError();
}

template <int DT, class Tile>
hipError_t start_stats(const CrossArgs& a, int nranks, hipStream_t s) {
    const uint32_t tiles_m = tiles_of(a.count, Tile::EM), tiles_n = tiles_of(a.rows, Tile::EN);
    const uint64_t blocks = tile_blocks(static_cast<uint64_t>(tiles_m) * tiles_n * nranks);
    if (blocks > kMostTiles<Tile>) return hipErrorInvalidValue;
    return by_rows<DT, Tile>(a, [&](auto whole) {
        hipLaunchKernelGGL((k_cross_stats<DT, Tile, whole.value>), dim3(static_cast<unsigned>(blocks)),
                           dim3(Tile::kThreads), 0, s, a, tiles_m, tiles_n, static_cast<uint32_t>(nranks));
    });
}

template <int DT>
hipError_t start_live(const CrossArgs& a, int nranks, hipStream_t s) {
    hipLaunchKernelGGL(k_cross_live, dim3(nranks), dim3(1024), 0, s, a,
                       DT == AR_FLOAT16 ? 8192.0f : DT == AR_BFLOAT16 ? 1.0f : 0.0f);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || a.rows == 0) return e;
    const dim3 grid(static_cast<unsigned>(std::min(a.rows, kMostBlocks)), nranks);
    hipLaunchKernelGGL((k_cross_gather<DT>), grid, dim3(256), 0, s, a, padded_cols(a.cols, elem_size<DT>()));
    return hipGetLastError();
}

template <int DT, class Tile>
hipError_t start_dz(const CrossArgs& a, int nranks, hipStream_t s) {
    const uint32_t tiles_m = tiles_of(a.piece, Tile::EM), tiles_n = tiles_of(a.rows, Tile::EN);
    const uint64_t blocks = tile_blocks(static_cast<uint64_t>(tiles_m) * tiles_n * nranks);
    if (blocks > kMostTiles<Tile>) return hipErrorInvalidValue;
    return by_rows<DT, Tile>(a, [&](auto whole) {
        hipLaunchKernelGGL((k_cross_dz<DT, Tile, whole.value>), dim3(static_cast<unsigned>(blocks)),
                           dim3(Tile::kThreads), 0, s, a, padded_cols(a.cols, elem_size<DT>()), tiles_m,
                           static_cast<uint32_t>(nranks));
    });
}

template <int DT, class Tile>
hipError_t start_dx(const CrossArgs& a, int nranks, bool add, hipStream_t s) {
    const uint32_t tiles_m = tiles_of(a.cols, Tile::EM), tiles_n = tiles_of(a.rows, Tile::EN);
    const uint64_t blocks = tile_blocks(static_cast<uint64_t>(tiles_m) * tiles_n * nranks * a.splits);
    if (blocks > kMostTiles<Tile>) return hipErrorInvalidValue;
    return by_rows<DT, Tile>(a, [&](auto whole) {
        hipLaunchKernelGGL((k_cross_dx<DT, Tile, whole.value>), dim3(static_cast<unsigned>(blocks)),
                           dim3(Tile::kThreads), 0, s, a, add ? 1 : 0, tiles_m, static_cast<uint32_t>(nranks));
    });
}

template <int DT, class Tile>
hipError_t start_dweight(const CrossArgs& a, int nranks, hipStream_t s) {
    const uint32_t tiles_m = tiles_of(a.cols, Tile::EM), tiles_n = tiles_of(a.count, Tile::EN);
    const uint64_t blocks = tile_blocks(static_cast<uint64_t>(tiles_m) * tiles_n * nranks);
    if (blocks > kMostTiles<Tile>) return hipErrorInvalidValue;
    hipLaunchKernelGGL((k_cross_dweight<DT, Tile>), dim3(static_cast<unsigned>(blocks)), dim3(Tile::kThreads), 0, s, a,
                       padded_cols(a.cols, elem_size<DT>()), tiles_m, tiles_n, static_cast<uint32_t>(nranks));
    return hipGetLastError();
}

template <int DT>
hipError_t start_align(const AlignArgs& a, int nranks, hipStream_t s) {
    const uint64_t vectors = a.count * (a.to_stride * elem_size<DT>() / kOperandBytes);
    if (vectors == 0) return hipSuccess;
    const dim3 grid(static_cast<unsigned>(std::min((vectors + 255) / 256, kMostBlocks)), nranks);
    hipLaunchKernelGGL((k_align<DT>), grid, dim3(256), 0, s, a);
    return hipGetLastError();
}

template <int DT>
hipError_t start_finish(const CrossArgs& a, int nranks, hipStream_t s) {
    const dim3 grid(static_cast<unsigned>(std::min(a.rows, kMostBlocks)), nranks);
    hipLaunchKernelGGL((k_cross_finish<DT>), grid, dim3(256), 0, s, a);
    return hipGetLastError();
}

// an expression with DT, a floating dtype
#define AR_BY_DTYPE(dtype, ...)                                                   \
    switch (dtype) {                                                              \
        case AR_FLOAT32: { constexpr int DT = AR_FLOAT32; return __VA_ARGS__; }   \
        case AR_BFLOAT16: { constexpr int DT = AR_BFLOAT16; return __VA_ARGS__; } \
        case AR_FLOAT16: { constexpr int DT = AR_FLOAT16; return __VA_ARGS__; }   \
        default: return hipErrorInvalidValue;                                     \
    }
template <int DT, class F>
hipError_t by_tile(CrossTile tile, const F& start) {
    switch (tile) {
        case CrossTile::kLarge: return start(LargeTile{});
        case CrossTile::kMedium: return start(MediumTile{});
        case CrossTile::kSmall: return start(SmallTile{});
        case CrossTile::kTiny: return start(TinyTile<DT>{});
    }
    return hipErrorInvalidValue;
}

}  // namespace

hipError_t launch_align(const AlignArgs& a, int nranks, ar_dtype_t dtype, hipStream_t s) {
    AR_BY_DTYPE(dtype, start_align<DT>(a, nranks, s))
}
hipError_t launch_cross_stats(const CrossArgs& a, int nranks, CrossTile tile, ar_dtype_t dtype, hipStream_t s) {
    AR_BY_DTYPE(dtype, by_tile<DT>(tile, [&](auto t) {
                    return start_stats<DT, decltype(t)>(a, nranks, s);
                }))
}
hipError_t launch_cross_loss(const CrossArgs& a, int nranks, hipStream_t s) {
    const uint64_t blocks = std::min<uint64_t>(tiles_of(a.rows, 16), 16 * kMostBlocks);
    hipLaunchKernelGGL(k_cross_loss, dim3(static_cast<unsigned>(blocks), nranks), dim3(256), 0, s, a);
    return hipGetLastError();
}
hipError_t launch_cross_live(const CrossArgs& a, int nranks, ar_dtype_t dtype, hipStream_t s) {
    AR_BY_DTYPE(dtype, start_live<DT>(a, nranks, s))
}
hipError_t launch_cross_dz(const CrossArgs& a, int nranks, ar_dtype_t dtype, hipStream_t s) {
    AR_BY_DTYPE(dtype, by_tile<DT>(pick_tile(a.piece, a.rows, nranks, dtype == AR_FLOAT32), [&](auto t) {
                    return start_dz<DT, decltype(t)>(a, nranks, s);
                }))
}
hipError_t launch_cross_dx(const CrossArgs& a, int nranks, bool add, CrossTile tile, ar_dtype_t dtype, hipStream_t s) {
    AR_BY_DTYPE(dtype, by_tile<DT>(tile, [&](auto t) {
                    return start_dx<DT, decltype(t)>(a, nranks, add, s);
                }))
}
hipError_t launch_cross_dweight(const CrossArgs& a, int nranks, ar_dtype_t dtype, hipStream_t s) {
    AR_BY_DTYPE(dtype, by_tile<DT>(pick_tile(a.cols, a.count, nranks, dtype == AR_FLOAT32), [&](auto t) {
                    return start_dweight<DT, decltype(t)>(a, nranks, s);
                }))
}
hipError_t launch_cross_finish(const CrossArgs& a, int nranks, ar_dtype_t dtype, hipStream_t s) {
    AR_BY_DTYPE(dtype, start_finish<DT>(a, nranks, s))
}

}  // namespace arimpl
