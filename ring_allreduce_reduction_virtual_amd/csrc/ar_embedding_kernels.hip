// HIP kernels of the embedding lookup and of its gradient (include/ar.h states
// the formulas).
//
// The lookup copies rows: the table's rows that tokens name are read, each row
// of the output is written once (8 x 4,096 tokens of 4,096 bf16 80 us, 5.6 TB/s
// of the 450 MB that reach memory).
//
// The gradient is a sum by token whose order must not depend on which
// workgroup comes first, so no row is added to with atomics.  The places are
// sorted by token, stably; the sorted order is cut into chunks of 8 or 32
// places, and a group of threads adds up each chunk's rows of dy.  A token
// whose places lie within one chunk is done there.  One that crosses a chunk's
// end leaves a partial sum in each chunk, so that in this launch a frequent
// token is spread over as many groups as it has chunks; a second launch joins
// the partial sums in order, one wavefront for a token's 256 columns, whose
// chain grows with the token's places (a rank's 32,768 places under a 1/k law
// 169 us for the whole gradient, all of one token 468).  The launch that sums also
// writes the zeros of rows that no token names.  Writing the table bounds it: 8 x
// 4,096 tokens into 8 x 32,768 rows of 4,096 bf16, 424 us for 2.4 GB (5.7 TB/s),
// the sort 12.6 and the join 14.8.

#include <hip/hip_runtime.h>

#include <type_traits>

#include "ar_embedding.h"
#include "ar_step_device.h"

namespace arimpl {
namespace {

__device__ __forceinline__ int64_t token_at(const char* tokens, uint64_t i, int wide) {
    return wide ? reinterpret_cast<const int64_t*>(tokens)[i] : reinterpret_cast<const int32_t*>(tokens)[i];
}

// Threads of a row: rows of up to 64 vectors of V elements have several to a wavefront.
template <int TPR>
constexpr int kRowsAtOnce = 256 / TPR;

template <int DT, int TDT, int TPR>
__global__ void __launch_bounds__(256) k_embedding(EmbeddingArgs a) {
    constexpr int V = 16 / elem_size<DT>();
    const int rank = blockIdx.y;
    const uint64_t step = static_cast<uint64_t>(gridDim.x) * kRowsAtOnce<TPR>;
    for (uint64_t row = static_cast<uint64_t>(blockIdx.x) * kRowsAtOnce<TPR> + threadIdx.x / TPR; row < a.rows;
         row += step) {
        const int64_t t = token_at(a.tokens[rank], row, a.wide_index);
        const bool known = t >= 0 && static_cast<uint64_t>(t) < a.vocab;
        const char* const from = a.table[rank] + (known ? static_cast<uint64_t>(t) : 0) * a.table_stride * elem_size<TDT>();
        char* const to = a.out[rank] + row * a.out_stride * elem_size<DT>();
        for (uint64_t c = (threadIdx.x % TPR) * V; c < a.cols; c += TPR * V) {
            Raw<TDT, V> r;
            if (known) load_at<false, false>(r, from, c, a.cols);
            float x[V];
#pragma unroll
            for (int j = 0; j < V; ++j) x[j] = known ? r.get(j) * a.scale : as_f(0x7fc00000u);
            Raw<DT, V> o;
            o.set_all(x);
            store_at<false, true>(o, to, c, a.cols);
        }
    }
}

// ---------------------------------------------------------------------------
// the sort
// ---------------------------------------------------------------------------

// A place's key: its token, or vocab (behind all tokens) when it takes no part.
__device__ __forceinline__ uint32_t key_at(const EmbeddingBackwardArgs& a, int rank, uint64_t i) {
    const int64_t t = token_at(a.tokens[rank], i, a.wide_index);
    const bool part = t >= 0 && static_cast<uint64_t>(t) < a.vocab && t != a.padding;
    return static_cast<uint32_t>(part ? static_cast<uint64_t>(t) : a.vocab);
}

// The lanes of the wavefront whose digit is this lane's.
__device__ __forceinline__ uint64_t same_digit(uint32_t digit, int bits) {
    uint64_t same = ~0ull;
    for (int b = 0; b < bits; ++b) {
        const bool set = (digit >> b) & 1u;
        const uint64_t with = __ballot(set);
        same &= set ? with : ~with;
    }
    return same;
}

// How many places of the wavefront's so far have this digit, this lane's among
// the lanes below it; `count` is the wavefront's own row of counters.
__device__ __forceinline__ uint32_t take_rank(uint32_t* count, uint32_t digit, int bits) {
    const uint64_t same = same_digit(digit, bits);
    const uint32_t below = __popcll(same & ((1ull << (threadIdx.x & 63)) - 1));
    const uint32_t before = count[digit];
    // every lane has read before the first lane of each digit writes
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    if (below == 0) count[digit] = before + __popcll(same);
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    return before + below;
}

// Sum of the wavefront's values up to and with this lane's.
__device__ __forceinline__ uint32_t sum_to_lane(uint32_t x) {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const uint32_t y = __shfl_up(x, d, 64);
        if (lane >= d) x += y;
    }
    return x;
}

// Turns the wavefronts' counters into what precedes each wavefront's places of
// a digit, and `digits` into what precedes the digit.  Called by all threads of
// the workgroup, with at least kDigits of them or a loop over the rest.
template <int THREADS>
__device__ __forceinline__ void scan_counts(uint32_t (*count)[kDigits], uint32_t* digits, uint32_t* totals) {
    constexpr int kWaves = THREADS / 64;
    uint32_t carry = 0;
    for (int d0 = 0; d0 < kDigits; d0 += THREADS) {
        const int d = d0 + static_cast<int>(threadIdx.x);
        uint32_t sum = 0;
        if (d < kDigits) {
#pragma unroll
            for (int w = 0; w < kWaves; ++w) {
                const uint32_t c = count[w][d];
                count[w][d] = sum;
                sum += c;
            }
        }
        const uint32_t to = sum_to_lane(sum);
        if ((threadIdx.x & 63) == 63) totals[threadIdx.x >> 6] = to;
        __syncthreads();
        uint32_t before = carry;
        for (int w = 0; w < kWaves; ++w) {
            if (w < static_cast<int>(threadIdx.x >> 6)) before += totals[w];
            carry += totals[w];
        }
        if (d < kDigits) digits[d] = before + to - sum;
        __syncthreads();
    }
}

// One rank's places in one workgroup, EACH a thread, all passes (4,096 places
// of 16-bit tokens on each of 8 ranks: 12 us).
template <int EACH>
__global__ void __launch_bounds__(kSortThreads) k_sort_one(EmbeddingBackwardArgs a) {
    constexpr int kWaves = kSortThreads / 64;
    __shared__ uint32_t count[kWaves][kDigits];
    __shared__ uint32_t digits[kDigits], totals[kWaves];
    __shared__ uint32_t keys[kSortThreads * EACH];
    __shared__ uint16_t places[kSortThreads * EACH];
    static_assert(kSortThreads * EACH <= 65536, "places of 16 bits");
    const int rank = blockIdx.x, wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const uint32_t n = static_cast<uint32_t>(a.rows);
    uint32_t key[EACH], place[EACH], at[EACH];
#pragma unroll
    for (int i = 0; i < EACH; ++i) {
        place[i] = (wave * EACH + i) * 64 + lane;
        key[i] = place[i] < n ? key_at(a, rank, place[i]) : 0xffffffffu;   // stays behind all others
    }
    const uint32_t mask = (1u << a.digit_bits) - 1;
    for (int pass = 0; pass < a.passes; ++pass) {
        const int shift = pass * a.digit_bits;
        for (int d = threadIdx.x; d < kWaves * kDigits; d += kSortThreads) (&count[0][0])[d] = 0;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < EACH; ++i) at[i] = take_rank(count[wave], (key[i] >> shift) & mask, a.digit_bits);
        __syncthreads();
        scan_counts<kSortThreads>(count, digits, totals);
#pragma unroll
        for (int i = 0; i < EACH; ++i) {
            const uint32_t d = (key[i] >> shift) & mask;
            const uint32_t to = digits[d] + count[wave][d] + at[i];
            keys[to] = key[i];
            places[to] = static_cast<uint16_t>(place[i]);
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < EACH; ++i) {
            const uint32_t from = (wave * EACH + i) * 64 + lane;
            key[i] = keys[from];
            place[i] = places[from];
        }
        __syncthreads();
    }
    uint32_t* const keys_to = a.keys + rank * sort_words(a.rows);
    uint32_t* const places_to = a.places + rank * sort_words(a.rows);
#pragma unroll
    for (int i = 0; i < EACH; ++i) {
        const uint32_t to = (wave * EACH + i) * 64 + lane;
        if (to < n) {
            keys_to[to] = key[i];
            places_to[to] = place[i];
        }
    }
}

// The key of a pass's i-th place: from the tokens, or from the pass before.
__device__ __forceinline__ uint32_t pass_key(const EmbeddingBackwardArgs& a, int rank, int pass, uint64_t i) {
    if (pass == 0) return key_at(a, rank, i);
    return a.keys[rank * sort_words(a.rows) + ((pass - 1) & 1) * a.rows + i];
}

__global__ void __launch_bounds__(kSortTileThreads) k_sort_count(EmbeddingBackwardArgs a, int pass) {
    __shared__ uint32_t count[kDigits];
    const int rank = blockIdx.y;
    const uint64_t tile = blockIdx.x;
    for (int d = threadIdx.x; d < kDigits; d += kSortTileThreads) count[d] = 0;
    __syncthreads();
    const uint32_t mask = (1u << a.digit_bits) - 1;
#pragma unroll
    for (int i = 0; i < kSortTileEach; ++i) {
        const uint64_t at = tile * kSortTile + i * kSortTileThreads + threadIdx.x;
        if (at < a.rows) atomicAdd(&count[(pass_key(a, rank, pass, at) >> (pass * a.digit_bits)) & mask], 1u);
    }
    __syncthreads();
    uint32_t* const to = a.counts + rank * a.tiles * kDigits + tile;
    for (int d = threadIdx.x; d < kDigits; d += kSortTileThreads) to[d * a.tiles] = count[d];
}

// Each count becomes the sum of those before it, digit by digit and tile by tile.
__global__ void __launch_bounds__(1024) k_sort_scan(EmbeddingBackwardArgs a) {
    __shared__ uint32_t totals[2][16];
    uint32_t* const count = a.counts + blockIdx.x * a.tiles * kDigits;
    const uint64_t n = a.tiles * kDigits;
    uint32_t carry = 0;
    int turn = 0;
    for (uint64_t first = 0; first < n; first += 4096) {
        uint32_t x[4], sum = 0;
        const uint64_t at = first + threadIdx.x * 4;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            x[k] = at + k < n ? count[at + k] : 0;
            sum += x[k];
        }
        const uint32_t to = sum_to_lane(sum);
        if ((threadIdx.x & 63) == 63) totals[turn][threadIdx.x >> 6] = to;
        __syncthreads();
        uint32_t before = carry + to - sum;
        for (int w = 0; w < 16; ++w) {
            if (w < static_cast<int>(threadIdx.x >> 6)) before += totals[turn][w];
            carry += totals[turn][w];
        }
        turn ^= 1;   // the next turn's totals go elsewhere: one barrier a turn
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if (at + k < n) count[at + k] = before;
            before += x[k];
        }
    }
}

__global__ void __launch_bounds__(kSortTileThreads) k_sort_place(EmbeddingBackwardArgs a, int pass) {
    constexpr int kWaves = kSortTileThreads / 64;
    __shared__ uint32_t count[kWaves][kDigits];
    const int rank = blockIdx.y, wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const uint64_t tile = blockIdx.x;
    uint32_t key[kSortTileEach], at[kSortTileEach];
    for (int d = threadIdx.x; d < kWaves * kDigits; d += kSortTileThreads) (&count[0][0])[d] = 0;
    __syncthreads();
    const uint32_t mask = (1u << a.digit_bits) - 1;
    const int shift = pass * a.digit_bits;
    const uint64_t first = tile * kSortTile + wave * kSortTileEach * 64 + lane;
#pragma unroll
    for (int i = 0; i < kSortTileEach; ++i)
        key[i] = first + i * 64 < a.rows ? pass_key(a, rank, pass, first + i * 64) : 0xffffffffu;
#pragma unroll
    for (int i = 0; i < kSortTileEach; ++i) {
        // past the last place: of the last digit, behind all others of the last tile
        at[i] = take_rank(count[wave], (key[i] >> shift) & mask, a.digit_bits);
    }
    __syncthreads();
    const uint32_t* const starts = a.counts + rank * a.tiles * kDigits + tile;
    for (int d = threadIdx.x; d < kDigits; d += kSortTileThreads) {
        uint32_t sum = starts[d * a.tiles];
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
            const uint32_t c = count[w][d];
            count[w][d] = sum;
            sum += c;
        }
    }
    __syncthreads();
    const uint64_t part = rank * sort_words(a.rows);
    const uint32_t* const places_from = a.places + part + ((pass + 1) & 1) * a.rows;
    uint32_t* const keys_to = a.keys + part + (pass & 1) * a.rows;
    uint32_t* const places_to = a.places + part + (pass & 1) * a.rows;
#pragma unroll
    for (int i = 0; i < kSortTileEach; ++i) {
        const uint64_t from = first + i * 64;
        if (from < a.rows) {
            const uint32_t to = count[wave][(key[i] >> shift) & mask] + at[i];
            keys_to[to] = key[i];
            places_to[to] = pass == 0 ? static_cast<uint32_t>(from) : places_from[from];
        }
    }
}

// ---------------------------------------------------------------------------
// the sums
// ---------------------------------------------------------------------------

template <int DT>
constexpr int kSumVec = 16 / elem_size<DT>();

// First place of the sorted keys that is not below v.
__device__ __forceinline__ uint64_t lower_bound(const uint32_t* keys, uint64_t n, uint32_t v) {
    uint64_t lo = 0;
    while (n > 0) {
        const uint64_t half = n / 2;
        const bool below = keys[lo + half] < v;
        lo = below ? lo + half + 1 : lo;
        n = below ? n - half - 1 : half;
    }
    return lo;
}

// A token's sums of V columns from c on, all but the first `skip` of them, to
// its row; a row of fewer than V columns up to its end.
template <int DT, int V>
__device__ __forceinline__ void write_row(const EmbeddingBackwardArgs& a, int rank, uint32_t token, uint64_t c, int skip,
                                          const float (&sum)[V]) {
    char* const to = a.dtable[rank] + token * a.dtable_stride * elem_size<DT>();
    float x[V];
#pragma unroll
    for (int j = 0; j < V; ++j) x[j] = sum[j] * a.scale;
    Raw<DT, V> r;
    if (a.accumulate) {
        load_at<false, false>(r, to, c, a.cols);
#pragma unroll
        for (int j = 0; j < V; ++j) x[j] += r.get(j);
    }
    r.set_all(x);
    if (skip == 0) {
        store_at<false, true>(r, to, c, a.cols);
    } else {
        r.store_from(to + c * elem_size<DT>(), skip);
    }
}

__device__ __forceinline__ float* partial_at(const EmbeddingBackwardArgs& a, int rank, uint64_t chunk, int which) {
    return a.partials + ((rank * a.chunks + chunk) * 2 + which) * a.cols;
}

// A wavefront's zeros, `n` elements from p: 16 bytes a lane from the first
// address that they fit, the elements before and behind one by one.
template <int DT>
__device__ __forceinline__ void write_zeros(char* p, uint64_t n) {
    constexpr int kEs = elem_size<DT>(), V = 16 / kEs;
    const uint32_t lane = threadIdx.x & 63;
    const uint32_t head = static_cast<uint32_t>((16 - (reinterpret_cast<uintptr_t>(p) & 15)) % 16 / kEs);
    if (n < V + head) {
        if (lane < n) store_elem<kEs, false>(p + lane * kEs, 0);
        return;
    }
    const uint64_t body = (n - head) / V * V;
    const uint32_t tail = static_cast<uint32_t>(n - head - body);
    const u32x4 zero = {0, 0, 0, 0};
    for (uint64_t c = lane * V; c < body; c += 64 * V) store16<false>(p + (head + c) * kEs, zero);
    if (lane < head) store_elem<kEs, false>(p + lane * kEs, 0);
    if (lane < tail) store_elem<kEs, false>(p + (head + body + lane) * kEs, 0);
}

// Rows of the table that a workgroup looks at, a quarter of them a wavefront.
// Measured, a table of 8 x 32,768 rows of 4,096 bf16 for 5 tokens (2.1 GB of
// zeros, which torch's fill writes in 315 us): 357 us; whole workgroups on a row
// at a time 371, with 32 rows 391, with 64 420, with nontemporal stores 392.
constexpr uint64_t kZeroRows = 16;

// Workgroups in turn: the ranks (neighbouring workgroups write different
// buffers), stretches of TPR * V columns, chunks, one for each group of TPR
// threads; behind all of these, rows of the table without a token, whole rows
// for a wavefront.
template <int DT, int TDT, int TPR>
__global__ void __launch_bounds__(256) k_embedding_sums(EmbeddingBackwardArgs a, uint32_t nranks, uint32_t stretches,
                                                        uint32_t sum_blocks, uint32_t zero_blocks) {
    constexpr int V = kSumVec<DT>;
    constexpr int kAhead = 8;   // rows on their way
    const uint32_t rank = blockIdx.x % nranks, turn = blockIdx.x / nranks;
    const uint32_t* const keys = a.keys + rank * sort_words(a.rows) + a.sorted * a.rows;
    const uint32_t* const places = a.places + rank * sort_words(a.rows) + a.sorted * a.rows;
    const uint32_t vocab = static_cast<uint32_t>(a.vocab);
    if (turn >= sum_blocks * stretches) {
        constexpr int kWaveRows = kZeroRows / 4;
        const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
        for (uint64_t first = (turn - sum_blocks * stretches) * kZeroRows + wave * kWaveRows; first < a.vocab;
             first += zero_blocks * kZeroRows) {
            bool empty = false;
            if (lane < kWaveRows && first + lane < a.vocab) {
                const uint32_t v = static_cast<uint32_t>(first + lane);
                const uint64_t at = lower_bound(keys, a.rows, v);
                empty = at >= a.rows || keys[at] != v;
            }
            for (uint64_t rows = __ballot(empty); rows != 0; rows &= rows - 1) {
                const uint64_t row = (first + __builtin_ctzll(rows)) * a.dtable_stride;
                write_zeros<TDT>(a.dtable[rank] + row * elem_size<TDT>(), a.cols);
            }
        }
        return;
    }
    // A vector that would cross the row's end is moved back to end there; its first
    // `skip` columns are the vector's before.
    uint64_t c = ((turn % stretches) * static_cast<uint64_t>(TPR) + threadIdx.x % TPR) * V;
    if (c >= a.cols) return;
    int skip = 0;
    if (a.cols >= V && c > a.cols - V) {
        skip = static_cast<int>(c - (a.cols - V));
        c = a.cols - V;
    }
    uint32_t group = threadIdx.x / TPR;
    if constexpr (TPR >= 64) group = __builtin_amdgcn_readfirstlane(group);
    const char* const dy = a.dy[rank] + c * elem_size<DT>();
    const uint64_t dy_stride = a.dy_stride * elem_size<DT>();
    const uint64_t step = static_cast<uint64_t>(sum_blocks) * kRowsAtOnce<TPR>;
    for (uint64_t chunk = static_cast<uint64_t>(turn / stretches) * kRowsAtOnce<TPR> + group; chunk < a.chunks;
         chunk += step) {
        const uint64_t first = chunk * a.chunk;
        const uint64_t end = std::min(a.rows, first + a.chunk);
        float sum[V];
#pragma unroll
        for (int j = 0; j < V; ++j) sum[j] = 0;
        uint32_t token = keys[first];
        bool begins = first == 0 || keys[first - 1] != token;   // in this chunk
        const bool goes_on = end < a.rows && keys[end] == keys[end - 1];
        const auto leave = [&](bool ends) {
            if (token >= vocab) return;
            if (begins && ends) {
                write_row<TDT>(a, rank, token, c, skip, sum);
            } else {
                float* const to = partial_at(a, rank, chunk, begins ? 1 : 0) + c;
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    if (j >= skip && c + j < a.cols) to[j] = sum[j];
                }
            }
        };
        for (uint64_t at = first; at < end; at += kAhead) {
            uint32_t key[kAhead], place[kAhead];
            Raw<DT, V> r[kAhead];
            // places past the end read the last one's row, which is not added
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                const uint64_t from = std::min(at + k, end - 1);
                key[k] = keys[from];
                place[k] = places[from];
            }
            if (a.cols >= V) {
#pragma unroll
                for (int k = 0; k < kAhead; ++k) r[k].template load<true>(dy + place[k] * dy_stride);
            } else {
#pragma unroll
                for (int k = 0; k < kAhead; ++k) r[k].load_some(dy + place[k] * dy_stride, static_cast<int>(a.cols));
            }
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                if (at + k >= end) break;
                if (key[k] != token) {
                    leave(true);
                    token = key[k];
                    begins = true;
#pragma unroll
                    for (int j = 0; j < V; ++j) sum[j] = 0;
                }
#pragma unroll
                for (int j = 0; j < V; ++j) sum[j] += r[k].get(j);
            }
        }
        leave(!goes_on);
    }
}

constexpr uint32_t kJoinGroup = 256;   // partial sums

// The tokens that cross the end of a chunk: a wavefront looks at one chunk's
// end and 256 columns; where a token begins in that chunk and goes on, it adds
// the partial sums up to the chunk where the token ends.
template <int TDT>
__global__ void __launch_bounds__(256) k_embedding_join(EmbeddingBackwardArgs a) {
    const int rank = blockIdx.z, lane = threadIdx.x & 63;
    const uint32_t* const keys = a.keys + rank * sort_words(a.rows) + a.sorted * a.rows;
    const uint64_t c = blockIdx.y * 256ull + lane * 4;
    for (uint64_t chunk = blockIdx.x * 4ull + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);; chunk += gridDim.x * 4ull) {
        const uint64_t first = chunk * a.chunk, end = first + a.chunk;
        if (end >= a.rows) return;
        const uint32_t token = keys[end - 1];
        if (token >= a.vocab || keys[end] != token || (first > 0 && keys[first - 1] == token)) continue;
        // chunks behind this one that the token reaches past: 64 ends looked at at a time
        uint64_t whole = 0;
        for (;;) {
            const uint64_t at = end + (whole + lane + 1) * a.chunk;   // the first place behind that chunk
            const uint64_t past = __ballot(at < a.rows && keys[at] == token);
            if (past != ~0ull) {
                whole += __builtin_ctzll(~past);
                break;
            }
            whole += 64;
        }
        const uint64_t last = chunk + 1 + whole;
        float sum[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) sum[j] = c + j < a.cols ? partial_at(a, rank, chunk, 1)[c + j] : 0.0f;
        // 16 at a time while there are as many: 32,768 places of one rank under a 1/k
        // law, 4,096 columns of bf16, 185 -> 172 us, all of one token 630 -> 475
        uint64_t k = chunk + 1;
        const auto add = [&](auto many) {
            float x[many.value][4];
#pragma unroll
            for (int i = 0; i < many.value; ++i) {
                const float* const from = partial_at(a, rank, k + i, 0);
#pragma unroll
                for (int j = 0; j < 4; ++j) x[i][j] = c + j < a.cols ? from[c + j] : 0.0f;
            }
#pragma unroll
            for (int i = 0; i < many.value; ++i) {
#pragma unroll
                for (int j = 0; j < 4; ++j) sum[j] += x[i][j];
            }
            k += many.value;
        };
        // Added in groups, the groups' sums in groups again, and what those give: one
        // chain would be off by as many roundings as there are partial sums, and after
        // some 2^24 alike would no longer grow.
        float groups[4] = {}, more[4] = {};
        uint32_t count = 0;
        for (uint64_t group = chunk;; group += kJoinGroup) {
            const uint64_t end_of_group = std::min(last + 1, group + kJoinGroup);
            while (k + 16 <= end_of_group) add(std::integral_constant<int, 16>{});
            while (k + 4 <= end_of_group) add(std::integral_constant<int, 4>{});
            while (k < end_of_group) add(std::integral_constant<int, 1>{});
            if (k > last) break;
            const bool full = ++count % kJoinGroup == 0;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                groups[j] += sum[j];
                sum[j] = 0;
                if (full) {
                    more[j] += groups[j];
                    groups[j] = 0;
                }
            }
        }
        if (count > 0) {   // else the sum as it is, the sign of a 0 with it
#pragma unroll
            for (int j = 0; j < 4; ++j) sum[j] = (more[j] + groups[j]) + sum[j];
        }
        if (c < a.cols) write_row<TDT>(a, rank, token, c, 0, sum);
    }
}

// Vectors of a row to threads of a row: all of one wavefront's or workgroup's
// threads work on rows as short as 8 vectors.
int row_threads(uint64_t cols, int vector) {
    const uint64_t need = (cols + vector - 1) / vector;
    return need <= 8 ? 8 : need <= 16 ? 16 : need <= 32 ? 32 : need <= 64 ? 64 : need <= 128 ? 128 : 256;
}

constexpr uint64_t kMostBlocks = 1u << 16;

template <int DT, int TDT, int TPR>
hipError_t start_embedding(const EmbeddingArgs& a, int nranks, hipStream_t s) {
    const uint64_t need = (a.rows + kRowsAtOnce<TPR> - 1) / kRowsAtOnce<TPR>;
    const dim3 grid(static_cast<unsigned>(std::min(need, kMostBlocks)), nranks);
    hipLaunchKernelGGL((k_embedding<DT, TDT, TPR>), grid, dim3(256), 0, s, a);
    return hipGetLastError();
}

template <int DT, int TDT>
hipError_t embedding_by_width(const EmbeddingArgs& a, int nranks, hipStream_t s) {
    switch (row_threads(a.cols, 16 / elem_size<DT>())) {
        case 8: return start_embedding<DT, TDT, 8>(a, nranks, s);
        case 16: return start_embedding<DT, TDT, 16>(a, nranks, s);
        case 32: return start_embedding<DT, TDT, 32>(a, nranks, s);
        case 64: return start_embedding<DT, TDT, 64>(a, nranks, s);
        case 128: return start_embedding<DT, TDT, 128>(a, nranks, s);
        default: return start_embedding<DT, TDT, 256>(a, nranks, s);
    }
}

hipError_t start_sort(const EmbeddingBackwardArgs& a, int nranks, hipStream_t s) {
    if (a.rows <= kSortOne) {
        const dim3 grid(nranks), block(kSortThreads);
        if (a.rows <= kSortThreads) {
            hipLaunchKernelGGL((k_sort_one<1>), grid, block, 0, s, a);
        } else if (a.rows <= kSortThreads * 4) {
            hipLaunchKernelGGL((k_sort_one<4>), grid, block, 0, s, a);
        } else {
            hipLaunchKernelGGL((k_sort_one<kSortEach>), grid, block, 0, s, a);
        }
        return hipGetLastError();
    }
    const dim3 tiles(static_cast<unsigned>(a.tiles), nranks);
    for (int pass = 0; pass < a.passes; ++pass) {
        hipLaunchKernelGGL(k_sort_count, tiles, dim3(kSortTileThreads), 0, s, a, pass);
        hipLaunchKernelGGL(k_sort_scan, dim3(nranks), dim3(1024), 0, s, a);
        hipLaunchKernelGGL(k_sort_place, tiles, dim3(kSortTileThreads), 0, s, a, pass);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

template <int DT, int TDT, int TPR>
hipError_t start_sums(const EmbeddingBackwardArgs& a, int nranks, hipStream_t s) {
    const uint64_t sums = (a.chunks + kRowsAtOnce<TPR> - 1) / kRowsAtOnce<TPR>;
    const uint64_t zeros = a.accumulate ? 0 : (a.vocab + kZeroRows - 1) / kZeroRows;
    const uint32_t stretches = static_cast<uint32_t>((a.cols + TPR * kSumVec<DT> - 1) / (TPR * kSumVec<DT>));
    const uint32_t sum_blocks = static_cast<uint32_t>(std::min(sums, std::max<uint64_t>(1, 4 * kMostBlocks / stretches)));
    const uint32_t zero_blocks = static_cast<uint32_t>(std::min(zeros, kMostBlocks));
    if (sum_blocks + zero_blocks == 0) return hipSuccess;
    const dim3 grid(nranks * (sum_blocks * stretches + zero_blocks));
    hipLaunchKernelGGL((k_embedding_sums<DT, TDT, TPR>), grid, dim3(256), 0, s, a, static_cast<uint32_t>(nranks),
                       stretches, sum_blocks, zero_blocks);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || a.chunks < 2) return e;
    const dim3 joins(static_cast<unsigned>(std::min((a.chunks + 3) / 4, 16 * kMostBlocks)),
                     static_cast<unsigned>((a.cols + 255) / 256), nranks);
    hipLaunchKernelGGL((k_embedding_join<TDT>), joins, dim3(256), 0, s, a);
    return hipGetLastError();
}

template <int DT, int TDT>
hipError_t backward_by_width(const EmbeddingBackwardArgs& a, int nranks, hipStream_t s) {
    if (a.rows > 0) {
        const hipError_t e = start_sort(a, nranks, s);
        if (e != hipSuccess) return e;
    }
    switch (row_threads(a.cols, kSumVec<DT>)) {
        case 8: return start_sums<DT, TDT, 8>(a, nranks, s);
        case 16: return start_sums<DT, TDT, 16>(a, nranks, s);
        case 32: return start_sums<DT, TDT, 32>(a, nranks, s);
        case 64: return start_sums<DT, TDT, 64>(a, nranks, s);
        case 128: return start_sums<DT, TDT, 128>(a, nranks, s);
        default: return start_sums<DT, TDT, 256>(a, nranks, s);
    }
}

}  // namespace

hipError_t launch_embedding(const EmbeddingArgs& a, int nranks, ar_dtype_t dtype, ar_dtype_t table, hipStream_t s) {
    const bool wide = table == AR_FLOAT32;
    switch (dtype) {
        case AR_FLOAT32: return embedding_by_width<AR_FLOAT32, AR_FLOAT32>(a, nranks, s);
        case AR_BFLOAT16:
            return wide ? embedding_by_width<AR_BFLOAT16, AR_FLOAT32>(a, nranks, s)
                        : embedding_by_width<AR_BFLOAT16, AR_BFLOAT16>(a, nranks, s);
        case AR_FLOAT16:
            return wide ? embedding_by_width<AR_FLOAT16, AR_FLOAT32>(a, nranks, s)
                        : embedding_by_width<AR_FLOAT16, AR_FLOAT16>(a, nranks, s);
        default: return hipErrorInvalidValue;
    }
}

hipError_t launch_embedding_backward(const EmbeddingBackwardArgs& a, int nranks, ar_dtype_t dtype, ar_dtype_t table,
                                     hipStream_t s) {
    const bool wide = table == AR_FLOAT32;
    switch (dtype) {
        case AR_FLOAT32: return backward_by_width<AR_FLOAT32, AR_FLOAT32>(a, nranks, s);
        case AR_BFLOAT16:
            return wide ? backward_by_width<AR_BFLOAT16, AR_FLOAT32>(a, nranks, s)
                        : backward_by_width<AR_BFLOAT16, AR_BFLOAT16>(a, nranks, s);
        case AR_FLOAT16:
            return wide ? backward_by_width<AR_FLOAT16, AR_FLOAT32>(a, nranks, s)
                        : backward_by_width<AR_FLOAT16, AR_FLOAT16>(a, nranks, s);
        default: return hipErrorInvalidValue;
    }
}

}  // namespace arimpl
