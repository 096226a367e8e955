// A tile of a matrix product on the matrix cores: out[m][n] = sum over k of
// A[m][k] B[n][k], float32 sums of 16-bit or float32 elements, kept in
// registers for the caller's epilogue.  Inline device code in an unnamed
// namespace, so each kernel source gets its own copy.
//
// A workgroup brings 128 or 256 bytes of k of each of its rows of A and B to shared
// memory at a time (global_load_lds: 16 bytes a lane, no registers in between),
// into one of several buffers while the matrix instructions work on another.  An
// operand may lie along k (rows of A or B) or across (rows of k); shared memory
// holds it as it lies, and 16-bit operands across k are turned on the way to
// the registers by ds_read_tr16_b64.  Both kinds exchange 16-byte chunks within
// a row by its number, so that the lanes that read at a time meet different
// banks.  Float32 operands whose rows do not lie on 16 bytes can be brought 4
// bytes a lane.
#pragma once

#include <type_traits>

#include "ar_step_device.h"

namespace arimpl {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

constexpr int kChunk = 16;
constexpr int kSquare = 16;   // of outputs, a matrix instruction's

// EM x EN outputs by WM x WN wavefronts, each TM x TN squares of 16, in steps of
// STEP bytes of k; BUFFERS steps in shared memory, one worked on, the others on
// their way.
template <int EM_, int EN_, int WM_, int WN_, int STEP_, int BUFFERS_>
struct TileOf {
    static constexpr int EM = EM_, EN = EN_, WM = WM_, WN = WN_, kStepBytes = STEP_, kBuffers = BUFFERS_;
    static constexpr int kThreads = WM * WN * 64;
    static constexpr int TM = EM / WM / kSquare, TN = EN / WN / kSquare;
    static constexpr int kBytes = (EM + EN) * kStepBytes;   // of one buffer
    static constexpr int kShared = kBuffers * kBytes;
};

// Most bytes from one row of an operand to the next: 256 rows' offsets are
// 32-bit numbers.
constexpr uint64_t kMostStride = 1u << 23;

// What out-of-range k reads.
__device__ const u32x4 kZeroChunk = {0, 0, 0, 0};

// An operand's part of a buffer: E rows of it (columns, when it lies across k).
template <int DT, int E, int kStepBytes, bool ALONG>
struct InShared {
    static constexpr int kEs = elem_size<DT>();
    static constexpr int kChunkElems = kChunk / kEs;
    static constexpr int kStep = kStepBytes / kEs;             // k at a time
    static_assert(kStepBytes == 128 || kStepBytes == 256, "the exchange of chunks");
    static constexpr int kRowChunks = ALONG ? kStepBytes / kChunk : E * kEs / kChunk;

    // which chunk of a row stands at a place, and where a chunk stands
    static __device__ __forceinline__ int swap(int row, int chunk) {
        if constexpr (ALONG) {
            return kStepBytes == 256 ? chunk ^ (row & 15) : chunk ^ ((row >> 1) & 7);
        } else if constexpr (kEs == 2) {
            return chunk ^ (((row & 3) << 2) & (kRowChunks - 1));
        } else {
            return chunk ^ (((row >> 2) & 3) << 2 & (kRowChunks - 1));
        }
    }

    // Where this lane reads in the operand's part of a buffer: for the T squares
    // from row (column) `first` on.  A lane's part of a square is 16 bytes along k,
    // by its sixteen of the wavefront: chunk 4 kk + lane / 16 of a step.
    template <int T>
    struct Lane {
        uint32_t at[ALONG ? 1 : T];
    };
    template <int T>
    static __device__ __forceinline__ Lane<T> lane(int first) {
        const int l = threadIdx.x & 63, group = l >> 4, j = l & 15;
        Lane<T> r;
        if constexpr (ALONG) {
            const int row = first + j;
            r.at[0] = row * kStepBytes + swap(row, group) * kChunk;
        } else if constexpr (kEs == 2) {
            const int k = group * 8 + j / 4;
#pragma unroll
            for (int t = 0; t < T; ++t) {
                const int chunk = (first + t * kSquare) / 8 + (j % 4) / 2;
                r.at[t] = k * E * kEs + swap(k, chunk) * kChunk + (j % 2) * 8;
            }
        } else {
#pragma unroll
            for (int t = 0; t < T; ++t) {
                const int m = first + t * kSquare + j;
                r.at[t] = group * 4 * E * kEs + swap(group * 4, m / 4) * kChunk + (m % 4) * 4;
            }
        }
        return r;
    }
    template <int T>
    static __device__ __forceinline__ u32x4 read(const char* part, const Lane<T>& r, int t, int kk) {
        if constexpr (ALONG) {
            // the rows of a square differ from the next one's by 16: the same exchange
            return *reinterpret_cast<const u32x4*>(part + t * kSquare * kStepBytes + (r.at[0] ^ (kk << 6)));
        } else if constexpr (kEs == 2) {
            typedef __attribute__((address_space(3))) s16x4 shared_s16x4;
            const char* const q = part + r.at[t] + kk * 32 * E * kEs;
            const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((shared_s16x4*)(q));
            const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((shared_s16x4*)(q + 4 * E * kEs));
            return __builtin_bit_cast(u32x4, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
        } else {
            const char* const q = part + r.at[t] + kk * 16 * E * kEs;
            u32x4 v;
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = *reinterpret_cast<const uint32_t*>(q + i * E * kEs);
            return v;
        }
    }
};

// One operand: E rows of it (columns, when it lies across k) from `first` on,
// of which those from `limit` on are not wanted (the last wanted one is read in
// their place: nothing of it reaches another output).  Its rows lie on 16 bytes,
// at most kMostStride apart.
template <int DT, int E, int THREADS, int kStepBytes, bool ALONG>
struct ChunkOperand : InShared<DT, E, kStepBytes, ALONG> {
    typedef InShared<DT, E, kStepBytes, ALONG> Shared;
    using Shared::kChunkElems, Shared::kEs, Shared::kRowChunks, Shared::kStep, Shared::swap;
    static constexpr int kLoads = E * kStepBytes / kChunk / THREADS;
    static_assert(E * kStepBytes % (kChunk * THREADS) == 0, "whole loads");
    static_assert(THREADS % kRowChunks == 0, "a thread keeps its chunk of a row");

    const char* base;          // of the step to bring next, the same in all lanes
    uint64_t advance;
    uint32_t offset[kLoads];   // from there: operands' rows lie at most kMostStride bytes apart

    __device__ __forceinline__ void start(const char* from, uint64_t stride, uint64_t first, uint64_t limit) {
        const int place = threadIdx.x % kRowChunks;
        // a tile past the limit has the last wanted row for all of its rows
        if (first >= limit) first = ALONG ? limit - 1 : (limit - 1) / kChunkElems * kChunkElems;
        base = from + (ALONG ? first * stride : first * kEs);
        // past the limit: the last wanted row, or the last wanted column's chunk
        const uint32_t last = static_cast<uint32_t>(std::min<uint64_t>(limit - 1 - first, E - 1));
#pragma unroll
        for (int j = 0; j < kLoads; ++j) {
            const uint32_t row = (j * THREADS + threadIdx.x) / kRowChunks, chunk = swap(row, place);
            if constexpr (ALONG) {
                offset[j] = std::min(row, last) * static_cast<uint32_t>(stride) + chunk * kChunk;
            } else {
                offset[j] = row * static_cast<uint32_t>(stride) + std::min(chunk, last / kChunkElems) * kChunk;
            }
        }
        advance = ALONG ? kStepBytes : kStep * stride;
    }

    // Brings the next step of k, of which `left` are in range (ALONG: rounded up
    // to whole chunks, whose rest must be zeros), to shared memory at `to`.  m0
    // says where in shared memory, and needs a wait before the load uses it; the
    // compiler keeps nothing there in kernels without indexed registers.
    __device__ __forceinline__ void issue(uint32_t to, int64_t left) {
        to = __builtin_amdgcn_readfirstlane(to + (threadIdx.x & ~63u) * kChunk);
        if (left >= kStep) {
#pragma unroll
            for (int j = 0; j < kLoads; ++j) {
                asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(to + j * THREADS * kChunk),
                             "v"(offset[j]), "s"(base)
                             : "memory");
            }
        } else {
#pragma unroll
            for (int j = 0; j < kLoads; ++j) {
                const int row = (j * THREADS + static_cast<int>(threadIdx.x)) / kRowChunks;
                const int k = ALONG ? swap(row, threadIdx.x % kRowChunks) * kChunkElems : row;
                const char* const q = k < left ? base + offset[j] : reinterpret_cast<const char*>(&kZeroChunk);
                asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(to + j * THREADS * kChunk),
                             "v"(q)
                             : "memory");
            }
        }
        base += advance;
    }
};

// The same of float32 operands in any place and any distance apart: 4 bytes a
// lane, whose addresses are made anew for each load.  Four times the load
// instructions: for products that reading the operands bounds.
template <int DT, int E, int THREADS, int kStepBytes, bool ALONG>
struct WordOperand : InShared<DT, E, kStepBytes, ALONG> {
    typedef InShared<DT, E, kStepBytes, ALONG> Shared;
    using Shared::kChunkElems, Shared::kEs, Shared::kRowChunks, Shared::kStep, Shared::swap;
    static constexpr int kWord = 4, kRowWords = kRowChunks * kChunk / kWord;
    static constexpr int kLoads = E * kStepBytes / kWord / THREADS;
    static_assert(kEs == kWord && E * kStepBytes % (kWord * THREADS) == 0, "whole loads");
    static_assert(THREADS % kRowWords == 0, "a thread keeps its word of a row");

    const char* base;   // of the step to bring next
    uint64_t stride, advance;
    uint32_t last;      // wanted row (column)

    __device__ __forceinline__ void start(const char* from, uint64_t stride_, uint64_t first, uint64_t limit) {
        if (first >= limit) first = limit - 1;
        stride = stride_;
        base = from + (ALONG ? first * stride : first * kEs);
        last = static_cast<uint32_t>(std::min<uint64_t>(limit - 1 - first, E - 1));
        advance = ALONG ? kStepBytes : kStep * stride;
    }

    // As above; k past `left` is 0 whatever lies there.
    __device__ __forceinline__ void issue(uint32_t to, int64_t left) {
        to = __builtin_amdgcn_readfirstlane(to + (threadIdx.x & ~63u) * kWord);
        const uint32_t word = threadIdx.x % kRowWords;
#pragma unroll
        for (int j = 0; j < kLoads; ++j) {
            const uint32_t row = (j * THREADS + threadIdx.x) / kRowWords;
            const uint32_t in = swap(row, word / kChunkElems) * kChunkElems + word % kChunkElems;   // its place in the row
            const uint32_t k = ALONG ? in : row, which = std::min(ALONG ? row : in, last);
            const char* q = base + (ALONG ? which : k) * stride + (ALONG ? k : which) * kWord;
            if (k >= left) q = reinterpret_cast<const char*>(&kZeroChunk);
            asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, off" ::"s"(to + j * THREADS * kWord), "v"(q)
                         : "memory");
        }
        base += advance;
    }
};

template <int DT, int E, int THREADS, int kStepBytes, bool WHOLE, bool ALONG>
using Operand = std::conditional_t<WHOLE, ChunkOperand<DT, E, THREADS, kStepBytes, ALONG>,
                                   WordOperand<DT, E, THREADS, kStepBytes, ALONG>>;

template <int DT>
__device__ __forceinline__ f32x4 multiply(u32x4 a, u32x4 b, f32x4 c) {
    if constexpr (DT == AR_BFLOAT16) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0,
                                                       0, 0);
    } else if constexpr (DT == AR_FLOAT16) {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0,
                                                      0);
    } else {
        // k in another order than in memory, the same for both
#pragma unroll
        for (int i = 0; i < 4; ++i) c = __builtin_amdgcn_mfma_f32_16x16x4f32(as_f(a[i]), as_f(b[i]), c, 0, 0, 0);
        return c;
    }
}

// Lane l of a square's sums has column n = l % 16 and rows 4 * (l / 16) to
// 4 * (l / 16) + 3.

// Waits until at most N of the wavefront's loads are on their way.
template <int N>
__device__ __forceinline__ void wait_loads() {
    static_assert(N < 64, "the counter's range");
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

// The sums of one tile, from k = 0 to `depth`.  `buffers`: Tile::kShared bytes
// of shared memory, free again when every wavefront has passed a barrier.
// WHOLE: the operands' rows lie on 16 bytes.
template <int DT, class Tile, bool WHOLE, bool A_ALONG, bool B_ALONG>
__device__ __forceinline__ void product(char* buffers, const char* a, uint64_t a_stride, uint64_t a_first,
                                        uint64_t a_limit, const char* b, uint64_t b_stride, uint64_t b_first,
                                        uint64_t b_limit, uint64_t depth, f32x4 (&sum)[Tile::TM][Tile::TN]) {
    typedef Operand<DT, Tile::EM, Tile::kThreads, Tile::kStepBytes, WHOLE, A_ALONG> A;
    typedef Operand<DT, Tile::EN, Tile::kThreads, Tile::kStepBytes, WHOLE, B_ALONG> B;
    // A step is worked off in parts: 64 bytes of k, and half of the squares of m.
    constexpr int kParts = Tile::kStepBytes / 32, kHalf = Tile::TM / 2;
    static_assert(Tile::TM % 2 == 0, "halves");
    constexpr int kStep = A::kStep;
#pragma unroll
    for (int i = 0; i < Tile::TM; ++i) {
#pragma unroll
        for (int j = 0; j < Tile::TN; ++j) sum[i][j] = f32x4{};
    }
    if (depth == 0) return;
    A oa;
    B ob;
    oa.start(a, a_stride, a_first, a_limit);
    ob.start(b, b_stride, b_first, b_limit);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const auto la = A::template lane<Tile::TM>((wave / Tile::WN) * Tile::TM * kSquare);
    const auto lb = B::template lane<Tile::TN>((wave % Tile::WN) * Tile::TN * kSquare);
    typedef __attribute__((address_space(3))) char shared_char;
    const uint32_t base = static_cast<uint32_t>(reinterpret_cast<uintptr_t>((shared_char*)buffers));
    constexpr uint32_t kA = Tile::EM * Tile::kStepBytes;
    // Steps past the last bring zeros that nothing reads, so that the number of
    // loads behind a step's is always the same.
    int64_t left = static_cast<int64_t>(depth);
    const auto bring_a = [&](uint32_t buffer) { oa.issue(base + buffer * Tile::kBytes, left); };
    const auto bring_b = [&](uint32_t buffer) {
        ob.issue(base + buffer * Tile::kBytes + kA, left);
        left -= kStep;
    };
    constexpr int kBehind = (Tile::kBuffers - 2) * (A::kLoads + B::kLoads);
#pragma unroll
    for (uint32_t k = 0; k + 1 < Tile::kBuffers; ++k) {
        bring_a(k);
        bring_b(k);
    }
    // A part is read while the matrix instructions work on the part before, the
    // next step's first one while they work on this step's last.
    u32x4 fa[2][kHalf], fb[2][Tile::TN];
    const auto read = [&](uint32_t buffer, int part) {
        const char* const pa = buffers + buffer * Tile::kBytes;
#pragma unroll
        for (int i = 0; i < kHalf; ++i) fa[part & 1][i] = A::template read<Tile::TM>(pa, la, (part & 1) * kHalf + i, part / 2);
        if (part % 2 == 0) {
#pragma unroll
            for (int j = 0; j < Tile::TN; ++j) fb[part / 2 & 1][j] = B::template read<Tile::TN>(pa + kA, lb, j, part / 2);
        }
    };
    const auto work = [&](int part) {
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = 0; i < kHalf; ++i) {
            const int m = (part & 1) * kHalf + i;
#pragma unroll
            for (int j = 0; j < Tile::TN; ++j) sum[m][j] = multiply<DT>(fa[part & 1][i], fb[part / 2 & 1][j], sum[m][j]);
        }
        __builtin_amdgcn_sched_barrier(0);
    };
    // Loads are issued in two halves, each before a part's matrix instructions: a
    // wavefront waits for the memory pipe to take them, and all of them at once
    // would keep the matrix cores waiting too.
    wait_loads<kBehind>();
    __syncthreads();
    uint32_t now = 0, free = Tile::kBuffers - 1;
    bring_a(free);
    read(0, 0);
    for (uint64_t k = kStep;; k += kStep) {
#pragma unroll
        for (int kk = 0; kk + 1 < kParts; ++kk) {
            read(now, kk + 1);
            if (kk == 0) bring_b(free);
            work(kk);
        }
        if (k < depth) {
            // the next step's loads have come, every wavefront's after the barrier; and
            // every wavefront has read all of this step, whose buffer is free
            wait_loads<kBehind>();
            __syncthreads();
            free = now;
            now = now + 1 == Tile::kBuffers ? 0 : now + 1;
            read(now, 0);
            bring_a(free);
        }
        work(kParts - 1);
        if (k >= depth) break;
    }
    // nothing may land in shared memory, or in the next workgroup's, after this
    wait_loads<0>();
}

// A launch's tiles to workgroups.  Workgroups go to the XCDs in turn; each XCD
// takes a stretch of neighbouring tiles, walked `kAcross` n-tiles wide, so that
// the tiles that it works on at a time share their operands in its L2.
constexpr uint32_t kAcross = 4;
struct TilePlace {
    uint32_t rank, part, m, n;
    bool valid;
    __device__ __forceinline__ TilePlace(uint32_t block, uint32_t tiles_m, uint32_t tiles_n, uint32_t ranks) : part(0) {
        uint32_t t = 0;
        valid = stretch(block, tiles_m * tiles_n * ranks, t);
        rank = t / (tiles_m * tiles_n);
        across(t % (tiles_m * tiles_n), tiles_m, tiles_n);
    }
    // The same when each rank (at most 64) has its own n side, of live[rank], in
    // tiles of `en`, and each of its tiles is made in `parts`.  The workgroups past
    // the last tile are then the launch's last, in every XCD alike: a batch half of
    // which is ignored leaves no XCD without work.
    __device__ __forceinline__ TilePlace(uint32_t block, uint32_t tiles_m, const uint32_t* live, uint32_t en,
                                         uint32_t parts, uint32_t ranks) {
        const uint32_t lane = threadIdx.x & 63, mine = lane < ranks ? (live[lane] + en - 1) / en : 0;
        const auto tiles_n = [&](uint32_t r) -> uint32_t { return __builtin_amdgcn_readlane(mine, r); };
        uint32_t all = 0, t = 0;
        for (uint32_t r = 0; r < ranks; ++r) all += tiles_n(r);
        valid = stretch(block, all * tiles_m * parts, t);
        if (!valid) return;
        for (rank = 0; rank + 1 < ranks; ++rank) {
            const uint32_t here = tiles_n(rank) * tiles_m * parts;
            if (t < here) break;
            t -= here;
        }
        const uint32_t each = tiles_n(rank) * tiles_m;
        part = t / each;
        across(t % each, tiles_m, tiles_n(rank));
    }

private:
    static __device__ __forceinline__ bool stretch(uint32_t block, uint32_t all, uint32_t& t) {
        const uint32_t each = (all + 7) / 8;
        t = (block & 7) * each + (block >> 3);
        return (block >> 3) < each && t < all;
    }
    __device__ __forceinline__ void across(uint32_t in, uint32_t tiles_m, uint32_t tiles_n) {
        const uint32_t group = in / (kAcross * tiles_m), rest = in % (kAcross * tiles_m);
        const uint32_t width = std::min(kAcross, tiles_n - group * kAcross);
        m = rest / width;
        n = group * kAcross + rest % width;
    }
};
inline uint64_t tile_blocks(uint64_t tiles) { return (tiles + 7) / 8 * 8; }

}  // namespace
}  // namespace arimpl
