// Attention of many query rows at once: over whole prompts packed one behind the other, and
// of a chunk of new tokens of every sequence over a paged key-value cache.
//   a_j = scale q . k_j,   out = sum_j exp(a_j) v_j / sum_j exp(a_j)
// for the q_heads / kv_heads = G query heads that share a key-value head.
//
// A row of the matrix products is a (token, head of the group) pair, so that the heads of a
// group share the keys that are loaded.  A unit of work is up to 256 consecutive rows of one
// (sequence, key-value head) and the keys that they see, in tiles of 128.  A persistent CTA
// per SM takes units, the long ones of a sequence first, every other round backwards.
//
//  * Two streams of work run side by side, each with its scores (128 x 128 fp32) and its output
//    (128 x D fp32) in tensor memory: while the tensor cores work for one, four warps turn the
//    scores of the other into probabilities.  The streams are the two halves of 256 rows over
//    the same keys, or, for 128 rows or fewer, even and odd tiles of the same rows' keys, joined
//    at the end.  D = 256 leaves room for one output and one stream, with two score tiles.
//  * Scores are tcgen05.mma of queries and keys in shared memory; the probabilities replace
//    their scores in tensor memory as 16-bit numbers and are the first operand of the product
//    with the values.  A row of scores is one thread's: 128 registers, no exchange.
//  * One pass: the running maximum that is subtracted is renewed, and the output rescaled,
//    only where the scores exceed it by more than `slack` (as a power of two).
//  * Keys and values come into a ring of stages by tensor maps, in boxes of 32, 16 or 8 rows (a
//    page's), where strides and page sizes allow it, else 16 bytes a lane.  E4M3 rows go into a
//    ring of their own and eight warps turn them into 16-bit ones.  Rows that no query of the
//    unit sees are zeros.
//  * Infinite and NaN values that a row does not see: units with such rows are taken again in a second
//    pass (see partly_seen), after all others, at the same speed.
//
// What bounds it, where rows and keys are many: the chain of a tile, scores, maximum, powers, product with the
// values, next scores, of which two run side by side.  At D = 128 a pair of tiles takes 3330 cycles; its
// products (32 of 128 x 128 x 16, 64 cycles each) take 2048 of them, and so does the shared memory's port (192 KB
// of operands and 64 KB of copies at 128 bytes a cycle).  Four warps take 1700 to 2000 cycles for a tile's
// probabilities, half of it powers, behind the other stream's products.  With D = 256 there is one chain, and the
// port takes 2560 cycles of its 4000.  8192 causal tokens of 32 heads of 128: 413 us, 1.33 PFLOP/s, 0.71 of what a
// library's matrix product reaches.  Calls of a few rows are bound by what a launch, the plan and cold code take.
#pragma once
#include <algorithm>
#include <atomic>
#include <type_traits>

#include "elem.cuh"
#include "kernels.h"
#include "launch.cuh"
#include "prompt_args.cuh"
#include "tc_ptx.cuh"

namespace w4a4 {
namespace prompt {

constexpr int kTile = 128;                 // keys of a tile, rows of a stream
constexpr uint64_t kWaitNs = 2000000000ull;
constexpr uint64_t kDrainNs = 10000000ull;  // of a kernel that gives up: copies that are under way have long landed
constexpr uint32_t kSuspendNs = 20000;
constexpr int kSoftmaxWarps = 8;
constexpr int kLostTiles = 16;

struct Sequence {
    int begin, rows, length;               // its rows [begin, begin + rows) of q and its keys
};

// A unit of work, or a piece of one: what the warps need to know of it.
struct Unit {
    int live;                              // 0: there are no more (of a pass), 1: of the first pass, else see partly_seen
    int b, head;                           // sequence, key-value head
    int row0, rows;                        // rows (token * G + head of the group) of the sequence
    int begin;                             // the sequence's first token in q
    int first, length;                     // its place among the keys, and how many there are
    int key0, end, tiles;                  // keys [key0, end), in tiles
    int tiles0;                            // of the first stream
    int shared;                            // the streams are halves of the rows
    int part;                              // where a piece of a unit goes, -1: the unit is whole
    int first_part, pieces;
};
static_assert(sizeof(Unit) == 64, "copied as four int4");

// 8-bit rows come into a ring of their own, from where they are turned into 16-bit ones.
template <int D, bool E4M3>
struct Plan {
    static constexpr int kDs = D < 128 ? D : 128;               // elements of a stage's rows
    static constexpr int kHalves = D / kDs;
    static constexpr int kPlanes = (kDs + 63) / 64;
    static constexpr int kStage = kPlanes * kTile * 128;
    static constexpr int kStreams = D == 256 ? 1 : 2;
    static constexpr int kQTile = kHalves * kStage;
    static constexpr int kQ = kStreams * kQTile;
    // Both rings fill the shared memory; 8-bit rows in flight gain less from room than 16-bit ones (D = 128, 64 sequences
    // of 4 tokens behind up to 8191, 32 heads for 8: 195 us with stages 3 + 4, 183 with those below).
    static constexpr int kStages = E4M3 ? (D == 64 ? 6 : 4) : D == 64 ? 11 : 5;
    static constexpr int kRawStages = E4M3 ? (D == 64 ? 10 : 2) : 0;
    static constexpr int kRawStage = kTile * kDs;
    static constexpr bool kRawSwizzled = kDs == 128;
    static constexpr int kRawRing = kRawStages > 0 ? kRawStages : 1;
    // warps: softmax, copies (twice as many to widen 8-bit rows: the same sequences took 236 us with four and 182
    // with eight when they were added), then one that plans, two that issue products, one for the ring of 8-bit rows
    static constexpr int kCopyWarps = E4M3 ? 8 : 4;
    static constexpr int kMmaWarp = kSoftmaxWarps + kCopyWarps, kPlanWarp = kMmaWarp + 1, kRawWarp = kMmaWarp + 3;
    static constexpr int kThreads = 32 * (kMmaWarp + 4);
    // registers of their threads: as many in all as a block of so many threads is launched with
    static constexpr int kLaunchRegs = E4M3 ? 96 : 128;
    static constexpr int kSoftmaxRegs = E4M3 ? 144 : 160, kCopyRegs = E4M3 ? 64 : 96, kOtherRegs = E4M3 ? 64 : 96;
    static_assert(32 * (kSoftmaxWarps * kSoftmaxRegs + kCopyWarps * kCopyRegs + 4 * kOtherRegs) <= kThreads * kLaunchRegs,
                  "an increase beyond what the block has would wait forever");
    static_assert(kThreads * kLaunchRegs <= 65536 && kThreads * (kLaunchRegs + 8) > 65536, "registers at launch");
    static constexpr int kRaw = kQ + kStages * kStage;
    static constexpr int kMl = kRaw + kRawStages * kRawStage;   // [2][128] maxima, then sums, of the streams
    static constexpr int kUnits = kMl + 2 * 2 * kTile * 4;      // [2] units
    static constexpr int kBars = kUnits + 2 * int(sizeof(Unit));
    static constexpr int kFlags = kBars + (2 * kStages + 22 + 2 * kRawStages) * 8;
    static constexpr int kLost = kFlags + 16;                   // [kLostTiles][4] keys of a tile on pages outside the pool
    static constexpr int kOrder = kLost + kLostTiles * 16;      // [64] sequences, see sort_sequences
    static constexpr int kThere = kOrder + 64;                  // [kRawStages][4] rows of a raw stage that are there
    static constexpr int kBytes = kThere + kRawStages * 16;
    // Copies are at most the rings ahead of the scores' products, and those two tiles ahead of
    // the probabilities.
    static_assert(kLostTiles >= (kStages + kRawStages) / 2 + 5, "a word is read before it is written again");
    static_assert(kThere % 16 == 0, "read four words at once");
    static_assert(kBytes <= 227 * 1024, "shared memory");
    static_assert(kStages >= 2 * kHalves, "the values of a tile and the keys of the next are waited for together");
    // tensor memory: a stream's scores (and probabilities) and its output
    static constexpr uint32_t scores(int buf) { return D == 256 ? 128 * buf : 256 * buf; }
    static constexpr uint32_t output(int stream) { return D == 256 ? 256 : 256 * stream + 128; }
};

__device__ __forceinline__ float ex2(float x) {  // 2 ulp; 2^-inf = 0
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
    return y;
}

// The same and its neighbours in the order in which they are written.
__device__ __forceinline__ uint64_t ex2_in_order(uint64_t x) {
    uint64_t y;
    asm volatile(
        "{\n.reg .f32 a, b;\nmov.b64 {a, b}, %1;\nex2.approx.ftz.f32 a, a;\nex2.approx.ftz.f32 b, b;\nmov.b64 %0, {a, b};\n}\n"
        : "=l"(y)
        : "l"(x));
    return y;
}
__device__ __forceinline__ uint64_t ffma2_in_order(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm volatile("fma.rn.f32x2 %0, %1, %2, %3;\n" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ uint64_t fadd2_in_order(uint64_t a, uint64_t b) {
    uint64_t d;
    asm volatile("add.rn.f32x2 %0, %1, %2;\n" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
template <class T>
__device__ __forceinline__ uint32_t down_in_order(float a, float b) {  // T::down
    uint32_t w;
    if constexpr (std::is_same_v<T, BF16>)
        asm volatile("cvt.rn.bf16x2.f32 %0, %1, %2;\n" : "=r"(w) : "f"(b), "f"(a));
    else
        asm volatile("cvt.rn.f16x2.f32 %0, %1, %2;\n" : "=r"(w) : "f"(b), "f"(a));
    return w;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;\n" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// A probability is 2^(its score - the subtracted maximum + lift), the maximum at most slack below the
// largest score so far.  fp16 ones are taken up to 2^15, so that weights down to 2^-38 of the largest
// keep the bits of their rounding: thousands of small ones beside one heavy key can make
// the output.  bf16 ones have fp32's range, and so have their values: up to 1, so that a product with a
// value is no larger than the value.
template <class T>
constexpr float slack = std::is_same_v<T, BF16> ? 8.f : 2.f;
template <class T>
constexpr float lift = std::is_same_v<T, BF16> ? -slack<T> : 13.f;

// One of each translation unit: there is one a head dimension.
static __device__ int g_prompt_status = 0;

// Where 16-byte piece c of a row is in a tile of planes of 128 rows of 128 bytes.
__device__ __forceinline__ uint32_t swizzled(int row, int c) {
    return (c >> 3) * (kTile * 128) + row * 128 + (((c & 7) ^ (row & 7)) << 4);
}

__device__ __forceinline__ Sequence sequence(const Args& A, int b, bool& bad) {
    Sequence s;
    const int from = A.starts[b], to = A.starts[b + 1];
    s.begin = max(0, min(from, A.tokens));
    const int end = max(s.begin, min(to, A.tokens));
    bad = from < 0 || to < from || to > A.tokens;
    s.rows = end - s.begin;
    s.length = s.rows;
    if (A.lengths) {
        const int n = A.lengths[b];
        s.length = max(0, min(n, A.keys.longest));
        bad |= n != s.length;
    }
    return s;
}

// Keys [lo, hi) that the row's token at `place` sees.
__device__ __forceinline__ void sees(const Args& A, int place, int length, int& lo, int& hi) {
    hi = A.causal ? max(0, min(place, length - 1) + 1) : length;
    // a place before token 0 sees nothing, whatever the window: clamped, since their difference can pass 31 bits
    lo = A.window > 0 ? max(0, max(-1, min(place, INT32_MAX - 1)) + 1 - A.window) : 0;
}

// Where key j's row of head `head` is, in keys (w = 0) or values (1); nullptr: on no page.
__device__ __forceinline__ const char* key_row(const Args& A, int b, int begin, int head, int j, int w) {
    const Keys& K = A.keys;
    const int64_t at = int64_t(head) * K.head_stride[w];
    if (!K.table) return K.pool[w] + at + int64_t(begin + j) * K.token_stride[w];
    const int p = K.by_page.quotient(j);
    const int page = K.table[b * K.table_stride + p];
    if (page < 0 || page >= K.pages) return nullptr;
    return K.pool[w] + at + page * K.page_stride[w] + int64_t(j - p * K.page_size) * K.token_stride[w];
}

template <class T, bool E4M3>
__device__ __forceinline__ float element(const char* row, int e) {
    if constexpr (E4M3) {
        __nv_fp8_e4m3 x;
        x.__x = *reinterpret_cast<const uint8_t*>(row + e);
        return float(x);
    } else {
        return T::up(*reinterpret_cast<const uint16_t*>(row + 2 * e)).x;
    }
}

// The keys among [lo, lo + 32) and below hi with an infinite or NaN value (a warp).
template <int D, bool E4M3, bool BF>
__device__ __forceinline__ uint32_t odd_keys(const Args& A, const Unit& U, int lo, int hi) {
    const int j = lo + int(threadIdx.x & 31);
    const char* const row = j < hi ? key_row(A, U.b, U.begin, U.head, j, 1) : nullptr;
    bool odd = false;
    for (int i = 0; row && i < D * (E4M3 ? 1 : 2) / 16; ++i) {
        const uint4 v = reinterpret_cast<const uint4*>(row)[i];
        for (const uint32_t w : {v.x, v.y, v.z, v.w})
            if constexpr (E4M3) {
                for (int s = 0; s < 32; s += 8) odd |= (w >> s & 0x7Fu) == 0x7Fu;
            } else {
                const uint32_t m = BF ? 0x7F80u : 0x7C00u;
                odd |= (w & m) == m || (w >> 16 & m) == m;
            }
    }
    return __ballot_sync(0xffffffffu, odd);
}
// Whether there are any among [lo, hi).
template <int D, bool E4M3, bool BF>
__device__ __noinline__ bool odd_values(const Args& A, const Unit& U, int lo, int hi) {
    for (; lo < hi; lo += 32)
        if (odd_keys<D, E4M3, BF>(A, U, lo, hi) != 0) return true;
    return false;
}

// Values of keys that a row does not see have a probability of zero, and their product is NaN where the
// value is infinite or NaN.  A unit with such a row among its outputs is taken again in a second pass, in which
// these values are zeros in the tiles that some row of the unit does not see whole; the rows that do see them have
// them added afterwards (the probability is not zero, so that the sum is what the value itself makes of it).
// A unit's `live` in that pass: 2 + 256 * its first tiles of that kind + 65536 * its last ones (four or so
// at most: a unit's rows are neighbours).
__device__ __forceinline__ bool partly_seen(int live, int t, int tiles) {
    return t < (live >> 8 & 0xFF) || t >= tiles - (live >> 16);
}
__device__ __forceinline__ int second_pass(const Args& A, const Unit& U) {
    int lo, hi, unused;
    sees(A, U.first + A.by_group.quotient(U.row0), U.length, unused, hi);
    sees(A, U.first + A.by_group.quotient(U.row0 + U.rows - 1), U.length, lo, unused);
    const int front = max(0, min(U.tiles, (lo - U.key0 + kTile - 1) / kTile));
    const int whole = hi >= U.end ? U.tiles : max(0, hi - U.key0) / kTile;
    return 2 | min(front, 255) << 8 | min(U.tiles - whole, 255) << 16;
}

// Zeros for the infinite and NaN elements of a stage, by the thread that issues its products: 20 us for a tile.
template <bool BF, int BYTES>
__device__ __noinline__ void clean_stage(uint8_t* stage) {
    constexpr uint32_t kExp = BF ? 0x7F807F80u : 0x7C007C00u, kOne = BF ? 0x00800080u : 0x04000400u;
    uint32_t* const words = reinterpret_cast<uint32_t*>(stage);
#pragma unroll 8
    for (int i = 0; i < BYTES / 16; ++i) {
        const uint4 v = reinterpret_cast<const uint4*>(stage)[i];
        // the sign bits: halves whose exponent is all ones
        if ((((v.x & kExp) + kOne | (v.y & kExp) + kOne | (v.z & kExp) + kOne | (v.w & kExp) + kOne) & 0x80008000u) == 0) continue;
        for (int k = 0; k < 4; ++k) {
            const uint32_t w = words[4 * i + k], odd = (w & kExp) + kOne;
            words[4 * i + k] = w & ~((odd & 0x8000u ? 0xFFFFu : 0u) | (odd & 0x80000000u ? 0xFFFF0000u : 0u));
        }
    }
    tc::fence_proxy_async_smem();
}

// Adds the infinite and NaN values of tiles that are partly seen to each lane's row (which sees keys [lo, hi), and some
// of them if `has`) of the output, elements [e0, e1), of type T or fp32.
template <int D, class T, bool E4M3>
__device__ __noinline__ void add_odd_values(const Args& A, const Unit& U, bool has, int lo, int hi, char* out, bool fp32,
                                            int e0, int e1) {
    for (int t = 0; t < U.tiles; ++t) {
        if (!partly_seen(U.live, t, U.tiles)) continue;
        const int end = min(U.key0 + (t + 1) * kTile, U.end);
        for (int j0 = U.key0 + t * kTile; j0 < end; j0 += 32)
            for (uint32_t odd = odd_keys<D, E4M3, std::is_same_v<T, BF16>>(A, U, j0, end); odd != 0; odd &= odd - 1) {
                const int j = j0 + __ffs(odd) - 1;
                const char* const row = key_row(A, U.b, U.begin, U.head, j, 1);
                for (int e = e0; has && j >= lo && j < hi && e < e1; ++e) {
                    const float v = element<T, E4M3>(row, e);
                    if (fabsf(v) < INFINITY) continue;
                    if (fp32) {
                        reinterpret_cast<float*>(out)[e] += v;
                    } else {
                        uint16_t& x = reinterpret_cast<uint16_t*>(out)[e];
                        x = uint16_t(T::down(T::up(x).x + v, 0.f));
                    }
                }
                __syncwarp();
            }
    }
}

// ---- the plan: which rows a unit has, and how units are split where they are few
// The first CTA's warp that makes the plan reports bad starts and lengths.
struct Share {
    int rows;          // of a unit
    int piece;         // tiles of a piece, 0: units are whole
};

// Tiles that a block of rows of this sequence sees at most.
__device__ __forceinline__ int most_tiles(const Args& A, const Sequence& s) {
    const int all = (s.length + kTile - 1) / kTile;
    if (A.window == 0) return all;
    const int64_t span = int64_t(A.window) + 256 / A.group + 1;
    return int(min(int64_t(all), (span + kTile - 1) / kTile + 1));
}
__device__ __forceinline__ int blocks_of(const Args& A, const Sequence& s, int rows) {
    return int((int64_t(s.rows) * A.group + rows - 1) / rows);
}

// n / d for d >= 1, exact: by a float division below 2^20 ((n + 1/2) / d is at least 1 / (2 d) from a
// whole number, the division and the conversion off by less than n / d * 2^-21), which takes a
// fifth of the time.
__device__ __forceinline__ int quotient(int n, int d) {
    return n < (1 << 20) ? int(__fdividef(n + 0.5f, float(d))) : n / d;
}

// f of every sequence, summed (a warp).  In fp32, exact below 2^24: what is decided by it is a
// matter of speed where it is larger.
template <class F>
__device__ __forceinline__ float sum_over_sequences(const Args& A, const Sequence& mine, F f) {
    const int lane = threadIdx.x & 31;
    float sum = lane < A.seqs ? f(mine) : 0.f;
    for (int b = lane + 32; b < A.seqs; b += 32) {
        bool bad;
        sum += f(sequence(A, b, bad));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    return sum;
}

// `mine`: the lane's sequence (of the first 32).
template <int D>
__device__ __forceinline__ Share share_out(const Args& A, const Sequence& mine) {
    constexpr int kStreams = Plan<D, false>::kStreams;
    const float ctas = gridDim.x;
    auto units_of = [&](int rows) {
        return A.kv_heads * sum_over_sequences(A, mine, [&](const Sequence& s) { return float(blocks_of(A, s, rows)); });
    };
    Share r{128, 0};
    // 256 rows a unit where there are units enough, or (below) tiles enough to split them into: 8192
    // causal tokens of 32 heads for 8 take 413 us and 464 with 128, eight texts of 1500 both ways with
    // 16 heads of 64 139 and 151, though the last round of their units is 5% full.
    float units = kStreams == 2 ? units_of(256) : 0.f;
    if (units >= ctas) r.rows = 256;
    if (!A.parts || r.rows == 256) return r;
    const float units128 = units_of(128);
    if (kStreams == 1) units = units128;
    const int wide = kStreams == 1 ? 128 : 256;
    for (int rows = wide; rows >= 128; rows -= 128) {
        const float n = rows == wide ? units : units128;
        if (n >= ctas) return r;
        const float tiles = A.kv_heads * sum_over_sequences(A, mine, [&](const Sequence& s) {
            return float(blocks_of(A, s, rows)) * most_tiles(A, s);
        });
        if (rows == 256 && tiles < 8 * ctas) continue;
        r.rows = rows;
        int piece = max(4, int(ceilf(tiles / ctas)));
        for (int tries = 0; tries < 8; ++tries) {
            const float all = A.kv_heads * sum_over_sequences(A, mine, [&](const Sequence& s) {
                return float(blocks_of(A, s, rows)) * max(1, quotient(most_tiles(A, s) + piece - 1, piece));
            });
            if (all <= ctas) {
                r.piece = piece;
                return r;
            }
            piece = max(piece + 1, int(piece * all / ctas));
        }
        return r;
    }
    return r;
}

// Sequences with the longest units first, for up to kSorted of them (two a lane): what is left for the last
// round is short then (six chunks of 417 tokens, the later ones behind more, D = 256: 89 us, 134 in
// the sequences' order; 64 of 4 tokens behind up to 8191, E4M3: 183 and 274).  More are taken as they come.
constexpr int kSorted = 64;
__device__ __forceinline__ void sort_sequences(const Args& A, const Sequence& mine, uint8_t* order) {
    const int lane = threadIdx.x & 31;
    Sequence s2{0, 0, 0};
    bool bad;
    if (lane + 32 < A.seqs) s2 = sequence(A, lane + 32, bad);
    const int key[2] = {mine.rows > 0 ? most_tiles(A, mine) : -1, s2.rows > 0 ? most_tiles(A, s2) : -1};
    int rank[2] = {0, 0};
    for (int k = 0; k < A.seqs; ++k) {
        const int other = __shfl_sync(0xffffffffu, k < 32 ? key[0] : key[1], k & 31);
#pragma unroll
        for (int i = 0; i < 2; ++i) rank[i] += other > key[i] || (other == key[i] && k < lane + 32 * i);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
        if (lane + 32 * i < A.seqs) order[rank[i]] = uint8_t(lane + 32 * i);
    __syncwarp();
}

// Where unit `want` is, for numbers that grow from call to call (a warp).
struct Walk {
    const uint8_t* order;    // of the sequences, nullptr: as they are
    const Sequence& mine;    // this lane's of the first 32, if they are as they are
    int base = -32, before = 0;  // sequences from `base` on, and the units before them
    int b = 0, pieces = 1, units = 0, upto = 0;  // of this lane's: number, pieces of a unit, units, those up to it
    Sequence s{0, 0, 0};
    __device__ __forceinline__ bool find(const Args& A, const Share& share, int want, Unit& U) {
        const int lane = threadIdx.x & 31;
        while (base < A.seqs) {
            const uint32_t beyond = __ballot_sync(0xffffffffu, upto > want - before);
            if (beyond == 0) {
                before += __shfl_sync(0xffffffffu, upto, 31);
                base += 32;
                b = base + lane;
                pieces = 1, units = 0;
                if (b < A.seqs) {
                    bool bad;
                    if (order) b = order[b];
                    s = order || base > 0 ? sequence(A, b, bad) : mine;
                    if (share.piece > 0) pieces = max(1, quotient(most_tiles(A, s) + share.piece - 1, share.piece));
                    units = blocks_of(A, s, share.rows) * A.kv_heads * pieces;
                }
                upto = units;  // (sequences that overlap, which is an error, can have more than 2^31 in all)
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int v = __shfl_up_sync(0xffffffffu, upto, o);
                    if (lane >= o) asm("add.sat.s32 %0, %0, %1;\n" : "+r"(upto) : "r"(v));
                }
                continue;
            }
            const int at = __ffs(beyond) - 1;
            auto of = [&](int v) { return __shfl_sync(0xffffffffu, v, at); };
            const int prior = __shfl_sync(0xffffffffu, upto, max(0, at - 1));
            fill(A, share, of(b), Sequence{of(s.begin), of(s.rows), of(s.length)}, of(units), of(pieces), want,
                 want - before - (at > 0 ? prior : 0), U);
            return true;
        }
        return false;
    }
    // The last blocks of a sequence, which see the most keys, come first.
    __device__ __forceinline__ void fill(const Args& A, const Share& share, int b, const Sequence& s, int units, int pieces,
                                         int want, int in, Unit& U) {
        const int per = A.kv_heads * pieces, back = quotient(in, per), rest = in - back * per;
        const int head = quotient(rest, pieces), piece = rest - head * pieces;
        const int block = quotient(units, per) - 1 - back;
        U.live = 1;
        U.b = b, U.head = head;
        U.row0 = block * share.rows;
        U.rows = min(share.rows, s.rows * A.group - U.row0);
        U.begin = s.begin, U.first = s.length - s.rows, U.length = s.length;
        if (!A.causal) U.first = 0;
        int lo, hi, unused, hi0;
        const int from = A.by_group.quotient(U.row0), to = A.by_group.quotient(U.row0 + U.rows - 1);
        sees(A, U.first + from, U.length, lo, unused);
        sees(A, U.first + to, U.length, unused, hi);
        lo = min(lo, hi) & ~(kTile - 1);
        int tiles = (hi - lo + kTile - 1) / kTile;
        U.part = -1;
        U.first_part = want - piece, U.pieces = pieces;
        if (pieces > 1) {
            const int t0 = min(tiles, piece * share.piece), t1 = min(tiles, t0 + share.piece);
            U.part = want;
            lo += t0 * kTile;
            tiles = t1 - t0;
            hi = min(hi, lo + tiles * kTile);
        }
        U.key0 = lo, U.end = hi, U.tiles = tiles;
        U.shared = U.rows > kTile;
        U.tiles0 = tiles;
        if (U.shared) {
            sees(A, U.first + A.by_group.quotient(U.row0 + kTile - 1), U.length, unused, hi0);
            U.tiles0 = max(0, min(tiles, (hi0 - lo + kTile - 1) / kTile));
        }
    }
};

template <int D, class T, bool E4M3>
__global__ void __launch_bounds__((Plan<D, E4M3>::kThreads), 1)
attention_kernel(const __grid_constant__ Args A, const __grid_constant__ CUtensorMap q_map,
                 const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map) {
    using namespace tc;
    using P = Plan<D, E4M3>;
    constexpr bool BF = std::is_same_v<T, BF16>;
    constexpr float kLift = lift<T>, kSlack = slack<T>;
    constexpr int kCopyWarps = P::kCopyWarps, kCopyThreads = 32 * kCopyWarps;
    constexpr int kMmaWarp = P::kMmaWarp, kPlanWarp = P::kPlanWarp, kRawWarp = P::kRawWarp;
    extern __shared__ __align__(1024) uint8_t smem[];
    int& abort_flag = *reinterpret_cast<int*>(smem + P::kFlags);
    int& never_abort = *reinterpret_cast<int*>(smem + P::kFlags + 4);
    uint32_t& tmem_base = *reinterpret_cast<uint32_t*>(smem + P::kFlags + 8);
    uint32_t& redo = *reinterpret_cast<uint32_t*>(smem + P::kFlags + 12);  // bit min(m, 31): unit m of the first pass is for the second
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    volatile int* abort = &abort_flag;
    const uint32_t base = smem_u32(smem);
    const uint32_t ring = base + P::kQ;
    const uint32_t bars = base + P::kBars;
    auto full = [&](int s) { return bars + 8 * s; };
    auto empty = [&](int s) { return bars + 8 * (P::kStages + s); };
    const uint32_t more = bars + 16 * P::kStages;
    const uint32_t q_full = more, q_free = more + 8, o_free = more + 16, pv_done = more + 24, all_done = more + 32;
    auto s_full = [&](int i) { return more + 40 + 8 * i; };
    auto p_full = [&](int i) { return more + 56 + 8 * i; };  // 2 * buffer + half of the keys
    auto o_full = [&](int i) { return more + 88 + 8 * i; };
    auto u_full = [&](int i) { return more + 104 + 8 * i; };
    auto u_free = [&](int i) { return more + 120 + 8 * i; };
    auto raw_full = [&](int s) { return more + 176 + 16 * s; };
    auto raw_empty = [&](int s) { return more + 184 + 16 * s; };
    const uint32_t ml_full = more + 136, ml_free = more + 144;
    auto turn = [&](int i) { return more + 152 + 8 * i; };
    Unit* units = reinterpret_cast<Unit*>(smem + P::kUnits);
    volatile uint32_t* lost = reinterpret_cast<volatile uint32_t*>(smem + P::kLost);

    if (tid == 0) {
        abort_flag = (base & 1023u) != 0;  // the swizzle's atoms start on 1024-byte boundaries
        never_abort = 0;
        redo = 0;
        // One arrival a copying warp; where its lanes copy all by themselves, one of each and one for the
        // warp's other words.
        for (int s = 0; s < P::kStages; ++s) {
            mbar_init(full(s), A.keys.box > 0 ? kCopyWarps : E4M3 ? 4 : 33 * 4);
            mbar_init(empty(s), 2);
        }
        mbar_init(q_full, kCopyThreads), mbar_init(q_free, 2);
        mbar_init(o_free, kSoftmaxWarps), mbar_init(pv_done, 1), mbar_init(all_done, P::kStreams);
        mbar_init(ml_full, kSoftmaxWarps), mbar_init(ml_free, kSoftmaxWarps);
        for (int i = 0; i < 2; ++i) {
            mbar_init(s_full(i), 1), mbar_init(p_full(2 * i), 4), mbar_init(p_full(2 * i + 1), 4), mbar_init(o_full(i), 1);
            mbar_init(turn(i), 1), mbar_init(u_full(i), 1), mbar_init(u_free(i), kSoftmaxWarps + kCopyWarps + P::kStreams + (E4M3 ? 1 : 0));
        }
        for (int s = 0; s < P::kRawStages; ++s) mbar_init(raw_full(s), 1), mbar_init(raw_empty(s), kCopyWarps);
        fence_mbar_init();
        mbar_arrive(turn(0));  // the first turn is the first stream's
    }
    if (warp == kMmaWarp) tmem_alloc(smem_u32(&tmem_base), 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_base;
    if (tid == 0 && A.keys.box > 0) prefetch_tensor_map(&k_map), prefetch_tensor_map(&v_map);
    if (tid == 32 && A.q_boxes) prefetch_tensor_map(&q_map);
    pdl_wait();
    pdl_launch_dependents();

    auto wait = [&](uint32_t bar, uint32_t parity) {
        if (warp_wait_parity_suspend(bar, parity, abort, kWaitNs, kSuspendNs)) return true;
        *abort = 1;
        return false;
    };
    // The same for what comes when a unit of so many tiles is done with.
    auto wait_for_unit = [&](uint32_t bar, uint32_t parity, int tiles) {
        if (warp_wait_parity_suspend(bar, parity, abort, A.wait_ns + tiles * A.tile_ns, kSuspendNs)) return true;
        *abort = 1;
        return false;
    };
    // The next unit, for every warp that works on it; nullptr: there are no more of this pass.  done_with gives
    // its place back.
    uint32_t n_unit = 0;
    auto done_with = [&]() {
        __syncwarp();
        if (lane == 0) mbar_arrive(u_free(n_unit & 1));
        ++n_unit;
    };
    auto unit = [&]() -> const Unit* {
        if (!wait(u_full(n_unit & 1), n_unit >> 1 & 1)) return nullptr;
        if (units[n_unit & 1].live) return units + (n_unit & 1);
        done_with();
        return nullptr;
    };
    // The end of a pass: whether a second one follows.
    auto pass_ends = [&]() {
        tc_fence_before();
        __syncthreads();
        return *static_cast<volatile uint32_t*>(&redo) != 0 && !*abort;
    };
    // What a warp does in both: one code for both passes, or (`twice`) a code each, where a loop around the first one costs
    // it registers.
    auto passes = [&](auto work) {
#pragma unroll 1
        for (int pass = 0; pass < 2; ++pass) {
            work(pass);
            if (!pass_ends()) return;
        }
    };
    auto twice = [&](auto work) {
        work(std::false_type{});
        if (!pass_ends()) return;
        work(std::true_type{});
        pass_ends();
    };

    auto plan = [&](int pass) {
        Sequence mine{0, 0, 0};
        bool any = false;
        if (lane < A.seqs) mine = sequence(A, lane, any);
        if (blockIdx.x == 0 && pass == 0) {
            for (int b = lane + 32; b < A.seqs; b += 32) {
                bool bad;
                sequence(A, b, bad);
                any |= bad;
            }
            if (any) atomicExch(&g_prompt_status, int(W4A4_ERR_INDEX));
        }
        uint8_t* const order = smem + P::kOrder;
        const bool sorted = A.seqs > 1 && A.seqs <= kSorted;
        if (sorted) sort_sequences(A, mine, order);
        const Share share = share_out<D>(A, mine);
        Walk walk{sorted ? order : nullptr, mine};
        int last = 0, before = 0;
        const uint32_t chosen = pass == 0 ? 0xffffffffu : redo;
        for (uint32_t m = 0;; ++m) {
            const int turn = int(m & 1 ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
            Unit U{};
            const bool live = walk.find(A, share, int(m * gridDim.x) + turn, U);
            if (live && !(chosen >> min(m, 31u) & 1)) continue;
            if (live && pass > 0) U.live = second_pass(A, U);
            const uint32_t n = n_unit++;
            const int tiles = before;  // of the unit whose place this one takes
            before = last, last = U.tiles;
            if (n == 0 && A.parts && lane == 0) {
                const bool part = live && U.part >= 0;
                A.parts_of[2 * blockIdx.x] = make_int4(U.begin, U.head, U.row0, U.rows);
                A.parts_of[2 * blockIdx.x + 1] = make_int4(U.first_part, part ? U.pieces : 0, 0, 0);
            }
            if (n >= 2 && !wait_for_unit(u_free(n & 1), (n >> 1 & 1) ^ 1, tiles)) return;
            if (lane == 0) {
                units[n & 1] = U;
                mbar_arrive(u_full(n & 1));
            }
            if (!live) return;
        }
    };

    // ---- queries, keys and values into shared memory
    uint32_t n_stage = 0, n_q = 0;  // copies of stages begun, units whose queries were copied
    uint32_t n_tile = 0;            // tiles of the units that are done with
    auto copy_queries = [&](const Unit& U) {
        if (n_q > 0 && !wait(q_free, (n_q - 1) & 1)) return false;
        ++n_q;
        if (A.q_boxes) {
            // (token, head) pairs side by side are a box of whole tokens.  Those behind the unit's rows,
            // another sequence's or none, are rows of scores that nobody reads.
            constexpr int kPlanes = P::kHalves * P::kPlanes;
            const int i = tid - 32 * kSoftmaxWarps, tiles = U.shared ? 2 : 1;
            if (i == 0)
                mbar_expect_tx(q_full, tiles * P::kQTile);
            else
                mbar_arrive(q_full);
            if (i < tiles * kPlanes) {
                const int h = i / kPlanes, plane = i - h * kPlanes;
                tma_load_4d(base + h * P::kQTile + plane * (kTile * 128), &q_map, 64 * plane, U.head * A.group,
                            U.begin + A.by_group.quotient(U.row0 + h * kTile), 0, q_full);
            }
            return true;
        }
        constexpr int kPieces = D * 2 / 16, kRounds = kTile * kPieces / kCopyThreads;
        for (int h = 0; h < (U.shared ? 2 : 1); ++h) {
            const uint32_t to = base + h * P::kQTile;
#pragma unroll 4
            for (int i = 0; i < kRounds; ++i) {
                const int id = i * kCopyThreads + tid - 32 * kSoftmaxWarps, row = id / kPieces, c = id - row * kPieces;
                const bool ok = h * kTile + row < U.rows;
                const int flat = ok ? U.row0 + h * kTile + row : 0, token = A.by_group.quotient(flat), g = flat - token * A.group;
                const char* src = A.q + 2 * ((U.begin + token) * A.q_token + (U.head * A.group + g) * A.q_head) + 16 * c;
                cp_async16_zfill(to + swizzled(row, c), src, ok ? 16 : 0);
            }
        }
        cp_async_mbar_arrive_noinc(q_full);
        return true;
    };
    // The place of the next copy in the ring, free to be written.
    auto next_stage = [&](int& st) {
        st = n_stage % P::kStages;
        if (n_stage >= P::kStages && !wait(empty(st), (n_stage / P::kStages - 1) & 1)) return false;
        ++n_stage;
        return true;
    };
    // Copies go in the order of use: the values of a tile behind the keys of the tile after it
    // (shared rows) or of the two after it.  copy_tiles(tiles, lag, look, send): look(u) prepares
    // tile u, send(kv, half, age) copies its keys (age 0) or the values of the tile `age` before.
    auto copy_tiles = [&](int tiles, int lag, auto look, auto send) {
        for (int u = 0; u < tiles + lag; ++u) {
            look(u);
#pragma unroll 1
            for (int half = 0; u >= lag && half < P::kHalves; ++half)
                if (!send(1, half, lag, u - lag)) return false;
#pragma unroll 1
            for (int half = 0; u < tiles && half < P::kHalves; ++half)
                if (!send(0, half, 0, u)) return false;
        }
        return true;
    };
    auto lag_of = [&](const Unit& U) { return P::kStreams == 2 && U.shared ? 1 : 2; };

    // 16 E4M3 elements, piece c of a row, as 16-bit ones into a stage.
    auto widen16 = [&](const uint4& raw, uint8_t* stage, int row, int c, bool rows_apart) {
        const uint32_t four[4] = {raw.x, raw.y, raw.z, raw.w};
        uint32_t two[8];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            e4m3x4_to_f16x2(four[k], two[2 * k], two[2 * k + 1]);
            if constexpr (BF) {  // exact: four significant bits
                const float2 f = F16::up(two[2 * k]), g = F16::up(two[2 * k + 1]);
                two[2 * k] = BF16::down(f.x, f.y), two[2 * k + 1] = BF16::down(g.x, g.y);
            }
        }
        // where eight lanes have pieces of one row, those of the second plane begin with the other half, so
        // that they hit all banks
        const bool odd = !rows_apart && (c >> 2 & 1);
        const uint4 lo = make_uint4(two[0], two[1], two[2], two[3]), hi = make_uint4(two[4], two[5], two[6], two[7]);
        *reinterpret_cast<uint4*>(stage + swizzled(row, 2 * c + odd)) = odd ? hi : lo;
        *reinterpret_cast<uint4*>(stage + swizzled(row, 2 * c + !odd)) = odd ? lo : hi;
    };

    // By the copy engine, each warp 32 rows of a tile, a box of K.box of them a lane; boxes that
    // are not all there by the warp's own loads.  (One warp for all of them has fewer instructions
    // but sends small boxes more slowly: 1.8 times the time for pages of 24, D = 256.)
    auto copy_boxes = [&]() {
        const Keys& K = A.keys;
        const int box = K.box, boxes = 32 / box, w = warp - kSoftmaxWarps, my = 32 * w + lane * box;
        const uint32_t all = (1u << boxes) - 1;
        for (;; done_with()) {
            const Unit* const U = unit();
            if (!U) return;
            if (U->tiles == 0) continue;
            const int key0 = U->key0, end = U->end, tiles = U->tiles, begin = U->begin, head = U->head;
            const int64_t table = U->b * K.table_stride;
            int page = 0, slot = 0;  // of this lane's box in the next tile
            auto look_up = [&](int tile) {
                const int j = key0 + tile * kTile + my;
                slot = begin + j;
                if (K.table && lane < boxes && tile < tiles && j < end) {
                    const int p = K.by_page.quotient(j);
                    slot = j - p * K.page_size;
                    page = K.table[table + p];
                }
            };
            look_up(0);
            if (!copy_queries(*U)) return;
            // of a tile and the two before it: this lane's page and slot, boxes that are all there, and that
            // are in part
            int pages[3] = {}, slots[3] = {};
            uint32_t whole[3] = {}, some[3] = {};
            auto look = [&](int u) {
#pragma unroll
                for (int k = 2; k > 0; --k)
                    pages[k] = pages[k - 1], slots[k] = slots[k - 1], whole[k] = whole[k - 1], some[k] = some[k - 1];
                if (u >= tiles) return;
                const int j = key0 + u * kTile + my;
                const bool in = lane < boxes && j < end, good = in && (!K.table || (page >= 0 && page < K.pages));
                some[0] = __ballot_sync(0xffffffffu, good), whole[0] = __ballot_sync(0xffffffffu, good && j + box <= end);
                pages[0] = page, slots[0] = slot;
                if (K.table) {
                    const uint32_t bad = __ballot_sync(0xffffffffu, in && !good);
                    if (lane == 0) {
                        uint32_t word = 0;
                        for (int k = 0; bad != 0 && k < boxes; ++k)
                            if (bad >> k & 1) word |= (0xffffffffu >> (32 - box)) << k * box;
                        lost[(n_tile + u) % kLostTiles * 4 + w] = word;
                        if (bad) atomicExch(&g_prompt_status, int(W4A4_ERR_INDEX));
                    }
                    look_up(u + 1);
                } else {
                    slot += kTile;
                }
            };
            auto send = [&](int kv, int half, int age, int tile) {
                int st;
                if (!next_stage(st)) return false;
                const uint32_t to = ring + st * P::kStage;
                const uint32_t there = age == 0 ? whole[0] : age == 1 ? whole[1] : whole[2];
                const int pg = age == 0 ? pages[0] : age == 1 ? pages[1] : pages[2];
                const int sl = age == 0 ? slots[0] : age == 1 ? slots[1] : slots[2];
                const uint32_t bytes = __popc(there) * box * 128 * P::kPlanes;
                if (lane == 0) {  // the warp's one arrival, or with rows of its own still to come (below) without it
                    if (there == all)
                        mbar_expect_tx(full(st), bytes);
                    else
                        mbar_expect_tx_only(full(st), bytes);
                }
                // lane 16 p + b: plane p of box b
                const int from = lane & 15, y = __shfl_sync(0xffffffffu, sl, from), z = __shfl_sync(0xffffffffu, pg, from);
                if (there >> from & 1 && lane < 16 * P::kPlanes)
                    tma_load_4d(to + (lane >> 4) * (kTile * 128) + (32 * w + from * box) * 128, kv ? &v_map : &k_map,
                                half * P::kDs + 64 * (lane >> 4), y, head, K.table ? z : 0, full(st));
                if (there != all) {
                    const uint32_t s = age == 0 ? some[0] : age == 1 ? some[1] : some[2];
                    const char* pool = K.pool[kv] + int64_t(head) * K.head_stride[kv] + half * P::kDs * 2;
                    constexpr int kPieces = P::kDs * 2 / 16;
                    for (int b = 0; b < boxes; ++b) {
                        if (there >> b & 1) continue;
                        const int have = s >> b & 1 ? end - (key0 + tile * kTile + 32 * w + b * box) : 0;
                        const int p = __shfl_sync(0xffffffffu, pg, b), y = __shfl_sync(0xffffffffu, sl, b);
                        const char* from = have > 0 ? pool + (K.table ? p * K.page_stride[kv] : 0) + int64_t(y) * K.token_stride[kv] : pool;
                        for (int i = lane; i < box * kPieces; i += 32) {
                            const int r = i / kPieces, c = i - r * kPieces;
                            cp_async16_zfill(to + swizzled(32 * w + b * box + r, c), r < have ? from + int64_t(r) * K.token_stride[kv] + 16 * c : pool,
                                             r < have ? 16 : 0);
                        }
                    }
                    cp_async_mbar_arrive(full(st));  // one more to wait for, until they are there
                    __syncwarp();
                    if (lane == 0) mbar_arrive(full(st));
                }
                return true;
            };
            if (!copy_tiles(tiles, lag_of(*U), look, send)) return;
            n_tile += tiles;
        }
    };

    // 8-bit rows by the copy engine, a box a lane, into their ring; pages behind a sequence's end
    // come as they are, pages outside the pool do not.
    uint32_t n_raw = 0;
    auto copy_raw = [&]() {
        const Keys& K = A.keys;
        const int box = K.box, boxes = box > 0 ? kTile / box : 0, my = lane * box;
        uint32_t* const there = reinterpret_cast<uint32_t*>(smem + P::kThere);
        for (;; done_with()) {
            const Unit* const U = unit();
            if (!U) return;
            if (U->tiles == 0 || box == 0) continue;
            const int key0 = U->key0, end = U->end, tiles = U->tiles, head = U->head;
            const int64_t table = U->b * K.table_stride;
            // of this lane's box in the next tile and the one after it: a look-up takes longer than a tile
            int page = -1, slot = 0, page2 = -1, slot2 = 0;
            auto look_up = [&](int tile, int& page, int& slot) {
                const int j = key0 + tile * kTile + my;
                page = -1;
                if (lane < boxes && tile < tiles && j < end) {
                    const int p = K.by_page.quotient(j);
                    slot = j - p * K.page_size;
                    page = K.table[table + p];
                }
            };
            look_up(0, page, slot);
            look_up(1, page2, slot2);
            int pages[3] = {}, slots[3] = {};   // of a tile and the two before it,
            uint32_t some[3] = {}, mine[3] = {};  // boxes on pages of the pool, and which of rows 32 lane .. + 31 are there
            auto look = [&](int u) {
#pragma unroll
                for (int k = 2; k > 0; --k) pages[k] = pages[k - 1], slots[k] = slots[k - 1], some[k] = some[k - 1], mine[k] = mine[k - 1];
                if (u >= tiles) return;
                const bool in = lane < boxes && key0 + u * kTile + my < end, good = in && page >= 0 && page < K.pages;
                some[0] = __ballot_sync(0xffffffffu, good), pages[0] = page, slots[0] = slot;
                const uint32_t bad = __ballot_sync(0xffffffffu, in && !good);
                if (lane < 4) {
                    uint32_t word = 0;
                    for (int k = 0; bad != 0 && k < 32; k += box)
                        if (bad >> quotient(32 * lane + k, box) & 1) word |= (0xffffffffu >> (32 - box)) << k;
                    lost[(n_tile + u) % kLostTiles * 4 + lane] = word;
                    const int have = end - (key0 + u * kTile + 32 * lane);
                    mine[0] = (have >= 32 ? 0xffffffffu : have > 0 ? (1u << have) - 1 : 0) & ~word;
                }
                if (bad && lane == 0) atomicExch(&g_prompt_status, int(W4A4_ERR_INDEX));
                page = page2, slot = slot2;
                look_up(u + 2, page2, slot2);
            };
            auto send = [&](int kv, int half, int age, int) {
                const int st = n_raw % P::kRawRing;
                if (n_raw >= P::kRawRing && !wait(raw_empty(st), (n_raw / P::kRawRing - 1) & 1)) return false;
                ++n_raw;
                const uint32_t s = age == 0 ? some[0] : age == 1 ? some[1] : some[2];
                const int pg = age == 0 ? pages[0] : age == 1 ? pages[1] : pages[2];
                const int sl = age == 0 ? slots[0] : age == 1 ? slots[1] : slots[2];
                if (lane < 4) there[4 * st + lane] = age == 0 ? mine[0] : age == 1 ? mine[1] : mine[2];
                __syncwarp();
                if (lane == 0) mbar_expect_tx(raw_full(st), __popc(s) * box * P::kDs);
                if (s >> lane & 1)
                    tma_load_4d(base + P::kRaw + st * P::kRawStage + my * P::kDs, kv ? &v_map : &k_map, half * P::kDs, sl, head, pg,
                                raw_full(st));
                return true;
            };
            if (!copy_tiles(tiles, lag_of(*U), look, send)) return;
            n_tile += tiles;
        }
    };
    // ... and turned into 16-bit rows by eight warps.
    uint32_t n_read = 0;
    auto widen = [&]() {
        const int t = tid - 32 * kSoftmaxWarps;
        for (;; done_with()) {
            const Unit* const U = unit();
            if (!U) return;
            if (U->tiles == 0) continue;
            const int stages = 2 * P::kHalves * U->tiles;
            if (!copy_queries(*U)) return;
            for (int x = 0; x < stages; ++x) {
                constexpr int kRowPieces = P::kDs / 16, kPieces = kTile * kRowPieces / kCopyThreads;
                const int from = n_read % P::kRawRing;
                if (!wait(raw_full(from), n_read / P::kRawRing & 1)) return;
                ++n_read;
                const uint8_t* src = smem + P::kRaw + from * P::kRawStage;
                // piece c of a row: eight lanes take eight rows' where rows are 128 bytes (and swizzled),
                // else what lies side by side
                auto place = [&](int i, int& row, int& c) {
                    const int id = i * kCopyThreads + t;
                    if constexpr (P::kRawSwizzled) {
                        row = (id & 7) | (id >> 6) << 3, c = id >> 3 & 7;
                        return row * 128 + ((c ^ (row & 7)) << 4);
                    } else {
                        row = id / kRowPieces, c = id - row * kRowPieces;
                        return 16 * id;
                    }
                };
                const uint32_t* const there = reinterpret_cast<const uint32_t*>(smem + P::kThere) + 4 * from;
                const uint4 rows = *reinterpret_cast<const uint4*>(there);
                uint4 raw[kPieces];
#pragma unroll
                for (int i = 0; i < kPieces; ++i) {
                    int row, c;
                    raw[i] = *reinterpret_cast<const uint4*>(src + place(i, row, c));
                }
                if ((rows.x & rows.y & rows.z & rows.w) != 0xffffffffu)
#pragma unroll
                    for (int i = 0; i < kPieces; ++i) {
                        int row, c;
                        place(i, row, c);
                        if (!(there[row >> 5] >> (row & 31) & 1)) raw[i] = make_uint4(0, 0, 0, 0);
                    }
                int st;  // waited for with the rows in registers, so that the next ones are on their way
                if (!next_stage(st)) return;
                // Read before the copy engine writes there again: the rows are not used until here, and while
                // products take the port of the shared memory the loads could come behind the next copy (D = 256:
                // eight rows of another tile, once in 200 units).  The fence costs 64 sequences of 4 tokens 5% (175 -> 183 us).
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(raw_empty(from));
                uint8_t* dst = smem + P::kQ + st * P::kStage;
#pragma unroll
                for (int i = 0; i < kPieces; ++i) {
                    int row, c;
                    place(i, row, c);
                    widen16(raw[i], dst, row, c, P::kRawSwizzled);
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(full(st));
            }
        }
    };

    // By loads of four warps, 32 rows of a tile each, where there are no tensor maps: pages that are
    // not whole times eight, strides that a map cannot have.  E4M3 rows are turned into 16-bit ones
    // on the way.
    auto copy_rows = [&]() {
        constexpr int kSize = E4M3 ? 1 : 2;
        constexpr int kPieces = P::kDs * kSize / 16;  // of a stage's row
        const Keys& K = A.keys;
        const int w = warp - kSoftmaxWarps;
        for (;; done_with()) {
            const Unit* const U = unit();
            if (!U) return;
            if (U->tiles == 0) continue;
            const int key0 = U->key0, end = U->end, tiles = U->tiles, begin = U->begin, head = U->head;
            const int64_t table = U->b * K.table_stride;
            int page = -1, slot = 0;  // of key 32 w + lane of the next tile
            auto look_up = [&](int tile) {
                const int j = key0 + tile * kTile + 32 * w + lane;
                page = -1;
                if (tile < tiles && j < end) {
                    const int p = K.by_page.quotient(j);
                    slot = j - p * K.page_size;
                    page = K.table[table + p];
                }
            };
            if (K.table) look_up(0);
            if (!copy_queries(*U)) return;
            if (w >= 4) continue;  // (of the warps that widen 8-bit rows)
            uint32_t ok[3] = {};              // of a tile and the two before it: keys that are there,
            int64_t k_off = 0, v_off[3] = {};  // and where this lane's is
            auto look = [&](int u) {
                ok[2] = ok[1], ok[1] = ok[0];
                v_off[2] = v_off[1], v_off[1] = v_off[0];
                if (u >= tiles) return;
                const int j0 = key0 + u * kTile + 32 * w;
                if (K.table) {
                    const bool good = page >= 0 && page < K.pages;
                    ok[0] = __ballot_sync(0xffffffffu, good);
                    const uint32_t bad = __ballot_sync(0xffffffffu, !good && j0 + lane < end);
                    if (lane == 0) {
                        if (bad) atomicExch(&g_prompt_status, int(W4A4_ERR_INDEX));
                        lost[(n_tile + u) % kLostTiles * 4 + w] = bad;
                    }
                    k_off = good ? page * K.page_stride[0] + int64_t(slot) * K.token_stride[0] : 0;
                    v_off[0] = good ? page * K.page_stride[1] + int64_t(slot) * K.token_stride[1] : 0;
                    look_up(u + 1);
                } else {
                    const int have = max(0, min(32, end - j0));
                    ok[0] = have == 32 ? 0xffffffffu : (1u << have) - 1;
                    if (lane < have) {
                        k_off = int64_t(begin + j0 + lane) * K.token_stride[0];
                        v_off[0] = int64_t(begin + j0 + lane) * K.token_stride[1];
                    }
                }
            };
            auto send = [&](int kv, int half, int age, int) {
                int st;
                if (!next_stage(st)) return false;
                const uint32_t to = ring + st * P::kStage;
                const uint32_t there = age == 0 ? ok[0] : age == 1 ? ok[1] : ok[2];
                const int64_t mine = kv == 0 ? k_off : age == 1 ? v_off[1] : v_off[2];
                const char* pool = K.pool[kv] + int64_t(head) * K.head_stride[kv] + half * P::kDs * kSize;
                auto source = [&](int r, int c) { return pool + 16 * c + __shfl_sync(0xffffffffu, mine, r); };
                if constexpr (!E4M3) {
#pragma unroll
                    for (int i = 0; i < kPieces; ++i) {
                        const int id = i * 32 + lane, r = id / kPieces, c = id - r * kPieces;
                        const char* src = source(r, c);
                        cp_async16_zfill(to + swizzled(32 * w + r, c), there >> r & 1 ? src : pool, there >> r & 1 ? 16 : 0);
                    }
                    cp_async_mbar_arrive_noinc(full(st));
                } else {
                    // (all at once do not fit the warp's registers)
                    constexpr int kAtOnce = kPieces % 4 == 0 ? 4 : 2;
#pragma unroll 1
                    for (int from = 0; from < kPieces; from += kAtOnce) {
                        uint4 raw[kAtOnce];
#pragma unroll
                        for (int i = 0; i < kAtOnce; ++i) {
                            const int id = (from + i) * 32 + lane, r = id / kPieces, c = id - r * kPieces;
                            const char* src = source(r, c);
                            raw[i] = there >> r & 1 ? ldg_stream_v4(src) : make_uint4(0, 0, 0, 0);
                        }
#pragma unroll
                        for (int i = 0; i < kAtOnce; ++i) {
                            const int id = (from + i) * 32 + lane, r = id / kPieces, c = id - r * kPieces, row = 32 * w + r;
                            widen16(raw[i], smem + (to - base), row, c, false);
                        }
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                }
                if (lane == 0) mbar_arrive(full(st));  // for the warp's word of `lost`, or its rows
                return true;
            };
            if (!copy_tiles(tiles, lag_of(*U), look, send)) return;
            n_tile += tiles;
        }
    };

    // The products of a stream, issued by one thread: the queue of the tensor cores holds two or
    // three, so what this thread does between the arrival of the probabilities and the next
    // scores leaves them idle, but for the other stream's.  With both streams' products from one
    // thread 8192 tokens of 32 heads of 128 took 450 us (413 now), and with descriptors that the
    // compiler sums up 690.
    uint32_t stages = 0;                                    // before this unit
    uint32_t turns = 0, n_o = 0, p_phase = 0, q_phase = 0;  // units with an output; bit i: the parity of p_full(i, .)
    auto multiply = [&](const int stream, auto second) {
        constexpr uint32_t kQk = idesc_m128_16bit(kTile, BF, false);
        constexpr uint32_t kPv = idesc_m128_16bit(P::kDs, BF, true);
        constexpr int kAhead = P::kStreams == 1 ? 2 : 1;  // tiles whose scores are under way
        // descriptors' low words (their high words are alike)
        const uint32_t keys0 = uint32_t(sdesc_sw128(ring)), values0 = uint32_t(sdesc_sw128(ring, kTile * 128));
        const uint32_t q0 = uint32_t(sdesc_sw128(base)), hi = uint32_t(sdesc_sw128(0) >> 32);
        auto wait1 = [&](uint32_t bar, uint32_t parity) {
            if (wait_parity_suspend(bar, parity, abort, kWaitNs, kSuspendNs)) return true;
            *abort = 1;
            return false;
        };
        for (;; ++n_unit) {
            const int i = n_unit & 1;
            if (!wait1(u_full(i), n_unit >> 1 & 1)) return;
            const Unit& U = units[i];
            const bool live = U.live != 0, shared = P::kStreams == 2 && U.shared;
            const int tiles = U.tiles, tiles0 = U.tiles0, kind = U.live;
            mbar_arrive(u_free(i));
            if (!live) {
                ++n_unit;
                return;
            }
            if (tiles == 0) continue;
            // this stream's tiles: `first`, `first` + `step`, ...
            const int first = P::kStreams == 2 && !shared ? stream : 0, step = P::kStreams == 2 && !shared ? 2 : 1;
            const int mine = shared ? (stream ? tiles : tiles0) : (tiles + step - 1 - first) / step;
            // where the copies of a tile's keys (values) are in their order
            auto keys_at = [&](int t) { return stages + P::kHalves * (shared ? 2 * t : max(0, 2 * t - 1)); };
            auto values_at = [&](int t) {
                return stages + P::kHalves * (shared || t == tiles - 1 ? 2 * t + 1 : 2 * t + 2);
            };
            auto ready = [&](uint32_t at) {
                if (!wait1(full(at % P::kStages), at / P::kStages & 1)) return false;
                if (!E4M3) fence_proxy_async_smem();  // copies of some went through the generic proxy
                return true;
            };
            // Both streams' threads go through all stages in their order and each gives every one back: a
            // thread that left the other's out would wait for a later use of the same place by a
            // parity that the use before the other's has too.
            auto release = [&](uint32_t at) {
                mma_commit(empty(at % P::kStages));
                if (P::kStreams == 1) mbar_arrive(empty(at % P::kStages));
            };
            auto see = [&](uint32_t at) {  // a stage of the other stream
                if (!wait1(full(at % P::kStages), at / P::kStages & 1)) return false;
                mbar_arrive(empty(at % P::kStages));
                return true;
            };
            const bool alternate = P::kStreams == 2 && !shared;
            auto see_keys = [&](int t) { return !alternate || t >= tiles || see(keys_at(t)); };
            auto see_values = [&](int t) { return !alternate || t >= tiles || see(values_at(t)); };
            if (!wait1(q_full, q_phase)) return;
            q_phase ^= 1;
            fence_proxy_async_smem();
            const uint32_t q = q0 + (shared && stream ? P::kQTile >> 4 : 0);
            auto keys_ready = [&](int x) {  // of this stream's x-th tile
                const uint32_t at = keys_at(first + x * step);
                return ready(at) && (P::kHalves == 1 || ready(at + 1));
            };
            auto scores = [&](int x) {
                const int buf = P::kStreams == 1 ? x & 1 : stream;
                const uint32_t at = keys_at(first + x * step);
#pragma unroll
                for (int half = 0; half < P::kHalves; ++half) {
                    mma_f16_rows<P::kDs / 16>(tmem + P::scores(buf), q + half * (P::kStage >> 4),
                                              keys0 + (at + half) % P::kStages * (P::kStage >> 4), hi, kQk, half > 0);
                }
                mma_commit(s_full(buf));
            };
            auto release_keys = [&](int x) {
                const uint32_t at = keys_at(first + x * step);
#pragma unroll
                for (int half = 0; half < P::kHalves; ++half) release(at + half);
                if (x == mine - 1) {
                    mma_commit(q_free);
                    if (P::kStreams == 1) mbar_arrive(q_free);
                }
            };
            if (mine == 0) mbar_arrive(q_free);
            // The streams take turns, so that the products of one end before the other's begin (side
            // by side each takes twice as long, and then both streams wait).  Both go through as many.
            const int other = P::kStreams == 1 ? 0 : shared ? (stream ? tiles0 : tiles) : (tiles + stream) / 2;
            auto my_turn = [&]() { return P::kStreams == 1 || (wait1(turn(stream), turns & 1) && ++turns); };
            auto pass = [&]() {
                if (P::kStreams == 2) mbar_arrive(turn(stream ^ 1));
            };
            if (stream == 1 && !see_keys(0)) return;
            for (int x = 0; x < min(kAhead, mine); ++x)
                if (!keys_ready(x)) return;
            if (!my_turn()) return;
            for (int x = 0; x < min(kAhead, mine); ++x) scores(x);
            pass();
            for (int x = 0; x < min(kAhead, mine); ++x) release_keys(x);
            if (stream == 0 ? !see_keys(1) : !see_values(0) || !see_keys(2)) return;
            for (int x = 0; x < max(mine, other); ++x) {
                if (x >= mine) {
                    if (!my_turn()) return;
                    pass();
                    continue;
                }
                const int buf = P::kStreams == 1 ? x & 1 : stream;
                const uint32_t at = values_at(first + x * step);
                for (int half = 0; half < P::kHalves; ++half) {
                    if (!ready(at + half)) return;
                    if (second && partly_seen(kind, first + x * step, tiles))
                        clean_stage<BF, P::kStage>(smem + P::kQ + (at + half) % P::kStages * P::kStage);
                }
                if (P::kStreams == 2 && x + kAhead < mine && !keys_ready(x + kAhead)) return;
                if (x == 0 && n_o > 0 && !wait1(o_free, (n_o - 1) & 1)) return;  // the last unit's output has been read
#pragma unroll
                for (int part = 0; part < 2; ++part) {
                    if (!wait1(p_full(2 * buf + part), p_phase >> buf & 1)) return;
                    if (part == 0 && !my_turn()) return;
                    tc_fence_after();
#pragma unroll
                    for (int half = 0; half < P::kHalves; ++half)
                        mma_f16_tmem_a_rows(tmem + P::output(stream) + half * P::kDs, tmem + P::scores(buf) + 32 * part,
                                            values0 + (at + half) % P::kStages * (P::kStage >> 4) + part * (64 * 128 >> 4), hi,
                                            kPv, x > 0 || part > 0);
                }
                p_phase ^= 1u << buf;
                if constexpr (P::kStreams == 1) mma_commit(pv_done);
                if (x == mine - 1) mma_commit(o_full(stream));
                if constexpr (P::kStreams == 1) {  // nobody waits for a turn: the values' room first
                    for (int half = 0; half < P::kHalves; ++half) release(at + half);
                    if (x + kAhead < mine && !keys_ready(x + kAhead)) return;
                }
                if (x + kAhead < mine) scores(x + kAhead);
                pass();
                if (x + kAhead < mine) release_keys(x + kAhead);
                if constexpr (P::kStreams == 2) release(at);
                if (!see_values(first + x * step + 1) || !see_keys(first + x * step + 3)) return;
            }
            for (int t = mine; shared && t < tiles; ++t) {  // tiles of the other stream alone
                if (!see(keys_at(t)) || !see(values_at(t))) return;
            }
            ++n_o;
            stages += 2 * P::kHalves * tiles;
        }
    };

    uint32_t s_phase = 0, o_phase = 0, n_ml = 0;  // bit i: the parity of s_full(i), o_full(i)
    auto softmax = [&]() {
        const int stream = warp >> 2, row = tid & 127;
        const uint32_t lanes = uint32_t(warp & 3) << 21;  // this warp's lanes of tensor memory
        float* ml = reinterpret_cast<float*>(smem + P::kMl);
        for (;; done_with()) {
            const Unit* const unit_n = unit();
            if (!unit_n) return;
            const Unit& U = *unit_n;
            const bool shared = P::kStreams == 2 && U.shared;
            // scores go by |scale|, keys' scale and log2 e; a negative scale turns their sign, and
            // a scale of zero makes them zero
            float scale2 = A.scale * 1.44269504088896341f, flip = 1.f;
            if (E4M3 && A.keys.scale[0]) scale2 *= A.keys.scale[0][U.head];
            if (!(scale2 > 0.f)) {
                flip = scale2 < 0.f ? -1.f : scale2 == 0.f ? 0.f : scale2;  // NaN stays
                scale2 = scale2 < 0.f ? -scale2 : 1.f;
            }
            int lo = 0, hi = INT32_MAX;
            if (const int local = (shared ? stream * kTile : 0) + row; local < U.rows)
                sees(A, U.first + A.by_group.quotient(U.row0 + local), U.length, lo, hi);
            const bool idle = (shared ? stream * kTile : 0) + (row & ~31) >= U.rows;  // none of the warp's rows is one
            const int mine = P::kStreams == 1 ? (stream == 0 ? U.tiles : 0)
                             : shared         ? (stream == 0 ? U.tiles0 : U.tiles)
                                              : (U.tiles + 1 - stream) / 2;
            float top = -INFINITY, sum = 0.f;  // what is subtracted (of the scores as they come), and the sum
            // The scores of the stream's i-th tile into probabilities.  They are loaded twice, once for
            // their maximum and once, half a tile at a time, for their powers: kept in between they
            // and their results were moved and spilled, 340 instructions of 900 for a warp's tile.
            auto probabilities = [&](uint32_t at, int buf, int i) {
                float m[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int part = 0; part < 2; ++part) {
                    float s[64];
                    tmem_ld32_at(at + 64 * part, s);
                    tmem_ld32_at(at + 64 * part + 32, s + 32);
                    tmem_wait_ld();
#pragma unroll
                    for (int c = 0; c < 64; c += 8)
#pragma unroll
                        for (int k = 0; k < 4; ++k) m[k] = max3(m[k], s[c + k], s[c + 4 + k]);
                }
                const float most = fmaxf(max3(m[0], m[1], m[2]), m[3]);
                const bool renew = i == 0 || (most - top) * scale2 > kSlack;
                if (__any_sync(0xffffffffu, renew)) {
                    // what is there so far was taken relative to the old maximum
                    const float by = i == 0 ? 0.f : renew ? ex2((top - most) * scale2) : 1.f;
                    if (renew) top = most;
                    sum = i == 0 ? 0.f : sum * by;
                    if (i > 0) {
                        if constexpr (P::kStreams == 1)  // the product before this one, still under way
                            if (!wait(pv_done, (n_tile + i - 1) & 1)) return false;
                        tc_fence_after();
                        const uint32_t o_at = tmem + lanes + P::output(P::kStreams == 1 ? 0 : stream);
#pragma unroll 1
                        for (int c = 0; c < D; c += 32) {
                            float o[32];
                            tmem_ld32(o_at + c, o);
                            tmem_wait_ld();
#pragma unroll
                            for (int k = 0; k < 32; ++k) o[k] *= by;
                            tmem_st32(o_at + c, o);
                        }
                    }
                }
                const float ref = (top == -INFINITY ? 0.f : top * scale2) - kLift;
                const uint64_t by2 = f2_pack(scale2, scale2), less = f2_pack(-ref, -ref);
                uint64_t sums[2] = {0, 0};
#pragma unroll
                for (int part = 0; part < 2; ++part) {
                    float s[64];
                    tmem_ld32_at(at + 64 * part, s);
                    tmem_ld32_at(at + 64 * part + 32, s + 32);
                    tmem_wait_ld();
                    // Pairs in a fixed order, each a few steps behind the last: ordered by the compiler
                    // the sums come last, with all powers kept until then.
                    uint32_t p[32];
                    uint64_t x[32], e[32];
#pragma unroll
                    for (int k = 0; k < 32 + 6; ++k) {
                        if (k < 32) x[k] = ffma2_in_order(f2_pack(s[2 * k], s[2 * k + 1]), by2, less);
                        if (k >= 2 && k - 2 < 32) e[k - 2] = ex2_in_order(x[k - 2]);
                        if (k >= 6) {
                            sums[k & 1] = fadd2_in_order(sums[k & 1], e[k - 6]);
                            const float2 y = f2_unpack(e[k - 6]);
                            p[k - 6] = down_in_order<T>(y.x, y.y);
                        }
                    }
                    tmem_st32_b32(at + 32 * part, p);
                    tmem_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(p_full(2 * buf + part));
                }
                const float2 x = f2_unpack(fadd2_b64(sums[0], sums[1]));
                sum += x.x + x.y;
                return true;
            };
            for (int i = 0; i < mine; ++i) {
                const int tile = P::kStreams == 1 || shared ? i : 2 * i + stream;
                const int buf = P::kStreams == 1 ? i & 1 : stream;
                // keys [a, b) of the tile are seen, but for those on pages outside the pool
                const int a = lo - U.key0 - tile * kTile, b = hi - U.key0 - tile * kTile;
                const bool all = __all_sync(0xffffffffu, a <= 0 && b >= kTile && flip == 1.f);
                const uint32_t at = tmem + lanes + P::scores(buf);
                if (!wait(s_full(buf), s_phase >> buf & 1)) return;
                s_phase ^= 1u << buf;
                tc_fence_after();
                if (idle) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane < 2) mbar_arrive(p_full(2 * buf + lane));
                    continue;
                }
                const volatile uint32_t* bad = lost + (n_tile + tile) % kLostTiles * 4;
                if (!all || (A.keys.table && (bad[0] | bad[1] | bad[2] | bad[3]) != 0)) {
                    // The scores as they count, in their place: few instructions, where a second form of
                    // what follows would have to be fetched for the one or two tiles that need it.
#pragma unroll 1
                    for (int c = 0; c < kTile; c += 16) {
                        float s[16];
                        tmem_ld16(at + c, s);
                        uint32_t bits = b - c >= 16 ? 0xffffu : (1u << max(b - c, 0)) - 1;
                        bits &= a - c >= 16 ? 0u : 0xffffu << max(a - c, 0);
                        if (A.keys.table) bits &= ~(bad[c >> 5] >> (c & 16));
                        tmem_wait_ld();
#pragma unroll
                        for (int k = 0; k < 16; ++k) s[k] = bits >> k & 1 ? s[k] * flip : -INFINITY;
                        tmem_st16(at + c, s);
                    }
                    tmem_wait_st();
                }
                if (!probabilities(at, buf, i)) return;
            }
            n_tile += U.tiles;

            // ---- the output: a stream's rows, or half of the elements of the rows that the
            // streams (or the only one) have worked on together
            const bool has0 = P::kStreams == 2 && shared ? U.tiles0 > 0 : U.tiles > 0;
            const bool has1 = P::kStreams == 2 && (shared ? U.tiles > 0 : U.tiles > 1);
            const bool reads0 = has0 && !(shared && stream == 1), reads1 = has1 && !(shared && stream == 0);
            bool counts0 = reads0, counts1 = reads1;  // this row saw one of the stream's keys
            float most = top == -INFINITY ? -INFINITY : top * scale2, w0 = 1.f, w1 = 1.f;
            if (!shared) {
                if (n_ml > 0 && !wait(ml_free, (n_ml - 1) & 1)) return;
                ml[stream * kTile + row] = most;
                ml[(2 + stream) * kTile + row] = sum;
                __syncwarp();
                if (lane == 0) mbar_arrive(ml_full);
                // (with one stream half of the warps have no tiles and wait here for the others'; two end together)
                if (!(P::kStreams == 1 ? wait_for_unit(ml_full, n_ml & 1, U.tiles) : wait(ml_full, n_ml & 1))) return;
                const float m0 = ml[row], m1 = ml[kTile + row];
                most = fmaxf(m0, m1);
                w0 = m0 == -INFINITY ? 0.f : ex2(m0 - most), w1 = m1 == -INFINITY ? 0.f : ex2(m1 - most);
                const float l0 = ml[2 * kTile + row], l1 = ml[3 * kTile + row];
                sum = l0 * w0 + l1 * w1;
                counts0 &= l0 != 0.f, counts1 &= l1 != 0.f;
                __syncwarp();
                if (lane == 0) mbar_arrive(ml_free);
                ++n_ml;
            }
            if (reads0 && !wait(o_full(0), o_phase & 1)) return;
            if (reads1 && !wait(o_full(1), o_phase >> 1 & 1)) return;
            o_phase ^= uint32_t(has0) | uint32_t(has1) << 1;
            tc_fence_after();
            const int local = (shared ? stream * kTile : 0) + row;
            const bool valid = local < U.rows;
            const int flat = U.row0 + local, token = A.by_group.quotient(valid ? flat : 0);
            const float v_scale = E4M3 && A.keys.scale[1] ? A.keys.scale[1][U.head] : 1.f;
            const int e0 = !shared && stream == 1 ? D / 2 : 0, e1 = shared || stream == 1 ? D : D / 2;
            const bool none = sum == 0.f;  // no key, or only scores of -inf
            const float by = U.part >= 0 ? 1.f : none ? 0.f : v_scale / sum;
            float* part = U.part >= 0 ? A.parts + int64_t(U.part) * kPartFloats : nullptr;
            const int h = U.head * A.group + flat - token * A.group;
            char* dst = part ? reinterpret_cast<char*>(part + local * D)
                             : A.out + 2 * ((U.begin + token) * A.o_token + h * A.o_head);
            float odd = 0.f;  // NaN once an element is infinite or NaN
            if (!idle) {
                w0 *= by, w1 *= by;
#pragma unroll 1
                for (int e = e0; e < e1; e += 16) {
                    float x[16], y[16];
                    if (reads0) tmem_ld16(tmem + lanes + P::output(0) + e, x);
                    if (reads1) tmem_ld16(tmem + lanes + P::output(P::kStreams - 1) + e, y);
                    tmem_wait_ld();
#pragma unroll
                    for (int k = 0; k < 16; ++k) {
                        // (a weight of zero too: infinite or NaN values among the keys that are seen stay)
                        x[k] = (counts0 ? x[k] * w0 : 0.f) + (counts1 ? y[k] * w1 : 0.f);
                        if (none) x[k] = 0.f;
                        odd = fmaf(x[k], 0.f, odd);
                    }
                    if (!valid) continue;
                    if (part) {
#pragma unroll
                        for (int k = 0; k < 16; k += 4)
                            *reinterpret_cast<float4*>(dst + 4 * (e + k)) = make_float4(x[k], x[k + 1], x[k + 2], x[k + 3]);
                    } else {
#pragma unroll
                        for (int k = 0; k < 16; k += 8)
                            *reinterpret_cast<uint4*>(dst + 2 * (e + k)) =
                                make_uint4(T::down(x[k], x[k + 1]), T::down(x[k + 2], x[k + 3]),
                                           T::down(x[k + 4], x[k + 5]), T::down(x[k + 6], x[k + 7]));
                    }
                }
            }
            if (U.tiles > 0) {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(o_free);
            }
            if (valid && (shared || stream == 0)) {
                if (part)
                    part[256 * 128 + local] = most, part[256 * 129 + local] = sum;
                else if (A.lse)
                    A.lse[int64_t(U.begin + token) * A.q_heads + h] =
                        none ? -INFINITY : 0.693147180559945309f * (most - kLift + log2f(sum));
            }
            if (U.live != 1) {
                if (!idle) add_odd_values<D, T, E4M3>(A, U, valid && !none, lo, hi, dst, part != nullptr, e0, e1);
            } else if (__any_sync(0xffffffffu, valid && odd != 0.f && sum < INFINITY)) {
                // keys that were in the tiles and that not every row of the warp sees
                const int last_lo = __reduce_max_sync(0xffffffffu, valid ? lo : 0);
                const int first_hi = __reduce_min_sync(0xffffffffu, valid ? hi : INT32_MAX);
                if (odd_values<D, E4M3, BF>(A, U, U.key0, min(U.end, last_lo)) ||
                    odd_values<D, E4M3, BF>(A, U, max(U.key0, first_hi), U.end))
                    if (lane == 0) atomicOr(&redo, 1u << min(n_unit, 31u));
            }
        }
    };

    if (warp < kSoftmaxWarps) {
        regs_inc<P::kSoftmaxRegs>();
        passes([&](int) { softmax(); });
    } else if (warp < kSoftmaxWarps + kCopyWarps) {
        regs_dec<P::kCopyRegs>();
        auto copies = [&](auto copy) {
            auto work = [&](auto) {
                copy();
                cp_async_commit();
                cp_async_wait<0>();
                if (*abort) {  // the copy engine's land before the shared memory goes away
                    for (uint32_t i = n_stage > P::kStages ? n_stage - P::kStages : 0; i < n_stage; ++i)
                        warp_wait_parity_suspend(full(i % P::kStages), i / P::kStages & 1, &never_abort, kDrainNs, kSuspendNs);
                    if (A.q_boxes && n_q > 0) warp_wait_parity_suspend(q_full, (n_q - 1) & 1, &never_abort, kDrainNs, kSuspendNs);
                }
            };
            // (64 sequences of 4 tokens, E4M3, D = 64: 147 us with one code, 139 with two; D = 128 183 and 195)
            if constexpr (E4M3 && D == 64)
                twice(work);
            else
                passes(work);
        };
        if (A.keys.box == 0) {
            copies(copy_rows);
        } else if constexpr (E4M3) {
            copies(widen);
        } else {
            copies(copy_boxes);
        }
    } else {
        regs_dec<P::kOtherRegs>();
        if (warp == kMmaWarp || (P::kStreams == 2 && warp == kMmaWarp + 2)) {
            // (a call to clean_stage in the first pass's code takes 2% of 2048 rows behind 30000)
            twice([&](auto second) {
                if (lane == 0) {
                    multiply((warp - kMmaWarp) >> 1, second);
                    // what has been issued ends before its operands and tensor memory go away
                    mma_commit(all_done);
                    wait_parity_suspend(all_done, second, &never_abort, kWaitNs, kSuspendNs);
                }
                __syncwarp();
            });
        } else if (warp == kPlanWarp) {
            passes(plan);
        } else if (E4M3 && warp == kRawWarp) {
            // (two codes for 2048 rows behind 30000 952 us, one 977)
            twice([&](auto) {
                copy_raw();
                if (*abort)
                    for (uint32_t i = n_raw > P::kRawRing ? n_raw - P::kRawRing : 0; i < n_raw; ++i)
                        warp_wait_parity_suspend(raw_full(i % P::kRawRing), i / P::kRawRing & 1, &never_abort, kDrainNs, kSuspendNs);
            });
        } else {
            passes([](int) {});
        }
    }
    if (warp == kMmaWarp) {
        tc_fence_after();
        tmem_relinquish();
        tmem_dealloc(tmem, 512);
    }
    if (tid == 0 && *abort) atomicExch(&g_prompt_status, int(W4A4_ERR_TIMEOUT));
}

// The parts of split units joined, in the order of their keys: part i of n takes the i-th
// n-th of the rows.  Four elements a thread.
template <int D, class T, bool E4M3>
__global__ void __launch_bounds__(256) join_kernel(const __grid_constant__ Args A) {
    constexpr float kLift = lift<T>;
    constexpr int kPer = D / 4, kRows = 256 / kPer;  // threads of a row, rows at a time
    pdl_wait();
    pdl_launch_dependents();
    const int4 a = A.parts_of[2 * blockIdx.x], b = A.parts_of[2 * blockIdx.x + 1];
    const int begin = a.x, head = a.y, row0 = a.z, rows = a.w, first = b.x, pieces = b.y;
    if (pieces == 0) return;
    const int me = int(blockIdx.x) - first;
    const int from = rows * me / pieces, to = rows * (me + 1) / pieces;
    const int e = threadIdx.x % kPer * 4;
    const float v_scale = E4M3 && A.keys.scale[1] ? A.keys.scale[1][head] : 1.f;
    for (int r = from + threadIdx.x / kPer; r < to && threadIdx.x < kPer * kRows; r += kRows) {
        const float* part = A.parts + int64_t(first) * kPartFloats;
        float most = -INFINITY;
        for (int i = 0; i < pieces; ++i) most = fmaxf(most, part[int64_t(i) * kPartFloats + 256 * 128 + r]);
        float sum = 0.f;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
        for (int i = 0; i < pieces; ++i) {
            const float* p = part + int64_t(i) * kPartFloats;
            const float m = p[256 * 128 + r], l = p[256 * 129 + r];
            const float4 x = *reinterpret_cast<const float4*>(p + r * D + e);
            if (l == 0.f) continue;  // the part saw nothing; scores that are all NaN leave m at -inf, but not l at zero
            const float w = m == -INFINITY ? 0.f : ex2(m - most);
            sum = fmaf(w, l, sum);
            o.x = fmaf(w, x.x, o.x), o.y = fmaf(w, x.y, o.y), o.z = fmaf(w, x.z, o.z), o.w = fmaf(w, x.w, o.w);
        }
        const bool none = sum == 0.f;
        const float by = none ? 0.f : v_scale / sum;
        if (none) o = make_float4(0.f, 0.f, 0.f, 0.f);
        const int flat = row0 + r, token = A.by_group.quotient(flat), h = head * A.group + flat - token * A.group;
        *reinterpret_cast<uint2*>(A.out + 2 * ((begin + token) * A.o_token + h * A.o_head + e)) =
            make_uint2(T::down(o.x * by, o.y * by), T::down(o.z * by, o.w * by));
        if (A.lse && e == 0)
            A.lse[int64_t(begin + token) * A.q_heads + h] =
                none ? -INFINITY : 0.693147180559945309f * (most - kLift + log2f(sum));
    }
}

// A map of [outer][middle][inner][dim] elements with these strides in bytes: boxes of 64 elements
// of inner_box x middle_box rows with the 128-byte swizzle, or of whole stage rows of bytes (swizzled if 128).
template <int D, bool BF>
bool encode(const char* p, bool bytes, int64_t inner, int64_t inner_stride, int64_t middle, int64_t middle_stride, int64_t outer,
            int64_t outer_stride, int inner_box, int middle_box, CUtensorMap& map) {
    const EncodeFn go = driver_encode();
    const cuuint64_t dims[4] = {D, cuuint64_t(inner), cuuint64_t(middle), cuuint64_t(outer)};
    auto stride = [](int64_t bytes, int64_t n) { return n > 1 ? cuuint64_t(bytes) : cuuint64_t(16); };  // of one: unused
    const cuuint64_t strides[3] = {stride(inner_stride, inner), stride(middle_stride, middle), stride(outer_stride, outer)};
    const cuuint32_t shape[4] = {cuuint32_t(bytes ? (D < 128 ? D : 128) : 64), cuuint32_t(inner_box), cuuint32_t(middle_box), 1};
    const cuuint32_t steps[4] = {1, 1, 1, 1};
    for (const cuuint64_t s : strides)
        if (s == 0) return false;  // rows that share memory
    return go && outer > 0 &&
           go(&map, bytes ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : BF ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
              4, const_cast<char*>(p), dims, strides, shape, steps, CU_TENSOR_MAP_INTERLEAVE_NONE,
              bytes && D < 128 ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, class T, bool E4M3>
w4a4_status run(Args& A, cudaStream_t s) {
    using P = Plan<D, E4M3>;
    auto kernel = attention_kernel<D, T, E4M3>;
    static std::atomic<uint64_t> ready{0};  // devices
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev < 0 || dev >= 64) return W4A4_ERR_CUDA;
    if (!(ready.load(std::memory_order_acquire) >> dev & 1)) {
        if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, P::kBytes) != cudaSuccess)
            return launch_status();
        ready.fetch_or(uint64_t(1) << dev, std::memory_order_release);
    }
    // A CTA per SM, or one per unit where there can be fewer.  Units are fewer than SMs if the
    // rows of all sequences are; then parts of them (of four tiles or more) are worth a second launch
    // where the cache can be long: 5 tokens behind 1500 of one sequence take 17.8 us, 22.9 whole;
    // behind 3000 19.8 and 37, with parts of two tiles 21.6; behind 700 15.5 either way.
    const int sms = std::min(device_sm_count(), kMaxParts);
    const int64_t rows = int64_t(A.tokens) * A.group;
    const int64_t most = A.kv_heads * ((rows + kTile - 1) / kTile + A.seqs);
    const int64_t least = A.kv_heads * ((rows + P::kStreams * kTile - 1) / (P::kStreams * kTile));
    const int64_t keys = A.window > 0 ? std::min(int64_t(A.keys.longest), int64_t(A.window) + A.tokens) : A.keys.longest;
    if (!(A.parts && least < sms && keys > 8 * kTile)) A.parts = nullptr;
    const int grid = A.parts ? sms : int(std::min(int64_t(sms), most));
    constexpr bool bf16 = std::is_same_v<T, BF16>;
    // Keys and values by the copy engine, eight rows or more a copy, where pages hold so many side by side.
    CUtensorMap maps[3] = {};
    const Keys& K = A.keys;
    const bool paged = K.table != nullptr;
    const int box = !paged ? 32 : K.page_size % 32 == 0 ? 32 : K.page_size % 16 == 0 ? 16 : K.page_size % 8 == 0 ? 8 : 0;
    auto rows_of = [&](int w) {
        return encode<D, bf16>(K.pool[w], E4M3, paged ? K.page_size : A.tokens, K.token_stride[w], A.kv_heads, K.head_stride[w],
                               paged ? K.pages : 1, K.page_stride[w], box, 1, maps[1 + w]);
    };
    A.keys.box = box > 0 && rows_of(0) && rows_of(1) ? box : 0;
    // ... and queries, where 128 rows are whole tokens.
    A.q_boxes = kTile % A.group == 0 && encode<D, bf16>(A.q, false, A.q_heads, 2 * A.q_head, A.tokens, 2 * A.q_token, 1, 0, A.group,
                                                        kTile / A.group, maps[0]);
    const char* text = !A.lengths ? (bf16 ? "prompt_attention bf16 tokens=%d seqs=%d heads=%d/%d dim=%d stages=%d grid=%d parts=%d"
                                          : "prompt_attention f16 tokens=%d seqs=%d heads=%d/%d dim=%d stages=%d grid=%d parts=%d")
                       : E4M3     ? "chunk_attention e4m3 tokens=%d seqs=%d heads=%d/%d dim=%d stages=%d grid=%d parts=%d"
                       : bf16     ? "chunk_attention bf16 tokens=%d seqs=%d heads=%d/%d dim=%d stages=%d grid=%d parts=%d"
                                  : "chunk_attention f16 tokens=%d seqs=%d heads=%d/%d dim=%d stages=%d grid=%d parts=%d";
    set_dispatch_ints(text, {A.tokens, A.seqs, A.q_heads, A.kv_heads, D, P::kStages, grid, A.parts != nullptr});
    w4a4_status st = launch<attention_kernel<D, T, E4M3>>(dim3(unsigned(grid)), P::kThreads, P::kBytes, s, A, maps[0], maps[1], maps[2]);
    if (st == W4A4_OK && A.parts) st = launch<join_kernel<D, T, E4M3>>(dim3(unsigned(grid)), 256, 0, s, A);
    return st;
}

// Entry of one head dimension.
template <int D>
w4a4_status run_dim(Args& A, bool bf16, bool e4m3, cudaStream_t s) {
    if (e4m3) return bf16 ? run<D, BF16, true>(A, s) : run<D, F16, true>(A, s);
    return bf16 ? run<D, BF16, false>(A, s) : run<D, F16, false>(A, s);
}

}  // namespace prompt
}  // namespace w4a4
