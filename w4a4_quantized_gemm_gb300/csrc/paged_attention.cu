// Attention of one new token per sequence over a paged key-value cache, split over
// the cache's length and joined:
//   a_j = scale q . k_j,   out = sum_j exp(a_j) v_j / sum_j exp(a_j)
// for the q_heads / kv_heads = G query heads that share a key-value head.
//
// Every cached byte is read once and used for 2 G flops, far below what the matrix
// units need to be the limit, so the bound is HBM traffic and the kernel is built to
// keep copies in flight:
//  * The work is cut into units: `span` tokens of one (sequence, group of key-value
//    heads, chunk of up to 16 of their query heads).  Each CTA of a grid that fills the
//    GPU once takes an equal, contiguous run of units, whatever the lengths.  The
//    lengths are read on the device, so a captured graph serves growing sequences.
//  * A CTA is four warps that share a unit out: 16 or 32 tokens of one key-value head
//    each (one head and consecutive tokens, or several heads and the same tokens, see
//    `together`).  A warp runs on its own: it copies its key and value rows into a ring
//    of stages in shared memory, the page table looked up three units ahead of the copy,
//    and keeps a running maximum, sum and output in registers (one pass).  Only the end
//    of a (sequence, head) synchronises the warps.
//  * The copies are 16 bytes a lane.  One bulk copy per row streams faster alone (4 GB in
//    256-byte rows: 7.1 TB/s against 6.8) but holds the issuing warp for tens of cycles a
//    row, and here the warp also has the arithmetic: 850 us instead of 692 on a batch of
//    4.3 GB, and only a third of the rate where rows are 64 bytes.
//  * Scores are m16n8k16 warp MMAs with 16 tokens as rows and 8 query heads as columns:
//    at one token per sequence there are G <= 16 useful columns, so the 128-row tcgen05
//    tile would stand idle.  The scores' transposed fragments are the probabilities
//    operand of the second product, whose rows are the head's elements.
//  * A run that ends inside a (sequence, head group) leaves its maximum, sum and output in
//    the workspace.  Parts are joined sixteen at a time, in token order, by the CTA that
//    completes the sixteen, and those by the CTA that completes the last.
#include <algorithm>
#include <atomic>

#include "elem.cuh"
#include "kernels.h"
#include "launch.cuh"
#include "tc_ptx.cuh"

namespace w4a4 {
namespace {

__device__ int g_attention_status = 0;

constexpr int kWarps = 4, kThreads = kWarps * 32;
constexpr int kPartRows = 32;           // rows of a part in the workspace
constexpr int kMaxSms = 160;
constexpr int kFewUnits = 8;            // runs shorter than this are single pieces
constexpr int kJoin = 16;               // parts that are joined at a time

enum Cache { kF16, kBF16, kE4M3 };

// Shared-memory plan of one head dimension, cache type and number NT of 8-head column
// tiles.  A row is padded to an odd number of 16-byte pieces: the eight rows of an
// ldmatrix then lie in different banks.  The stage that a warp has just used also
// holds its output when the warps are joined.
template <int D, int CT, int NT>
struct Plan {
    static constexpr int kSize = CT == kE4M3 ? 1 : 2;
    static constexpr int kRowBytes = D * kSize;
    static constexpr int kPieces = kRowBytes / 16;
    static constexpr int kRow = (kPieces | 1) * 16;                 // bytes of a row in shared memory
    // Tokens of a warp's step: 32 where a row is short, to halve the steps' fixed cost
    static constexpr int kTokens = CT == kE4M3 || D == 64 ? 32 : 16;
    static constexpr int kStage = 2 * kTokens * kRow;               // keys, then values
    static constexpr int kPerSM = kStage > 10000 ? 1 : kStage < 6000 ? 3 : 2;  // CTAs
    static constexpr int kRoom = 228 * 1024 / kPerSM - 1280;        // of an SM, less 1 KB a CTA and the static part
    static constexpr int kChunk = 8 * NT;                           // query heads of a chunk
    static constexpr int kFixed = 2 * kWarps * kChunk * 4;          // the warps' maxima and sums
    static constexpr int kStages = (kRoom - kFixed) / (kWarps * (kStage + 4));
    static constexpr int kOutRow = D + 4;                           // floats of a joined row
    static constexpr int kRing = kWarps * kStages * kStage;
    static constexpr int kBytes = kRing + kFixed + kWarps * kStages * 4;
    static_assert(kStages >= 2 && kBytes <= 227 * 1024 - 256, "shared memory");
    static_assert(kPerSM <= (D == 64 ? 3 : D == 256 ? 1 : 2), "max_ctas");
    static_assert(8 * NT * kOutRow * 4 <= kStage, "a stage holds a warp's output");
};

// Division by a number that the host knows, 1 <= d < 2^31: n / d = n * mul >> shift for
// 0 <= n < 2^31, mul = ceil(2^shift / d), shift = 31 + ceil(log2 d).  (A division takes a
// hundred and fifty cycles, and a short sequence's way through the kernel has a dozen.)
struct Divisor {
    uint32_t mul, shift;
    explicit Divisor(int d = 1) {
        shift = 31;
        while ((1ll << (shift - 31)) < d) ++shift;
        mul = uint32_t(((1ull << shift) + d - 1) / d);
    }
    __device__ __forceinline__ int quotient(int n) const { return int(uint64_t(uint32_t(n)) * mul >> shift); }
};

struct Args {
    w4a4_kv_cache c;
    int page_stride[2], token_stride[2], head_stride[2];  // of keys and values, in bytes
    int longest;  // tokens a row of the page table holds
    const void* q;
    void* out;
    float* lse;
    const int32_t* lengths;
    int32_t* arrived;  // [seqs][heads] joined sixteens that have arrived; zero between calls, as is
    int32_t* joined;   // [2 * CTAs] parts of the sixteen that opens with this one that have arrived
    float* parts;      // [2][2 * CTAs][kPartRows * D outputs, kPartRows maxima, kPartRows sums]: parts, then joins
    int64_t joined_at;  // from a part to where its sixteen's join goes, in floats
    int64_t q_token, q_head, o_token, o_head;
    float scale_log2;
    int q_heads, group, chunks, window;
    int together;    // head chunks of a unit: 1, 2 or 4
    int heads;       // kv_heads * chunks / together: units' head groups of a sequence
    int rows;        // query heads of a chunk (the last of a key-value head may have fewer)
    int span_log2;   // log2 of the tokens of a unit
    Divisor by_page, by_ctas, by_chunks, by_rows, by_items;  // page size, grid, chunks, rows, items
    int items;       // outputs of a unit, four elements each
    bool q_bf16;
};

__device__ __forceinline__ void ldmatrix4_trans(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];\n"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t a) {  // of 16-bit elements, over the warp
    uint32_t d;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;\n" : "=r"(d) : "r"(a));
    return d;
}
__device__ __forceinline__ void mma_bf16_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};\n"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <int CT>
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if constexpr (CT == kBF16)
        mma_bf16_16816(d, a, b0, b1);
    else
        mma_f16_16816(d, a, b0, b1);
}
// Four E4M3 bytes -> two fp16 pairs (bytes 0, 1 and 2, 3), exact.
__device__ __forceinline__ void e4m3x4_to_f16x2(uint32_t four, uint32_t& low, uint32_t& high) {
    asm("{\n.reg .b16 a, b;\nmov.b32 {a, b}, %2;\ncvt.rn.f16x2.e4m3x2 %0, a;\ncvt.rn.f16x2.e4m3x2 %1, b;\n}\n"
        : "=r"(low), "=r"(high)
        : "r"(four));
}
__device__ __forceinline__ float exp2_approx(float x) {  // 2 ulp; 2^-inf = 0
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float ref_of(float top) {  // what is subtracted: nothing while every score is -inf
    return top == -INFINITY ? 0.f : top;
}
__device__ __forceinline__ int add_acq_rel(int32_t* p, int v) {
    int old;
    asm volatile("atom.add.acq_rel.gpu.global.s32 %0, [%1], %2;\n" : "=r"(old) : "l"(p), "r"(v) : "memory");
    return old;
}

// n / d for 0 <= n <= 2^20 and d >= 1: (n + 1/2) / d is at least 1 / (2 d) away from a whole
// number, the division off by 2 ulp and the rounding of d, together less than n / d * 2^-21.
// (An integer division takes a hundred cycles and more, and a short sequence's way through
// the kernel had four: 300 sequences of up to 300 tokens, one head: 13.4 us with
// them, 13.1 with these.)
__device__ __forceinline__ int small_quotient(int n, int d) { return int(__fdividef(n + 0.5f, float(d))); }

// How the units are shared out: the first `more` CTAs take each + 1, the others each.
struct Share {
    int each, more;
    __device__ __forceinline__ int start(int c) const { return each * c + min(c, more); }
    __device__ __forceinline__ int owner(int unit) const {
        if (each == 1 && more == 0) return unit;
        const int longer = more * (each + 1);
        return unit < longer ? unit / (each + 1) : more + (unit - longer) / each;
    }
};

// Tokens of sequence b that take part: [lo, lo + n).
__device__ __forceinline__ void range_of(const Args& A, int b, int& lo, int& n) {
    const int len = max(0, min(A.lengths[b], A.longest));
    lo = A.window > 0 ? max(0, len - A.window) : 0;
    n = len - lo;
}

__device__ __forceinline__ int tiles_of(const Args& A, int n) { return int((uint32_t(n) + (1u << A.span_log2) - 1) >> A.span_log2); }

// A place in the sequence of units: tile `tile` of (sequence b, head group hc).
struct Cursor {
    int b, hc, tile, tiles, lo, n;
    __device__ __forceinline__ void enter(const Args& A) {
        range_of(A, b, lo, n);
        tiles = tiles_of(A, n);
    }
    __device__ __forceinline__ void advance(const Args& A) {  // to the next unit, if there is one
        if (++tile < tiles) return;
        tile = 0;
        if (++hc < A.heads) return;
        hc = 0;
        do {
            if (++b >= A.c.seqs) return;
            enter(A);
        } while (n == 0);
    }
};

// Scale of a row of queries for the fp16 MMA of E4M3 caches: bf16 queries can lie
// outside fp16's range, so a row is multiplied by the power of two that brings its
// largest element into [2^13, 2^14) (exact for elements down to 2^-28 of it) and the
// scores by its inverse.  Beside an infinite element every finite one has to stay finite,
// and no more: its scores are infinities or NaN.
__device__ __forceinline__ float row_shift(float top) {
    if (!(top > 0.f)) return 1.f;
    const int e = isinf(top) ? 127 : max(ilogbf(top), -100);
    return exp2f(float(13 - e));
}

template <int D, int CT, int NT>
__global__ void __launch_bounds__(kThreads, Plan<D, CT, NT>::kPerSM) paged_attention_kernel(const Args A) {
    using P = Plan<D, CT, NT>;
    // bf16 probabilities have fp32's range: no lift, and the maximum may be further behind
    constexpr float kLift = CT == kBF16 ? 0.f : 13.f, kSlack = CT == kBF16 ? 8.f : 2.f;
    constexpr int kChunk = P::kChunk, kTokens = P::kTokens, kSubs = kTokens / 16, kSteps = D / 16;
    extern __shared__ __align__(128) uint8_t smem[];
    float* warp_max = reinterpret_cast<float*>(smem + P::kRing);  // [kWarps][kChunk]
    float* warp_sum = warp_max + kWarps * kChunk;                 // [kWarps][kChunk]
    uint32_t* masks = reinterpret_cast<uint32_t*>(warp_sum + kWarps * kChunk);  // [kWarps][kStages]
    __shared__ int scan[kWarps];
    __shared__ int found[6];
    __shared__ int s_last;

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int quad = lane >> 2, in_quad = lane & 3;
    pdl_wait();
    pdl_launch_dependents();
    const int B = A.c.seqs;

    // ---- this CTA's run of units: a scan over the sequences' tile counts.  Up to 32
    // sequences each warp does it for itself, a lane a sequence; more are shared out to the
    // CTA's threads, several in a row to each beyond 128.
    // A run of few units, though, is one piece of one (sequence, head group), so that a CTA
    // has one part to leave and one join to take part in: pieces of at most `piece` units,
    // the least for which there are CTAs enough (8 sequences of 700 tokens: 10.8 us, 12.3
    // with runs over two (sequence, head group)s; 200 windows of 588 tokens, 8-bit, D = 96: 15.5
    // and 20.3 us, both with the rows in HBM).
    int first, count;
    Share share;
    int piece = 0, c0 = 0, c1 = 0;  // piece > 0: the CTAs that share this one's (sequence, head group)
    Cursor at;
    int seq_tiles;  // tiles of the sequences before at.b
    {
        const bool few = B <= 32;
        const int per = few ? 1 : (B + kThreads - 1) / kThreads, me = few ? lane : tid;
        const int b0 = min(B, me * per), b1 = min(B, b0 + per);
        int mine = 0, first_tiles = 0, lo = 0, n = 0;
        bool bad = false, empty = false;
        for (int b = b0; b < b1; ++b) {
            const int len = A.lengths[b];
            bad |= len < 0 || len > A.longest;
            range_of(A, b, lo, n);
            empty |= n == 0;
            mine += tiles_of(A, n);
            if (b == b0) first_tiles = mine;
        }
        if (bad && blockIdx.x == 0) atomicExch(&g_attention_status, int(W4A4_ERR_INDEX));
        // inclusive scan over the sequences, and their sum
        auto scan_of = [&](int v, int& all) {
            for (int o = 1; o < min(B, 32); o <<= 1) {
                const int u = __shfl_up_sync(0xffffffffu, v, o);
                if (lane >= o) v += u;
            }
            if (few) {
                all = __shfl_sync(0xffffffffu, v, min(B, 32) - 1);
                return v;
            }
            __syncthreads();
            if (lane == 31) scan[warp] = v;
            __syncthreads();
            all = 0;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                if (w < warp) v += scan[w];
                all += scan[w];
            }
            return v;
        };
        int total;
        const int upto = scan_of(mine, total);
        int before = upto - mine;
        total *= A.heads;
        // sequences without tokens: zeros, from whichever CTA their number falls to
        if (few ? __any_sync(0xffffffffu, empty) : __syncthreads_or(empty))
            for (int b = blockIdx.x; b < B; b += gridDim.x) {
                int l, tokens;
                range_of(A, b, l, tokens);
                if (tokens > 0) continue;
                for (int i = tid; i < A.q_heads * (D / 8); i += kThreads) {
                    const int h = i / (D / 8), e = i % (D / 8) * 8;
                    *reinterpret_cast<uint4*>(static_cast<char*>(A.out) + 2 * (b * A.o_token + h * A.o_head + e)) =
                        make_uint4(0, 0, 0, 0);
                }
                if (A.lse)
                    for (int h = tid; h < A.q_heads; h += kThreads) A.lse[int64_t(b) * A.q_heads + h] = -INFINITY;
            }
        if (total == 0) return;
        const int ctas = gridDim.x, c = blockIdx.x;
        share.each = total < ctas ? 1 : A.by_ctas.quotient(total);
        share.more = total < ctas ? 0 : total - share.each * ctas;
        int pieces = 0, upto_pieces = 0;  // of this thread's sequences, of those up to them; of a head group
        auto pieces_of = [&](int tiles) { return small_quotient(tiles + piece - 1, piece); };
        if (total > ctas && share.each < kFewUnits) {
            // the (sequence, head group)s with tokens, or all where a thread has several sequences
            const int groups = (few       ? __popc(__ballot_sync(0xffffffffu, mine > 0))
                                : per > 1 ? B
                                          : __syncthreads_count(mine > 0)) * A.heads;
            if (groups <= ctas) {
                piece = share.each + (share.more > 0);
                for (int tries = 0; tries < 8; ++tries) {
                    pieces = pieces_of(first_tiles);
                    for (int b = b0 + 1; b < b1; ++b) {
                        int l, k;
                        range_of(A, b, l, k);
                        pieces += pieces_of(tiles_of(A, k));
                    }
                    int all;
                    upto_pieces = scan_of(pieces, all);
                    if (all * A.heads <= ctas) {
                        if (c >= all * A.heads) return;
                        break;
                    }
                    piece = tries < 7 ? max(piece + 1, A.by_ctas.quotient(piece * all * A.heads)) : 0;
                }
            }
        }
        if (piece == 0 && c >= total) return;
        // the thread that has this CTA's first unit tells the others of its sequence
        first = share.start(c);
        count = share.start(c + 1) - first;
        int from = (upto_pieces - pieces) * A.heads;  // pieces before the sequence's
        const bool here = piece > 0 ? from <= c && c < upto_pieces * A.heads
                                    : before * A.heads <= first && first < upto * A.heads;
        int b = b0;
        if (here && per > 1)
            for (; b < b1; ++b) {
                range_of(A, b, lo, n);
                mine = tiles_of(A, n);
                if (piece > 0) {
                    pieces = pieces_of(mine);
                    if (c < from + pieces * A.heads) break;
                    from += pieces * A.heads;
                } else if (first < (before + mine) * A.heads) {
                    break;
                }
                before += mine;
            }
        int in = piece > 0 ? c - from : first - before * A.heads;  // into the sequence's pieces, or units
        if (few) {
            at.b = __ffs(__ballot_sync(0xffffffffu, here)) - 1;
            seq_tiles = __shfl_sync(0xffffffffu, before, at.b);
            at.lo = __shfl_sync(0xffffffffu, lo, at.b);
            at.n = __shfl_sync(0xffffffffu, n, at.b);
            at.tiles = __shfl_sync(0xffffffffu, mine, at.b);
            pieces = __shfl_sync(0xffffffffu, pieces, at.b);
            in = __shfl_sync(0xffffffffu, in, at.b);
        } else {
            if (here) found[0] = b, found[1] = before, found[2] = lo, found[3] = n, found[4] = pieces, found[5] = in;
            __syncthreads();
            at.b = found[0], seq_tiles = found[1], at.lo = found[2], at.n = found[3], pieces = found[4], in = found[5];
            at.tiles = tiles_of(A, at.n);
        }
        const int of = piece > 0 ? pieces : at.tiles;
        at.hc = in < (1 << 20) ? small_quotient(in, of) : in / of;
        at.tile = in - at.hc * of;
        if (piece > 0) {
            const int k = at.tile;
            c0 = c - k, c1 = c0 + pieces - 1;
            const int least = small_quotient(at.tiles, pieces), more = at.tiles - least * pieces;
            at.tile = least * k + min(k, more);
            count = least + (k < more);
            first = seq_tiles * A.heads + at.hc * at.tiles + at.tile;
        }
    }

    // ---- the warp's ring of stages
    const int sharers = kWarps / A.together;  // warps of a head chunk (a power of two)
    const int my_tokens = (warp & (sharers - 1)) * kTokens, my_chunk = (warp * A.together) / kWarps;
    const uint32_t ring = smem_u32(smem) + warp * P::kStages * P::kStage;
    uint32_t* my_masks = masks + warp * P::kStages;
    // The page table is read three units ahead of the copy: `next`, `after` and `later` are
    // the next units to copy, `ahead` the place of the one whose look-up comes next.
    struct Ahead {
        int page, slot, kvh;  // of token lane % kTokens; the unit's key-value head
        bool in_range;
    };
    Cursor ahead = at;
    int to_put = count, to_look = count;
    auto look_up = [&](Ahead& u) {
        u.in_range = false;
        if (to_look <= 0) return;
        const int j = (ahead.tile << A.span_log2) + my_tokens + (lane & (kTokens - 1));
        u.in_range = j < ahead.n;
        u.kvh = A.by_chunks.quotient(ahead.hc * A.together + my_chunk);
        if (u.in_range) {
            const int tok = ahead.lo + j, p = A.by_page.quotient(tok);
            u.slot = tok - p * A.c.page_size;
            u.page = A.c.page_table[ahead.b * A.c.table_stride + p];
        }
        if (--to_look > 0) ahead.advance(A);
    };
    Ahead next, after, later;
    look_up(next);
    look_up(after);
    look_up(later);

    // ---- running softmax of this warp's tokens: columns 8 t + 2 (lane % 4) + {0, 1} are
    // query heads; out[m][t] is rows (elements of the head) 16 m + quad and + 8
    uint32_t qf[kSteps][NT][2];
    float out[kSteps][NT][4];
    float top[NT][2], sum[NT][2], factor[NT][2];
    int kvh = 0, in_group = 0;  // this warp's key-value head, and its chunk's first query head in the group
    bool fresh = true;
    // The queries of a place are requested before its first rows are copied, or while the
    // place before it is joined: behind the copies they would take microseconds.
    auto load_q = [&](const Cursor& to) {
        const int v = to.hc * A.together + my_chunk;
        kvh = A.by_chunks.quotient(v);
        in_group = (v - kvh * A.chunks) * kChunk;
        const int rows = min(kChunk, A.group - in_group);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const int row = 8 * t + quad;
            const char* src = static_cast<const char*>(A.q) +
                              2 * (to.b * A.q_token + (kvh * A.group + in_group + row) * A.q_head);
#pragma unroll
            for (int s = 0; s < kSteps; ++s) {
                // The MMA's k-columns 2 (lane % 4) + {0, 1} and those + 8 stand for these
                // elements; E4M3 keys come four consecutive elements to a lane, so there both
                // pairs are taken from four consecutive ones.
                const int e = CT == kE4M3 ? 16 * s + 4 * in_quad : 16 * s + 2 * in_quad;
                qf[s][t][0] = qf[s][t][1] = 0;
                if (row < rows) {
                    qf[s][t][0] = *reinterpret_cast<const uint32_t*>(src + 2 * e);
                    qf[s][t][1] = *reinterpret_cast<const uint32_t*>(src + 2 * (e + (CT == kE4M3 ? 2 : 8)));
                }
            }
        }
    };
    load_q(at);
    auto copy_unit = [&](int stage) {
        const bool ok = next.in_range && next.page >= 0 && next.page < A.c.pages;
        if (next.in_range && !ok) atomicExch(&g_attention_status, int(W4A4_ERR_INDEX));
        const uint32_t mask = __ballot_sync(0xffffffffu, ok) & (kTokens == 32 ? 0xffffffffu : 0xffffu);
        if (lane == 0) my_masks[stage] = mask;
        if (mask) {
            const uint32_t dst = ring + stage * P::kStage;
            auto row_of = [&](int kv) {
                const int64_t off = int64_t(next.page) * A.page_stride[kv] + int64_t(next.slot) * A.token_stride[kv] +
                                    int64_t(next.kvh) * A.head_stride[kv];
                return reinterpret_cast<unsigned long long>(kv ? A.c.v : A.c.k) + (ok ? off : 0);
            };
            // with 16 tokens, lanes 0-15 address the keys of their token, lanes 16-31 the values
            const unsigned long long mine = row_of(kTokens == 32 || lane < 16 ? 0 : 1);
            const unsigned long long other = kTokens == 32 ? row_of(1) : mine;
#pragma unroll
            for (int i = 0; i < 2 * kTokens * P::kPieces / 32; ++i) {  // a warp's width of pieces at a time
                const int piece = i * 32 + lane, r = piece / P::kPieces, c = piece % P::kPieces;
                const char* src = reinterpret_cast<const char*>(
                    __shfl_sync(0xffffffffu, kTokens == 32 && i >= P::kPieces ? other : mine, r & 31));
                tc::cp_async16_zfill(dst + r * P::kRow + c * 16, src + c * 16, (mask >> (r & (kTokens - 1)) & 1) * 16);
            }
        }
        --to_put;
        next = after;
        after = later;
        look_up(later);
    };

    int stage = 0, fill = 0;
    for (int it = 1 - P::kStages; it < count; ++it) {  // the first kStages - 1 steps only copy
        if (to_put > 0) copy_unit(fill);
        cp_async_commit();
        if (++fill == P::kStages) fill = 0;
        if (it < 0) continue;

        if (fresh) {
            fresh = false;
            const float ks = CT == kE4M3 && A.c.k_scale ? A.c.k_scale[kvh] : 1.f;
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                float shift = 1.f;
                if (CT == kE4M3 && A.q_bf16) {
                    float big = 0.f;
#pragma unroll
                    for (int s = 0; s < kSteps; ++s)
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const float2 f = BF16::up(qf[s][t][i]);
                            big = fmaxf(big, fmaxf(fabsf(f.x), fabsf(f.y)));
                        }
                    big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 1));
                    big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 2));
                    shift = row_shift(big);
#pragma unroll
                    for (int s = 0; s < kSteps; ++s)
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const float2 f = BF16::up(qf[s][t][i]);
                            qf[s][t][i] = F16::down(f.x * shift, f.y * shift);
                        }
                }
                const float mine = A.scale_log2 * ks / shift;  // of head quad; the scores' columns are other heads
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    factor[t][j] = CT == kE4M3 ? __shfl_sync(0xffffffffu, mine, (2 * in_quad + j) * 4) : mine;
                    top[t][j] = -INFINITY, sum[t][j] = 0.f;
                }
#pragma unroll
                for (int m = 0; m < kSteps; ++m)
#pragma unroll
                    for (int j = 0; j < 4; ++j) out[m][t][j] = 0.f;
            }
        }

        cp_async_wait<P::kStages - 1>();
        __syncwarp();
        const uint32_t mask = my_masks[stage];
        const uint32_t keys = ring + stage * P::kStage, values = keys + kTokens * P::kRow;
        if (mask) {
            float s[kSubs][NT][4];  // tokens 16 u + quad (two heads), then + 8
#pragma unroll
            for (int u = 0; u < kSubs; ++u) {
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int j = 0; j < 4; ++j) s[u][t][j] = 0.f;
                const uint32_t base = keys + (16 * u + (lane & 15)) * P::kRow + (lane >> 4) * 16;
                if constexpr (CT == kE4M3) {
                    // an 8x8 b16 matrix is 8 tokens x 16 E4M3 elements: one k-step
#pragma unroll
                    for (int st = 0; st < kSteps; st += 2) {
                        uint32_t r[4];
                        tc::ldsm_x4(r, base + st * 16);
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            uint32_t a[4];
                            e4m3x4_to_f16x2(r[2 * h], a[0], a[2]);
                            e4m3x4_to_f16x2(r[2 * h + 1], a[1], a[3]);
#pragma unroll
                            for (int t = 0; t < NT; ++t) mma<CT>(s[u][t], a, qf[st + h][t][0], qf[st + h][t][1]);
                        }
                    }
                } else {
                    float odd[NT][4] = {};  // two chains of MMAs, so that neither waits for every result
#pragma unroll
                    for (int st = 0; st < kSteps; st += 2) {
                        uint32_t a[4], b[4];
                        tc::ldsm_x4(a, base + st * 32);
                        tc::ldsm_x4(b, base + st * 32 + 32);
#pragma unroll
                        for (int t = 0; t < NT; ++t) {
                            mma<CT>(s[u][t], a, qf[st][t][0], qf[st][t][1]);
                            mma<CT>(odd[t], b, qf[st + 1][t][0], qf[st + 1][t][1]);
                        }
                    }
#pragma unroll
                    for (int t = 0; t < NT; ++t)
#pragma unroll
                        for (int j = 0; j < 4; ++j) s[u][t][j] += odd[t][j];
                }
            }
            // Scores in units of log2, tokens that do not take part at -inf.  The subtracted
            // maximum is only renewed when a score exceeds it by more than kSlack, so that the
            // reduction over the warp and the rescaling of the output are left out of most
            // steps.  What is subtracted (`top`) lies kLift below the maximum: an fp16
            // probability then goes up to 2^(kLift + kSlack) = 2^15, and is a normal number down
            // to 2^-27 of the largest instead of 2^-14.  (Unlifted, tokens at 2^-25 were lost,
            // and thousands of them beside one heavy token can make the output.)
            constexpr uint32_t kFull = kTokens == 32 ? 0xffffffffu : 0xffffu;
            bool over = false;
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float limit = top[t][j & 1] + (kLift + kSlack);
#pragma unroll
                    for (int u = 0; u < kSubs; ++u) {
                        s[u][t][j] *= factor[t][j & 1];
                        if (mask != kFull && !(mask >> (16 * u + 8 * (j >> 1) + quad) & 1)) s[u][t][j] = -INFINITY;
                        over |= s[u][t][j] > limit;
                    }
                }
            if (__any_sync(0xffffffffu, over)) {
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        float m = -INFINITY;
#pragma unroll
                        for (int u = 0; u < kSubs; ++u) m = fmaxf(m, fmaxf(s[u][t][j], s[u][t][j + 2]));
#pragma unroll
                        for (int o = 4; o < 32; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
                        m = fmaxf(top[t][j], m - kLift);
                        const float fade = exp2_approx(top[t][j] - ref_of(m));
                        top[t][j] = m;
                        sum[t][j] *= fade;
#pragma unroll
                        for (int i = 0; i < kSteps; ++i) {
                            out[i][t][j] *= fade;
                            out[i][t][j + 2] *= fade;
                        }
                    }
            }
            // Probabilities [token][head] as the product's second operand.  Rounded to its type they
            // would add 0.7 (fp16) to 1 (bf16) of the outputs' own rounding to their error, so with
            // 16-bit caches what the rounding leaves goes in as a second operand, in the shadow of
            // HBM (128 sequences of 8192 tokens, fp16: 689 us with one operand, 693 with both; D = 256
            // in groups of 16, the most: 1083 and 1113).  An 8-bit cache keeps the one rounding to
            // fp16, 2^-11 beside the 2^-4 of its values: there the instructions are nearer to the
            // limit (E4M3, D = 64: 103 and 108 us, D = 256: 348 and 366).
            constexpr int kParts = CT == kE4M3 ? 1 : 2;
            uint32_t pf[kSubs][NT][kParts][2];
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                const float r0 = ref_of(top[t][0]), r1 = ref_of(top[t][1]);
#pragma unroll
                for (int u = 0; u < kSubs; ++u)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const float a = exp2_approx(s[u][t][2 * h] - r0), b = exp2_approx(s[u][t][2 * h + 1] - r1);
                        sum[t][0] += a;
                        sum[t][1] += b;
                        const uint32_t p = CT == kBF16 ? BF16::down(a, b) : F16::down(a, b);
                        pf[u][t][0][h] = transpose8x8(p);
                        if constexpr (kParts == 2) {
                            const float2 of = CT == kBF16 ? BF16::up(p) : F16::up(p);
                            pf[u][t][1][h] = transpose8x8(CT == kBF16 ? BF16::down(a - of.x, b - of.y)
                                                                      : F16::down(a - of.x, b - of.y));
                        }
                    }
            }
#pragma unroll
            for (int u = 0; u < kSubs; ++u) {
                if constexpr (CT == kE4M3) {
                    // a register holds (token, d), (token, d + 1), (token + 1, d), (token + 1, d + 1):
                    // the even and the odd elements of a 16-byte piece are the MMA's rows 0-7 and 8-15
                    const uint32_t base = values + (16 * u + (lane & 15)) * P::kRow + (lane >> 4) * 16;
#pragma unroll
                    for (int m = 0; m < kSteps; m += 2) {
                        uint32_t r[4];
                        ldmatrix4_trans(r, base + m * 16);
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            uint32_t a[4];
                            e4m3x4_to_f16x2(prmt(r[2 * h], 0u, 0x3120u), a[0], a[1]);
                            e4m3x4_to_f16x2(prmt(r[2 * h + 1], 0u, 0x3120u), a[2], a[3]);
#pragma unroll
                            for (int t = 0; t < NT; ++t) mma<CT>(out[m + h][t], a, pf[u][t][0][0], pf[u][t][0][1]);
                        }
                    }
                } else {
                    const uint32_t base =
                        values + (16 * u + (lane & 7) + (lane >> 4) * 8) * P::kRow + (lane >> 3 & 1) * 16;
#pragma unroll
                    for (int m = 0; m < kSteps; ++m) {
                        uint32_t a[4];
                        ldmatrix4_trans(a, base + m * 32);
#pragma unroll
                        for (int t = 0; t < NT; ++t)
#pragma unroll
                            for (int i = 0; i < kParts; ++i) mma<CT>(out[m][t], a, pf[u][t][i][0], pf[u][t][i][1]);
                    }
                }
            }
        }
        __syncwarp();
        const int used = stage;
        if (++stage == P::kStages) stage = 0;

        if (at.tile + 1 < at.tiles && it + 1 < count) {
            ++at.tile;
            continue;
        }

        // ---- the end of this CTA's part of (sequence, head group): join the warps.  Each
        // leaves its output as [head][element] in the stage it has just used.
        fresh = true;
        float* mine = reinterpret_cast<float*>(smem + (warp * P::kStages + used) * P::kStage);
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) sum[t][j] += __shfl_xor_sync(0xffffffffu, sum[t][j], o);
                const int head = 8 * t + 2 * in_quad + j;
                if (quad == 0) {
                    warp_max[warp * kChunk + head] = top[t][j];
                    warp_sum[warp * kChunk + head] = sum[t][j];
                }
                float* row = mine + head * P::kOutRow;
#pragma unroll
                for (int m = 0; m < kSteps; ++m) {
                    if constexpr (CT == kE4M3) {
                        *reinterpret_cast<float2*>(row + 16 * m + 2 * quad) = make_float2(out[m][t][j], out[m][t][j + 2]);
                    } else {
                        row[16 * m + quad] = out[m][t][j];
                        row[16 * m + quad + 8] = out[m][t][j + 2];
                    }
                }
            }
        const Cursor was = at;
        const int seg = seq_tiles * A.heads + was.hc * was.tiles;  // its first unit
        if (it + 1 < count) {
            at.tile = at.tiles;
            at.advance(A);
            if (at.b != was.b) seq_tiles += was.tiles;
            load_q(at);
        }
        __syncthreads();

        const bool whole = seg >= first && seg + was.tiles <= first + count;
        int first_slot = 0;  // of c0: 1 if its run starts with another (sequence, head group)
        if (!whole && piece == 0) {
            c0 = share.owner(seg);
            c1 = share.owner(seg + was.tiles - 1);
            first_slot = share.start(c0) < seg ? 1 : 0;
        }
        constexpr int kPart = kPartRows * (D + 2);
        auto slot_of = [&](int c) { return 2 * c + (c == c0 ? first_slot : 0); };
        auto part_of = [&](int c) { return A.parts + int64_t(slot_of(c)) * kPart; };
        // Row r is query head `row` of the unit's head chunk `chunk`, which a last chunk may lack.
        const int items = A.items;
        auto chunk_of = [&](int r) { return A.together == 1 ? 0 : A.by_rows.quotient(r); };
        auto write = [&](int r, int e, const float4& o, float m, float l) {
            const int chunk = chunk_of(r), v = was.hc * A.together + chunk, head = A.by_chunks.quotient(v);
            const int in = (v - head * A.chunks) * kChunk + r - chunk * A.rows;  // in the head's group
            if (in >= A.group) return;
            const int h = head * A.group + in;
            const float vs = CT == kE4M3 && A.c.v_scale ? A.c.v_scale[head] : 1.f;
            const float inv = __fdividef(vs, l);  // 2 ulp
            uint32_t* dst = reinterpret_cast<uint32_t*>(static_cast<char*>(A.out) + 2 * (was.b * A.o_token + h * A.o_head + e));
            // without weight: zeros, although a weight of zero times an infinite value or a NaN is in o
            const bool none = l == 0.f;
            const float x0 = none ? 0.f : o.x * inv, x1 = none ? 0.f : o.y * inv, x2 = none ? 0.f : o.z * inv,
                        x3 = none ? 0.f : o.w * inv;
            *reinterpret_cast<uint2*>(dst) = A.q_bf16 ? make_uint2(BF16::down(x0, x1), BF16::down(x2, x3))
                                                      : make_uint2(F16::down(x0, x1), F16::down(x2, x3));
            if (A.lse && e == 0) A.lse[int64_t(was.b) * A.q_heads + h] = (m + log2f(l)) * 0.693147180559945309f;
        };
        auto leave = [&](float* part, int r, int e, const float4& o, float m, float l) {
            *reinterpret_cast<float4*>(part + r * D + e) = o;
            if (e == 0) part[kPartRows * D + r] = m, part[kPartRows * D + kPartRows + r] = l;
        };
#pragma unroll 1
        for (int i = tid; i < items; i += kThreads) {
            const int r = i / (D / 4), e = i % (D / 4) * 4, chunk = chunk_of(r), row = r - chunk * A.rows;
            float wm[kWarps], wl[kWarps];
            float4 wo[kWarps];
            float m = -INFINITY, l = 0.f;
#pragma unroll
            for (int k = 0; k < kWarps; ++k) {
                const int w = chunk * sharers + k;
                wm[k] = -INFINITY, wl[k] = 0.f;
                wo[k] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (k < sharers) {
                    wm[k] = warp_max[w * kChunk + row], wl[k] = warp_sum[w * kChunk + row];
                    wo[k] = *reinterpret_cast<const float4*>(smem + (w * P::kStages + used) * P::kStage +
                                                             (row * P::kOutRow + e) * 4);
                }
                m = fmaxf(m, wm[k]);
            }
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int k = 0; k < kWarps; ++k) {
                const float f = exp2_approx(wm[k] - ref_of(m));
                l += f * wl[k];
                o.x += f * wo[k].x, o.y += f * wo[k].y, o.z += f * wo[k].z, o.w += f * wo[k].w;
            }
            if (whole)
                write(r, e, o, m, l);
            else
                leave(part_of(blockIdx.x), r, e, o, m, l);
        }
        __syncthreads();
        if (!whole) {
            const int n = c1 - c0 + 1, sixteens = (n + kJoin - 1) / kJoin;
            const int c_first = c0 + (int(blockIdx.x) - c0) / kJoin * kJoin;  // of this CTA's sixteen
            const int in_sixteen = min(kJoin, c1 + 1 - c_first);
            // The barrier puts the CTA's writes before thread 0's release; the CTA that counts
            // the last part has acquired all of them.
            auto arrive = [&](int32_t* counter, int parts) {
                if (tid == 0) {
                    s_last = add_acq_rel(counter, 1) == parts - 1;
                    if (s_last) *counter = 0;
                }
                __syncthreads();
                return s_last != 0;
            };
            // Level 0 joins the parts of this CTA's sixteen, level 1 the joined sixteens.  A thread
            // takes four elements of a row over all parts, or over every ways-th where there
            // are fewer elements than threads.
            float* meet = reinterpret_cast<float*>(smem + used * P::kStage);  // [ways][items][6]
            const int width = min(items, kThreads), ways = A.by_items.quotient(kThreads);
            const int my_way = A.by_items.quotient(tid), my_item = tid - my_way * width;
            for (int level = 0; level < 2; ++level) {
                if (!(level == 0 ? arrive(A.joined + slot_of(c_first), in_sixteen)
                                 : arrive(A.arrived + int64_t(was.b) * A.heads + was.hc, sixteens)))
                    break;
                const int from = level == 0 ? c_first : c0;
                const int step = level == 0 ? 1 : kJoin, parts = level == 0 ? in_sixteen : sixteens;
                const bool last = level == 1 || sixteens == 1;
                for (int i0 = 0; i0 < items; i0 += kThreads) {
                    const int i = i0 + my_item, way = my_way;
                    const int r = i / (D / 4), e = i % (D / 4) * 4;
                    float m = -INFINITY, l = 0.f;
                    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (i < items && way < ways) {
                        constexpr int kBatch = 8;
#pragma unroll 1
                        for (int p0 = way; p0 < parts; p0 += ways * kBatch) {
                            float pm[kBatch], pl[kBatch];
                            float4 po[kBatch];
#pragma unroll
                            for (int k = 0; k < kBatch; ++k) {
                                const int p = p0 + k * ways;
                                pm[k] = -INFINITY, pl[k] = 0.f;
                                po[k] = make_float4(0.f, 0.f, 0.f, 0.f);
                                if (p < parts) {
                                    const float* part = part_of(from + p * step) + (level ? A.joined_at : 0);
                                    po[k] = __ldcg(reinterpret_cast<const float4*>(part + r * D + e));
                                    pm[k] = __ldcg(part + kPartRows * D + r);
                                    pl[k] = __ldcg(part + kPartRows * D + kPartRows + r);
                                }
                            }
                            float now = m;
#pragma unroll
                            for (int k = 0; k < kBatch; ++k) now = fmaxf(now, pm[k]);
                            const float fade = exp2_approx(m - ref_of(now));
                            m = now;
                            l *= fade, o.x *= fade, o.y *= fade, o.z *= fade, o.w *= fade;
#pragma unroll
                            for (int k = 0; k < kBatch; ++k) {
                                const float f = exp2_approx(pm[k] - ref_of(m));
                                l += f * pl[k];
                                o.x += f * po[k].x, o.y += f * po[k].y, o.z += f * po[k].z, o.w += f * po[k].w;
                            }
                        }
                    }
                    if (ways > 1) {
                        float* at_me = meet + tid * 6;
                        at_me[0] = m, at_me[1] = l, at_me[2] = o.x, at_me[3] = o.y, at_me[4] = o.z, at_me[5] = o.w;
                        __syncthreads();
                        if (tid < items)
#pragma unroll 1
                            for (int w = 1; w < ways; ++w) {
                                const float* v = meet + (tid + w * items) * 6;
                                const float now = fmaxf(m, v[0]);
                                const float f = exp2_approx(m - ref_of(now)), g = exp2_approx(v[0] - ref_of(now));
                                m = now;
                                l = l * f + g * v[1];
                                o.x = o.x * f + g * v[2], o.y = o.y * f + g * v[3];
                                o.z = o.z * f + g * v[4], o.w = o.w * f + g * v[5];
                            }
                    }
                    if (i < items && way == 0) {
                        if (last)
                            write(r, e, o, m, l);
                        else
                            leave(part_of(c_first) + A.joined_at, r, e, o, m, l);
                    }
                }
                __syncthreads();
                if (last) break;
            }
        }

    }
}

// CTAs of a launch at most: as many as the plan of any cache type puts on an SM.
constexpr int max_ctas(int head_dim) { return kMaxSms * (head_dim == 64 ? 3 : head_dim == 256 ? 1 : 2); }
int most_groups(int q_heads, int kv_heads) { return kv_heads * ((q_heads / kv_heads + 7) / 8); }  // of a sequence
constexpr size_t part_floats(int head_dim) { return size_t(kPartRows) * (head_dim + 2); }
// The workspace: room for the parts and the joins of any head dimension, then the counters
// of first joins, then those of last ones.  Where the counters start depends on no shape,
// so that one buffer serves calls of all shapes: no part is ever written where another
// call counts, and every counter is zero between calls.
constexpr size_t parts_bytes(int head_dim) { return 4 * max_ctas(head_dim) * part_floats(head_dim) * 4; }
constexpr size_t kPartsRoom = std::max({parts_bytes(64), parts_bytes(96), parts_bytes(128), parts_bytes(256)});
constexpr int kMostCtas = std::max({max_ctas(64), max_ctas(96), max_ctas(128), max_ctas(256)});

template <int D, int CT, int NT>
w4a4_status launch_n(Args& A, cudaStream_t s) {
    using P = Plan<D, CT, NT>;
    static std::atomic<uint64_t> ready{0};  // devices on which the kernel's shared-memory limit has been raised
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev < 0 || dev >= 64 || !(ready.load(std::memory_order_relaxed) >> dev & 1)) {
        if (cudaFuncSetAttribute(paged_attention_kernel<D, CT, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 P::kBytes) != cudaSuccess)
            return launch_status();
        if (dev >= 0 && dev < 64) ready.fetch_or(uint64_t(1) << dev);
    }
    const int64_t longest = int64_t(A.c.max_pages) * A.c.page_size;
    const int64_t keys = A.window > 0 && A.window < longest ? A.window : longest;
    int64_t full = P::kPerSM * int64_t(device_sm_count());  // CTAs the GPU holds at once
    if (full > max_ctas(D)) full = max_ctas(D);
    A.chunks = (A.group + P::kChunk - 1) / P::kChunk;
    A.rows = A.group < P::kChunk ? A.group : P::kChunk;
    A.by_chunks = Divisor(A.chunks);
    A.by_rows = Divisor(A.rows);
    const int chunks = A.c.kv_heads * A.chunks;  // of a sequence
    // Head chunks side by side: the warps take two or four of them and the same tokens.
    //  * Chunks of one head read the same rows, which then come from HBM once (64 sequences
    //    of 8192 tokens, fp16, D = 256, groups of 16: 1113 us, one at a time 1397).
    //  * Rows of adjacent heads make one longer row of what the warps fetch together: 64
    //    sequences of 8192 tokens, E4M3, D = 64: 103 us, one head at a time 140 us; E4M3,
    //    D = 256: 353 and 409 us; fp16, D = 96: 275 and 352 us, D = 256: 703 and 707 us.  Not
    //    at D = 128 of a 16-bit type (128 sequences: 689 and 693 us; in groups of 16 heads
    //    366 and 345 us).
    //  * Neither where there is less work: it makes (sequence, head group) pairs fewer and
    //    their splits, so the joins, longer (8 x 5000 tokens, fp16, D = 128: 40 and 35 us; 2
    //    x 642, E4M3, D = 256, groups of 16: 32 and 12.4 us).  What work there is goes by
    //    the page table's width, since the lengths are on the device: where the rules above
    //    hold, short sequences in a table with room for long ones take the first time.
    //  * With sequences of one step, and more of them than CTAs, no warp is left without
    //    tokens (128 sequences of 4 tokens: 5.1 and 9.1 us).
    A.together = 1;
    const bool adjacent = (CT == kE4M3 || D != 128) && A.c.k_head_stride == D && A.c.v_head_stride == D;
    const int64_t work = int64_t(A.c.seqs) * chunks * keys;
    const bool much = work > 64 * full * kWarps * P::kTokens;
    if (((adjacent || A.chunks > 1) && much) || (keys <= P::kTokens && int64_t(A.c.seqs) * chunks > full))
        while (A.together < kPartRows / P::kChunk && A.together < kWarps && chunks % (2 * A.together) == 0)
            A.together *= 2;
    A.heads = chunks / A.together;
    A.items = A.together * A.rows * (D / 4);
    A.by_items = Divisor(A.items < kThreads ? A.items : kThreads);
    A.span_log2 = A.together == 1 ? 2 : A.together == 2 ? 1 : 0;
    A.span_log2 += P::kTokens == 32 ? 5 : 4;
    const int64_t span = int64_t(1) << A.span_log2;
    // As many CTAs as the GPU holds, or one per unit where there can be fewer.
    const int64_t units = int64_t(A.c.seqs) * A.heads * ((keys + span - 1) / span);
    if (units > INT32_MAX) return W4A4_ERR_UNSUPPORTED_SHAPE;
    const int64_t grid = units < 1 ? 1 : units < full ? units : full;
    A.by_ctas = Divisor(int(grid));
    set_dispatch_ints(CT == kF16    ? "paged_attention f16 seqs=%d heads=%d/%d dim=%d stages=%d heads/unit=%d grid=%d"
                      : CT == kBF16 ? "paged_attention bf16 seqs=%d heads=%d/%d dim=%d stages=%d heads/unit=%d grid=%d"
                                    : "paged_attention e4m3 seqs=%d heads=%d/%d dim=%d stages=%d heads/unit=%d grid=%d",
                      {A.c.seqs, A.q_heads, A.c.kv_heads, D, P::kStages, A.together, int(grid)});
    return launch<paged_attention_kernel<D, CT, NT>>(dim3(unsigned(grid)), kThreads, P::kBytes, s, A);
}

template <int D, int CT>
w4a4_status launch_c(Args& A, cudaStream_t s) {
    // 16 heads a chunk where the group has more than 8; at D = 256 their output alone would
    // take 128 registers, and two chunks of 8 side by side are faster (64 sequences of 8192
    // tokens, groups of 16, fp16: 1113 us against 1934)
    if constexpr (D < 256)
        if (A.group > 8) return launch_n<D, CT, 2>(A, s);
    return launch_n<D, CT, 1>(A, s);
}

template <int D>
w4a4_status launch_d(Args& A, cudaStream_t s) {
    return A.c.dtype == W4A4_F16    ? launch_c<D, kF16>(A, s)
           : A.c.dtype == W4A4_BF16 ? launch_c<D, kBF16>(A, s)
                                    : launch_c<D, kE4M3>(A, s);
}

}  // namespace

w4a4_status attention_read_and_clear_status() { return take_status_word(g_attention_status); }

size_t attention_workspace_bytes(int seqs, int q_heads, int kv_heads) {
    return kPartsRoom + align256((2 * kMostCtas + size_t(seqs) * most_groups(q_heads, kv_heads)) * 4);
}

w4a4_status launch_paged_attention(const w4a4_kv_cache& c, const w4a4_paged_attention_args& a, cudaStream_t s) {
    Args A;
    A.c = c;
    A.q = a.q, A.out = a.out, A.lse = a.lse, A.lengths = a.lengths;
    A.q_heads = a.q_heads;
    A.group = a.q_heads / c.kv_heads;
    A.window = a.window;
    A.longest = c.max_pages * c.page_size;
    const int size = c.dtype == W4A4_E4M3 ? 1 : 2;  // strides are at most 2^29 elements
    A.page_stride[0] = int(c.k_page_stride * size), A.page_stride[1] = int(c.v_page_stride * size);
    A.token_stride[0] = int(c.k_token_stride * size), A.token_stride[1] = int(c.v_token_stride * size);
    A.head_stride[0] = int(c.k_head_stride * size), A.head_stride[1] = int(c.v_head_stride * size);
    A.by_page = Divisor(c.page_size);
    A.parts = static_cast<float*>(a.workspace);
    A.joined_at = 2 * max_ctas(c.head_dim) * int64_t(part_floats(c.head_dim));
    A.joined = reinterpret_cast<int32_t*>(static_cast<char*>(a.workspace) + kPartsRoom);
    A.arrived = A.joined + 2 * kMostCtas;
    A.q_token = a.q_token_stride, A.q_head = a.q_head_stride;
    A.o_token = a.out_token_stride, A.o_head = a.out_head_stride;
    A.scale_log2 = a.scale * 1.44269504088896341f;
    A.q_bf16 = a.dtype == W4A4_BF16;
    switch (c.head_dim) {
        case 64: return launch_d<64>(A, s);
        case 96: return launch_d<96>(A, s);
        case 128: return launch_d<128>(A, s);
        default: return launch_d<256>(A, s);
    }
}

}  // namespace w4a4
