// Attention of one new token per sequence over a paged key-value cache, split over
// the cache's length and joined:
//   a_j = scale q . k_j,   out = sum_j exp(a_j) v_j / sum_j exp(a_j)
// for the q_heads / kv_heads = G query heads that share a key-value head.
//
// Every cached byte is read once and used for 2 G flops, far below what the matrix
// units need to be the limit, so the bound is HBM traffic and the kernel is built to
// keep copies in flight:
//  * The work is cut into units of 64 tokens of one (sequence, key-value head,
//    chunk of up to 16 of its query heads), in that order, and each CTA of a grid that
//    fills the GPU once takes an equal, contiguous run of units, whatever the lengths.
//    The lengths are read on the device, so a captured graph serves growing sequences.
//  * A CTA is four warps; a warp takes 16 tokens of each unit and runs on its own: it
//    copies its key and value rows into a ring of stages in shared memory (16-byte
//    asynchronous copies, rows looked up in the page table one stage ahead of the
//    copy) and keeps a running maximum, sum and output in registers (one pass).
//    Only the end of a (sequence, head) synchronises the warps.
//  * Scores are m16n8k16 warp MMAs with the query heads as rows: at one token per
//    sequence a tile has at most 16 useful rows, so the 128-row tcgen05 tile would
//    stand idle and cost an extra trip through tensor memory.
//  * A run that ends inside a (sequence, head) leaves its maximum, sum and output in
//    the workspace; the CTA that comes last joins the parts in token order.
#include <atomic>

#include "elem.cuh"
#include "kernels.h"

namespace w4a4 {
namespace {

__device__ int g_attention_status = 0;

constexpr int kWarps = 4, kThreads = kWarps * 32;
constexpr int kKeys = 16;               // tokens of a unit that a warp takes
constexpr int kUnit = kWarps * kKeys;   // tokens of a unit
constexpr int kRows = 16;               // query heads of a chunk (rows of the MMA)
constexpr int kMaxCtas = 320;           // CTAs of a launch at most (two per SM)

enum Cache { kF16, kBF16, kE4M3 };

// Shared-memory plan of one head dimension and cache type.  A row is padded to an
// odd number of 16-byte pieces: the eight rows of an ldmatrix then lie in different
// banks.   The rings take
// what two CTAs per SM leave (one at D = 256 of a 16-bit type).
template <int D, int CT, bool WIDE>
struct Plan {
    static constexpr int kSize = CT == kE4M3 ? 1 : 2;
    static constexpr int kChunks = D * kSize / 16;                  // 16-byte pieces of a row
    static constexpr int kRow = (kChunks | 1) * 16;                 // bytes of a row in shared memory
    static constexpr int kStage = 2 * kKeys * kRow;                 // keys, then values
    static constexpr int kPerSM = kStage > 10000 ? 1 : 2;           // CTAs per SM
    static constexpr int kOutRows = WIDE ? 16 : 8;
    static constexpr int kMerge = 2 * kOutRows * D * 4;             // two warps' outputs
    static constexpr int kRoom = 228 * 1024 / kPerSM - 1280;        // of an SM, less 1 KB a CTA and the static part
    static constexpr int kStages = (kRoom - kMerge - 2 * kWarps * kRows * 4) / (kWarps * (kStage + 4));
    static constexpr int kRing = kWarps * kStages * kStage;
    static constexpr int kBytes = kRing + kMerge + (2 * kWarps * kRows + kWarps * kStages) * 4;
    static_assert(kStages >= 2 && kBytes <= 227 * 1024 - 256, "shared memory");
};

struct Args {
    w4a4_kv_cache c;
    const void* q;
    void* out;
    float* lse;
    const int32_t* lengths;
    int32_t* arrived;  // [seqs][heads] parts that have arrived; zero between calls
    float* parts;      // [2 * CTAs][kRows * D outputs, kRows maxima, kRows sums]
    int64_t q_token, q_head, o_token, o_head;
    float scale_log2;
    int q_heads, group, chunks, heads, window;  // heads = kv_heads * chunks
    bool q_bf16;
};

__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];\n"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];\n"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
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
// Two E4M3 bytes (low 16 bits) -> fp16 pair, exact.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t two) {
    uint32_t d;
    asm("{\n.reg .b16 t;\ncvt.u16.u32 t, %1;\ncvt.rn.f16x2.e4m3x2 %0, t;\n}\n" : "=r"(d) : "r"(two));
    return d;
}
__device__ __forceinline__ float exp2_approx(float x) {  // 2 ulp; 2^-inf = 0
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
    return y;
}
// 16 bytes global -> shared; `bytes` of them (0 or 16) are read, the rest is zero.
__device__ __forceinline__ void cp_async16_zfill(uint32_t dst, const void* src, int bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}

// Tokens of sequence b that take part: [lo, lo + n).
__device__ __forceinline__ void range_of(const Args& A, int b, int& lo, int& n) {
    int len = A.lengths[b];
    len = max(0, min(len, A.c.max_pages * A.c.page_size));
    lo = A.window > 0 ? max(0, len - A.window) : 0;
    n = len - lo;
}

// A place in the sequence of units: tile `tile` of (sequence b, head chunk hc).
struct Cursor {
    int b, hc, tile, tiles, lo, n;
    __device__ __forceinline__ void enter(const Args& A) {
        range_of(A, b, lo, n);
        tiles = (n + kUnit - 1) / kUnit;
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
// scores by its inverse.
__device__ __forceinline__ float row_shift(float top) {
    if (!(top > 0.f) || isinf(top)) return 1.f;
    const int e = max(ilogbf(top), -100);
    return exp2f(float(13 - e));
}

template <int D, int CT, bool WIDE>
__global__ void __launch_bounds__(kThreads, Plan<D, CT, WIDE>::kPerSM) paged_attention_kernel(const Args A) {
    using P = Plan<D, CT, WIDE>;
    extern __shared__ __align__(128) uint8_t smem[];
    float* merge = reinterpret_cast<float*>(smem + P::kRing);
    float* warp_max = merge + P::kMerge / 4;        // [kWarps][kRows]
    float* warp_sum = warp_max + kWarps * kRows;    // [kWarps][kRows]
    uint32_t* masks = reinterpret_cast<uint32_t*>(warp_sum + kWarps * kRows);  // [kWarps][kStages]
    __shared__ int64_t scan[kWarps];
    __shared__ int64_t s_prefix, s_total;
    __shared__ int s_seq, s_last;

    pdl_wait();
    pdl_launch_dependents();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int quad = lane >> 2, in_quad = lane & 3;
    const int B = A.c.seqs;

    // ---- this CTA's run of units: a scan over the sequences' tile counts
    int64_t first, count, total;
    Cursor at;
    int64_t seq_tiles;  // tiles of the sequences before at.b
    {
        const int per = (B + kThreads - 1) / kThreads;
        const int b0 = min(B, tid * per), b1 = min(B, b0 + per);
        int64_t mine = 0;
        bool bad = false;
        for (int b = b0; b < b1; ++b) {
            const int len = A.lengths[b];
            bad |= len < 0 || len > A.c.max_pages * A.c.page_size;
            int lo, n;
            range_of(A, b, lo, n);
            mine += (n + kUnit - 1) / kUnit;
        }
        if (bad && blockIdx.x == 0) atomicExch(&g_attention_status, int(W4A4_ERR_INDEX));
        int64_t upto = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t v = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += v;
        }
        if (lane == 31) scan[warp] = upto;
        __syncthreads();
        for (int w = 0; w < warp; ++w) upto += scan[w];
        if (tid == kThreads - 1) s_total = upto;
        __syncthreads();
        total = s_total * A.heads;
        const int64_t ctas = min(int64_t(gridDim.x), total);
        // sequences without tokens: zeros, from whichever CTA their number falls to
        for (int b = blockIdx.x; b < B; b += gridDim.x) {
            int lo, n;
            range_of(A, b, lo, n);
            if (n > 0) continue;
            for (int i = tid; i < A.q_heads * (D / 8); i += kThreads) {
                const int h = i / (D / 8), e = i % (D / 8) * 8;
                *reinterpret_cast<uint4*>(static_cast<char*>(A.out) + 2 * (b * A.o_token + h * A.o_head + e)) =
                    make_uint4(0, 0, 0, 0);
            }
            if (A.lse)
                for (int h = tid; h < A.q_heads; h += kThreads) A.lse[int64_t(b) * A.q_heads + h] = -INFINITY;
        }
        if (blockIdx.x >= ctas) return;
        first = total * blockIdx.x / ctas;
        count = total * (blockIdx.x + 1) / ctas - first;
        const int64_t tile = first / A.heads;  // compared with whole sequences: heads * tiles units each
        int64_t before = upto - mine;
        if (mine > 0 && before <= tile && tile < upto) {
            for (int b = b0; b < b1; ++b) {
                int lo, n;
                range_of(A, b, lo, n);
                const int t = (n + kUnit - 1) / kUnit;
                if (tile < before + t) {
                    s_seq = b;
                    s_prefix = before;
                    break;
                }
                before += t;
            }
        }
        __syncthreads();
        at.b = s_seq;
        seq_tiles = s_prefix;
        at.enter(A);
        const int64_t in = first - seq_tiles * A.heads;
        at.hc = int(in / at.tiles);
        at.tile = int(in - int64_t(at.hc) * at.tiles);
    }
    const int64_t ctas = min(int64_t(gridDim.x), total);

    // ---- the warp's ring of stages
    uint8_t* ring = smem + warp * P::kStages * P::kStage;
    const uint32_t ring_addr = smem_u32(ring);
    Cursor put = at;
    int64_t to_put = count;
    int page = 0, slot = 0;  // of token lane % 16 of the next unit to copy
    bool in_range = false;
    auto look_up = [&] {
        const int j = put.tile * kUnit + warp * kKeys + (lane & 15);
        in_range = to_put > 0 && j < put.n;
        if (in_range) {
            const int tok = put.lo + j, p = tok / A.c.page_size;
            slot = tok - p * A.c.page_size;
            page = A.c.page_table[put.b * A.c.table_stride + p];
        }
    };
    auto copy_unit = [&](int stage) {
        const bool ok = in_range && page >= 0 && page < A.c.pages;
        if (in_range && !ok) atomicExch(&g_attention_status, int(W4A4_ERR_INDEX));
        const uint32_t mask = __ballot_sync(0xffffffffu, ok) & 0xffffu;
        if (lane == 0) masks[warp * P::kStages + stage] = mask;
        if (mask) {
            const int kvh = put.hc / A.chunks;
            // lanes 0-15 address the keys of their token, lanes 16-31 the values
            const bool keys = lane < 16;
            const int64_t off = !ok ? 0
                                : keys ? page * A.c.k_page_stride + slot * A.c.k_token_stride + kvh * A.c.k_head_stride
                                       : page * A.c.v_page_stride + slot * A.c.v_token_stride + kvh * A.c.v_head_stride;
            const char* row = static_cast<const char*>(keys ? A.c.k : A.c.v) + off * P::kSize;
            const uint32_t dst = ring_addr + stage * P::kStage;
#pragma unroll
            for (int i = 0; i < P::kChunks; ++i) {  // 32 rows of kChunks pieces, a warp's width at a time
                const int piece = i * 32 + lane, r = piece / P::kChunks, c = piece % P::kChunks;
                const char* src = reinterpret_cast<const char*>(
                    __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(row), r));
                cp_async16_zfill(dst + r * P::kRow + c * 16, src + c * 16, (mask >> (r & 15) & 1) * 16);
            }
        }
        if (to_put > 0) {
            --to_put;
            if (to_put > 0) put.advance(A);
            look_up();
        }
    };
    look_up();
#pragma unroll
    for (int s = 0; s < P::kStages - 1; ++s) {
        if (to_put > 0) copy_unit(s);
        cp_async_commit();
    }

    // ---- running softmax of this warp's tokens for the chunk's heads: rows quad and
    // quad + 8 (WIDE) of the tile; out[t] are the MMA accumulators of 8 columns each
    constexpr int kSteps = D / 16;
    uint32_t qf[kSteps][WIDE ? 4 : 2];
    float out[D / 8][4];
    float top[2], sum[2], factor[2];
    int rows = 0;
    bool fresh = true;

    int stage = 0;
    for (int64_t it = 0; it < count; ++it) {
        const int fill = stage == 0 ? P::kStages - 1 : stage - 1;
        if (to_put > 0) copy_unit(fill);
        cp_async_commit();

        const int kvh = at.hc / A.chunks, row0 = kvh * A.group + (at.hc - kvh * A.chunks) * kRows;
        if (fresh) {
            fresh = false;
            rows = min(kRows, (kvh + 1) * A.group - row0);
#pragma unroll
            for (int t = 0; t < D / 8; ++t)
#pragma unroll
                for (int j = 0; j < 4; ++j) out[t][j] = 0.f;
            const float ks = CT == kE4M3 && A.c.k_scale ? A.c.k_scale[kvh] : 1.f;
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                top[half] = -INFINITY, sum[half] = 0.f;
                if (half == 1 && !WIDE) continue;
                const int row = quad + 8 * half;
                const char* src = static_cast<const char*>(A.q) + 2 * (at.b * A.q_token + (row0 + row) * A.q_head);
                float shift = 1.f;
#pragma unroll
                for (int s = 0; s < kSteps; ++s) {
                    // The MMA's columns 2 (lane % 4) + {0, 1} and those + 8 stand for these
                    // elements; E4M3 rows come four consecutive elements to a lane, so
                    // there both pairs are taken from four consecutive ones.
                    const int e = CT == kE4M3 ? 16 * s + 4 * in_quad : 16 * s + 2 * in_quad;
                    uint32_t lo = 0, hi = 0;
                    if (row < rows) {
                        lo = *reinterpret_cast<const uint32_t*>(src + 2 * e);
                        hi = *reinterpret_cast<const uint32_t*>(src + 2 * (e + (CT == kE4M3 ? 2 : 8)));
                    }
                    qf[s][WIDE ? half : 0] = lo;
                    qf[s][WIDE ? 2 + half : 1] = hi;
                }
                if (CT == kE4M3 && A.q_bf16) {
                    float big = 0.f;
#pragma unroll
                    for (int s = 0; s < kSteps; ++s)
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const float2 f = BF16::up(qf[s][WIDE ? 2 * i + half : i]);
                            big = fmaxf(big, fmaxf(fabsf(f.x), fabsf(f.y)));
                        }
                    big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 1));
                    big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 2));
                    shift = row_shift(big);
#pragma unroll
                    for (int s = 0; s < kSteps; ++s)
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            uint32_t& w = qf[s][WIDE ? 2 * i + half : i];
                            const float2 f = BF16::up(w);
                            w = F16::down(f.x * shift, f.y * shift);
                        }
                }
                factor[half] = A.scale_log2 * ks / shift;
            }
        }

        cp_async_wait<P::kStages - 1>();
        __syncwarp();
        const uint32_t mask = masks[warp * P::kStages + stage];
        if (mask) {
            const uint32_t keys = ring_addr + stage * P::kStage, values = keys + kKeys * P::kRow;
            float s[2][4] = {};  // scores of tokens 0-7 and 8-15
            if constexpr (CT == kE4M3) {
                // an 8x8 b16 matrix is 8 tokens x 16 E4M3 elements: one k-step
                const uint32_t base = keys + ((lane & 7) + (lane & 8)) * P::kRow + (lane >> 4) * 16;
#pragma unroll
                for (int st = 0; st < kSteps; st += 2) {
                    uint32_t r[4];
                    ldmatrix4(r, base + st * 16);
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        const uint32_t a[4] = {qf[st + u][0], WIDE ? qf[st + u][1] : 0u, qf[st + u][WIDE ? 2 : 1],
                                               WIDE ? qf[st + u][3 % (WIDE ? 4 : 2)] : 0u};
#pragma unroll
                        for (int t = 0; t < 2; ++t)
                            mma<CT>(s[t], a, e4m3x2_to_f16x2(r[2 * u + t] & 0xffffu), e4m3x2_to_f16x2(r[2 * u + t] >> 16));
                    }
                }
            } else {
                const uint32_t base = keys + ((lane & 7) + (lane >> 4) * 8) * P::kRow + (lane >> 3 & 1) * 16;
#pragma unroll
                for (int st = 0; st < kSteps; ++st) {
                    uint32_t r[4];
                    ldmatrix4(r, base + st * 32);
                    const uint32_t a[4] = {qf[st][0], WIDE ? qf[st][1] : 0u, qf[st][WIDE ? 2 : 1],
                                           WIDE ? qf[st][3 % (WIDE ? 4 : 2)] : 0u};
                    mma<CT>(s[0], a, r[0], r[1]);
                    mma<CT>(s[1], a, r[2], r[3]);
                }
            }
            uint32_t pf[4] = {0u, 0u, 0u, 0u};  // probabilities as the A operand
#pragma unroll
            for (int half = 0; half < (WIDE ? 2 : 1); ++half) {
                float mx = -INFINITY;
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        float& v = s[t][2 * half + j];
                        v = mask >> (8 * t + 2 * in_quad + j) & 1 ? v * factor[half] : -INFINITY;
                        mx = fmaxf(mx, v);
                    }
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
                const float now = fmaxf(top[half], mx);
                const float ref = now == -INFINITY ? 0.f : now;  // all scores -inf so far: nothing, not NaN
                const float fade = exp2_approx(top[half] - ref);
                top[half] = now;
                float add = 0.f;
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    const float a = exp2_approx(s[t][2 * half] - ref), b = exp2_approx(s[t][2 * half + 1] - ref);
                    add += a + b;
                    pf[2 * t + half] = CT == kBF16 ? BF16::down(a, b) : F16::down(a, b);
                }
                sum[half] = sum[half] * fade + add;
#pragma unroll
                for (int t = 0; t < D / 8; ++t) {
                    out[t][2 * half] *= fade;
                    out[t][2 * half + 1] *= fade;
                }
            }
            const uint32_t base = values + (lane & 15) * P::kRow + (lane >> 4) * 16;
#pragma unroll
            for (int c = 0; c < P::kChunks; c += 2) {
                uint32_t r[4];
                ldmatrix4_trans(r, base + c * 16);
                if constexpr (CT == kE4M3) {
                    // a register holds (token, d), (token, d + 1), (token + 1, d), (token + 1, d + 1):
                    // the even and the odd elements of a 16-byte piece are two MMA tiles
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        const uint32_t lo = prmt(r[2 * u], 0u, 0x3120u), hi = prmt(r[2 * u + 1], 0u, 0x3120u);
                        mma<CT>(out[2 * (c + u)], pf, e4m3x2_to_f16x2(lo & 0xffffu), e4m3x2_to_f16x2(hi & 0xffffu));
                        mma<CT>(out[2 * (c + u) + 1], pf, e4m3x2_to_f16x2(lo >> 16), e4m3x2_to_f16x2(hi >> 16));
                    }
                } else {
                    mma<CT>(out[c], pf, r[0], r[1]);
                    mma<CT>(out[c + 1], pf, r[2], r[3]);
                }
            }
        }
        __syncwarp();
        if (++stage == P::kStages) stage = 0;

        if (at.tile + 1 < at.tiles && it + 1 < count) {
            ++at.tile;
            continue;
        }

        // ---- the end of this CTA's part of (sequence, head chunk): join the warps
        fresh = true;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            sum[half] += __shfl_xor_sync(0xffffffffu, sum[half], 1);
            sum[half] += __shfl_xor_sync(0xffffffffu, sum[half], 2);
            if (in_quad == 0) {
                warp_max[warp * kRows + quad + 8 * half] = top[half];
                warp_sum[warp * kRows + quad + 8 * half] = sum[half];
            }
        }
        __syncthreads();
        float all_max[2], all_sum[2];
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const int row = quad + 8 * half;
            float m = -INFINITY, l = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) m = fmaxf(m, warp_max[w * kRows + row]);
            const float ref = m == -INFINITY ? 0.f : m;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) l += warp_sum[w * kRows + row] * exp2_approx(warp_max[w * kRows + row] - ref);
            all_max[half] = m, all_sum[half] = l;
            const float f = exp2_approx(top[half] - ref);
#pragma unroll
            for (int t = 0; t < D / 8; ++t) {
                out[t][2 * half] *= f;
                out[t][2 * half + 1] *= f;
            }
        }
        // warps 2 and 3 hand over to 0 and 1, then 1 to 0; a lane meets its own layout
        auto give = [&](int to) {
            float* buf = merge + to * P::kOutRows * D;
#pragma unroll
            for (int t = 0; t < D / 8; ++t)
#pragma unroll
                for (int half = 0; half < (WIDE ? 2 : 1); ++half)
                    *reinterpret_cast<float2*>(buf + ((t * (WIDE ? 2 : 1) + half) * 32 + lane) * 2) =
                        make_float2(out[t][2 * half], out[t][2 * half + 1]);
        };
        auto take = [&](int from) {
            const float* buf = merge + from * P::kOutRows * D;
#pragma unroll
            for (int t = 0; t < D / 8; ++t)
#pragma unroll
                for (int half = 0; half < (WIDE ? 2 : 1); ++half) {
                    const float2 v = *reinterpret_cast<const float2*>(buf + ((t * (WIDE ? 2 : 1) + half) * 32 + lane) * 2);
                    out[t][2 * half] += v.x;
                    out[t][2 * half + 1] += v.y;
                }
        };
        if (warp >= 2) give(warp - 2);
        __syncthreads();
        if (warp < 2) take(warp);
        if (warp == 1) give(1);
        __syncthreads();

        const int64_t seg = seq_tiles * A.heads + int64_t(at.hc) * at.tiles;  // its first unit
        const int64_t c0 = ((seg + 1) * ctas - 1) / total;
        const int64_t c1 = ((seg + at.tiles) * ctas - 1) / total;
        const bool whole = c0 == c1;
        auto slot_of = [&](int64_t c) {  // a CTA's first and last (sequence, head) may be shared
            return A.parts + (2 * c + (c == c0 && total * c / ctas < seg ? 1 : 0)) * (kRows * D + 2 * kRows);
        };
        const float vs = CT == kE4M3 && A.c.v_scale ? A.c.v_scale[kvh] : 1.f;
        // Columns of accumulator pair t: 8 t + 2 (lane % 4) + {0, 1}; for E4M3 values
        // pair t holds the even (t even) or odd elements of 16-byte piece t / 2.
        if (warp == 0) {
            take(1);
#pragma unroll
            for (int half = 0; half < (WIDE ? 2 : 1); ++half) {
                const int row = quad + 8 * half;
                if (row >= rows) continue;
                if (whole) {
                    const float inv = all_sum[half] == 0.f ? 0.f : vs / all_sum[half];
                    char* dst = static_cast<char*>(A.out) + 2 * (at.b * A.o_token + (row0 + row) * A.o_head);
                    auto down = [&](float x, float y) { return A.q_bf16 ? BF16::down(x, y) : F16::down(x, y); };
#pragma unroll
                    for (int t = 0; t < D / 8; t += 2) {
                        const float x0 = out[t][2 * half] * inv, x1 = out[t][2 * half + 1] * inv;
                        const float y0 = out[t + 1][2 * half] * inv, y1 = out[t + 1][2 * half + 1] * inv;
                        if constexpr (CT == kE4M3) {
                            *reinterpret_cast<uint2*>(dst + 2 * (8 * t + 4 * in_quad)) = make_uint2(down(x0, y0), down(x1, y1));
                        } else {
                            *reinterpret_cast<uint32_t*>(dst + 2 * (8 * t + 2 * in_quad)) = down(x0, x1);
                            *reinterpret_cast<uint32_t*>(dst + 2 * (8 * t + 8 + 2 * in_quad)) = down(y0, y1);
                        }
                    }
                    if (A.lse && in_quad == 0)
                        A.lse[int64_t(at.b) * A.q_heads + row0 + row] =
                            (all_max[half] + log2f(all_sum[half])) * 0.693147180559945309f;
                } else {
                    float* dst = slot_of(blockIdx.x) + row * D;
#pragma unroll
                    for (int t = 0; t < D / 8; t += 2) {
                        if constexpr (CT == kE4M3) {
                            *reinterpret_cast<float4*>(dst + 8 * t + 4 * in_quad) = make_float4(
                                out[t][2 * half], out[t + 1][2 * half], out[t][2 * half + 1], out[t + 1][2 * half + 1]);
                        } else {
                            *reinterpret_cast<float2*>(dst + 8 * t + 2 * in_quad) =
                                make_float2(out[t][2 * half], out[t][2 * half + 1]);
                            *reinterpret_cast<float2*>(dst + 8 * t + 8 + 2 * in_quad) =
                                make_float2(out[t + 1][2 * half], out[t + 1][2 * half + 1]);
                        }
                    }
                    if (in_quad == 0) {
                        float* stat = slot_of(blockIdx.x) + kRows * D + row;
                        stat[0] = all_max[half];
                        stat[kRows] = all_sum[half];
                    }
                }
            }
        }
        if (!whole) {
            // The parts' writes come before the count; the last CTA reads them after it.
            if (warp == 0) {
                __threadfence();
                __syncwarp();
                if (lane == 0) {
                    int32_t* count_at = A.arrived + int64_t(at.b) * A.heads + at.hc;
                    const int parts = int(c1 - c0) + 1;
                    const bool last = atomicAdd(count_at, 1) == parts - 1;
                    if (last) *count_at = 0;
                    s_last = last;
                    __threadfence();
                }
            }
            __syncthreads();
            if (s_last) {
                for (int row = warp; row < rows; row += kWarps) {  // a warp joins a row
                    float m = -INFINITY;
                    for (int64_t c = c0 + lane; c <= c1; c += 32) m = fmaxf(m, __ldcg(slot_of(c) + kRows * D + row));
#pragma unroll
                    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
                    const float ref = m == -INFINITY ? 0.f : m;
                    float l = 0.f;
                    float acc[D / 32] = {};
#pragma unroll 4
                    for (int64_t c = c0; c <= c1; ++c) {
                        const float* part = slot_of(c);
                        const float w = exp2_approx(__ldcg(part + kRows * D + row) - ref);
                        l += w * __ldcg(part + kRows * D + kRows + row);
#pragma unroll
                        for (int i = 0; i < D / 32; ++i) acc[i] += w * __ldcg(part + row * D + i * 32 + lane);
                    }
                    const float inv = l == 0.f ? 0.f : vs / l;
                    uint16_t* dst = static_cast<uint16_t*>(A.out) + at.b * A.o_token + (row0 + row) * A.o_head;
#pragma unroll
                    for (int i = 0; i < D / 32; ++i) {
                        const float x = acc[i] * inv;
                        dst[i * 32 + lane] = uint16_t(A.q_bf16 ? BF16::down(x, 0.f) : F16::down(x, 0.f));
                    }
                    if (A.lse && lane == 0)
                        A.lse[int64_t(at.b) * A.q_heads + row0 + row] = (m + log2f(l)) * 0.693147180559945309f;
                }
            }
            __syncthreads();
        }

        if (it + 1 < count) {
            const int was = at.b, tiles = at.tiles;
            at.advance(A);
            if (at.b != was) seq_tiles += tiles;
        }
    }
}

size_t counters_bytes(int seqs, int heads) { return align256(size_t(seqs) * heads * 4); }
int chunks_of(int group) { return (group + kRows - 1) / kRows; }

template <int D, int CT, bool WIDE>
w4a4_status launch_w(const Args& A, cudaStream_t s) {
    using P = Plan<D, CT, WIDE>;
    // CUDA keeps a kernel's shared-memory limit per device; setting it again is cheap but not free
    static std::atomic<uint64_t> ready{0};
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev < 0 || dev >= 64 || !(ready.load() >> dev & 1)) {
        if (cudaFuncSetAttribute(paged_attention_kernel<D, CT, WIDE>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 P::kBytes) != cudaSuccess)
            return launch_status();
        if (dev >= 0 && dev < 64) ready.fetch_or(uint64_t(1) << dev);
    }
    // As many CTAs as the GPU holds at once, or one per unit where there can be fewer.
    const int64_t longest = int64_t(A.c.max_pages) * A.c.page_size;
    const int64_t keys = A.window > 0 && A.window < longest ? A.window : longest;
    const int64_t units = int64_t(A.c.seqs) * A.heads * ((keys + kUnit - 1) / kUnit);
    int64_t grid = P::kPerSM * device_sm_count();
    if (grid > kMaxCtas) grid = kMaxCtas;
    if (grid > units) grid = units > 0 ? units : 1;
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attr[1];
    cfg.attrs = attr;
    cfg.numAttrs = add_pdl_attr(attr, 0);
    cfg.gridDim = dim3(unsigned(grid));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = P::kBytes;
    cfg.stream = s;
    cudaLaunchKernelEx(&cfg, paged_attention_kernel<D, CT, WIDE>, A);
    set_dispatch("paged_attention mma.m16n8k16 seqs=%d heads=%d/%d dim=%d %s stages=%d grid=%d", A.c.seqs, A.q_heads,
                 A.c.kv_heads, D, CT == kF16 ? "f16" : CT == kBF16 ? "bf16" : "e4m3", P::kStages, int(grid));
    return launch_status();
}

template <int D, int CT>
w4a4_status launch_c(const Args& A, cudaStream_t s) {
    return A.group > 8 ? launch_w<D, CT, true>(A, s) : launch_w<D, CT, false>(A, s);
}

template <int D>
w4a4_status launch_d(const Args& A, cudaStream_t s) {
    return A.c.dtype == W4A4_F16    ? launch_c<D, kF16>(A, s)
           : A.c.dtype == W4A4_BF16 ? launch_c<D, kBF16>(A, s)
                                    : launch_c<D, kE4M3>(A, s);
}

}  // namespace

w4a4_status attention_read_and_clear_status() { return take_index_status(g_attention_status); }

size_t attention_workspace_bytes(int seqs, int q_heads, int kv_heads, int head_dim) {
    const int heads = kv_heads * chunks_of(q_heads / kv_heads);
    return counters_bytes(seqs, heads) + size_t(2) * kMaxCtas * (kRows * head_dim + 2 * kRows) * 4;
}

w4a4_status launch_paged_attention(const w4a4_kv_cache& c, const w4a4_paged_attention_args& a, cudaStream_t s) {
    Args A;
    A.c = c;
    A.q = a.q, A.out = a.out, A.lse = a.lse, A.lengths = a.lengths;
    A.group = a.q_heads / c.kv_heads;
    A.chunks = chunks_of(A.group);
    A.heads = c.kv_heads * A.chunks;
    A.q_heads = a.q_heads;
    A.window = a.window;
    A.arrived = static_cast<int32_t*>(a.workspace);
    A.parts = reinterpret_cast<float*>(static_cast<char*>(a.workspace) + counters_bytes(c.seqs, A.heads));
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
