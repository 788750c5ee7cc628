// Attention of many query rows at once: over whole prompts packed one behind the other, and
// of a chunk of new tokens of every sequence over a paged key-value cache.
//   a_j = scale q . k_j,   out = sum_j exp(a_j) v_j / sum_j exp(a_j)
//
// One warp takes one (row, query head) and goes over the keys that the row sees, one at a
// time, with the running maximum, sum and output in registers.
#include <type_traits>

#include "elem.cuh"
#include "kernels.h"
#include "launch.cuh"

namespace w4a4 {
namespace {

__device__ int g_prompt_status = 0;

enum Kind { kF16, kBF16, kE4M3 };

// Keys and values: rows of the packed prompts (table NULL), or of a paged cache.
struct Keys {
    const char* pool[2];         // keys, values
    int64_t page_stride[2];      // in bytes, and so below
    int token_stride[2], head_stride[2];
    const float* scale[2];       // of E4M3 rows, per key-value head
    const int32_t* table;
    int64_t table_stride;
    int page_size, pages, longest;
};

struct Args {
    Keys keys;
    const char* q;
    char* out;
    float* lse;
    const int32_t *starts, *lengths;
    int64_t q_token, q_head, o_token, o_head;  // elements
    float scale;
    int tokens, seqs, q_heads, group, window;
    bool causal;
};

struct Sequence {
    int begin, rows, length;  // its rows [begin, begin + rows) and its keys
};
__device__ __forceinline__ Sequence sequence(const Args& A, int b, bool& bad) {
    Sequence s;
    const int from = A.starts[b], to = A.starts[b + 1];
    s.begin = max(0, min(from, A.tokens));
    const int end = max(s.begin, min(to, A.tokens));
    bad = from < 0 || to < from || to > A.tokens;
    s.rows = end - s.begin;
    s.length = s.rows;
    if (A.lengths) {
        s.length = max(0, min(A.lengths[b], A.keys.longest));
        bad |= A.lengths[b] != s.length;
    }
    return s;
}

template <class T>
__device__ __forceinline__ float up1(const char* p) {
    if constexpr (T::kSize == 2)
        return T::up(*reinterpret_cast<const uint16_t*>(p)).x;
    else
        return 0.f;
}

template <class T, bool E4M3, int D>
__global__ void __launch_bounds__(128) prompt_attention_kernel(const Args A) {
    pdl_wait();
    pdl_launch_dependents();
    constexpr int kPer = D / 32;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int h = blockIdx.y, g = h / A.group;
    const Keys& K = A.keys;
    for (int b = blockIdx.z; b < A.seqs; b += gridDim.z) {
        bool bad;
        const Sequence s = sequence(A, b, bad);
        if (bad && threadIdx.x == 0) atomicExch(&g_prompt_status, int(W4A4_ERR_INDEX));
        for (int i = blockIdx.x * 4 + warp; i < s.rows; i += gridDim.x * 4) {
            const int place = s.length - s.rows + i;  // of the row among the keys
            const int hi = A.causal ? min(s.length, max(0, place + 1)) : s.length;
            const int lo = A.causal && A.window > 0 ? max(0, place + 1 - A.window) : 0;
            float q[kPer], o[kPer] = {}, m = -INFINITY, l = 0.f;
            const int64_t row = s.begin + i;
#pragma unroll
            for (int e = 0; e < kPer; ++e) q[e] = up1<T>(A.q + 2 * (row * A.q_token + h * A.q_head + lane + 32 * e));
            float scale = A.scale, v_scale = 1.f;
            if (E4M3 && K.scale[0]) scale *= K.scale[0][g];
            if (E4M3 && K.scale[1]) v_scale = K.scale[1][g];
            for (int j = lo; j < hi; ++j) {
                const char* at[2];
                bool ok = true;
                int slot = s.begin + j;
                int64_t page = 0;
                if (K.table) {
                    const int p = j / K.page_size;
                    slot = j - p * K.page_size;
                    page = K.table[b * K.table_stride + p];
                    ok = page >= 0 && page < K.pages;
                }
                if (!ok) {
                    if (lane == 0) atomicExch(&g_prompt_status, int(W4A4_ERR_INDEX));
                    continue;
                }
#pragma unroll
                for (int w = 0; w < 2; ++w)
                    at[w] = K.pool[w] + page * K.page_stride[w] + int64_t(slot) * K.token_stride[w] + int64_t(g) * K.head_stride[w];
                auto value = [&](int w, int e) {
                    if constexpr (E4M3) {
                        __nv_fp8_e4m3 x;
                        x.__x = *reinterpret_cast<const uint8_t*>(at[w] + lane + 32 * e);
                        return float(x);
                    } else {
                        return up1<T>(at[w] + 2 * (lane + 32 * e));
                    }
                };
                float a = 0.f;
#pragma unroll
                for (int e = 0; e < kPer; ++e) a = fmaf(q[e], value(0, e), a);
#pragma unroll
                for (int x = 16; x > 0; x >>= 1) a += __shfl_xor_sync(0xffffffffu, a, x);
                a *= scale;
                const float top = fmaxf(m, a), ref = top == -INFINITY ? 0.f : top;
                const float keep = expf(m - ref), p = expf(a - ref);
                l = l * keep + p;
#pragma unroll
                for (int e = 0; e < kPer; ++e) o[e] = o[e] * keep + p * value(1, e);
                m = top;
            }
            const float by = l == 0.f ? 0.f : v_scale / l;
#pragma unroll
            for (int e = 0; e < kPer; ++e) {
                const uint32_t w = T::down(l == 0.f ? 0.f : o[e] * by, 0.f);
                *reinterpret_cast<uint16_t*>(A.out + 2 * (row * A.o_token + h * A.o_head + lane + 32 * e)) = uint16_t(w);
            }
            if (A.lse && lane == 0) A.lse[row * A.q_heads + h] = l == 0.f ? -INFINITY : m + logf(l);
        }
    }
}

template <class T, bool E4M3>
w4a4_status launch_d(const Args& A, int dim, cudaStream_t s) {
    const int rows = (A.tokens + 3) / 4;
    const dim3 grid(unsigned(rows < 4096 ? rows : 4096), unsigned(A.q_heads), unsigned(A.seqs < 64 ? A.seqs : 64));
    constexpr bool bf16 = std::is_same_v<T, BF16>;
    const char* text = !A.lengths ? (bf16 ? "prompt_attention bf16 tokens=%d seqs=%d heads=%d/%d dim=%d"
                                          : "prompt_attention f16 tokens=%d seqs=%d heads=%d/%d dim=%d")
                       : E4M3     ? "chunk_attention e4m3 tokens=%d seqs=%d heads=%d/%d dim=%d"
                       : bf16     ? "chunk_attention bf16 tokens=%d seqs=%d heads=%d/%d dim=%d"
                                  : "chunk_attention f16 tokens=%d seqs=%d heads=%d/%d dim=%d";
    set_dispatch_ints(text, {A.tokens, A.seqs, A.q_heads, A.q_heads / A.group, dim});
    switch (dim) {
        case 64: return launch<prompt_attention_kernel<T, E4M3, 64>>(grid, 128, 0, s, A);
        case 96: return launch<prompt_attention_kernel<T, E4M3, 96>>(grid, 128, 0, s, A);
        case 128: return launch<prompt_attention_kernel<T, E4M3, 128>>(grid, 128, 0, s, A);
        default: return launch<prompt_attention_kernel<T, E4M3, 256>>(grid, 128, 0, s, A);
    }
}

}  // namespace

w4a4_status prompt_read_and_clear_status() { return take_status_word(g_prompt_status); }

w4a4_status launch_prompt_attention(const w4a4_prompt_attention_args& a, cudaStream_t s) {
    Args A{};
    A.keys.pool[0] = static_cast<const char*>(a.k), A.keys.pool[1] = static_cast<const char*>(a.v);
    A.keys.token_stride[0] = int(2 * a.k_token_stride), A.keys.token_stride[1] = int(2 * a.v_token_stride);
    A.keys.head_stride[0] = int(2 * a.k_head_stride), A.keys.head_stride[1] = int(2 * a.v_head_stride);
    A.q = static_cast<const char*>(a.q), A.out = static_cast<char*>(a.out), A.lse = a.lse, A.starts = a.starts;
    A.q_token = a.q_token_stride, A.q_head = a.q_head_stride, A.o_token = a.out_token_stride, A.o_head = a.out_head_stride;
    A.scale = a.scale;
    A.tokens = a.tokens, A.seqs = a.seqs, A.q_heads = a.q_heads, A.group = a.q_heads / a.kv_heads, A.window = a.window;
    A.causal = a.causal != 0;
    return a.dtype == W4A4_F16 ? launch_d<F16, false>(A, a.head_dim, s) : launch_d<BF16, false>(A, a.head_dim, s);
}

w4a4_status launch_chunk_attention(const w4a4_kv_cache& c, const w4a4_chunk_attention_args& a, cudaStream_t s) {
    Args A{};
    const bool e4m3 = c.dtype == W4A4_E4M3;
    const int size = e4m3 ? 1 : 2;
    A.keys.pool[0] = static_cast<const char*>(c.k), A.keys.pool[1] = static_cast<const char*>(c.v);
    A.keys.page_stride[0] = size * c.k_page_stride, A.keys.page_stride[1] = size * c.v_page_stride;
    A.keys.token_stride[0] = int(size * c.k_token_stride), A.keys.token_stride[1] = int(size * c.v_token_stride);
    A.keys.head_stride[0] = int(size * c.k_head_stride), A.keys.head_stride[1] = int(size * c.v_head_stride);
    A.keys.scale[0] = c.k_scale, A.keys.scale[1] = c.v_scale;
    A.keys.table = c.page_table, A.keys.table_stride = c.table_stride;
    A.keys.page_size = c.page_size, A.keys.pages = c.pages, A.keys.longest = c.max_pages * c.page_size;
    A.q = static_cast<const char*>(a.q), A.out = static_cast<char*>(a.out), A.lse = a.lse;
    A.starts = a.starts, A.lengths = a.lengths;
    A.q_token = a.q_token_stride, A.q_head = a.q_head_stride, A.o_token = a.out_token_stride, A.o_head = a.out_head_stride;
    A.scale = a.scale;
    A.tokens = a.tokens, A.seqs = c.seqs, A.q_heads = a.q_heads, A.group = a.q_heads / c.kv_heads, A.window = a.window;
    A.causal = a.causal != 0;
    if (a.dtype == W4A4_F16) return e4m3 ? launch_d<F16, true>(A, c.head_dim, s) : launch_d<F16, false>(A, c.head_dim, s);
    return e4m3 ? launch_d<BF16, true>(A, c.head_dim, s) : launch_d<BF16, false>(A, c.head_dim, s);
}

}  // namespace w4a4
