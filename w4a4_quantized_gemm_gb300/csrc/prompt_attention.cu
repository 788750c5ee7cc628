// Entry of the attentions over packed prompts and of chunks over a paged cache
// (prompt_attention.cuh).
#include "prompt_attention.cuh"

namespace w4a4 {
namespace {

using prompt::Args;

template <class T, bool E4M3>
w4a4_status launch_d(Args& A, int dim, cudaStream_t s) {
    switch (dim) {
        case 64: return prompt::run<64, T, E4M3>(A, s);
        case 96: return prompt::run<96, T, E4M3>(A, s);
        case 128: return prompt::run<128, T, E4M3>(A, s);
        default: return prompt::run<256, T, E4M3>(A, s);
    }
}

}  // namespace

w4a4_status prompt_read_and_clear_status() { return take_status_word(prompt::g_prompt_status); }

w4a4_status launch_prompt_attention(const w4a4_prompt_attention_args& a, cudaStream_t s) {
    Args A;
    A.keys.pool[0] = static_cast<const char*>(a.k), A.keys.pool[1] = static_cast<const char*>(a.v);
    A.keys.token_stride[0] = int(2 * a.k_token_stride), A.keys.token_stride[1] = int(2 * a.v_token_stride);
    A.keys.head_stride[0] = int(2 * a.k_head_stride), A.keys.head_stride[1] = int(2 * a.v_head_stride);
    A.keys.longest = a.tokens;
    A.q = static_cast<const char*>(a.q), A.out = static_cast<char*>(a.out), A.lse = a.lse, A.starts = a.starts;
    A.q_token = a.q_token_stride, A.q_head = a.q_head_stride, A.o_token = a.out_token_stride, A.o_head = a.out_head_stride;
    A.scale = a.scale;
    A.tokens = a.tokens, A.seqs = a.seqs, A.q_heads = a.q_heads, A.kv_heads = a.kv_heads, A.window = a.window;
    A.group = a.q_heads / a.kv_heads, A.by_group = Divisor(A.group);
    A.causal = a.causal != 0;
    return a.dtype == W4A4_F16 ? launch_d<F16, false>(A, a.head_dim, s) : launch_d<BF16, false>(A, a.head_dim, s);
}

w4a4_status launch_chunk_attention(const w4a4_kv_cache& c, const w4a4_chunk_attention_args& a, cudaStream_t s) {
    Args A;
    const bool e4m3 = c.dtype == W4A4_E4M3;
    const int size = e4m3 ? 1 : 2;
    A.keys.pool[0] = static_cast<const char*>(c.k), A.keys.pool[1] = static_cast<const char*>(c.v);
    A.keys.page_stride[0] = size * c.k_page_stride, A.keys.page_stride[1] = size * c.v_page_stride;
    A.keys.token_stride[0] = int(size * c.k_token_stride), A.keys.token_stride[1] = int(size * c.v_token_stride);
    A.keys.head_stride[0] = int(size * c.k_head_stride), A.keys.head_stride[1] = int(size * c.v_head_stride);
    A.keys.scale[0] = c.k_scale, A.keys.scale[1] = c.v_scale;
    A.keys.table = c.page_table, A.keys.table_stride = c.table_stride;
    A.keys.page_size = c.page_size, A.keys.by_page = Divisor(c.page_size);
    A.keys.pages = c.pages, A.keys.longest = c.max_pages * c.page_size;
    A.q = static_cast<const char*>(a.q), A.out = static_cast<char*>(a.out), A.lse = a.lse;
    A.starts = a.starts, A.lengths = a.lengths;
    A.parts = static_cast<float*>(a.workspace);
    A.parts_of = reinterpret_cast<int4*>(A.parts + int64_t(prompt::kMaxParts) * prompt::kPartFloats);
    A.q_token = a.q_token_stride, A.q_head = a.q_head_stride, A.o_token = a.out_token_stride, A.o_head = a.out_head_stride;
    A.scale = a.scale;
    A.tokens = a.tokens, A.seqs = c.seqs, A.q_heads = a.q_heads, A.kv_heads = c.kv_heads, A.window = a.window;
    A.group = a.q_heads / c.kv_heads, A.by_group = Divisor(A.group);
    A.causal = a.causal != 0;
    if (attention_parts_bytes() < sizeof(float) * prompt::kMaxParts * prompt::kPartFloats + 32 * prompt::kMaxParts)
        return W4A4_ERR_WORKSPACE;
    if (a.dtype == W4A4_F16) return e4m3 ? launch_d<F16, true>(A, c.head_dim, s) : launch_d<F16, false>(A, c.head_dim, s);
    return e4m3 ? launch_d<BF16, true>(A, c.head_dim, s) : launch_d<BF16, false>(A, c.head_dim, s);
}

}  // namespace w4a4
