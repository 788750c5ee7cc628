// Entry of the attentions over packed prompts and of chunks over a paged cache
// (prompt_attention.cuh).
#include <atomic>

#include "kernels.h"
#include "prompt_args.cuh"

namespace w4a4 {
namespace {

using prompt::Args;

std::atomic<uint64_t> g_wait_ns{0}, g_tile_ns{0};

w4a4_status run(Args& A, int dim, bool bf16, bool e4m3, cudaStream_t s) {
    A.wait_ns = g_wait_ns.load(std::memory_order_relaxed), A.tile_ns = g_tile_ns.load(std::memory_order_relaxed);
    if (A.wait_ns == 0) A.wait_ns = 2000000000ull, A.tile_ns = 20000;  // a tile takes 1 to 2 us
    switch (dim) {
        case 64: return prompt::run_64(A, bf16, e4m3, s);
        case 96: return prompt::run_96(A, bf16, e4m3, s);
        case 128: return prompt::run_128(A, bf16, e4m3, s);
        default: return prompt::run_256(A, bf16, e4m3, s);
    }
}

}  // namespace

void set_prompt_wait_ns(uint64_t ns, uint64_t tile_ns) {
    g_wait_ns.store(ns, std::memory_order_relaxed), g_tile_ns.store(tile_ns, std::memory_order_relaxed);
}

w4a4_status prompt_read_and_clear_status() {
    w4a4_status first = W4A4_OK;  // every word is read: reading clears it
    for (const w4a4_status st : {prompt::status_64(), prompt::status_96(), prompt::status_128(), prompt::status_256()})
        if (first == W4A4_OK) first = st;
    return first;
}

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
    return run(A, a.head_dim, a.dtype == W4A4_BF16, false, s);
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
    return run(A, c.head_dim, a.dtype == W4A4_BF16, e4m3, s);
}

}  // namespace w4a4
