// What the kernels of prompt_attention.cuh are given, and their entries, one a head dimension.
#pragma once
#include "common.cuh"

namespace w4a4 {
namespace prompt {

constexpr int kMaxParts = 156;             // of a call
constexpr int kPartFloats = 256 * 130;     // of one: [rows][D] outputs, [256] maxima, [256] sums

// Keys and values: rows of the packed prompts (table NULL), or of a paged cache.
struct Keys {
    const char* pool[2] = {};              // keys, values
    int64_t page_stride[2] = {};           // in bytes, and so below
    int token_stride[2] = {}, head_stride[2] = {};
    const float* scale[2] = {};            // of E4M3 rows, per key-value head
    const int32_t* table = nullptr;
    int64_t table_stride = 0;
    int page_size = 1, pages = 0, longest = 0;
    int box = 0;                           // keys that one copy of the tensor maps brings, 0: there are no maps
    Divisor by_page;
};

struct Args {
    Keys keys;
    const char* q;
    char* out;
    float* lse;
    const int32_t *starts, *lengths = nullptr;
    float* parts = nullptr;                // NULL: units are not split
    int4* parts_of = nullptr;              // [kMaxParts][2]: (begin, head, row0, rows), (first part, parts of the unit)
    int64_t q_token, q_head, o_token, o_head;  // elements
    float scale;
    int tokens, seqs, q_heads, kv_heads, group, window;
    bool causal;
    Divisor by_group;
    uint64_t wait_ns = 0, tile_ns = 0;     // to wait for a unit to be done with, and more for each of its tiles
    bool q_boxes = false;                  // queries come by the copy engine: 128 rows are whole tokens
};

w4a4_status run_64(Args& A, bool bf16, bool e4m3, cudaStream_t s);
w4a4_status run_96(Args& A, bool bf16, bool e4m3, cudaStream_t s);
w4a4_status run_128(Args& A, bool bf16, bool e4m3, cudaStream_t s);
w4a4_status run_256(Args& A, bool bf16, bool e4m3, cudaStream_t s);
w4a4_status status_64();
w4a4_status status_96();
w4a4_status status_128();
w4a4_status status_256();

}  // namespace prompt
}  // namespace w4a4
