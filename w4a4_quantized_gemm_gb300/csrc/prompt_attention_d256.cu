// Prompt and chunk attention of 256-wide heads.
#include "prompt_attention.cuh"

namespace w4a4 {
namespace prompt {

w4a4_status run_256(Args& A, bool bf16, bool e4m3, cudaStream_t s) { return run_dim<256>(A, bf16, e4m3, s); }
w4a4_status status_256() { return take_status_word(g_prompt_status); }

}  // namespace prompt
}  // namespace w4a4
