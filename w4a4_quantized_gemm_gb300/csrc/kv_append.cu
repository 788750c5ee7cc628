// Appending the keys and values of new tokens to a paged cache, with the per-head
// RMSNorm of q and k and the position rotation on the way ("W4A4 CUDA Kernel for
// Voice Clone", 3.4: the step between the qkv linear and attention).
//
// A head x of D elements becomes x' = x / sqrt(mean x^2 + eps) * gain and then, for
// the pairs (a, b) of the first rot_dim elements, (x'_a c - x'_b n, x'_b c + x'_a n)
// with c, n the cosine and sine of the token's position times the pair's frequency.
// Every byte is read once and written once, so the bound is HBM traffic.
//
// One CTA of 128 threads takes one token (a slice of its heads when there are few
// tokens): the heads of a token share position, page and rotation, which are
// looked up once and stay in registers.  A head belongs to D / 8 lanes, 16 bytes
// each (a 16-lane group with four idle lanes at D = 96); the partner of a pair is
// in the same lane (interleaved) or in a lane of the same group, reached by a
// shuffle; the sum of squares is a shuffle reduction over the group.
#include "elem.cuh"
#include "kernels.h"

namespace w4a4 {
namespace {

__device__ int g_append_status = 0;

constexpr int kThreads = 128;

template <class T, bool E4M3, int LPH>  // LPH: lanes of a head's group (8, 16 or 32)
__global__ void __launch_bounds__(kThreads) kv_append_kernel(const w4a4_kv_cache c, const w4a4_kv_append_args a) {
    pdl_wait();
    pdl_launch_dependents();
    const int t = blockIdx.x, lane = threadIdx.x % LPH, group = threadIdx.x / LPH;
    constexpr int kGroups = kThreads / LPH;
    const int D = c.head_dim, e = lane * 8;  // this lane's elements e .. e + 7
    const bool has = e < D;

    // The token's place.  Anything outside its table makes it a padding token.
    const int seq = a.seqs ? a.seqs[t] : t;
    const int pos = a.positions[t];
    bool live = seq >= 0;
    int64_t page = 0;
    int slot = 0;
    if (live) {
        bool ok = seq < c.seqs && pos >= 0 && (!a.rope || pos < a.rope_rows);
        const int at = ok ? pos / c.page_size : 0;
        ok = ok && at < c.max_pages;
        if (ok) {
            page = c.page_table[int64_t(seq) * c.table_stride + at];
            slot = pos - at * c.page_size;
            ok = page >= 0 && page < c.pages;
        }
        if (!ok) {
            live = false;
            if (threadIdx.x == 0) atomicExch(&g_append_status, int(W4A4_ERR_INDEX));
        }
    }

    // This lane's rotation: pairs (i, i + R/2) use the cosines of eight consecutive
    // i, interleaved pairs those of four.
    const int R = a.rope && live ? a.rot_dim : 0;
    const bool turns = e < R, inter = a.interleaved != 0;
    const bool upper = !inter && e >= R / 2;  // this lane holds the b of its pairs
    float cs[8], sn[8];
    if (turns) {
        const float* row = a.rope + int64_t(pos) * R;
        const int i = inter ? e / 2 : (upper ? e - R / 2 : e);
        const float4* pc = reinterpret_cast<const float4*>(row + i);
        const float4* ps = reinterpret_cast<const float4*>(row + R / 2 + i);
        const float4 c0 = pc[0], s0 = ps[0];
        float4 c1 = c0, s1 = s0;
        if (!inter) c1 = pc[1], s1 = ps[1];
        cs[0] = c0.x, cs[1] = c0.y, cs[2] = c0.z, cs[3] = c0.w, cs[4] = c1.x, cs[5] = c1.y, cs[6] = c1.z, cs[7] = c1.w;
        sn[0] = s0.x, sn[1] = s0.y, sn[2] = s0.z, sn[3] = s0.w, sn[4] = s1.x, sn[5] = s1.y, sn[6] = s1.z, sn[7] = s1.w;
    }
    // Half-split partner's lane inside the group (its own lane where nothing turns).
    const int partner = (threadIdx.x & 31) - lane + (turns && !inter ? (upper ? lane - R / 16 : lane + R / 16) : lane);

    const int rows = a.q_heads + 2 * c.kv_heads;
    // The loop bound is the warp's first group's, so that every lane takes part in
    // each shuffle; `valid` masks the memory accesses.
    const int first = blockIdx.y * kGroups + group;
    const int step = gridDim.y * kGroups;
    const int warp_first = blockIdx.y * kGroups + (threadIdx.x & ~31) / LPH;
    for (int base = 0; warp_first + base < rows; base += step) {
        const int row = first + base;
        const bool valid = has && row < rows;
        const bool is_q = row < a.q_heads, is_v = row >= a.q_heads + c.kv_heads;
        const int h = is_q ? row : (is_v ? row - a.q_heads - c.kv_heads : row - a.q_heads);
        const void* src = is_q ? a.q : (is_v ? a.v : a.k);
        const int64_t from = is_q ? t * a.q_token_stride + h * a.q_head_stride
                             : is_v ? t * a.v_token_stride + h * a.v_head_stride
                                    : t * a.k_token_stride + h * a.k_head_stride;
        float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        if (valid && live) load8<T>(src, from + e, x);
        const void* gain = is_q ? a.q_gain : a.k_gain;
        if (a.q_gain || a.k_gain) {
            float ss = 0.f;
#pragma unroll
            for (int j = 0; j < 8; ++j) ss += x[j] * x[j];
#pragma unroll
            for (int o = LPH / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
            if (!is_v && gain && valid && live) {
                const float inv = 1.f / sqrtf(ss / float(D) + a.eps);
                float g[8];
                load8<T>(gain, e, g);
#pragma unroll
                for (int j = 0; j < 8; ++j) x[j] = x[j] * inv * g[j];
            }
        }
        if (inter) {
            if (turns && !is_v) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float p = x[2 * j], q = x[2 * j + 1];
                    x[2 * j] = p * cs[j] - q * sn[j];
                    x[2 * j + 1] = q * cs[j] + p * sn[j];
                }
            }
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float o = __shfl_sync(0xffffffffu, x[j], partner);
                if (turns && !is_v) x[j] = upper ? x[j] * cs[j] + o * sn[j] : x[j] * cs[j] - o * sn[j];
            }
        }
        if (!valid) continue;
        if (is_q) {
            store8<T>(a.q_out, t * a.out_token_stride + h * a.out_head_stride + e, x);
        } else if (live) {
            void* pool = is_v ? c.v : c.k;
            const int64_t to = is_v ? page * c.v_page_stride + slot * c.v_token_stride + h * c.v_head_stride
                                    : page * c.k_page_stride + slot * c.k_token_stride + h * c.k_head_stride;
            if constexpr (E4M3) {
                const float* scales = is_v ? c.v_scale : c.k_scale;
                const float s = scales ? scales[h] : 1.f;
                uint2 o;
                o.x = e4m3x2(x[0] / s, x[1] / s) | e4m3x2(x[2] / s, x[3] / s) << 16;
                o.y = e4m3x2(x[4] / s, x[5] / s) | e4m3x2(x[6] / s, x[7] / s) << 16;
                *reinterpret_cast<uint2*>(static_cast<char*>(pool) + to + e) = o;
            } else {
                store8<T>(pool, to + e, x);
            }
        }
    }
}

__global__ void rope_table_kernel(float* rope, int64_t n, int half, double log2_theta) {
    pdl_wait();
    pdl_launch_dependents();
    for (int64_t i = int64_t(blockIdx.x) * blockDim.x + threadIdx.x; i < n; i += int64_t(gridDim.x) * blockDim.x) {
        const int64_t p = i / half;
        const int j = int(i - p * half);
        double s, co;
        sincos(double(p) * exp2(-log2_theta * double(j) / double(half)), &s, &co);
        rope[p * 2 * half + j] = float(co);
        rope[p * 2 * half + half + j] = float(s);
    }
}

template <class T, bool E4M3>
void launch_t(const w4a4_kv_cache& c, const w4a4_kv_append_args& a, cudaStream_t s) {
    const int lph = c.head_dim <= 64 ? 8 : c.head_dim <= 128 ? 16 : 32;
    const int groups = kThreads / lph, rows = a.q_heads + 2 * c.kv_heads;
    // Few tokens: a token's heads are spread over CTAs until two per SM have work.
    const int most = (rows + groups - 1) / groups, want = (2 * device_sm_count() + a.tokens - 1) / a.tokens;
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attr[1];
    cfg.attrs = attr;
    cfg.numAttrs = add_pdl_attr(attr, 0);
    cfg.gridDim = dim3(unsigned(a.tokens), unsigned(most < want ? most : want));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    if (lph == 8)
        cudaLaunchKernelEx(&cfg, kv_append_kernel<T, E4M3, 8>, c, a);
    else if (lph == 16)
        cudaLaunchKernelEx(&cfg, kv_append_kernel<T, E4M3, 16>, c, a);
    else
        cudaLaunchKernelEx(&cfg, kv_append_kernel<T, E4M3, 32>, c, a);
    set_dispatch("kv_append tokens=%d heads=%d+2x%d dim=%d %s grid=%dx%u", a.tokens, a.q_heads, c.kv_heads, c.head_dim,
                 E4M3 ? "e4m3 cache" : "16-bit cache", a.tokens, cfg.gridDim.y);
}

}  // namespace

w4a4_status append_read_and_clear_status() { return take_index_status(g_append_status); }

void launch_kv_append(const w4a4_kv_cache& c, const w4a4_kv_append_args& a, cudaStream_t s) {
    const bool e4m3 = c.dtype == W4A4_E4M3;
    if (a.dtype == W4A4_F16)
        e4m3 ? launch_t<F16, true>(c, a, s) : launch_t<F16, false>(c, a, s);
    else
        e4m3 ? launch_t<BF16, true>(c, a, s) : launch_t<BF16, false>(c, a, s);
}

void launch_rope_table(float* rope, int rows, int rot_dim, double theta, cudaStream_t s) {
    const int64_t n = int64_t(rows) * (rot_dim / 2), blocks = (n + 255) / 256;
    const int64_t most = 8 * device_sm_count();
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attr[1];
    cfg.attrs = attr;
    cfg.numAttrs = add_pdl_attr(attr, 0);
    cfg.gridDim = dim3(unsigned(blocks < most ? blocks : most));
    cfg.blockDim = dim3(256);
    cfg.stream = s;
    cudaLaunchKernelEx(&cfg, rope_table_kernel, rope, n, rot_dim / 2, log2(theta));
    set_dispatch("rope_table rows=%d rot_dim=%d", rows, rot_dim);
}

}  // namespace w4a4
