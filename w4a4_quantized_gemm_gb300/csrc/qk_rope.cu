// Queries and keys of a prompt normalised and rotated by their positions where no cache
// takes the keys ("W4A4 CUDA Kernel for Voice Clone", 3.4: the step between the qkv
// linear and attention).
//
// A head x of D elements becomes x' = x / sqrt(mean x^2 + eps) * gain and then, for the
// pairs (a, b) of the first rot_dim elements, (x'_a c - x'_b n, x'_b c + x'_a n) with c, n
// the cosine and sine of the token's position times the pair's frequency.  Every byte is
// read once and written once, so the bound is HBM traffic.
//
// A CTA takes one token, or a slice of its heads when there are few: they share position and
// rotation, which are looked up once and stay in registers.  A head belongs to D / 16 lanes
// (eight with two idle ones at D = 96), each with the two 16-byte pieces that hold both
// elements of its pairs, so the rotation needs no exchange, the sum of squares is a shuffle
// reduction, and a row may be its own output.
#include "elem.cuh"
#include "kernels.h"
#include "launch.cuh"

namespace w4a4 {
namespace {

__device__ int g_rope_status = 0;

// Many tokens: one warp a CTA in at most 78 registers, so that an SM holds 26, and HBM enough
// loads; few, which all fit at once: two warps.
constexpr int kFew = 5;  // tokens per SM up to which they are few
constexpr int threads_of(bool many) { return many ? 32 : 64; }
constexpr int per_sm(bool many) { return many ? 26 : 10; }  // CTAs that an SM holds
constexpr int kAhead = 2;  // heads whose pieces a lane holds at once

template <class T, int LPH, bool MANY>  // LPH: lanes of a head's group (4, 8 or 16)
__global__ void __launch_bounds__(threads_of(MANY), per_sm(MANY)) qk_rope_kernel(const w4a4_qk_rope_args a) {
    pdl_wait();
    pdl_launch_dependents();
    constexpr int kGroups = threads_of(MANY) / LPH;
    const int t = blockIdx.x, lane = threadIdx.x % LPH, group = threadIdx.x / LPH;
    const int D = a.head_dim, R = a.rope ? a.rot_dim : 0;
    const bool has = lane < D / 16, inter = a.interleaved != 0;
    // This lane's elements e0 .. + 7 and e1 .. + 7: a pair's halves while they are rotated
    // ones, else two neighbouring pieces of the rest.
    const bool turns = lane < R / 16;
    const int e0 = turns ? 8 * lane : 16 * lane, e1 = turns ? e0 + R / 2 : e0 + 8;

    const int rows = a.q_heads + a.kv_heads, step = gridDim.y * kGroups, first = blockIdx.y * kGroups + group;
    uint4 raw[kAhead][2];
    auto load = [&](int base) {
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int row = first + base + u * step;
            raw[u][0] = raw[u][1] = make_uint4(0, 0, 0, 0);
            if (!has || row >= rows) continue;
            const bool is_q = row < a.q_heads;
            const char* src = static_cast<const char*>(is_q ? a.q : a.k);
            src += 2 * (is_q ? t * a.q_token_stride + row * a.q_head_stride
                             : t * a.k_token_stride + (row - a.q_heads) * a.k_head_stride);
            raw[u][0] = *reinterpret_cast<const uint4*>(src + 2 * e0);
            raw[u][1] = *reinterpret_cast<const uint4*>(src + 2 * e1);
        }
    };
    load(0);  // before anything else: the look-ups hide behind it

    const int pos = a.positions ? a.positions[t] : 0;
    bool live = pos >= 0;
    if (live && a.rope && pos >= a.rope_rows) {
        live = false;
        if (threadIdx.x == 0) atomicExch(&g_rope_status, int(W4A4_ERR_INDEX));
    }
    // The cosines of eight consecutive pairs (half-split), or of the four pairs of each piece
    // (interleaved).
    float cs[8], sn[8];
    if (turns && live) {
        const float* row = a.rope + int64_t(pos) * R;
        const int i0 = inter ? e0 / 2 : e0, i1 = inter ? e1 / 2 : e0 + 4;
        *reinterpret_cast<float4*>(cs) = *reinterpret_cast<const float4*>(row + i0);
        *reinterpret_cast<float4*>(cs + 4) = *reinterpret_cast<const float4*>(row + i1);
        *reinterpret_cast<float4*>(sn) = *reinterpret_cast<const float4*>(row + R / 2 + i0);
        *reinterpret_cast<float4*>(sn + 4) = *reinterpret_cast<const float4*>(row + R / 2 + i1);
    }
    const float per_head = 1.f / float(D);
    // The loop bound is the warp's first group's, so that every lane takes part in each shuffle.
    const int warp_first = blockIdx.y * kGroups + (threadIdx.x & ~31) / LPH;
    for (int base = 0; warp_first + base < rows; base += kAhead * step) {
        if (base) load(base);
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int row = first + base + u * step;
            if (warp_first + base + u * step >= rows) break;
            const bool is_q = row < a.q_heads, here = has && row < rows;
            float x[8], y[8];
            up8<T>(raw[u][0], x);
            up8<T>(raw[u][1], y);
            if (a.q_gain || a.k_gain) {
                float ss = 0.f;
#pragma unroll
                for (int j = 0; j < 8; ++j) ss += x[j] * x[j] + y[j] * y[j];
#pragma unroll
                for (int o = LPH / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
                const void* gain = is_q ? a.q_gain : a.k_gain;
                if (gain && here) {
                    const float inv = rsqrtf(ss * per_head + a.eps);  // 2 ulp
                    float g[8], h[8];
                    load8<T>(gain, e0, g);
                    load8<T>(gain, e1, h);
#pragma unroll
                    for (int j = 0; j < 8; ++j) x[j] = x[j] * inv * g[j], y[j] = y[j] * inv * h[j];
                }
            }
            if (!here) continue;
            if (!live) {
#pragma unroll
                for (int j = 0; j < 8; ++j) x[j] = y[j] = 0.f;
            } else if (turns && inter) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float p = x[2 * j], q = x[2 * j + 1], r = y[2 * j], s = y[2 * j + 1];
                    x[2 * j] = p * cs[j] - q * sn[j];
                    x[2 * j + 1] = q * cs[j] + p * sn[j];
                    y[2 * j] = r * cs[4 + j] - s * sn[4 + j];
                    y[2 * j + 1] = s * cs[4 + j] + r * sn[4 + j];
                }
            } else if (turns) {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float p = x[j], q = y[j];
                    x[j] = p * cs[j] - q * sn[j];
                    y[j] = q * cs[j] + p * sn[j];
                }
            }
            void* dst = is_q ? a.q_out : a.k_out;
            const int64_t to = is_q ? t * a.q_out_token_stride + row * a.q_out_head_stride
                                    : t * a.k_out_token_stride + (row - a.q_heads) * a.k_out_head_stride;
            store8<T>(dst, to + e0, x);
            store8<T>(dst, to + e1, y);
        }
    }
}

template <class T, bool MANY>
w4a4_status launch_m(const w4a4_qk_rope_args& a, cudaStream_t s) {
    const int lph = a.head_dim <= 64 ? 4 : a.head_dim <= 128 ? 8 : 16;
    const int groups = threads_of(MANY) / lph, rows = a.q_heads + a.kv_heads;
    // A token's heads are spread over as many CTAs as the GPU holds at once.
    const int most = (rows + groups - 1) / groups, full = per_sm(MANY) * device_sm_count();
    const int want = full / a.tokens > 1 ? full / a.tokens : 1;
    const dim3 grid(unsigned(a.tokens), unsigned(most < want ? most : want));
    set_dispatch_ints("qk_rope tokens=%d heads=%d+%d dim=%d threads=%d grid=%dx%d",
                      {a.tokens, a.q_heads, a.kv_heads, a.head_dim, threads_of(MANY), a.tokens, int(grid.y)});
    if (lph == 4) return launch<qk_rope_kernel<T, 4, MANY>>(grid, threads_of(MANY), 0, s, a);
    if (lph == 8) return launch<qk_rope_kernel<T, 8, MANY>>(grid, threads_of(MANY), 0, s, a);
    return launch<qk_rope_kernel<T, 16, MANY>>(grid, threads_of(MANY), 0, s, a);
}

template <class T>
w4a4_status launch_t(const w4a4_qk_rope_args& a, cudaStream_t s) {
    return a.tokens > kFew * device_sm_count() ? launch_m<T, true>(a, s) : launch_m<T, false>(a, s);
}

}  // namespace

w4a4_status rope_read_and_clear_status() { return take_status_word(g_rope_status); }

w4a4_status launch_qk_rope(const w4a4_qk_rope_args& a, cudaStream_t s) {
    return a.dtype == W4A4_F16 ? launch_t<F16>(a, s) : launch_t<BF16>(a, s);
}

}  // namespace w4a4
