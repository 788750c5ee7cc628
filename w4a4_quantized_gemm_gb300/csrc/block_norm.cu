// The residual stream between two blocks of a decoder layer in one pass over a row:
//   r' = r + scale * gate (.) post(y),   x = pre(r')
// post and pre each nothing, an RMSNorm or a LayerNorm.  Four separate steps (norm,
// gate, add, norm) would move a row ten times; here y and r are read once and r' and
// x written once, which is the HBM bound.
//
// One CTA per row.  A thread keeps CH chunks of eight elements of y and r in
// registers (fp32) through both norms, so the reductions are the only exchanges:
// each is a warp shuffle and one pass through shared memory.  The variance of a
// LayerNorm is summed about the mean in a second reduction, not as a difference of
// squares, so that a row with a large mean keeps its digits.
#include "elem.cuh"
#include "kernels.h"

namespace w4a4 {
namespace {

// Sum over the CTA, the same bits in every thread (fixed order).  `slot` alternates
// between consecutive calls, so one barrier per call separates its reads from the
// next call's writes.
template <int NT>
__device__ __forceinline__ float block_sum(float v, float (*red)[NT / 32], int slot) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if constexpr (NT == 32) return v;
    if ((threadIdx.x & 31) == 0) red[slot][threadIdx.x >> 5] = v;
    __syncthreads();
    float t = 0.f;
#pragma unroll
    for (int w = 0; w < NT / 32; ++w) t += red[slot][w];
    return t;
}

// z -> norm(z) in place; chunk c of this thread is elements (c * NT + tid) * 8 ..
// and takes part while that is below W.
template <class T, int NT, int CH>
__device__ __forceinline__ void normalise(float (&z)[CH][8], int kind, const void* gain, const void* bias, int W,
                                          float eps, float (*red)[NT / 32], int& slot) {
    if (kind == W4A4_NORM_NONE) return;
    const float n = 1.f / float(W);
    float mean = 0.f;
    if (kind == W4A4_NORM_LAYER) {
        float s = 0.f;
#pragma unroll
        for (int c = 0; c < CH; ++c)
#pragma unroll
            for (int j = 0; j < 8; ++j) s += z[c][j];
        mean = block_sum<NT>(s, red, slot) * n;
        slot ^= 1;
    }
    float ss = 0.f;
#pragma unroll
    for (int c = 0; c < CH; ++c)
        if ((c * NT + int(threadIdx.x)) * 8 < W)
#pragma unroll
            for (int j = 0; j < 8; ++j) ss += (z[c][j] - mean) * (z[c][j] - mean);
    const float inv = 1.f / sqrtf(block_sum<NT>(ss, red, slot) * n + eps);
    slot ^= 1;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        const int k = (c * NT + threadIdx.x) * 8;
        if (k >= W) continue;
        float g[8], b[8];
        if (gain) load8<T>(gain, k, g);
        if (kind == W4A4_NORM_LAYER && bias) load8<T>(bias, k, b);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            float v = (z[c][j] - mean) * inv;
            if (gain) v *= g[j];
            if (kind == W4A4_NORM_LAYER && bias) v += b[j];
            z[c][j] = v;
        }
    }
}

template <class T, class R, int NT, int CH>
__global__ void __launch_bounds__(NT) block_norm_kernel(const w4a4_block_norm_args a) {
    __shared__ float red[2][NT / 32];
    pdl_wait();
    pdl_launch_dependents();
    const int64_t m = blockIdx.x;
    const int W = a.width;
    const int64_t gate_at = a.rows_per_gate ? m / a.rows_per_gate * a.gate_stride : 0;
    float y[CH][8], r[CH][8];
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        const int k = (c * NT + threadIdx.x) * 8;
        if (k < W) {
            load8<T>(a.y, m * a.y_stride + k, y[c]);
            load8<R>(a.r, m * a.r_stride + k, r[c]);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) y[c][j] = r[c][j] = 0.f;
        }
    }
    int slot = 0;
    normalise<T, NT, CH>(y, a.post, a.post_gain, a.post_bias, W, a.eps, red, slot);
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        const int k = (c * NT + threadIdx.x) * 8;
        if (k >= W) continue;
        float g[8];
        if (a.gate) load8<T>(a.gate, gate_at + k, g);
#pragma unroll
        for (int j = 0; j < 8; ++j) r[c][j] += a.scale * (a.gate ? g[j] * y[c][j] : y[c][j]);
        store8<R>(a.r_out, m * a.r_out_stride + k, r[c]);
    }
    if (!a.x) return;
    normalise<T, NT, CH>(r, a.pre, a.pre_gain, a.pre_bias, W, a.eps, red, slot);
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        const int k = (c * NT + threadIdx.x) * 8;
        if (k < W) store8<T>(a.x, m * a.x_stride + k, r[c]);
    }
}

template <class T, class R, int NT, int CH>
void launch_k(const w4a4_block_norm_args& a, cudaStream_t s) {
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attr[1];
    cfg.attrs = attr;
    cfg.numAttrs = add_pdl_attr(attr, 0);
    cfg.gridDim = dim3(unsigned(a.rows));
    cfg.blockDim = dim3(NT);
    cfg.stream = s;
    cudaLaunchKernelEx(&cfg, block_norm_kernel<T, R, NT, CH>, a);
    set_dispatch("block_norm rows=%d width=%d threads=%d chunks/thread=%d", a.rows, a.width, NT, CH);
}

template <class T, class R>
void launch_r(const w4a4_block_norm_args& a, cudaStream_t s) {
    const int chunks = a.width / 8;
    if (chunks <= 32)
        launch_k<T, R, 32, 1>(a, s);
    else if (chunks <= 128)
        launch_k<T, R, 128, 1>(a, s);
    else if (chunks <= 256)
        launch_k<T, R, 256, 1>(a, s);
    else if (chunks <= 512)
        launch_k<T, R, 256, 2>(a, s);
    else if (chunks <= 1024)
        launch_k<T, R, 512, 2>(a, s);
    else
        launch_k<T, R, 512, 4>(a, s);
}

}  // namespace

void launch_block_norm(const w4a4_block_norm_args& a, cudaStream_t s) {
    if (a.dtype == W4A4_F16)
        a.res_dtype == W4A4_F32 ? launch_r<F16, F32>(a, s) : launch_r<F16, F16>(a, s);
    else
        a.res_dtype == W4A4_F32 ? launch_r<BF16, F32>(a, s) : launch_r<BF16, BF16>(a, s);
}

}  // namespace w4a4
