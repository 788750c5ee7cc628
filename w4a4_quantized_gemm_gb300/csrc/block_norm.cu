// The residual stream between two blocks of a decoder layer in one pass over a row:
//   r' = r + scale * gate (.) post(y),   x = pre(r')
// post and pre each nothing, an RMSNorm or a LayerNorm.  Four separate steps (norm,
// gate, add, norm) would move a row ten times; here y and r are read once and r' and
// x written once, which is the HBM bound.
//
// A CTA takes every grid-th row (narrow rows: several at a time), a thread the same
// columns of each: CH chunks of eight
// elements in registers (fp32) through both norms.  The gains, biases and a shared gate
// are read once for all rows (packed, in registers), and the next row is requested
// before this one is worked on.  The arithmetic is done on pairs (f32x2), and a missing
// gain or bias is a vector of ones or zeros rather than a choice per element: one row
// per CTA in scalar fp32 took 54 instructions an element, which were the bound.  At
// 8192 x 4096 (bf16 on an fp32 stream, two LayerNorms, gate rows) 65 us, 6.2 TB/s of the
// 403 MB that have to move; that first form 90 us.
//
// The statistics are the only exchanges: a warp's sums by shuffles, the warps' through
// shared memory behind one barrier.  A LayerNorm sums about a pivot that belongs to the
// row, the mean of the first eight elements that the warp holds:
//   mean = p + sum(z - p) / n,   sum (z - mean)^2 = sum (z - p)^2 - (sum(z - p))^2 / n,
// so that both sums go through the shuffles side by side instead of the squares after the
// mean (4096 rows of 4096, fp16, two LayerNorms: 31.1 -> 27.7 us).  The difference is safe:
// eight of the h <= 1024 elements (32 lanes of four chunks) have the mean p, so
// (p - mean)^2 is at most h / 8 times the variance and the difference loses at most seven
// of fp32's 24 bits, however large the mean.  The warps' moments are joined in the same
// way about the first warp's mean, where that ratio is at most 16, the warps.
#include <atomic>

#include "elem.cuh"
#include "kernels.h"
#include "launch.cuh"
#include "tc_ptx.cuh"

namespace w4a4 {
namespace {

template <int N>  // over each group of N lanes (a power of two)
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
    for (int o = N / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// This thread's place among the NC threads of its row (more than a warp: the whole CTA).
template <int NC>
__device__ __forceinline__ int column() {
    return NC > 32 ? threadIdx.x : threadIdx.x % NC;
}

// Pairs of fp32 in a 64-bit register.
__device__ __forceinline__ uint64_t pair(float a, float b) {
    return uint64_t(__float_as_uint(b)) << 32 | __float_as_uint(a);
}
__device__ __forceinline__ uint64_t both(float a) { return pair(a, a); }
__device__ __forceinline__ float lo(uint64_t p) { return __uint_as_float(uint32_t(p)); }
__device__ __forceinline__ float hi(uint64_t p) { return __uint_as_float(uint32_t(p >> 32)); }
template <class T>
__device__ __forceinline__ uint64_t up2(uint32_t w) {
    const float2 f = T::up(w);
    return pair(f.x, f.y);
}
template <class T>
__device__ __forceinline__ uint32_t down2(uint64_t p) { return T::down(lo(p), hi(p)); }
__device__ __forceinline__ uint32_t word(const uint4& v, int i) {
    return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
}

// 16 bytes that are read once: not kept in L1, where they would displace the vectors.
__device__ __forceinline__ uint4 ld_once(const void* p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];\n"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p)
                 : "memory");
    return v;
}
// Eight fp32: one 32-byte access where the row allows it (two 16-byte ones at a stride
// of 32 bytes would each touch half of every sector).
__device__ __forceinline__ void ld_once8(const float* p, bool wide, uint4 (&v)[2]) {
    if (wide)
        asm volatile("ld.global.L1::no_allocate.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n"
                     : "=r"(v[0].x), "=r"(v[0].y), "=r"(v[0].z), "=r"(v[0].w), "=r"(v[1].x), "=r"(v[1].y),
                       "=r"(v[1].z), "=r"(v[1].w)
                     : "l"(p)
                     : "memory");
    else
        v[0] = ld_once(p), v[1] = ld_once(p + 4);
}

// A thread's chunks of a vector [W] of a 16-bit type; `fill` (two elements) where there
// is none.  Held in registers for all rows, or read where they are used (512 threads of
// four chunks: too many to hold).
template <class T, int NC, int CH>
struct Vector {
    static constexpr bool kHeld = CH <= 2 || NC == 32;
    const char* at;
    uint32_t fill;
    uint4 v[kHeld ? CH : 1];
    __device__ __forceinline__ uint4 read(int c, int W) const {
        const int k = (c * NC + column<NC>()) * 8;
        return at && k < W ? *reinterpret_cast<const uint4*>(at + 2 * k) : make_uint4(fill, fill, fill, fill);
    }
    __device__ __forceinline__ void init(const void* p, float missing, int W) {
        at = static_cast<const char*>(p);
        fill = T::down(missing, missing);
        if constexpr (kHeld)
#pragma unroll
            for (int c = 0; c < CH; ++c) v[c] = read(c, W);
    }
    __device__ __forceinline__ uint4 get(int c, int W) {
        if constexpr (kHeld) {
            // opaque, or the compiler converts it once for all rows and holds twice the registers
            asm volatile("" : "+r"(v[c].x), "+r"(v[c].y), "+r"(v[c].z), "+r"(v[c].w));
            return v[c];
        }
        return read(c, W);
    }
};

// z -> norm(z) in place; chunk c of this thread is elements (c * NC + column) * 8 ..
// and takes part while that is below W (the others are zero).  NC threads, in one or
// several warps, have a row and get the same statistics (fixed order).  LAYER: one of the
// row's norms is a LayerNorm (an RMSNorm beside it takes the mean and the bias as zero);
// without it the mean, the bias and their work are left out (fp16, 4096 x 12288: 115 us with
// them, 88 without).
template <class T, int NC, int CH, bool LAYER>
__device__ __forceinline__ void normalise(uint64_t (&z)[CH][4], int kind, Vector<T, NC, CH>& gain,
                                          Vector<T, NC, CH>& bias, int W, float eps, float4* red) {
    if (kind == W4A4_NORM_NONE) return;
    constexpr int kWarps = NC > 32 ? NC / 32 : 1, kLanes = NC < 32 ? NC : 32;
    constexpr int kSlots = kWarps <= 4 ? 4 : kWarps <= 8 ? 8 : 16;  // lanes that join the warps' moments
    const int warp = kWarps > 1 ? threadIdx.x >> 5 : 0, lane = threadIdx.x & 31;
    const float n = 1.f / float(W);
    float mean = 0.f, v;
    auto takes_part = [&](int c) { return (c * NC + column<NC>()) * 8 < W; };
    if (LAYER && kind == W4A4_NORM_LAYER) {
        int h = 0;  // elements of this warp that take part
#pragma unroll
        for (int c = 0; c < CH; ++c) h += min(8 * kLanes, max(0, W - (c * NC + warp * 32) * 8));
        float held = float(h);
        const uint64_t e = tc::fadd2_b64(tc::fadd2_b64(z[0][0], z[0][1]), tc::fadd2_b64(z[0][2], z[0][3]));
        float pivot = __shfl_sync(0xffffffffu, (lo(e) + hi(e)) * 0.125f, 0, kLanes);
        uint64_t s = 0, q = 0;
        const uint64_t off = both(-pivot);
#pragma unroll
        for (int c = 0; c < CH; ++c)
            if (takes_part(c))
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint64_t d = tc::fadd2_b64(z[c][i], off);
                    s = tc::fadd2_b64(s, d);
                    q = tc::ffma2_b64(d, d, q);
                }
        float sum = group_sum<kLanes>(lo(s) + hi(s));
        v = group_sum<kLanes>(lo(q) + hi(q));
        if constexpr (kWarps > 1) {
            mean = sum / fmaxf(held, 1.f);
            if (lane == 0) red[warp] = make_float4(pivot + mean, held, v - sum * mean, 0.f);
            __syncthreads();
            // lane w of each kSlots takes warp w's moments: the same sums, in the same order, in all
            const int w = lane % kSlots;
            const float4 of = w < kWarps ? red[w] : make_float4(0.f, 0.f, 0.f, 0.f);
            pivot = red[0].x;
            const float d = of.x - pivot;
            sum = group_sum<kSlots>(of.y * d);
            v = group_sum<kSlots>(of.z + of.y * d * d);
        }
        mean = pivot + sum * n;
        v -= sum * sum * n;
        v = v < 0.f ? 0.f : v;  // a NaN stays
    } else {
        uint64_t q = 0;
#pragma unroll
        for (int c = 0; c < CH; ++c)
#pragma unroll
            for (int i = 0; i < 4; ++i) q = tc::ffma2_b64(z[c][i], z[c][i], q);
        v = group_sum<kLanes>(lo(q) + hi(q));
        if constexpr (kWarps > 1) {
            if (lane == 0) red[warp].z = v;
            __syncthreads();
            const int w = lane % kSlots;
            v = group_sum<kSlots>(w < kWarps ? red[w].z : 0.f);
        }
    }
    const float factor = rsqrtf(v * n + eps);  // 2 ulp
    const uint64_t inv = both(factor), less = both(-mean * factor);
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        const uint4 g = gain.get(c, W);
        if constexpr (LAYER) {
            const uint4 b = bias.get(c, W);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                z[c][i] = tc::ffma2_b64(tc::ffma2_b64(z[c][i], inv, less), up2<T>(word(g, i)), up2<T>(word(b, i)));
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) z[c][i] = tc::fmul2_b64(tc::fmul2_b64(z[c][i], inv), up2<T>(word(g, i)));
        }
    }
}

template <class T, class R, int NT, int NC, int CH, bool LAYER>  // NT threads, NC to a row
__global__ void __launch_bounds__(NT, CH == 2 && NT % 96 ? 512 / NT : 1) block_norm_kernel(const w4a4_block_norm_args a) {
    // a norm's partial sums; two sets that rows alternate between, so that a row's
    // barriers separate its reads from the next use of the set
    __shared__ float4 red[2][2][NT / 32];
    pdl_wait();
    pdl_launch_dependents();
    const int W = a.width;
    const bool wide = R::kSize == 4 && ((reinterpret_cast<uintptr_t>(a.r) | reinterpret_cast<uintptr_t>(a.r_out)) & 31) == 0 &&
                      ((a.r_stride | a.r_out_stride) & 7) == 0;
    const bool row_gate = a.gate && a.rows_per_gate;
    Vector<T, NC, CH> post_gain, post_bias, pre_gain, pre_bias, gate;
    uint4 ny[CH], nr[CH][R::kSize / 2], ng[CH];  // the next row, as it is in memory
#pragma unroll
    for (int c = 0; c < CH; ++c)  // chunks past the row stay zero
        ny[c] = ng[c] = nr[c][0] = nr[c][R::kSize / 2 - 1] = make_uint4(0, 0, 0, 0);
    constexpr uint32_t kRows = NT / NC;  // of a CTA at a time
    const uint32_t rows = a.rows, step = gridDim.x * kRows, mine = NT > NC ? threadIdx.x / NC : 0;
    auto request = [&](uint32_t m) {
        const char* y = static_cast<const char*>(a.y) + 2 * (m * a.y_stride);
        const char* r = static_cast<const char*>(a.r) + R::kSize * (m * a.r_stride);
        const char* gates = static_cast<const char*>(a.gate);
        if (row_gate) gates += 2 * (m / uint32_t(a.rows_per_gate) * a.gate_stride);
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int k = (c * NC + column<NC>()) * 8;
            if (k >= W || (kRows > 1 && m >= rows)) continue;
            ny[c] = ld_once(y + 2 * k);
            if constexpr (R::kSize == 4)
                ld_once8(reinterpret_cast<const float*>(r) + k, wide, nr[c]);
            else
                nr[c][0] = ld_once(r + 2 * k);
            if (row_gate) ng[c] = *reinterpret_cast<const uint4*>(gates + 2 * k);
        }
    };
    request(blockIdx.x * kRows + mine);
    post_gain.init(a.post_gain, 1.f, W);
    post_bias.init(a.post == W4A4_NORM_LAYER ? a.post_bias : nullptr, 0.f, W);
    pre_gain.init(a.pre_gain, 1.f, W);
    pre_bias.init(a.pre == W4A4_NORM_LAYER ? a.pre_bias : nullptr, 0.f, W);
    gate.init(row_gate ? nullptr : a.gate, 1.f, W);
    const uint64_t scale = both(a.scale);
    int set = 0;
    // a warp's last rows may be missing: its lanes stay for the shuffles
    for (uint32_t first = blockIdx.x * kRows; first < rows; first += step, set ^= 1) {
        const uint32_t m = first + mine;
        const bool row = kRows == 1 || m < rows;
        char* r_row = static_cast<char*>(a.r_out) + R::kSize * (m * a.r_out_stride);
        char* x_row = static_cast<char*>(a.x) + 2 * (m * a.x_stride);
        uint64_t y[CH][4], r[CH][4];
        uint4 g[CH];
#pragma unroll
        for (int c = 0; c < CH; ++c) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                y[c][i] = up2<T>(word(ny[c], i));
                if constexpr (R::kSize == 4)
                    r[c][i] = uint64_t(word(nr[c][i / 2], i % 2 * 2 + 1)) << 32 | word(nr[c][i / 2], i % 2 * 2);
                else
                    r[c][i] = up2<R>(word(nr[c][0], i));
            }
            g[c] = ng[c];
        }
        if (first + step < rows) request(m + step);
        normalise<T, NC, CH, LAYER>(y, a.post, post_gain, post_bias, W, a.eps, red[set][0]);
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int k = (c * NC + column<NC>()) * 8;
            if (a.gate) {
                if (!row_gate) g[c] = gate.get(c, W);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    r[c][i] = tc::ffma2_b64(tc::fmul2_b64(scale, up2<T>(word(g[c], i))), y[c][i], r[c][i]);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) r[c][i] = tc::ffma2_b64(scale, y[c][i], r[c][i]);
            }
            if (k < W && row) {
                char* dst = r_row + R::kSize * k;
                if constexpr (R::kSize == 4) {
                    if (wide) {
                        const uint32_t w[8] = {uint32_t(r[c][0]), uint32_t(r[c][0] >> 32), uint32_t(r[c][1]),
                                               uint32_t(r[c][1] >> 32), uint32_t(r[c][2]), uint32_t(r[c][2] >> 32),
                                               uint32_t(r[c][3]), uint32_t(r[c][3] >> 32)};
                        tc::st_global_v8(dst, w);
                    } else {
                        reinterpret_cast<ulonglong2*>(dst)[0] = make_ulonglong2(r[c][0], r[c][1]);
                        reinterpret_cast<ulonglong2*>(dst)[1] = make_ulonglong2(r[c][2], r[c][3]);
                    }
                } else {
                    *reinterpret_cast<uint4*>(dst) =
                        make_uint4(down2<R>(r[c][0]), down2<R>(r[c][1]), down2<R>(r[c][2]), down2<R>(r[c][3]));
                }
            } else if (k >= W) {  // the rest of a row takes part in no statistics
#pragma unroll
                for (int i = 0; i < 4; ++i) r[c][i] = 0;
            }
        }
        if (!a.x) continue;
        normalise<T, NC, CH, LAYER>(r, a.pre, pre_gain, pre_bias, W, a.eps, red[set][1]);
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int k = (c * NC + column<NC>()) * 8;
            if (k < W && row)
                *reinterpret_cast<uint4*>(x_row + 2 * k) =
                    make_uint4(down2<T>(r[c][0]), down2<T>(r[c][1]), down2<T>(r[c][2]), down2<T>(r[c][3]));
        }
    }
}

template <class T, class R, int NT, int NC, int CH, bool LAYER>
w4a4_status launch_k(const w4a4_block_norm_args& a, cudaStream_t s) {
    static std::atomic<int> per_sm{0};  // CTAs that an SM holds (registers), the same on every device
    int n = per_sm.load(std::memory_order_relaxed);
    if (n == 0) {
        if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, block_norm_kernel<T, R, NT, NC, CH, LAYER>, NT, 0) != cudaSuccess ||
            n < 1)
            n = 1;
        per_sm.store(n, std::memory_order_relaxed);
    }
    const int64_t full = n * int64_t(device_sm_count()), ctas = (int64_t(a.rows) * NC + NT - 1) / NT;
    const unsigned grid = unsigned(ctas < full ? ctas : full);
    set_dispatch_ints("block_norm rows=%d width=%d threads=%d chunks/thread=%d grid=%d",
                      {a.rows, a.width, NT, CH, int(grid)});
    return launch<block_norm_kernel<T, R, NT, NC, CH, LAYER>>(dim3(grid), NT, 0, s, a);
}

template <class T, class R, bool LAYER>
w4a4_status launch_l(const w4a4_block_norm_args& a, cudaStream_t s) {
    const int chunks = a.width / 8;
    // Narrow rows share a warp, and a CTA has four: 8192 rows of 64 (fp16) take 1.9 us, one
    // row to a CTA of one warp 4.9 us.  (8192 of 512 take 7.8 us, two warps to a row 7.7, but
    // with the rows in L2 5.1 and 5.9.)
    // Up to 1024 a warp has a row to itself where there are rows enough, without barriers:
    // 8192 of 1024, LayerNorms, 14.3 us, four warps to a row 17.1 us; but 700 take 3.2 and 2.8.
    // Above that two chunks a thread, and thread counts between the powers of two: with 128
    // threads only, 4096 rows of 1200 (fp16, LayerNorms) take 13.7 us, with 96 threads 11.9; of
    // 2560 25.4 us with 256 threads and 22.6 with 192, of 5120 53 us with 512 and 45.2 with 384.
    if (chunks <= 8)
        return launch_k<T, R, 128, 8, 1, LAYER>(a, s);
    else if (chunks <= 16)
        return launch_k<T, R, 128, 16, 1, LAYER>(a, s);
    else if (chunks <= 32)
        return launch_k<T, R, 128, 32, 1, LAYER>(a, s);
    else if (chunks <= 64)
        return launch_k<T, R, 128, 32, 2, LAYER>(a, s);
    else if (chunks <= 128 && a.rows > 8 * device_sm_count())
        return launch_k<T, R, 128, 32, 4, LAYER>(a, s);
    else if (chunks <= 128)
        return launch_k<T, R, 128, 128, 1, LAYER>(a, s);
    else if (chunks <= 192)
        return launch_k<T, R, 96, 96, 2, LAYER>(a, s);
    else if (chunks <= 256)
        return launch_k<T, R, 128, 128, 2, LAYER>(a, s);
    else if (chunks <= 384)
        return launch_k<T, R, 192, 192, 2, LAYER>(a, s);
    else if (chunks <= 512)
        return launch_k<T, R, 256, 256, 2, LAYER>(a, s);
    else if (chunks <= 768)
        return launch_k<T, R, 384, 384, 2, LAYER>(a, s);
    else if (chunks <= 1024)
        return launch_k<T, R, 512, 512, 2, LAYER>(a, s);
    else
        return launch_k<T, R, 512, 512, 4, LAYER>(a, s);
}

template <class T, class R>
w4a4_status launch_r(const w4a4_block_norm_args& a, cudaStream_t s) {
    return a.post == W4A4_NORM_LAYER || a.pre == W4A4_NORM_LAYER ? launch_l<T, R, true>(a, s) : launch_l<T, R, false>(a, s);
}

}  // namespace

w4a4_status launch_block_norm(const w4a4_block_norm_args& a, cudaStream_t s) {
    if (a.dtype == W4A4_F16) return a.res_dtype == W4A4_F32 ? launch_r<F16, F32>(a, s) : launch_r<F16, F16>(a, s);
    return a.res_dtype == W4A4_F32 ? launch_r<BF16, F32>(a, s) : launch_r<BF16, BF16>(a, s);
}

}  // namespace w4a4
