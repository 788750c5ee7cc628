// Appending the keys and values of new tokens to a paged cache, with the per-head
// RMSNorm of q and k and the position rotation on the way ("W4A4 CUDA Kernel for
// Voice Clone", 3.4: the step between the qkv linear and attention).
//
// A head x of D elements becomes x' = x / sqrt(mean x^2 + eps) * gain and then, for
// the pairs (a, b) of the first rot_dim elements, (x'_a c - x'_b n, x'_b c + x'_a n)
// with c, n the cosine and sine of the token's position times the pair's frequency.
// Every byte is read once and written once, so the bound is HBM traffic.
//
// One CTA takes one token (a slice of its heads when there are few
// tokens): the heads of a token share position, page and rotation, which are looked up
// once and stay in registers.  A head belongs to D / 16 lanes (eight with two idle ones
// at D = 96), each with the two 16-byte pieces that hold both elements of its pairs, so
// the rotation needs no exchange; the sum of squares is a shuffle reduction over the
// lanes.  A lane's pieces of up to two heads are loaded before anything else is done:
// HBM needs about 40 KB in flight per SM, and the first loads then cover the look-ups.
#include "elem.cuh"
#include "kernels.h"
#include "launch.cuh"

namespace w4a4 {
namespace {

__device__ int g_append_status = 0;

// Two forms.  Many tokens: one warp a CTA in at most 78 registers, so that an SM holds 26
// (8192 tokens of 48 heads of 128, fp16: 34.0 us, 6.1 TB/s; two warps without the limit
// 40 us).  Few, which all fit at once: the gains of q and k are requested with the first
// heads and kept, 700 tokens of 32 heads 4.7 us instead of 4.9, one token 2.4 us either way.
constexpr int kFew = 5;  // tokens per SM up to which they are few
constexpr int threads_of(bool many) { return many ? 32 : 64; }
constexpr int per_sm(bool many) { return many ? 26 : 10; }  // CTAs that an SM holds
constexpr int kAhead = 2;  // heads whose pieces a lane holds at once

// Quotients by a head's scale: x / s = x hi + x lo with 1 / s = hi + lo to 2^-46, hi rounded
// towards zero and lo of its sign.  The sum is rounded once, so a quotient that lies halfway
// between two E4M3 values is found exactly, which hi alone misses; infinities, NaN and s = 0
// come out as the division's.  8192 tokens of 32 + 2 x 8 heads of 128 take 33.1 us, 35.8 with a
// division itself, 32.7 with hi alone; 4096 of 16 + 2 x 16 of 64 take 10.4, 12.1 and 9.5
// (inputs in L2).  A scale far from one is brought nearer by a power of two, and x with it, so
// that 1 / s is a normal number.
struct Quotients {
    float by, hi, lo;
    __device__ __forceinline__ explicit Quotients(float s) {
        by = fabsf(s) < 0x1p-100f ? 0x1p64f : fabsf(s) > 0x1p100f ? 0x1p-64f : 1.f;
        s *= by;
        hi = __frcp_rz(s);
        lo = hi * fmaxf(fmaf(-hi, s, 1.f), 0x1p-60f);  // not zero: x may be infinite
    }
    __device__ __forceinline__ void of(float (&x)[8]) const {
        if (by != 1.f)
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] *= by;
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = fmaf(x[j], hi, x[j] * lo);
    }
};

// One 8-element piece to the cache, in its type.
template <class T, bool E4M3>
__device__ __forceinline__ void store_piece(void* pool, int64_t at, const float (&x)[8]) {
    if constexpr (E4M3) {
        uint2 o;
        o.x = e4m3x2(x[0], x[1]) | e4m3x2(x[2], x[3]) << 16;
        o.y = e4m3x2(x[4], x[5]) | e4m3x2(x[6], x[7]) << 16;
        *reinterpret_cast<uint2*>(static_cast<char*>(pool) + at) = o;
    } else {
        store8<T>(pool, at, x);
    }
}

template <class T, bool E4M3, int LPH, bool MANY>  // LPH: lanes of a head's group (4, 8 or 16)
__global__ void __launch_bounds__(threads_of(MANY), per_sm(MANY)) kv_append_kernel(const w4a4_kv_cache c, const w4a4_kv_append_args a) {
    pdl_wait();
    pdl_launch_dependents();
    const int t = blockIdx.x, lane = threadIdx.x % LPH, group = threadIdx.x / LPH;
    constexpr int kGroups = threads_of(MANY) / LPH;
    const int D = c.head_dim, R = a.rope ? a.rot_dim : 0;
    const bool has = lane < D / 16, inter = a.interleaved != 0;
    // This lane's elements e[0] .. + 7 and e[1] .. + 7: a pair's halves while they are
    // rotated ones, else two neighbouring pieces of the rest.
    const bool turns = lane < R / 16;
    const int e0 = turns ? 8 * lane : 16 * lane, e1 = turns ? e0 + R / 2 : e0 + 8;

    const int rows = a.q_heads + 2 * c.kv_heads;  // queries, keys, values
    const int step = gridDim.y * kGroups;
    const int first = blockIdx.y * kGroups + group;
    uint4 raw[kAhead][2];
    auto load = [&](int base) {
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int row = first + base + u * step;
            raw[u][0] = raw[u][1] = make_uint4(0, 0, 0, 0);
            if (!has || row >= rows) continue;
            const bool is_q = row < a.q_heads, is_v = row >= a.q_heads + c.kv_heads;
            const char* src = static_cast<const char*>(is_q ? a.q : is_v ? a.v : a.k);
            src += 2 * (is_q ? t * a.q_token_stride + row * a.q_head_stride
                        : is_v ? t * a.v_token_stride + (row - a.q_heads - c.kv_heads) * a.v_head_stride
                               : t * a.k_token_stride + (row - a.q_heads) * a.k_head_stride);
            raw[u][0] = *reinterpret_cast<const uint4*>(src + 2 * e0);
            raw[u][1] = *reinterpret_cast<const uint4*>(src + 2 * e1);
        }
    };
    load(0);

    // This lane's gains, of q and of k.
    const bool norms = a.q_gain || a.k_gain;
    const float per_head = 1.f / float(D);
    uint4 gains[4] = {};
    if (!MANY && norms && has) {
        const char *qg = static_cast<const char*>(a.q_gain), *kg = static_cast<const char*>(a.k_gain);
        if (qg) gains[0] = *reinterpret_cast<const uint4*>(qg + 2 * e0), gains[1] = *reinterpret_cast<const uint4*>(qg + 2 * e1);
        if (kg) gains[2] = *reinterpret_cast<const uint4*>(kg + 2 * e0), gains[3] = *reinterpret_cast<const uint4*>(kg + 2 * e1);
    }

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
    // This lane's rotation: the cosines of eight consecutive pairs (half-split), or of
    // the four pairs of each of its pieces (interleaved).
    float cs[8], sn[8];
    if (turns && live) {
        const float* row = a.rope + int64_t(pos) * R;
        const int i0 = inter ? e0 / 2 : e0, i1 = inter ? e1 / 2 : e0 + 4;
        const float4 c0 = *reinterpret_cast<const float4*>(row + i0), c1 = *reinterpret_cast<const float4*>(row + i1);
        const float4 s0 = *reinterpret_cast<const float4*>(row + R / 2 + i0),
                     s1 = *reinterpret_cast<const float4*>(row + R / 2 + i1);
        cs[0] = c0.x, cs[1] = c0.y, cs[2] = c0.z, cs[3] = c0.w, cs[4] = c1.x, cs[5] = c1.y, cs[6] = c1.z, cs[7] = c1.w;
        sn[0] = s0.x, sn[1] = s0.y, sn[2] = s0.z, sn[3] = s0.w, sn[4] = s1.x, sn[5] = s1.y, sn[6] = s1.z, sn[7] = s1.w;
    }

    // The loop bound is the warp's first group's, so that every lane takes part in each shuffle.
    const int warp_first = blockIdx.y * kGroups + (threadIdx.x & ~31) / LPH;
    for (int base = 0; warp_first + base < rows; base += kAhead * step) {
        if (base) load(base);
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int row = first + base + u * step;
            if (warp_first + base + u * step >= rows) break;
            const bool is_q = row < a.q_heads, is_v = row >= a.q_heads + c.kv_heads;
            float x[8], y[8];
            up8<T>(raw[u][0], x);
            up8<T>(raw[u][1], y);
            if (norms) {
                float ss = 0.f;
#pragma unroll
                for (int j = 0; j < 8; ++j) ss += x[j] * x[j] + y[j] * y[j];
#pragma unroll
                for (int o = LPH / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
                if (is_q ? a.q_gain != nullptr : !is_v && a.k_gain) {
                    const float inv = rsqrtf(ss * per_head + a.eps);  // 2 ulp
                    float g[8], h[8];
                    if constexpr (MANY) {
                        const void* gain = is_q ? a.q_gain : a.k_gain;
                        load8<T>(gain, e0 < D ? e0 : 0, g);
                        load8<T>(gain, e1 < D ? e1 : 0, h);
                    } else {
                        up8<T>(is_q ? gains[0] : gains[2], g);
                        up8<T>(is_q ? gains[1] : gains[3], h);
                    }
#pragma unroll
                    for (int j = 0; j < 8; ++j) x[j] = x[j] * inv * g[j], y[j] = y[j] * inv * h[j];
                }
            }
            if (!has || row >= rows) continue;
            if (turns && live && !is_v) {
                if (inter) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float p = x[2 * j], q = x[2 * j + 1], r = y[2 * j], s = y[2 * j + 1];
                        x[2 * j] = p * cs[j] - q * sn[j];
                        x[2 * j + 1] = q * cs[j] + p * sn[j];
                        y[2 * j] = r * cs[4 + j] - s * sn[4 + j];
                        y[2 * j + 1] = s * cs[4 + j] + r * sn[4 + j];
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const float p = x[j], q = y[j];
                        x[j] = p * cs[j] - q * sn[j];
                        y[j] = q * cs[j] + p * sn[j];
                    }
                }
            }
            if (is_q) {
                if (!live)
#pragma unroll
                    for (int j = 0; j < 8; ++j) x[j] = y[j] = 0.f;
                const int64_t to = t * a.out_token_stride + row * a.out_head_stride;
                store8<T>(a.q_out, to + e0, x);
                store8<T>(a.q_out, to + e1, y);
            } else if (live) {
                const int h = row - a.q_heads - (is_v ? c.kv_heads : 0);
                void* pool = is_v ? c.v : c.k;
                const int64_t to = is_v ? page * c.v_page_stride + slot * c.v_token_stride + h * c.v_head_stride
                                        : page * c.k_page_stride + slot * c.k_token_stride + h * c.k_head_stride;
                const float* scales = is_v ? c.v_scale : c.k_scale;
                if (E4M3 && scales) {
                    const Quotients per(scales[h]);
                    per.of(x);
                    per.of(y);
                }
                store_piece<T, E4M3>(pool, to + e0, x);
                store_piece<T, E4M3>(pool, to + e1, y);
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

template <class T, bool E4M3, bool MANY>
w4a4_status launch_m(const w4a4_kv_cache& c, const w4a4_kv_append_args& a, cudaStream_t s) {
    const int lph = c.head_dim <= 64 ? 4 : c.head_dim <= 128 ? 8 : 16;
    const int groups = threads_of(MANY) / lph, rows = a.q_heads + 2 * c.kv_heads;
    // A token's heads are spread over as many CTAs as the GPU holds at once.
    const int most = (rows + groups - 1) / groups, full = per_sm(MANY) * device_sm_count();
    int want = full / a.tokens > 1 ? full / a.tokens : 1;
    // Many tokens that fill the GPU once or twice but for a quarter or more of the last time:
    // two CTAs a token, where it has heads enough to repay the second look-up.  Of 48 heads of
    // 128 (fp16), 2500 tokens take 16.4 us, 17.4 with one; 6000 tokens 29.4 and 31.6; but 4200
    // (full and a little) 21.4 and 20.3, and 2500 tokens of 24 heads of 64 7.7 and 7.0.
    const int over = a.tokens % full;
    if (MANY && want == 1 && a.tokens < 2 * full && over > full / 8 && over <= full * 3 / 4 && most > 3 * kAhead) want = 2;
    const dim3 grid(unsigned(a.tokens), unsigned(most < want ? most : want));
    set_dispatch_ints(E4M3 ? "kv_append tokens=%d heads=%d+2x%d dim=%d e4m3 cache threads=%d grid=%dx%d"
                           : "kv_append tokens=%d heads=%d+2x%d dim=%d 16-bit cache threads=%d grid=%dx%d",
                      {a.tokens, a.q_heads, c.kv_heads, c.head_dim, threads_of(MANY), a.tokens, int(grid.y)});
    if (lph == 4) return launch<kv_append_kernel<T, E4M3, 4, MANY>>(grid, threads_of(MANY), 0, s, c, a);
    if (lph == 8) return launch<kv_append_kernel<T, E4M3, 8, MANY>>(grid, threads_of(MANY), 0, s, c, a);
    return launch<kv_append_kernel<T, E4M3, 16, MANY>>(grid, threads_of(MANY), 0, s, c, a);
}

template <class T, bool E4M3>
w4a4_status launch_t(const w4a4_kv_cache& c, const w4a4_kv_append_args& a, cudaStream_t s) {
    return a.tokens > kFew * device_sm_count() ? launch_m<T, E4M3, true>(c, a, s) : launch_m<T, E4M3, false>(c, a, s);
}

}  // namespace

w4a4_status append_read_and_clear_status() { return take_status_word(g_append_status); }

w4a4_status launch_kv_append(const w4a4_kv_cache& c, const w4a4_kv_append_args& a, cudaStream_t s) {
    const bool e4m3 = c.dtype == W4A4_E4M3;
    if (a.dtype == W4A4_F16) return e4m3 ? launch_t<F16, true>(c, a, s) : launch_t<F16, false>(c, a, s);
    return e4m3 ? launch_t<BF16, true>(c, a, s) : launch_t<BF16, false>(c, a, s);
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
    set_dispatch_ints("rope_table rows=%d rot_dim=%d", {rows, rot_dim});
}

}  // namespace w4a4
