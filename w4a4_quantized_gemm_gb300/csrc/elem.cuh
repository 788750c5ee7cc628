// Element types of the operators around the linears: fp16 and bf16 activations,
// fp32 residual streams, E4M3 cache rows.  Values are handled eight at a time
// (16 bytes of a 16-bit type), in fp32, and rounded once, to nearest even.
#pragma once
#include <cuda_bf16.h>

#include "common.cuh"

namespace w4a4 {

struct F16 {
    static constexpr int kSize = 2;
    static __device__ __forceinline__ float2 up(uint32_t w) {
        return __half22float2(*reinterpret_cast<const __half2*>(&w));
    }
    static __device__ __forceinline__ uint32_t down(float a, float b) {
        const __half2 h = __floats2half2_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
};
struct BF16 {
    static constexpr int kSize = 2;
    static __device__ __forceinline__ float2 up(uint32_t w) {  // a bf16 is the upper half of its fp32 value
        return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
    }
    static __device__ __forceinline__ uint32_t down(float a, float b) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
};
struct F32 {
    static constexpr int kSize = 4;
};

// Two fp32 -> two E4M3 bytes (a in the low one): nearest even, saturating, NaN kept.
__device__ __forceinline__ uint32_t e4m3x2(float a, float b) {
    return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}

// Four E4M3 bytes -> two fp16 pairs (bytes 0, 1 and 2, 3), exact.
__device__ __forceinline__ void e4m3x4_to_f16x2(uint32_t four, uint32_t& low, uint32_t& high) {
    asm("{\n.reg .b16 a, b;\nmov.b32 {a, b}, %2;\ncvt.rn.f16x2.e4m3x2 %0, a;\ncvt.rn.f16x2.e4m3x2 %1, b;\n}\n"
        : "=r"(low), "=r"(high)
        : "r"(four));
}

// Eight consecutive elements of a row, 16-byte aligned.
template <class T>
__device__ __forceinline__ void up8(const uint4& w, float (&x)[8]) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = T::up(u[i]);
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
    }
}
template <class T>
__device__ __forceinline__ uint4 down8(const float (&x)[8]) {
    return make_uint4(T::down(x[0], x[1]), T::down(x[2], x[3]), T::down(x[4], x[5]), T::down(x[6], x[7]));
}
template <class T>
__device__ __forceinline__ void load8(const void* row, int64_t i, float (&x)[8]) {
    const char* p = static_cast<const char*>(row) + i * T::kSize;
    if constexpr (T::kSize == 4) {
        const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
        x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
    } else {
        up8<T>(*reinterpret_cast<const uint4*>(p), x);
    }
}
template <class T>
__device__ __forceinline__ void store8(void* row, int64_t i, const float (&x)[8]) {
    char* p = static_cast<char*>(row) + i * T::kSize;
    if constexpr (T::kSize == 4) {
        reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
        reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
    } else {
        *reinterpret_cast<uint4*>(p) = down8<T>(x);
    }
}

// Reads and clears the status a kernel left in its device word (host).
template <class Symbol>
w4a4_status take_status_word(const Symbol& word) {
    int v = 0;
    if (cudaMemcpyFromSymbol(&v, word, sizeof(int)) != cudaSuccess) {
        cudaGetLastError();
        return W4A4_ERR_CUDA;
    }
    if (v != 0) {
        const int zero = 0;
        cudaMemcpyToSymbol(word, &zero, sizeof(int));
        return w4a4_status(v);
    }
    return W4A4_OK;
}

}  // namespace w4a4
