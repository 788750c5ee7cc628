// Launch of a kernel through the driver's entry point.  The runtime's launch looks the
// kernel up and checks its own state first: 2.0 us of host time against 1.7 on the Grace
// host, where a decode step's short kernels take 1.4 to 2.5 us on the GPU.
#pragma once
#include <cuda.h>

#include <atomic>

#include "common.cuh"

namespace w4a4 {

using LaunchFn = CUresult (*)(const CUlaunchConfig*, CUfunction, void**, void**);

inline LaunchFn driver_launch() {
    static const LaunchFn fn = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult found{};
        if (cudaGetDriverEntryPointByVersion("cuLaunchKernelEx", &p, 12000, cudaEnableDefault, &found) != cudaSuccess ||
            found != cudaDriverEntryPointSuccess) {
            cudaGetLastError();
            p = nullptr;
        }
        return reinterpret_cast<LaunchFn>(p);
    }();
    return fn;
}

// cuTensorMapEncodeTiled, or nullptr.
using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                              const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
inline EncodeFn driver_encode() {
    static const EncodeFn fn = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult found{};
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &found) != cudaSuccess ||
            found != cudaDriverEntryPointSuccess) {
            cudaGetLastError();
            p = nullptr;
        }
        return reinterpret_cast<EncodeFn>(p);
    }();
    return fn;
}

// Kernel<<<grid, threads, smem, stream>>>(args...) with programmatic dependent launch
// (add_pdl_attr).  The kernel's handle is kept per device.
template <auto Kernel, class... A>
w4a4_status launch(dim3 grid, unsigned threads, unsigned smem, cudaStream_t stream, const A&... args) {
    static std::atomic<CUfunction> handles[64];
    int dev = 0;
    cudaGetDevice(&dev);
    const LaunchFn go = driver_launch();
    if (!go || dev < 0 || dev >= 64) return W4A4_ERR_CUDA;
    CUfunction fn = handles[dev].load(std::memory_order_acquire);
    if (!fn) {
        cudaFunction_t f = nullptr;
        if (cudaGetFuncBySymbol(&f, reinterpret_cast<const void*>(Kernel)) != cudaSuccess) return launch_status();
        fn = reinterpret_cast<CUfunction>(f);
        handles[dev].store(fn, std::memory_order_release);
    }
    cudaLaunchAttribute pdl[1];
    CUlaunchAttribute attr{};
    attr.id = CU_LAUNCH_ATTRIBUTE_PROGRAMMATIC_STREAM_SERIALIZATION;
    attr.value.programmaticStreamSerializationAllowed = 1;
    CUlaunchConfig cfg{};
    cfg.gridDimX = grid.x, cfg.gridDimY = grid.y, cfg.gridDimZ = grid.z;
    cfg.blockDimX = threads, cfg.blockDimY = 1, cfg.blockDimZ = 1;
    cfg.sharedMemBytes = smem;
    cfg.hStream = stream;
    cfg.attrs = &attr;
    cfg.numAttrs = add_pdl_attr(pdl, 0);
    void* params[] = {const_cast<void*>(static_cast<const void*>(&args))...};
    CUresult done = go(&cfg, fn, params, nullptr);
    if (done == CUDA_ERROR_INVALID_CONTEXT) {
        // The driver's entry point needs a context on the calling thread, and none of the cached
        // look-ups above has bound one: a thread whose first CUDA call this is.
        if (cudaSetDevice(dev) != cudaSuccess) return launch_status();
        done = go(&cfg, fn, params, nullptr);
    }
    return done == CUDA_SUCCESS ? W4A4_OK : W4A4_ERR_CUDA;
}

}  // namespace w4a4
