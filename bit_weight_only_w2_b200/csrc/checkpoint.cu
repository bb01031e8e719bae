// 8-bit copies of activations: store (bf16 -> e4m3 codes and block exponents) and load. Both are
// streams through memory: a thread handles eight values on 16- and 8-byte accesses, kPer pieces at a
// CTA's stride, all asked for before the first is used (one piece a thread kept too few bytes in
// flight: 51 us for 4608 x 12288, floor 26).
#include <cuda_runtime.h>

#include <cstdint>

#include "adapter_internal.h"
#include "checkpoint.cuh"
#include "sm100_ptx.cuh"
#include "tcgen05_ptx.cuh"

namespace lowbit {
namespace {

constexpr int kThreads = 256;

constexpr int kPer = 4;

__global__ void __launch_bounds__(kThreads)
    checkpoint_store_kernel(const uint4* __restrict__ x, int64_t n8, uint2* __restrict__ codes, uint8_t* __restrict__ exps) {
    grid_dependency_wait();
    grid_launch_dependents();
    const int64_t i0 = static_cast<int64_t>(blockIdx.x) * (kThreads * kPer) + threadIdx.x;
    uint4 v[kPer];
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        const int64_t i = i0 + j * kThreads;
        v[j] = i < n8 ? ldg_nc_v4(x + i) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        const int64_t i = i0 + j * kThreads;
        uint8_t ex;
        // (n8 is a multiple of 4: a block's four lanes are all inside or all outside)
        const uint2 c = checkpoint_encode8(v[j], ex);
        if (i < n8) {
            codes[i] = c;
            if ((i & 3) == 0) exps[i >> 2] = ex;
        }
    }
}

__global__ void __launch_bounds__(kThreads)
    checkpoint_load_kernel(const uint2* __restrict__ codes, const uint8_t* __restrict__ exps, int64_t n8, uint4* __restrict__ x) {
    grid_dependency_wait();
    grid_launch_dependents();
    const int64_t i0 = static_cast<int64_t>(blockIdx.x) * (kThreads * kPer) + threadIdx.x;
    uint2 c[kPer];
    uint32_t e[kPer];
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        const int64_t i = i0 + j * kThreads;
        c[j] = i < n8 ? __ldg(codes + i) : make_uint2(0, 0);
        e[j] = i < n8 ? __ldg(exps + (i >> 2)) : 0;
    }
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        const int64_t i = i0 + j * kThreads;
        if (i < n8) x[i] = checkpoint_decode8(c[j], e[j]);
    }
}

template <class... Args>
lowbit_status launch(void (*kernel)(Args...), int64_t n8, cudaStream_t stream, Args... args) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3(static_cast<unsigned>((n8 + kThreads * kPer - 1) / (kThreads * kPer)), 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (take_injected_failure(kInjectLaunch)) return LOWBIT_ERR_CUDA;
    return cudaLaunchKernelEx(&cfg, kernel, args...) == cudaSuccess ? LOWBIT_OK : LOWBIT_ERR_CUDA;
}

}  // namespace

lowbit_status checkpoint_store_launch(const void* x, int64_t count, uint8_t* codes, uint8_t* exps, cudaStream_t s) {
    return launch(checkpoint_store_kernel, count / 8, s, static_cast<const uint4*>(x), count / 8,
                  reinterpret_cast<uint2*>(codes), exps);
}
lowbit_status checkpoint_load_launch(const uint8_t* codes, const uint8_t* exps, int64_t count, void* x, cudaStream_t s) {
    return launch(checkpoint_load_kernel, count / 8, s, reinterpret_cast<const uint2*>(codes), exps, count / 8,
                  static_cast<uint4*>(x));
}

}  // namespace lowbit
