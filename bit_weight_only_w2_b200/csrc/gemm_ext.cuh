// Launch of the tensor-memory kernel's adapter and gradient variants (kExtAdapter, kExtGrad): tensor
// maps and launch. Included by one translation unit per code width and direction,
// so that the instantiations build in parallel.
#pragma once

#include <atomic>

#include "adapter_internal.h"
#include "gemm_kernel.cuh"

namespace lowbit {
namespace {

// Shared-memory opt-in of a kernel, once per device (one bit per device that has it).
template <int BITS, int GS, int BT, bool PAIR, int EXT>
bool ext_allow_smem() {
    using C = Cfg<BITS, GS, BT, PAIR, EXT>;
    static std::atomic<uint64_t> devices{0};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return false;
    const uint64_t bit = dev < 64 ? (uint64_t(1) << dev) : 0;
    if (bit && (devices.load(std::memory_order_acquire) & bit)) return true;
    if (cudaFuncSetAttribute(lowbit_gemm_kernel<BITS, GS, BT, PAIR, EXT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             C::kSmemBytes) != cudaSuccess)
        return false;
    devices.fetch_or(bit, std::memory_order_acq_rel);
    return true;
}

// Clusters of `ks` CTA pairs that the current device holds at once (asked once per device and ks).
template <int BITS, int GS, int EXT>
int pair_clusters(int ks) {
    using C = Cfg<BITS, GS, 256, true, EXT>;
    constexpr int kDevices = 16;
    static std::atomic<int> cached[kDevices][5];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || !ext_allow_smem<BITS, GS, 256, true, EXT>()) return 0;
    const bool keep = dev < kDevices;
    if (keep && cached[dev][ks].load(std::memory_order_relaxed) > 0) return cached[dev][ks].load(std::memory_order_relaxed);
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = ks;
    cfg.gridDim = dim3(2, 1, ks);
    cfg.blockDim = dim3(C::kThreads, 1, 1);
    cfg.dynamicSmemBytes = C::kSmemBytes;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, lowbit_gemm_kernel<BITS, GS, 256, true, EXT>, &cfg) != cudaSuccess) {
        cudaGetLastError();
        n = 0;
    }
    if (keep && n > 0) cached[dev][ks].store(n, std::memory_order_relaxed);
    return n;
}

template <int BITS, int GS, int BT, bool PAIR, int EXT>
lowbit_status ext_launch(const ExtProblem& e, const ExtBuffers& b, int rows, int ksplit, cudaStream_t stream) {
    using C = Cfg<BITS, GS, BT, PAIR, EXT>;
    auto kernel = lowbit_gemm_kernel<BITS, GS, BT, PAIR, EXT>;
    const void* fn = reinterpret_cast<const void*>(kernel);
    if (!ext_allow_smem<BITS, GS, BT, PAIR, EXT>()) return LOWBIT_ERR_CUDA;
    const ExtWorkspace& w = b.w;
    const uint64_t M = e.M, R = e.rows;
    const uint64_t red_words = EXT == kExtGrad ? uint64_t(e.red + 127) / 128 * 128 * BITS / 32 : uint64_t(e.red) * BITS / 32;
    const CUtensorMapSwizzle wswz = C::kWRowBytes == 16   ? CU_TENSOR_MAP_SWIZZLE_NONE
                                    : C::kWRowBytes == 32 ? CU_TENSOR_MAP_SWIZZLE_32B
                                                          : CU_TENSOR_MAP_SWIZZLE_64B;
    CUtensorMap mx, mw, ms, mz, my;
    ExtParams p = {};
    const uint32_t xbox[3] = {64, static_cast<uint32_t>(C::kXRows), 2};
    const uint64_t xdims[3] = {64, M, static_cast<uint64_t>(w.red64) / 64};
    const uint64_t xstr[2] = {static_cast<uint64_t>(w.red64) * 2, 128};
    bool ok = make_map_3d(&mx, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, b.at<void>(w.xh), xdims, xstr, xbox,
                          CU_TENSOR_MAP_SWIZZLE_128B);
    ok = ok && make_map_2d(&mw, CU_TENSOR_MAP_DATA_TYPE_UINT32, 4, e.words, red_words, R, red_words * 4,
                           C::kWordsPerRow, rows, wswz);
    ok = ok && make_map_2d(&ms, CU_TENSOR_MAP_DATA_TYPE_UINT16, 2, e.scales, e.N, e.K / GS, uint64_t(e.N) * 2,
                           kBlockN, C::kGroupsPerStage, CU_TENSOR_MAP_SWIZZLE_NONE);
    mz = ms;
    if (BITS == 4)
        ok = ok && make_map_2d(&mz, CU_TENSOR_MAP_DATA_TYPE_UINT16, 2, e.zeros, e.N, e.K / GS, uint64_t(e.N) * 2,
                               kBlockN, C::kGroupsPerStage, CU_TENSOR_MAP_SWIZZLE_NONE);
    ok = ok && make_map_2d(&my, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, e.out, R, M, R * 2, rows, BT,
                           CU_TENSOR_MAP_SWIZZLE_NONE);
    if (e.ad.num > 0) {
        const uint64_t pdims[3] = {64, M, static_cast<uint64_t>(w.p_cols) / 64};
        const uint64_t pstr[2] = {static_cast<uint64_t>(w.p_cols) * 2, 128};
        const uint32_t pbox[3] = {64, static_cast<uint32_t>(C::kXRows), C::kPHalves};
        ok = ok && make_map_3d(&p.map_p, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, b.at<void>(w.pslots), pdims, pstr, pbox,
                               CU_TENSOR_MAP_SWIZZLE_128B);
        p.adapters = true;
        p.tile_slots = e.ad.index ? b.at<int>(w.tile_slots) : nullptr;
        p.slot_side = b.at<int>(w.slot_side);
        p.slot_pitch = static_cast<int>(w.slot_pitch);
        p.rank_log2 = slot_log2(e.ad.rank);
        // the weight side, (R, N, L) or (K, R, L): ranks past R read as zero
        const uint64_t rk = e.ad.rank, in = EXT == kExtGrad ? R : rk, mid = EXT == kExtGrad ? rk : R;
        const uint64_t sdims[3] = {in, mid, static_cast<uint64_t>(e.ad.num)};
        const uint64_t sstr[2] = {in * 2, in * mid * 2};
        p.chunk_log2 = side_chunk_log2(EXT == kExtGrad, p.rank_log2, C::kSlotCols);
        const uint32_t chunk = 1u << p.chunk_log2;
        const uint32_t fbox[3] = {chunk, kBlockN, 1}, gbox[3] = {64, chunk, 1};
        const CUtensorMapSwizzle fswz = chunk == 16   ? CU_TENSOR_MAP_SWIZZLE_32B
                                        : chunk == 32 ? CU_TENSOR_MAP_SWIZZLE_64B
                                                      : CU_TENSOR_MAP_SWIZZLE_128B;
        ok = ok && (EXT == kExtGrad
                        ? make_map_3d(&p.map_side, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, e.ad.A, sdims, sstr, gbox,
                                      CU_TENSOR_MAP_SWIZZLE_128B)
                        : make_map_3d(&p.map_side, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, e.ad.B, sdims, sstr, fbox, fswz));
    }
    p.status = device_status_address();
    if (!ok || !p.status) return LOWBIT_ERR_CUDA;
    p.M = static_cast<int>(e.M);
    p.N = static_cast<int>(e.rows);
    p.K = static_cast<int>(e.red);
    p.num_kb = static_cast<int>((e.red + kBlockK - 1) / kBlockK);
    p.rows = rows;
    p.wtx_bytes = static_cast<uint32_t>(C::kWTxFixed + rows * C::kWRowBytes);
    p.m_tiles = static_cast<int>(w.m_tiles);
    p.n_tiles = static_cast<int>(PAIR ? e.rows / (2 * rows) : (e.rows + rows - 1) / rows);
    p.num_tiles = p.m_tiles * p.n_tiles;
    p.Y = static_cast<__nv_bfloat16*>(e.out);
    p.rowmul = b.at<float>(w.rowmul);
    if (ksplit > p.num_kb) ksplit = p.num_kb;
    const int kbps = (p.num_kb + ksplit - 1) / ksplit;
    ksplit = (p.num_kb + kbps - 1) / kbps;     // every rank gets at least one k-block
    // 256-token tiles over a multiple of 256 weight rows run on CTA pairs, split ones if the GPU holds
    // all of their clusters at once (a split grid is not persistent)
    if constexpr (BT == 256 && !PAIR) {
        const int pair_tiles = static_cast<int>(w.m_tiles * (e.rows / (2 * kBlockN)));
        if (e.rows % (2 * kBlockN) == 0 && (ksplit == 1 || (ksplit <= 4 && pair_tiles <= pair_clusters<BITS, GS, EXT>(ksplit))))
            return ext_launch<BITS, GS, BT, true, EXT>(e, b, rows, ksplit, stream);
    }
    p.kb_per_split = ksplit > 1 ? kbps : p.num_kb;
    p.ksplit = ksplit;

    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attrs[2];
    int na = 0;
    attrs[na].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attrs[na].val.programmaticStreamSerializationAllowed = 1;
    ++na;
    if (PAIR && ksplit > 1) {
        cfg.gridDim = dim3(2 * p.num_tiles, 1, ksplit);
    } else if (PAIR) {
        int pairs = cluster_capacity(fn, 2, C::kThreads, C::kSmemBytes, true);
        if (pairs > num_sms() / 2) pairs = num_sms() / 2;
        if (pairs < 1) pairs = 1;
        cfg.gridDim = dim3(2 * (p.num_tiles < pairs ? p.num_tiles : pairs), 1, 1);
    } else if (ksplit > 1) {
        cfg.gridDim = dim3(p.num_tiles, 1, ksplit);
    } else {
        const int slots = num_sms() * C::kCtasPerSm;
        cfg.gridDim = dim3(p.num_tiles < slots ? p.num_tiles : slots, 1, 1);
    }
    if (PAIR || ksplit > 1) {
        attrs[na].id = cudaLaunchAttributeClusterDimension;
        attrs[na].val.clusterDim.x = PAIR ? 2 : 1;
        attrs[na].val.clusterDim.y = 1;
        attrs[na].val.clusterDim.z = ksplit;
        ++na;
    }
    cfg.blockDim = dim3(C::kThreads, 1, 1);
    cfg.dynamicSmemBytes = C::kSmemBytes;
    cfg.stream = stream;
    cfg.attrs = attrs;
    cfg.numAttrs = na;
    if (take_injected_failure(kInjectLaunch)) return LOWBIT_ERR_CUDA;
    return cudaLaunchKernelEx(&cfg, kernel, mx, mw, ms, mz, my, p) == cudaSuccess ? LOWBIT_OK : LOWBIT_ERR_CUDA;
}

template <int BITS, int GS, int EXT>
lowbit_status ext_dispatch(const ExtProblem& e, const ExtBuffers& b, cudaStream_t stream) {
    const int rows = kBlockN, ksplit = b.w.product_split;
    switch (b.w.tile_tokens) {
        case 32: return ext_launch<BITS, GS, 32, false, EXT>(e, b, rows, ksplit, stream);
        case 64: return ext_launch<BITS, GS, 64, false, EXT>(e, b, rows, ksplit, stream);
        case 128: return ext_launch<BITS, GS, 128, false, EXT>(e, b, rows, ksplit, stream);
        case 256: return ext_launch<BITS, GS, 256, false, EXT>(e, b, rows, ksplit, stream);
        default: return LOWBIT_ERR_UNSUPPORTED;
    }
}

}  // namespace
}  // namespace lowbit

// Defines ext_gemm_b<BITS> (EXT = kExtAdapter) or ext_grad_b<BITS> (kExtGrad).
#define LOWBIT_EXT_ENTRY(NAME, BITS, EXT)                                                       \
    namespace lowbit {                                                                          \
    lowbit_status NAME(const ExtProblem& e, const ExtBuffers& b, cudaStream_t stream) {         \
        return e.group_size == 64 ? ext_dispatch<BITS, 64, EXT>(e, b, stream)                   \
                                  : ext_dispatch<BITS, 128, EXT>(e, b, stream);                 \
    }                                                                                           \
    }
