// The tensor-memory GEMM's X conversion pass, its host side (tile choice, tensor maps, launch) and
// the device status word. The kernel itself, with the reasons for its design, is in
// gemm_kernel.cuh.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <atomic>
#include <mutex>

#include <cstdint>
#include <cstdio>

#include "adapter_internal.h"
#include "capacity_cache.h"
#include "lowbit_internal.h"
#include "sm100_ptx.cuh"
#include "tcgen05_ptx.cuh"
#include "gemm_kernel.cuh"

namespace lowbit {

__device__ unsigned g_device_status = 0;
__device__ __forceinline__ unsigned* status_word() { return &g_device_status; }

// ---------------------------------------------------------------------------------------------
// X conversion pass: bf16 [M][K] -> fp16 [M][K] with a power-of-two factor per row.
// ---------------------------------------------------------------------------------------------
// One CTA per row: finds the largest |x| of the row (from the bf16 bits), picks e so that the
// row's largest value scaled by 2^-e lies in [2^15, 2^16) -- inside fp16's range, with every value
// within 2^29 of it still an fp16 normal -- writes the row times 2^-e as fp16 (exact) and
// rowmul[row] = 2^e, which the GEMM epilogue multiplies back (exact). Rows that are all zero,
// or hold an infinity or NaN, keep e = 0 (non-finite values convert as they are).
__device__ __forceinline__ uint32_t absmax_bf16x8(const uint4& v, uint32_t m) {
    m = max(m, max(v.x & 0x7FFFu, (v.x >> 16) & 0x7FFFu));
    m = max(m, max(v.y & 0x7FFFu, (v.y >> 16) & 0x7FFFu));
    m = max(m, max(v.z & 0x7FFFu, (v.z >> 16) & 0x7FFFu));
    m = max(m, max(v.w & 0x7FFFu, (v.w >> 16) & 0x7FFFu));
    return m;
}
__device__ __forceinline__ uint32_t bf16x2_to_f16x2(uint32_t w, float scale) {
    return pack_f16x2(__uint_as_float(w << 16) * scale, __uint_as_float(w & 0xFFFF0000u) * scale);
}

constexpr int kConvThreads = 256;

// One CTA per row of X. PER > 0: the row is held in registers (PER 16-byte chunks per thread,
// K <= 2048 * PER), so X is read from memory once; PER == 0: any K, the row is read twice.
template <int PER>
__global__ void __launch_bounds__(kConvThreads) convert_x_kernel(const uint4* __restrict__ X, int K8,
                                                                 uint4* __restrict__ Xh, float* __restrict__ rowmul) {
    grid_dependency_wait();
    grid_launch_dependents();
    const int row = blockIdx.x;
    const uint4* src = X + static_cast<size_t>(row) * K8;
    uint4* dst = Xh + static_cast<size_t>(row) * K8;
    uint32_t mx = 0;
    uint4 v[PER > 0 ? PER : 1];
    if (PER > 0) {
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            const int i = threadIdx.x + j * kConvThreads;
            v[j] = i < K8 ? ldg_nc_v4(src + i) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int j = 0; j < PER; ++j) mx = absmax_bf16x8(v[j], mx);
    } else {
        for (int i = threadIdx.x; i < K8; i += kConvThreads) mx = absmax_bf16x8(src[i], mx);
    }
    mx = __reduce_max_sync(0xffffffffu, mx);
    __shared__ uint32_t warp_max[kConvThreads / 32];
    if ((threadIdx.x & 31) == 0) warp_max[threadIdx.x >> 5] = mx;
    __syncthreads();
    mx = 0;
#pragma unroll
    for (int w = 0; w < kConvThreads / 32; ++w) mx = max(mx, warp_max[w]);
    const int E = static_cast<int>(mx >> 7);            // biased exponent of the largest |x|
    int e = (mx == 0 || E >= 255) ? 0 : E - 142;          // largest |x| * 2^-e in [2^15, 2^16)
    e = max(-100, min(112, e));
    const float scale = __int_as_float((127 - e) << 23);  // 2^-e
    auto cvt = [&](const uint4& a) {
        uint4 o;
        o.x = bf16x2_to_f16x2(a.x, scale);
        o.y = bf16x2_to_f16x2(a.y, scale);
        o.z = bf16x2_to_f16x2(a.z, scale);
        o.w = bf16x2_to_f16x2(a.w, scale);
        return o;
    };
    if (PER > 0) {
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            const int i = threadIdx.x + j * kConvThreads;
            if (i < K8) dst[i] = cvt(v[j]);
        }
    } else {
        for (int i = threadIdx.x; i < K8; i += kConvThreads) dst[i] = cvt(src[i]);
    }
    if (threadIdx.x == 0) rowmul[row] = __int_as_float((127 + e) << 23);   // 2^e
}

lowbit_status launch_convert_x(const GemmProblem& g, cudaStream_t stream) {
    const WorkspaceLayout ws = workspace_layout(g.M, g.K);
    cudaLaunchConfig_t ccfg = {};
    cudaLaunchAttribute cattr[1];
    cattr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    cattr[0].val.programmaticStreamSerializationAllowed = 1;
    ccfg.gridDim = dim3(static_cast<unsigned>(g.M), 1, 1);
    ccfg.blockDim = dim3(kConvThreads, 1, 1);
    ccfg.stream = stream;
    ccfg.attrs = cattr;
    ccfg.numAttrs = 1;
    const int K8 = static_cast<int>(g.K / 8);
    if (take_injected_failure(kInjectLaunch)) return LOWBIT_ERR_CUDA;
    const uint4* x = static_cast<const uint4*>(g.X);
    uint4* xh = static_cast<uint4*>(g.workspace);
    float* rm = reinterpret_cast<float*>(static_cast<uint8_t*>(g.workspace) + ws.rowmul_offset);
    cudaError_t e;
    if (K8 <= kConvThreads) e = cudaLaunchKernelEx(&ccfg, convert_x_kernel<1>, x, K8, xh, rm);
    else if (K8 <= 2 * kConvThreads) e = cudaLaunchKernelEx(&ccfg, convert_x_kernel<2>, x, K8, xh, rm);
    else if (K8 <= 4 * kConvThreads) e = cudaLaunchKernelEx(&ccfg, convert_x_kernel<4>, x, K8, xh, rm);
    else if (K8 <= 8 * kConvThreads) e = cudaLaunchKernelEx(&ccfg, convert_x_kernel<8>, x, K8, xh, rm);
    else e = cudaLaunchKernelEx(&ccfg, convert_x_kernel<0>, x, K8, xh, rm);
    return e == cudaSuccess ? LOWBIT_OK : LOWBIT_ERR_CUDA;
}

// One CTA waits on a barrier that nothing arrives on, with the GEMM's bounded wait: the wait
// gives up after `limit` clocks and records the timeout in the device status word.
__global__ void bounded_wait_selftest_kernel(long long limit) {
    __shared__ uint64_t bar;
    __shared__ int abort_flag;
    if (threadIdx.x == 0) {
        mbar_init(&bar, 1);
        abort_flag = 0;
        fence_mbar_init();
    }
    __syncthreads();
    if (threadIdx.x == 0) mbar_wait(&bar, 0, &abort_flag, &g_device_status, limit);
}

lowbit_status selftest_bounded_wait(long long limit_cycles, cudaStream_t stream) {
    bounded_wait_selftest_kernel<<<1, 32, 0, stream>>>(limit_cycles);
    return cudaGetLastError() == cudaSuccess ? LOWBIT_OK : LOWBIT_ERR_CUDA;
}

// One thread asks to store one element past a one-element array. The store happens only when
// the index is in range, so nothing is ever written out of bounds; in debug builds the index
// check in front of it records the failure in the status word, as the GEMM kernels' checks do.
__device__ unsigned g_selftest_cell[1];
__global__ void index_check_selftest_kernel(int index) {
    const bool ok = index >= 0 && index < 1;
    if (dcheck(ok, &g_device_status) && ok) g_selftest_cell[index] = 1u;
}

lowbit_status selftest_index_check(cudaStream_t stream) {
    if (!kDebugChecks) return LOWBIT_ERR_UNSUPPORTED;
    index_check_selftest_kernel<<<1, 1, 0, stream>>>(1);
    return cudaGetLastError() == cudaSuccess ? LOWBIT_OK : LOWBIT_ERR_CUDA;
}

// ---------------------------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------------------------
namespace {

PFN_cuTensorMapEncodeTiled_v12000 get_encode_fn();

// Tensor maps are a pure function of their arguments (address, geometry, box, swizzle), so
// encoded maps are kept in a small direct-mapped cache: a linear called again with the same
// buffers skips the driver's encode.
struct MapKey {
    uint64_t base;
    uint64_t dims[3];
    uint64_t strides[2];
    uint32_t box[3];
    int dtype, rank, swz;
    bool operator==(const MapKey& o) const {
        return base == o.base && dims[0] == o.dims[0] && dims[1] == o.dims[1] && dims[2] == o.dims[2] &&
               strides[0] == o.strides[0] && strides[1] == o.strides[1] && box[0] == o.box[0] &&
               box[1] == o.box[1] && box[2] == o.box[2] && dtype == o.dtype && rank == o.rank && swz == o.swz;
    }
};

bool encode_cached(CUtensorMap* map, CUtensorMapDataType dtype, int rank, const void* base, const uint64_t* dims,
                   const uint64_t* strides, const uint32_t* box, CUtensorMapSwizzle swz) {
    if (take_injected_failure(kInjectEncode)) return false;
    constexpr int kSlots = 1024;
    struct Slot {
        bool used;
        MapKey key;
        CUtensorMap map;
    };
    static Slot* slots = new Slot[kSlots]();
    static std::mutex mu;
    MapKey k = {};
    k.base = reinterpret_cast<uint64_t>(base);
    for (int i = 0; i < rank; ++i) {
        k.dims[i] = dims[i];
        k.box[i] = box[i];
    }
    for (int i = 0; i + 1 < rank; ++i) k.strides[i] = strides[i];
    k.dtype = static_cast<int>(dtype);
    k.rank = rank;
    k.swz = static_cast<int>(swz);
    uint64_t h = k.base * 0x9E3779B97F4A7C15ull;
    for (int i = 0; i < 3; ++i) h ^= (k.dims[i] + 0x632BE59BD9B4E019ull * (k.box[i] + 1)) * (2 * i + 3);
    h ^= (k.strides[0] * 31 + k.strides[1]) ^ (static_cast<uint64_t>(k.dtype) << 40) ^
         (static_cast<uint64_t>(k.swz) << 48) ^ (static_cast<uint64_t>(rank) << 56);
    h ^= h >> 29;
    Slot& sl = slots[h % kSlots];
    {
        std::lock_guard<std::mutex> lock(mu);
        if (sl.used && sl.key == k) {
            *map = sl.map;
            return true;
        }
    }
    auto fn = get_encode_fn();
    if (!fn) return false;
    cuuint64_t d[3], st[2];
    cuuint32_t b[3], estr[3] = {1, 1, 1};
    for (int i = 0; i < rank; ++i) {
        d[i] = dims[i];
        b[i] = box[i];
    }
    for (int i = 0; i + 1 < rank; ++i) st[i] = strides[i];
    auto encode = [&] {
        return fn(map, dtype, rank, const_cast<void*>(base), d, st, b, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, swz,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    };
    CUresult r = encode();
    int dev = 0;
    // A host thread that has done no CUDA work yet has no context, and this driver call binds none (the
    // runtime's launches do): selecting its device does, also under a stream capture.
    if (r == CUDA_ERROR_INVALID_CONTEXT && cudaGetDevice(&dev) == cudaSuccess && cudaSetDevice(dev) == cudaSuccess)
        r = encode();
    if (r != CUDA_SUCCESS) return false;
    std::lock_guard<std::mutex> lock(mu);
    sl.used = true;
    sl.key = k;
    sl.map = *map;
    return true;
}

// The driver's tensor-map encoder, looked up once (a function-local static: initialised exactly
// once even when several host threads make their first call at the same time).
PFN_cuTensorMapEncodeTiled_v12000 get_encode_fn() {
    static const PFN_cuTensorMapEncodeTiled_v12000 fn = []() -> PFN_cuTensorMapEncodeTiled_v12000 {
        cudaDriverEntryPointQueryResult q;
        void* f = nullptr;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &f, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
        cudaGetLastError();
        return nullptr;
    }();
    return fn;
}

// X as a 3-D tensor (64 k, M rows, K/64 k-atoms) so that one box covers a whole 128-wide k-block
// of BT token rows in the 128-byte-swizzled layout [k half][row][64 k] the MMA reads.
bool make_map_x3d(CUtensorMap* map, const void* base, uint64_t M, uint64_t K, uint32_t box_rows) {
    const uint64_t dims[3] = {64, M, K / 64};
    const uint64_t strides[2] = {K * 2, 128};
    const uint32_t box[3] = {64, box_rows, 2};
    return encode_cached(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, base, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

}  // namespace

bool make_map_3d(CUtensorMap* map, CUtensorMapDataType dtype, const void* base, const uint64_t (&dims)[3],
                 const uint64_t (&strides)[2], const uint32_t (&box)[3], CUtensorMapSwizzle swz) {
    return encode_cached(map, dtype, 3, base, dims, strides, box, swz);
}

bool make_map_2d(CUtensorMap* map, CUtensorMapDataType dtype, int elem_bytes, const void* base, uint64_t inner,
                 uint64_t outer, uint64_t row_bytes, uint32_t box_inner, uint32_t box_outer,
                 CUtensorMapSwizzle swz) {
    (void)elem_bytes;
    const uint64_t dims[2] = {inner, outer};
    const uint64_t strides[1] = {row_bytes};
    const uint32_t box[2] = {box_inner, box_outer};
    return encode_cached(map, dtype, 2, base, dims, strides, box, swz);
}

int cluster_capacity(const void* kernel, int ks, int threads, int smem_bytes, bool along_x) {
    static CapacityCache cache;
    int dev = 0;
    cudaGetDevice(&dev);
    return cache.get(kernel, dev, ks, along_x, [&] {
        int n = 0;
        cudaLaunchConfig_t cfg = {};
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = along_x ? ks : 1;
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = along_x ? 1 : ks;
        cfg.gridDim = along_x ? dim3(ks, 1, 1) : dim3(1, 1, ks);
        cfg.blockDim = dim3(threads, 1, 1);
        cfg.dynamicSmemBytes = smem_bytes;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess || n <= 0) {
            cudaGetLastError();
            n = num_sms() / ks;
        }
        return n;
    });
}

// SM count of the current device (cached per device; 148 if the query fails).
int num_sms() {
    static std::atomic<int> sms[64];
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev < 0 || dev >= 64) dev = 0;
    int n = sms[dev].load(std::memory_order_relaxed);
    if (n <= 0) {
        if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) {
            cudaGetLastError();
            n = 148;
        }
        sms[dev].store(n, std::memory_order_relaxed);
    }
    return n;
}

namespace {

// rows: weight rows per CTA tile (0 = automatic: 128, or a CTA pair's 256 where that applies).
template <int BITS, int GS, int BT, bool PAIR = false>
lowbit_status launch(const GemmProblem& g, int rows, int ksplit_request, cudaStream_t stream, bool convert_x) {
    using C = Cfg<BITS, GS, BT, PAIR>;
    auto kernel = lowbit_gemm_kernel<BITS, GS, BT, PAIR>;
    const bool auto_rows = rows == 0;
    if (auto_rows || PAIR) rows = kBlockN;
    // the shared-memory opt-in is per device: one bit per device that has it
    static std::atomic<uint64_t> attr_devices{0};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return LOWBIT_ERR_CUDA;
    const uint64_t bit = dev < 64 ? (uint64_t(1) << dev) : 0;
    if (!bit || !(attr_devices.load(std::memory_order_acquire) & bit)) {
        if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes) != cudaSuccess)
            return LOWBIT_ERR_CUDA;
        attr_devices.fetch_or(bit, std::memory_order_acq_rel);
    }
    CUtensorMap mx, mw, ms, mz;
    const int K = static_cast<int>(g.K), N = static_cast<int>(g.N), M = static_cast<int>(g.M);
    const CUtensorMapSwizzle wswz = C::kWRowBytes == 16   ? CU_TENSOR_MAP_SWIZZLE_NONE
                                    : C::kWRowBytes == 32 ? CU_TENSOR_MAP_SWIZZLE_32B
                                                          : CU_TENSOR_MAP_SWIZZLE_64B;
    const WorkspaceLayout ws = workspace_layout(g.M, g.K);
    void* xh = g.workspace;
    float* rowmul = reinterpret_cast<float*>(static_cast<uint8_t*>(g.workspace) + ws.rowmul_offset);
    bool ok = make_map_x3d(&mx, xh, M, K, C::kXRows);
    ok = ok && make_map_2d(&mw, CU_TENSOR_MAP_DATA_TYPE_UINT32, 4, g.Wp, uint64_t(K) * BITS / 32, N,
                           uint64_t(K) * BITS / 8, C::kWordsPerRow, rows, wswz);
    ok = ok && make_map_2d(&ms, CU_TENSOR_MAP_DATA_TYPE_UINT16, 2, g.scales, N, K / GS, uint64_t(N) * 2, kBlockN,
                           C::kGroupsPerStage, CU_TENSOR_MAP_SWIZZLE_NONE);
    if (BITS == 4)
        ok = ok && make_map_2d(&mz, CU_TENSOR_MAP_DATA_TYPE_UINT16, 2, g.zeros, N, K / GS, uint64_t(N) * 2,
                               kBlockN, C::kGroupsPerStage, CU_TENSOR_MAP_SWIZZLE_NONE);
    else
        mz = ms;
    // Y as (N, M) with a box of one tile, [BT tokens][rows]: the store of each CTA's last tile
    CUtensorMap my;
    ok = ok && make_map_2d(&my, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, g.Y, N, M, uint64_t(N) * 2, rows, BT,
                           CU_TENSOR_MAP_SWIZZLE_NONE);
    if (!ok) return LOWBIT_ERR_CUDA;

    KernelParams p;
    p.M = M;
    p.N = N;
    p.K = K;
    p.num_kb = (K + kBlockK - 1) / kBlockK;
    p.rows = rows;
    p.wtx_bytes = static_cast<uint32_t>(C::kWTxFixed + rows * C::kWRowBytes);
    p.m_tiles = (M + BT - 1) / BT;
    p.n_tiles = PAIR ? N / (2 * rows) : (N + rows - 1) / rows;
    p.num_tiles = p.m_tiles * p.n_tiles;
    p.Y = static_cast<__nv_bfloat16*>(g.Y);
    p.rowmul = rowmul;
    int ksplit = PAIR ? 1 : ksplit_request;
    if (ksplit < 0) {
        // Automatic: the largest split that leaves every rank at least 24 k-blocks (3072 of K)
        // and keeps all clusters resident at once (the split grid is not persistent, so a
        // second wave would double the time); cluster placement is limited by the GPC layout.
        ksplit = 1;
        const int slots = num_sms() * C::kCtasPerSm;
        for (int ks = 8; ks >= 2; --ks) {
            if (p.num_kb / ks < 24 || p.num_tiles * ks > slots) continue;
            if (p.num_tiles <= cluster_capacity(reinterpret_cast<const void*>(kernel), ks, C::kThreads,
                                                C::kSmemBytes)) {
                ksplit = ks;
                break;
            }
        }
    }
    if (ksplit < 1) ksplit = 1;
    if (ksplit > 8) ksplit = 8;
    // An unsplit grid of 256-token tiles over a multiple of 256 weight rows runs on CTA pairs.
    if constexpr (BT == 256 && !PAIR) {
        if (auto_rows && ksplit == 1 && N % (2 * kBlockN) == 0)
            return launch<BITS, GS, BT, true>(g, 0, 1, stream, convert_x);
    }
    if (ksplit > p.num_kb) ksplit = p.num_kb;
    int kbps = (p.num_kb + ksplit - 1) / ksplit;
    ksplit = (p.num_kb + kbps - 1) / kbps;     // every rank gets at least one k-block
    p.kb_per_split = ksplit > 1 ? kbps : p.num_kb;
    p.ksplit = ksplit;

    // X -> fp16 copy in the workspace, then the GEMM; both launched as programmatic dependents
    // of whatever precedes them on the stream.
    if (convert_x && launch_convert_x(g, stream) != LOWBIT_OK) return LOWBIT_ERR_CUDA;

    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attrs[2];
    int na = 0;
    attrs[na].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attrs[na].val.programmaticStreamSerializationAllowed = 1;
    ++na;
    if (PAIR) {
        // persistent grid of CTA pairs, the two CTAs of a pair adjacent along x (clusters of 2)
        int pairs = cluster_capacity(reinterpret_cast<const void*>(kernel), 2, C::kThreads, C::kSmemBytes, true);
        if (pairs > num_sms() / 2) pairs = num_sms() / 2;
        if (pairs < 1) pairs = 1;
        cfg.gridDim = dim3(2 * (p.num_tiles < pairs ? p.num_tiles : pairs), 1, 1);
        attrs[na].id = cudaLaunchAttributeClusterDimension;
        attrs[na].val.clusterDim.x = 2;
        attrs[na].val.clusterDim.y = 1;
        attrs[na].val.clusterDim.z = 1;
        ++na;
    } else if (ksplit > 1) {
        cfg.gridDim = dim3(p.num_tiles, 1, ksplit);
        attrs[na].id = cudaLaunchAttributeClusterDimension;
        attrs[na].val.clusterDim.x = 1;
        attrs[na].val.clusterDim.y = 1;
        attrs[na].val.clusterDim.z = ksplit;
        ++na;
    } else {
        const int slots = num_sms() * C::kCtasPerSm;
        cfg.gridDim = dim3(p.num_tiles < slots ? p.num_tiles : slots, 1, 1);
    }
    cfg.blockDim = dim3(C::kThreads, 1, 1);
    cfg.dynamicSmemBytes = C::kSmemBytes;
    cfg.stream = stream;
    cfg.attrs = attrs;
    cfg.numAttrs = na;
    if (take_injected_failure(kInjectLaunch)) return LOWBIT_ERR_CUDA;
    cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, mx, mw, ms, mz, my, p);
    return e == cudaSuccess ? LOWBIT_OK : LOWBIT_ERR_CUDA;
}

// Token-tile width for M rows.
int pick_bt(int64_t M) {
    if (M <= 16) return 16;
    if (M <= 32) return 32;
    if (M <= 64) return 64;
    if (M <= 128) return 128;
    return 256;
}

int ctas_per_sm_for(int bt) { return bt <= 64 ? 2 : 1; }

template <int BITS, int GS>
lowbit_status launch_bits_gs(const GemmProblem& g, int bt, int rows, int ksplit, cudaStream_t s, bool cx) {
    switch (bt) {
        case 16: return launch<BITS, GS, 16>(g, rows, ksplit, s, cx);
        case 32: return launch<BITS, GS, 32>(g, rows, ksplit, s, cx);
        case 64: return launch<BITS, GS, 64>(g, rows, ksplit, s, cx);
        case 128: return launch<BITS, GS, 128>(g, rows, ksplit, s, cx);
        case 256:
            if (rows == 2 * kBlockN) return launch<BITS, GS, 256, true>(g, 0, 1, s, cx);
            return launch<BITS, GS, 256>(g, rows, ksplit, s, cx);
        default: return LOWBIT_ERR_UNSUPPORTED;
    }
}

}  // namespace

// Chooses the launch configuration (tile_tokens, tile_rows, ksplit), each 0 = automatic:
//   * one token tile and small M (weight streaming, HBM-bound): either "flat" tiles of
//     ceil(N / #SMs) rows (a multiple of 8) with the whole K per CTA and no reduction, or 128-row
//     tiles with K split over a cluster, whichever reads fewer X bytes per weight byte;
//   * few tiles otherwise: 128-row tiles with K split over a cluster;
//   * many tiles: 128-row tiles on a persistent grid.
bool uses_x_copy(const GemmProblem& g) { return !smallm_supported(g); }

lowbit_status gemm_launch(const GemmProblem& g, int force_bt, int force_rows, int force_split,
                          cudaStream_t stream, bool convert_x) {
    // tile_tokens == 1 selects the small-M warp-MMA kernel with X as the 16-row operand, 8 the
    // one with weights as the 16-row operand (M <= 8); automatic: 8 for M <= 8, else 1 up to 16
    if (force_bt == 1 || force_bt == 8) return smallm_launch(g, force_rows, force_split, force_bt == 8, stream);
    if (!force_bt && !force_rows && !force_split && smallm_supported(g))
        return smallm_launch(g, 0, 0, g.M <= 8, stream);
    const int bt = force_bt ? force_bt : pick_bt(g.M);
    const int sms = num_sms();
    const int64_t num_kb = (g.K + kBlockK - 1) / kBlockK;
    const int64_t m_tiles = (g.M + bt - 1) / bt;
    int rows = force_rows ? force_rows : kBlockN;
    int ksplit = force_split;
    if (!force_rows && !force_split) {
        const int64_t slots = static_cast<int64_t>(sms) * ctas_per_sm_for(bt);
        const int64_t tiles128 = m_tiles * ((g.N + kBlockN - 1) / kBlockN);
        int64_t flat_rows = ((g.N + sms - 1) / sms + 7) / 8 * 8;
        // X bytes read per packed-weight byte by one CTA: 2 * bt / (rows * bits / 8)
        const double x_per_w = (2.0 * bt) / (static_cast<double>(flat_rows) * g.bits / 8.0);
        ksplit = 1;
        if (bt <= 64 && m_tiles == 1 && flat_rows < kBlockN && x_per_w <= 1.25) {
            rows = static_cast<int>(flat_rows);
        } else if (bt <= 64 && m_tiles == 1) {
            if (tiles128 * 2 <= slots && num_kb >= 4) {
                int64_t s = sms / tiles128;   // small M: one CTA per SM
                if (s > 8) s = 8;
                if (s > num_kb / 2) s = num_kb / 2;
                ksplit = static_cast<int>(s < 1 ? 1 : s);
            }
        } else {
            ksplit = -1;   // chosen by the launch from the cluster capacity
        }
    }
    if (!ksplit) ksplit = 1;
    // 256 rows: one tile per CTA pair (256-token tiles, N a multiple of 256, no K split)
    const bool pair_rows = force_rows == 2 * kBlockN;
    if (pair_rows && (bt != 256 || g.N % (2 * kBlockN) != 0 || ksplit > 1)) return LOWBIT_ERR_UNSUPPORTED;
    if (!pair_rows && (rows < 8 || rows > kBlockN || rows % 8)) return LOWBIT_ERR_UNSUPPORTED;   // (ksplit -1: automatic)
    if (!force_rows && rows == kBlockN) rows = 0;   // automatic: the launch may use CTA pairs
    switch (g.bits * 1000 + g.group_size) {
        case 1064: return launch_bits_gs<1, 64>(g, bt, rows, ksplit, stream, convert_x);
        case 1128: return launch_bits_gs<1, 128>(g, bt, rows, ksplit, stream, convert_x);
        case 2064: return launch_bits_gs<2, 64>(g, bt, rows, ksplit, stream, convert_x);
        case 2128: return launch_bits_gs<2, 128>(g, bt, rows, ksplit, stream, convert_x);
        case 4064: return launch_bits_gs<4, 64>(g, bt, rows, ksplit, stream, convert_x);
        case 4128: return launch_bits_gs<4, 128>(g, bt, rows, ksplit, stream, convert_x);
        default: return LOWBIT_ERR_UNSUPPORTED;
    }
}

unsigned* device_status_address() {
    constexpr int kMaxDevices = 64;
    static std::atomic<unsigned*> ptrs[kMaxDevices];
    static std::mutex mu;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return nullptr;
    unsigned* p = ptrs[dev].load(std::memory_order_acquire);
    if (p) return p;
    std::lock_guard<std::mutex> lock(mu);
    p = ptrs[dev].load(std::memory_order_relaxed);
    if (!p) {
        void* ptr = nullptr;
        if (cudaGetSymbolAddress(&ptr, g_device_status) != cudaSuccess) return nullptr;
        p = static_cast<unsigned*>(ptr);
        ptrs[dev].store(p, std::memory_order_release);
    }
    return p;
}

namespace {
lowbit_status status_of_word(unsigned v) {
    if (v & kDevErrTimeout) return LOWBIT_ERR_TIMEOUT;
    if (v & kDevErrCheck) return LOWBIT_ERR_DEVICE_CHECK;
    return LOWBIT_OK;
}
}  // namespace

lowbit_status read_device_status(int clear) {
    unsigned v = 0;
    if (cudaDeviceSynchronize() != cudaSuccess) return LOWBIT_ERR_CUDA;
    if (cudaMemcpyFromSymbol(&v, g_device_status, sizeof(v)) != cudaSuccess) return LOWBIT_ERR_CUDA;
    if (clear && v) {
        const unsigned zero = 0;
        if (cudaMemcpyToSymbol(g_device_status, &zero, sizeof(zero)) != cudaSuccess) return LOWBIT_ERR_CUDA;
    }
    return status_of_word(v);
}

// Stream-ordered read and clear: the copy of the word and the clearing store are queued on
// `stream`, so only the work queued there before them is waited for.
lowbit_status read_stream_status(cudaStream_t stream) {
    unsigned* word = device_status_address();
    if (!word) return LOWBIT_ERR_CUDA;
    unsigned v = 0;
    if (cudaMemcpyAsync(&v, word, sizeof(v), cudaMemcpyDeviceToHost, stream) != cudaSuccess ||
        cudaMemsetAsync(word, 0, sizeof(unsigned), stream) != cudaSuccess ||
        cudaStreamSynchronize(stream) != cudaSuccess)
        return LOWBIT_ERR_CUDA;
    return status_of_word(v);
}

}  // namespace lowbit
