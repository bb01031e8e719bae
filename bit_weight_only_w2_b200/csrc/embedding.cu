// Lookup of vocabulary rows by token, and its gradient by sorted tokens.
//
// Lookup: y[t] = multiplier * E[token t] (zeros for a token outside the table), one pass: a warp takes 1024 columns of a
// token, four 16-byte pieces a lane, all requested before the first is used. Rows of bf16 are bound by memory. Packed rows
// are decoded on the way: the four words of a block hold the pairs of four (ternary: eight) neighbouring 8-column pieces,
// which as many lanes read together; that is bound by the issue of instructions (16384 tokens of 2560 ternary columns: 78 % of
// the slots, DRAM 17 % of its rate, since most of Y is still in L2 at the end).
//
// Gradient: dE[v] = multiplier * the sum of dy[t] over the tokens t of v, of stretches in the tokens' order that are joined in
// that order, whatever the timing:
//   1. the tokens are sorted by row (stable radix sort, digits of up to 9 bits): up to kSortMost tokens in one CTA,
//      more in tiles of kTile, with a launch for the digits' counts and one for the moves of each digit, and one for the
//      counts' sums between them where there are more than kFewTiles tiles (the sort of 32768 tokens in one CTA took
//      140 us; in tiles all of the gradient of 32000 x 512 takes 35). Beside the sort dE is filled with zeros;
//   2. a CTA adds up kRun tokens of the sorted list for 1024 columns, in fp32: a row whose tokens all lie in the run is
//      stored at once; the parts of rows that go over a run's ends are kept in fp32;
//   3. the parts are joined in order by the CTA of the run that such a row begins in.
// Runs of equal length bound the work of step 2 however often a token repeats; step 3 is a CTA's per 256 columns of the row,
// whose parts it reads: 100000 tokens of one row take 250 us for 300 x 2560, of all rows alike 154 (72 columns: 102 and 50).
// The zeros bound a whole table (131072 x 2560: 115 of 180 us with 32768 tokens). Few rows (tokens added to a frozen table), or few tokens on a small table, take
// one launch instead.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <atomic>

#include "sm100_ptx.cuh"
#include "vocab_internal.h"

namespace lowbit {
namespace {

constexpr int kThreads = 256;

template <class... P, class... A>
lowbit_status launch_after(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t stream, A... args) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (take_injected_failure(kInjectLaunch)) return LOWBIT_ERR_CUDA;
    return cudaLaunchKernelEx(&cfg, kernel, args...) == cudaSuccess ? LOWBIT_OK : LOWBIT_ERR_CUDA;
}

__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ float2 f32x2(uint32_t v) { return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xFFFF0000u)); }

// ---------------------------------------------------------------------------------------------
// Lookup
// ---------------------------------------------------------------------------------------------
constexpr int kPieces = 4;   // of 8 columns, per lane

// The 8 values of piece c (columns 8c .. 8c + 7) of a packed row, as code values.
template <int BITS>
struct Codes {
    uint4 w;
    __device__ __forceinline__ void load(const uint32_t* row, int c) {
        if (BITS == 1)
            w.x = __ldg(row + (c >> 2));
        else
            w = __ldg(reinterpret_cast<const uint4*>(row) + (BITS == 2 ? c >> 3 : c >> 2));
    }
    __device__ __forceinline__ void values(int c, float (&v)[8]) const {
        if (BITS == 1) {   // plain order: pairs 4 (c % 4) .. + 3 of the word
            const uint32_t x = w.x >> (4 * (c & 3));
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                v[2 * q] = (x >> q) & 1 ? 1.f : -1.f;
                v[2 * q + 1] = (x >> (16 + q)) & 1 ? 1.f : -1.f;
            }
        } else {           // block order: pair p of the block's word q holds columns 8p + 2q and 8p + 2q + 1
            const int shift = BITS == 2 ? 2 * (c & 7) : 4 * (c & 3);
            const uint32_t words[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const uint32_t x = words[q] >> shift, mask = (1 << BITS) - 1;
                v[2 * q] = static_cast<float>(x & mask);
                v[2 * q + 1] = static_cast<float>((x >> 16) & mask);
                if (BITS == 2) {
                    v[2 * q] -= 1.f;
                    v[2 * q + 1] -= 1.f;
                }
            }
        }
    }
};

template <int BITS>
__global__ void __launch_bounds__(kThreads) embedding_kernel(const void* __restrict__ rows, const __half* __restrict__ scales,
                                                             const __half* __restrict__ zeros, const int32_t* __restrict__ tokens,
                                                             int64_t units, int segs, int K8, int64_t N, int group_log2, float multiplier,
                                                             uint4* __restrict__ out) {
    grid_launch_dependents();
    grid_dependency_wait();
    const int lane = threadIdx.x & 31;
    const int64_t unit = int64_t(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
    if (unit >= units) return;
    const int64_t t = unit / segs;
    const int c0 = static_cast<int>(unit - t * segs) * (32 * kPieces) + lane;
    const int token = __ldg(tokens + t);
    const bool has = token >= 0 && token < N;
    uint4* dst = out + t * K8;
    if (!has) {
#pragma unroll
        for (int i = 0; i < kPieces; ++i)
            if (c0 + 32 * i < K8) dst[c0 + 32 * i] = make_uint4(0, 0, 0, 0);
        return;
    }
    if constexpr (BITS == kDense) {
        const uint4* src = static_cast<const uint4*>(rows) + int64_t(token) * K8;
        uint4 v[kPieces];
#pragma unroll
        for (int i = 0; i < kPieces; ++i)
            if (c0 + 32 * i < K8) v[i] = __ldg(src + c0 + 32 * i);
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            if (c0 + 32 * i >= K8) continue;
            uint32_t* w = reinterpret_cast<uint32_t*>(&v[i]);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const float2 f = f32x2(w[q]);
                w[q] = bf16x2(f.x * multiplier, f.y * multiplier);
            }
            dst[c0 + 32 * i] = v[i];
        }
    } else {
        const uint32_t* src = static_cast<const uint32_t*>(rows) + int64_t(token) * (K8 * BITS / 4);
        Codes<BITS> w[kPieces];
        float s[kPieces], z[kPieces];
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            const int c = c0 + 32 * i;
            if (c < K8) {
                const int64_t at = int64_t(c >> (group_log2 - 3)) * N + token;
                w[i].load(src, c);
                s[i] = __half2float(scales[at]);
                z[i] = BITS == 4 ? __half2float(zeros[at]) : 0.f;
            }
        }
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            const int c = c0 + 32 * i;
            if (c >= K8) continue;
            float v[8];
            w[i].values(c, v);
            // (q - z) is exact in fp32; its product with the scale and that with the multiplier are rounded to fp32,
            // 2^-24 each, before the one rounding to bf16
#pragma unroll
            for (int q = 0; q < 8; ++q) v[q] = (v[q] - z[i]) * s[i] * multiplier;
            dst[c] = make_uint4(bf16x2(v[0], v[1]), bf16x2(v[2], v[3]), bf16x2(v[4], v[5]), bf16x2(v[6], v[7]));
        }
    }
}

// ---------------------------------------------------------------------------------------------
// Gradient: the sort. Keys are rows of dE (tokens outside them: `rows`, which puts them last).
// ---------------------------------------------------------------------------------------------
constexpr int kSortThreads = 1024, kSortWarps = 32;
constexpr int kSortItems = 2;                            // per thread, at most
constexpr int kSortMost = kSortThreads * kSortItems;     // tokens of one CTA
constexpr int kDigitBits = 9, kMaxDigits = 1 << kDigitBits;

struct SortPlan {
    int passes, bits;   // digits of `bits` bits
};
SortPlan sort_plan(int64_t rows) {   // keys 0 .. rows
    int bits = 1;
    while ((int64_t(1) << bits) <= rows) ++bits;
    const int passes = (bits + kDigitBits - 1) / kDigitBits;
    return SortPlan{passes, (bits + passes - 1) / passes};
}

__device__ __forceinline__ uint32_t key_of(int token, int64_t first, int64_t rows) {
    const int64_t at = int64_t(token) - first;
    return static_cast<uint32_t>(at >= 0 && at < rows ? at : rows);
}

// The lanes of the warp with this lane's digit.
__device__ __forceinline__ uint32_t peers_of(uint32_t digit, int bits) {
    uint32_t m = 0xffffffffu;
    for (int b = 0; b < bits; ++b) {
        const uint32_t v = __ballot_sync(0xffffffffu, (digit >> b) & 1u);
        m &= (digit >> b) & 1u ? v : ~v;
    }
    return m;
}

// One CTA sorts every token: each warp keeps the order of its own stretch of the list, so the digits' counts, warp by
// warp, give each token its place. Keys and positions are held in registers while shared memory is rewritten.
template <int ITEMS>
__device__ void sort_in_cta(const int32_t* tokens, int T, int64_t first, int64_t rows, SortPlan plan, uint32_t* keys_out,
                            uint32_t* pos_out, uint8_t* smem) {
    uint32_t* keys = reinterpret_cast<uint32_t*>(smem);
    uint16_t* pos = reinterpret_cast<uint16_t*>(keys + kSortThreads * ITEMS);
    uint16_t* count = pos + kSortThreads * ITEMS;               // [warp][digit]
    uint32_t* start = reinterpret_cast<uint32_t*>(count + kSortWarps * kMaxDigits);   // [digit]
    uint32_t* sums = start + kMaxDigits;                        // [kMaxDigits / 32]
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t below = (1u << lane) - 1u;
    const int base = warp * 32 * ITEMS + lane;
    uint32_t key[ITEMS];
    uint16_t at[ITEMS];
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
        const int t = base + 32 * i;
        key[i] = t < T ? key_of(tokens[t], first, rows) : 0xffffffffu;   // (past the end: behind everything)
        at[i] = static_cast<uint16_t>(t);
    }
    const uint32_t digits = 1u << plan.bits;
    for (int pass = 0; pass < plan.passes; ++pass) {
        const int shift = pass * plan.bits;
        for (int i = threadIdx.x; i < kSortWarps * kMaxDigits; i += kSortThreads) count[i] = 0;
        __syncthreads();
        uint16_t rank[ITEMS];
        uint16_t* mine = count + warp * kMaxDigits;
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
            const uint32_t d = (key[i] >> shift) & (digits - 1);
            const uint32_t peers = peers_of(d, plan.bits);
            const uint16_t before = mine[d];
            __syncwarp();
            rank[i] = static_cast<uint16_t>(before + __popc(peers & below));
            if ((peers & below) == 0) mine[d] = static_cast<uint16_t>(before + __popc(peers));
            __syncwarp();
        }
        __syncthreads();
        // per digit: the warps' counts to their sums so far, and the digits' starts
        if (threadIdx.x < kMaxDigits) {
            uint32_t total = 0;
            for (int w = 0; w < kSortWarps; ++w) {
                const uint32_t c = count[w * kMaxDigits + threadIdx.x];
                count[w * kMaxDigits + threadIdx.x] = static_cast<uint16_t>(total);
                total += c;
            }
            uint32_t incl = total;
#pragma unroll
            for (int o = 1; o < 32; o *= 2) {
                const uint32_t v = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += v;
            }
            if (lane == 31) sums[warp] = incl;
            start[threadIdx.x] = incl - total;
        }
        __syncthreads();
        if (threadIdx.x < kMaxDigits) {
            uint32_t before = 0;
            for (int w = 0; w < warp; ++w) before += sums[w];
            start[threadIdx.x] += before;
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
            const uint32_t d = (key[i] >> shift) & (digits - 1);
            const uint32_t to = start[d] + count[warp * kMaxDigits + d] + rank[i];
            keys[to] = key[i];
            pos[to] = at[i];
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
            key[i] = keys[base + 32 * i];
            at[i] = pos[base + 32 * i];
        }
        __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
        const int t = base + 32 * i;
        if (t < T) {
            keys_out[t] = key[i];
            pos_out[t] = at[i];
        }
    }
}

// Beside the sorting CTAs of a launch the others fill a part of dE with zeros, whatever its rows hold later: a plain
// stream of stores by neighbouring threads (131072 x 2560 in 115 us, 5.8 TB/s; row by row, only those without tokens, 172).
struct Zeros {
    uint4* out;
    int64_t from, to;   // 16-byte pieces
};
__device__ __forceinline__ void fill(const Zeros& z, int cta, int ctas) {
    for (int64_t i = z.from + int64_t(cta) * kSortThreads + threadIdx.x; i < z.to; i += int64_t(ctas) * kSortThreads)
        z.out[i] = make_uint4(0, 0, 0, 0);
}

template <int ITEMS>
__global__ void __launch_bounds__(kSortThreads) sort_small_kernel(const int32_t* __restrict__ tokens, int T, int64_t first, int64_t rows,
                                                                  SortPlan plan, uint32_t* __restrict__ keys, uint32_t* __restrict__ pos,
                                                                  Zeros zeros) {
    extern __shared__ __align__(16) uint8_t smem[];
    grid_launch_dependents();
    grid_dependency_wait();
    if (blockIdx.x > 0) return fill(zeros, blockIdx.x - 1, gridDim.x - 1);
    sort_in_cta<ITEMS>(tokens, T, first, rows, plan, keys, pos, smem);
}

// More tokens: tiles of kTile tokens. count: the digits' counts of each tile, [digit][tile].
constexpr int kTileItems = 2, kTile = kSortThreads * kTileItems;
constexpr int kFewTiles = 64;

__global__ void __launch_bounds__(kSortThreads) sort_count_kernel(const int32_t* __restrict__ tokens, const uint32_t* __restrict__ keys,
                                                                  int64_t T, int64_t first, int64_t rows, int shift, int bits,
                                                                  uint32_t* __restrict__ counts, int tiles, Zeros zeros) {
    grid_launch_dependents();
    grid_dependency_wait();
    if (static_cast<int>(blockIdx.x) >= tiles) return fill(zeros, blockIdx.x - tiles, gridDim.x - tiles);
    __shared__ uint32_t hist[kMaxDigits];
    for (int d = threadIdx.x; d < kMaxDigits; d += kSortThreads) hist[d] = 0;
    __syncthreads();
    const int64_t base = int64_t(blockIdx.x) * kTile;
    for (int i = threadIdx.x; i < kTile; i += kSortThreads)
        if (base + i < T) {
            const uint32_t k = tokens ? key_of(tokens[base + i], first, rows) : keys[base + i];
            atomicAdd(&hist[(k >> shift) & ((1u << bits) - 1)], 1u);
        }
    __syncthreads();
    for (int d = threadIdx.x; d < 1 << bits; d += kSortThreads) counts[int64_t(d) * tiles + blockIdx.x] = hist[d];
}

// Exclusive sums of n counts, one CTA.
__global__ void __launch_bounds__(kSortThreads) sort_scan_kernel(uint32_t* __restrict__ counts, int64_t n) {
    grid_launch_dependents();
    grid_dependency_wait();
    __shared__ uint32_t sums[kSortWarps];
    __shared__ uint32_t carry;
    if (threadIdx.x == 0) carry = 0;
    __syncthreads();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int64_t base = 0; base < n; base += kSortThreads * 4) {
        uint32_t v[4], total = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t at = base + threadIdx.x * 4 + i;
            v[i] = at < n ? counts[at] : 0;
            total += v[i];
        }
        uint32_t incl = total;
#pragma unroll
        for (int o = 1; o < 32; o *= 2) {
            const uint32_t u = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += u;
        }
        if (lane == 31) sums[warp] = incl;
        __syncthreads();
        uint32_t before = carry + incl - total;
        for (int w = 0; w < warp; ++w) before += sums[w];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t at = base + threadIdx.x * 4 + i;
            if (at < n) counts[at] = before;
            before += v[i];
        }
        __syncthreads();
        if (threadIdx.x == kSortThreads - 1) carry = before;
        __syncthreads();
    }
}

__global__ void __launch_bounds__(kSortThreads) sort_move_kernel(const int32_t* __restrict__ tokens, const uint32_t* __restrict__ keys,
                                                                 const uint32_t* __restrict__ pos, int64_t T, int64_t first, int64_t rows,
                                                                 int shift, int bits, const uint32_t* __restrict__ counts, int tiles,
                                                                 uint32_t* __restrict__ keys_out, uint32_t* __restrict__ pos_out,
                                                                 Zeros zeros) {
    grid_launch_dependents();
    grid_dependency_wait();
    if (static_cast<int>(blockIdx.x) >= tiles) return fill(zeros, blockIdx.x - tiles, gridDim.x - tiles);
    __shared__ uint16_t count[kSortWarps * kMaxDigits];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t below = (1u << lane) - 1u;
    for (int i = threadIdx.x; i < kSortWarps * kMaxDigits; i += kSortThreads) count[i] = 0;
    __syncthreads();
    const int64_t base = int64_t(blockIdx.x) * kTile + warp * 32 * kTileItems + lane;
    uint32_t key[kTileItems], at[kTileItems];
    uint16_t rank[kTileItems];
    uint16_t* mine = count + warp * kMaxDigits;
#pragma unroll
    for (int i = 0; i < kTileItems; ++i) {
        const int64_t t = base + 32 * i;
        key[i] = at[i] = 0;
        if (t < T) {
            key[i] = tokens ? key_of(tokens[t], first, rows) : keys[t];
            at[i] = pos ? pos[t] : static_cast<uint32_t>(t);
        }
        const uint32_t d = (key[i] >> shift) & ((1u << bits) - 1);
        const uint32_t live = __ballot_sync(0xffffffffu, t < T), peers = peers_of(d, bits) & live;
        const uint16_t before = mine[d];
        __syncwarp();
        rank[i] = static_cast<uint16_t>(before + __popc(peers & below));
        if (t < T && (peers & below) == 0) mine[d] = static_cast<uint16_t>(before + __popc(peers));
        __syncwarp();
    }
    // The tile's starts: from sort_scan_kernel, or where the tiles are few summed up here, a digit a thread.
    __shared__ uint32_t start[kMaxDigits];
    __shared__ uint32_t sums[kMaxDigits / 32];
    if (tiles <= kFewTiles && threadIdx.x < kMaxDigits) {
        uint32_t total = 0, mine_before = 0;
        if (static_cast<int>(threadIdx.x) < 1 << bits) {
#pragma unroll 8
            for (int t = 0; t < tiles; ++t) {
                if (t == static_cast<int>(blockIdx.x)) mine_before = total;
                total += counts[int64_t(threadIdx.x) * tiles + t];
            }
        }
        uint32_t incl = total;
#pragma unroll
        for (int o = 1; o < 32; o *= 2) {
            const uint32_t v = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += v;
        }
        if (lane == 31) sums[warp] = incl;
        start[threadIdx.x] = incl - total + mine_before;
    }
    __syncthreads();
    if (tiles <= kFewTiles && threadIdx.x < kMaxDigits) {
        uint32_t before = 0;
        for (int w = 0; w < warp; ++w) before += sums[w];
        start[threadIdx.x] += before;
    }
    for (int d = threadIdx.x; d < 1 << bits; d += kSortThreads) {
        uint32_t total = 0;
        for (int w = 0; w < kSortWarps; ++w) {
            const uint32_t c = count[w * kMaxDigits + d];
            count[w * kMaxDigits + d] = static_cast<uint16_t>(total);
            total += c;
        }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kTileItems; ++i) {
        const int64_t t = base + 32 * i;
        if (t < T) {
            const uint32_t d = (key[i] >> shift) & ((1u << bits) - 1);
            const int64_t to = int64_t(tiles <= kFewTiles ? start[d] : counts[int64_t(d) * tiles + blockIdx.x]) + count[warp * kMaxDigits + d] + rank[i];
            keys_out[to] = key[i];
            pos_out[to] = at[i];
        }
    }
}

// ---------------------------------------------------------------------------------------------
// Gradient: the sums
// ---------------------------------------------------------------------------------------------
constexpr int kRun = 32;            // sorted tokens per CTA
constexpr int kSumThreads = 128;    // 8 columns each

struct Sum {
    float v[8];
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = 0.f;
    }
    __device__ __forceinline__ void add(const uint4& a) {
        const float2 f0 = f32x2(a.x), f1 = f32x2(a.y), f2 = f32x2(a.z), f3 = f32x2(a.w);
        v[0] += f0.x; v[1] += f0.y; v[2] += f1.x; v[3] += f1.y;
        v[4] += f2.x; v[5] += f2.y; v[6] += f3.x; v[7] += f3.y;
    }
    __device__ __forceinline__ uint4 rounded(float m) const {
        return make_uint4(bf16x2(v[0] * m, v[1] * m), bf16x2(v[2] * m, v[3] * m), bf16x2(v[4] * m, v[5] * m), bf16x2(v[6] * m, v[7] * m));
    }
};

// parts [2][runs][K]: a run's part of a row that began in an earlier run, and of one that it begins and does not end.
__global__ void __launch_bounds__(kSumThreads) sum_runs_kernel(const uint32_t* __restrict__ keys, const uint32_t* __restrict__ pos, int64_t T,
                                                               uint32_t rows, const uint4* __restrict__ dy, int K8, float multiplier,
                                                               uint4* __restrict__ out, float4* __restrict__ parts, int64_t runs) {
    grid_launch_dependents();
    grid_dependency_wait();
    const int64_t run = blockIdx.x, i0 = run * kRun;
    const int n = static_cast<int>(T - i0 < kRun ? T - i0 : kRun);
    const int lane = threadIdx.x & 31;
    // every warp holds the run's keys and positions, one a lane
    const uint32_t my_key = lane < n ? keys[i0 + lane] : 0xffffffffu;
    const uint32_t my_pos = lane < n ? pos[i0 + lane] : 0;
    if (__shfl_sync(0xffffffffu, my_key, 0) >= rows) return;   // (tokens outside the rows come last)
    const uint32_t before = i0 > 0 ? keys[i0 - 1] : 0xffffffffu, after = i0 + n < T ? keys[i0 + n] : 0xffffffffu;
    const int c = blockIdx.y * kSumThreads + threadIdx.x;
    const bool live = c < K8;
    Sum s;
    s.zero();
    uint4 v[8];   // eight tokens' pieces in flight
#pragma unroll 1
    for (int i = 0; i < n; i += 8) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint32_t at = __shfl_sync(0xffffffffu, my_pos, (i + j) & 31);
            const uint32_t k = __shfl_sync(0xffffffffu, my_key, (i + j) & 31);
            v[j] = make_uint4(0, 0, 0, 0);
            if (live && i + j < n && k < rows) v[j] = __ldg(dy + int64_t(at) * K8 + c);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int e = i + j;
            const uint32_t k = __shfl_sync(0xffffffffu, my_key, e & 31), next = __shfl_sync(0xffffffffu, my_key, (e + 1) & 31);
            const uint32_t here = __shfl_sync(0xffffffffu, my_key, 0);
            if (e >= n || k >= rows) continue;
            s.add(v[j]);
            const bool last = e + 1 == n;
            if (!last && next == k) continue;
            // the row's tokens of this run end here
            const bool began = !(k == here && before == k), ends = !(last && after == k);
            if (live) {
                if (began && ends) {
                    out[int64_t(k) * K8 + c] = s.rounded(multiplier);
                } else {
                    float4* to = parts + ((began ? runs : 0) + run) * (2 * int64_t(K8)) + 2 * c;
                    to[0] = make_float4(s.v[0], s.v[1], s.v[2], s.v[3]);
                    to[1] = make_float4(s.v[4], s.v[5], s.v[6], s.v[7]);
                }
            }
            s.zero();
        }
    }
}

// 256 columns a CTA, eight warps that each add an eighth of the row's parts, joined in order.
constexpr int kJoinWarps = 8;
__device__ __forceinline__ bool join_warps(Sum& s, float (&sh)[kJoinWarps][32][9]) {   // true for warp 0: s is the sum
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
    for (int i = 0; i < 8; ++i) sh[warp][lane][i] = s.v[i];
    __syncthreads();
    if (warp > 0) return false;
    for (int w = 1; w < kJoinWarps; ++w)
#pragma unroll
        for (int i = 0; i < 8; ++i) s.v[i] += sh[w][lane][i];
    return true;
}

__global__ void __launch_bounds__(32 * kJoinWarps) join_runs_kernel(const uint32_t* __restrict__ keys, int64_t T, uint32_t rows, int K8,
                                                                    float multiplier, const float4* __restrict__ parts, int64_t runs,
                                                                    uint4* __restrict__ out) {
    grid_launch_dependents();
    grid_dependency_wait();
    const int64_t run = blockIdx.x, end = (run + 1) * kRun;
    if (end >= T) return;                                  // the last run's rows end in it
    const uint32_t k = keys[end - 1];
    if (k >= rows || keys[end] != k) return;               // no row goes over this run's end
    if (keys[run * kRun] == k && run > 0 && keys[run * kRun - 1] == k) return;   // it began in an earlier run
    // the last run with tokens of the row: keys ascend, so the runs that begin with k are neighbours; 32 probes at a time
    int64_t lo = run + 1, hi = runs - 1;
    while (lo < hi) {
        const int64_t step = (hi - lo + 31) / 32, probe = lo + step * (1 + (threadIdx.x & 31));
        const int in = __popc(__ballot_sync(0xffffffffu, probe <= hi && keys[probe * kRun] == k));
        lo += step * in;
        hi = min(hi, lo + step - 1);
    }
    __shared__ float sh[kJoinWarps][32][9];
    const int warp = threadIdx.x >> 5, c = blockIdx.y * 32 + (threadIdx.x & 31);
    const int64_t count = lo - run + 1, per = (count + kJoinWarps - 1) / kJoinWarps;
    Sum s;
    s.zero();
    if (c < K8) {
#pragma unroll 4
        for (int64_t r = run + warp * per; r < run + min(count, (warp + 1) * per); ++r) {
            const float4* from = parts + ((r == run ? runs : 0) + r) * (2 * int64_t(K8)) + 2 * c;
            const float4 a = from[0], b = from[1];
            s.v[0] += a.x; s.v[1] += a.y; s.v[2] += a.z; s.v[3] += a.w;
            s.v[4] += b.x; s.v[5] += b.y; s.v[6] += b.z; s.v[7] += b.w;
        }
    }
    if (join_warps(s, sh) && c < K8) out[int64_t(k) * K8 + c] = s.rounded(multiplier);
}

// Few rows: a CTA takes 256 columns of one row, finds its tokens (kept in order: each of the eight warps looks through
// an eighth of the list and adds what it finds) and joins the warps' sums in order. T tokens read from L2 by each CTA,
// 3 us for 1537 tokens and 24 rows of 2560 where the sort, sums and joins take 12.
__global__ void __launch_bounds__(32 * kJoinWarps) sum_few_rows_kernel(const int32_t* __restrict__ tokens, int T, int64_t first,
                                                                       const uint4* __restrict__ dy, int K8, float multiplier,
                                                                       uint4* __restrict__ out) {
    grid_launch_dependents();
    grid_dependency_wait();
    __shared__ float sh[kJoinWarps][32][9];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, c = blockIdx.y * 32 + lane;
    const int64_t want = first + blockIdx.x;
    const int per = ((T + kJoinWarps - 1) / kJoinWarps + 31) / 32 * 32, t1 = min(T, (warp + 1) * per);
    Sum s;
    s.zero();
#pragma unroll 4
    for (int t0 = warp * per; t0 < t1; t0 += 32) {
        const int token = t0 + lane < t1 ? __ldg(tokens + t0 + lane) : -1;
        uint32_t found = __ballot_sync(0xffffffffu, token >= 0 && token == want);
        while (found) {   // eight tokens' loads in flight
            uint4 v[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int t = t0 + __ffs(found) - 1;
                v[j] = make_uint4(0, 0, 0, 0);
                if (found && c < K8) v[j] = __ldg(dy + int64_t(t) * K8 + c);
                found &= found - 1;   // (0 stays 0)
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) s.add(v[j]);
        }
    }
    if (join_warps(s, sh) && c < K8) out[int64_t(blockIdx.x) * K8 + c] = s.rounded(multiplier);
}

// Few tokens: a CTA takes 256 columns of 32 rows, whose tokens it marks in shared memory. A warp adds up a row of up to
// kAlone tokens by itself; a row of more takes all eight warps, an eighth of the list each, joined in order.
// One launch of 6 to 14 us where the sort, sums and joins take 14 (256 tokens, 1 to 16 MB); but it fills zeros row by row,
// at half the rate (82 MB: 39 us, 25 with the sort).
constexpr int kFewTokens = 256, kAlone = 24;
constexpr int64_t kSmallTable = int64_t(8) << 20;   // values
bool few_tokens(int64_t T, int64_t rows, int64_t K) { return T <= kFewTokens && rows <= kSmallTable / K; }
__global__ void __launch_bounds__(32 * kJoinWarps) sum_few_tokens_kernel(const int32_t* __restrict__ tokens, int T, int64_t first,
                                                                         int64_t rows, const uint4* __restrict__ dy, int K8,
                                                                         float multiplier, uint4* __restrict__ out) {
    grid_launch_dependents();
    grid_dependency_wait();
    __shared__ uint8_t key[kFewTokens];   // row of a token among the 32, or 32
    __shared__ int count[32];
    __shared__ float sh[kJoinWarps][32][9];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, c = blockIdx.y * 32 + lane;
    const int64_t row0 = int64_t(blockIdx.x) * 32;
    const int n = static_cast<int>(rows - row0 < 32 ? rows - row0 : 32);
    if (threadIdx.x < 32) count[threadIdx.x] = 0;
    __syncthreads();
    const int padded = (T + 255) / 256 * 256;
    for (int t = threadIdx.x; t < padded; t += 32 * kJoinWarps) {
        const int64_t at = t < T ? int64_t(tokens[t]) - first - row0 : -1;
        const bool in = at >= 0 && at < n;
        key[t] = static_cast<uint8_t>(in ? at : 32);
        if (in) atomicAdd(&count[at], 1);
    }
    __syncthreads();
    auto add_up = [&](Sum& s, int r, int t0, int t1) {
        s.zero();
        for (; t0 < t1; t0 += 32) {
            uint32_t found = __ballot_sync(0xffffffffu, key[t0 + lane] == r);
            while (found) {   // eight tokens' loads in flight
                uint4 v[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int t = t0 + __ffs(found) - 1;
                    v[j] = make_uint4(0, 0, 0, 0);
                    if (found && c < K8) v[j] = __ldg(dy + int64_t(t) * K8 + c);
                    found &= found - 1;   // (0 stays 0)
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) s.add(v[j]);
            }
        }
    };
    uint4* to = out + row0 * K8 + c;
    Sum s;
    for (int r = warp; r < n; r += kJoinWarps) {
        if (count[r] > kAlone) continue;
        if (count[r] > 0) {
            add_up(s, r, 0, padded);
            if (c < K8) to[int64_t(r) * K8] = s.rounded(multiplier);
        } else if (c < K8) {
            to[int64_t(r) * K8] = make_uint4(0, 0, 0, 0);
        }
    }
    for (int r = 0; r < n; ++r) {
        if (count[r] <= kAlone) continue;
        add_up(s, r, warp * (padded / kJoinWarps), (warp + 1) * (padded / kJoinWarps));
        if (join_warps(s, sh) && c < K8) to[int64_t(r) * K8] = s.rounded(multiplier);
        __syncthreads();
    }
}

// Few: as many CTAs as the GPU holds at once, each with a list it looks through in a few microseconds. 4096 tokens, one in
// twenty on 24 rows of 2560 (100 rows): 5.9 (8.4) us, sorted 14.1 (14.7); 8192: 9.7 (15.3) and 15.1 (16.3); 16384: 17.5 (27.9)
// and 18.8 (19.8). The limit keeps away from where they meet, since tokens that are all on the rows take longer.
bool few_rows(int64_t T, int64_t rows, int64_t K) { return T <= 4096 && rows * ((K + 255) / 256) <= 148 * 8; }

struct GradLayout {
    int64_t runs, tiles;
    size_t keys, pos, keys2, pos2, counts, parts, total;
};
GradLayout grad_layout(int64_t T, int64_t rows, int64_t K) {
    GradLayout l = {};
    l.runs = (T + kRun - 1) / kRun;
    if (few_rows(T, rows, K) || few_tokens(T, rows, K)) {
        l.total = 256;
        return l;
    }
    size_t at = 0;
    auto take = [&](size_t bytes) {
        const size_t here = at;
        at += (bytes + 255) / 256 * 256;
        return here;
    };
    l.keys = take(T * 4);
    l.pos = take(T * 4);
    if (T > kSortMost) {
        l.tiles = (T + kTile - 1) / kTile;
        l.keys2 = take(T * 4);
        l.pos2 = take(T * 4);
        l.counts = take((size_t(1) << sort_plan(rows).bits) * l.tiles * 4);
    }
    l.parts = take(2 * static_cast<size_t>(l.runs) * K * 4);
    l.total = at;
    return l;
}

// CTAs that fill zeros: two an SM, each with four pieces a thread at least.
unsigned fill_ctas(const Zeros& z) {
    const int64_t n = (z.to - z.from + 4 * kSortThreads - 1) / (4 * kSortThreads);
    return static_cast<unsigned>(n < 2 * 148 ? n : 2 * 148);
}

template <int ITEMS>
lowbit_status sort_small(const int32_t* tokens, int64_t T, int64_t first, int64_t rows, SortPlan plan, uint32_t* keys, uint32_t* pos,
                         const Zeros& zeros, cudaStream_t stream) {
    constexpr size_t smem = size_t(kSortThreads) * ITEMS * 6 + kSortWarps * kMaxDigits * 2 + kMaxDigits * 4 + 256;
    static_assert(smem <= 232448, "shared memory");
    static std::atomic<uint64_t> devices{0};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return LOWBIT_ERR_CUDA;
    const uint64_t bit = dev < 64 ? (uint64_t(1) << dev) : 0;
    if (!bit || !(devices.load(std::memory_order_acquire) & bit)) {
        if (cudaFuncSetAttribute(sort_small_kernel<ITEMS>, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem)) != cudaSuccess)
            return LOWBIT_ERR_CUDA;
        devices.fetch_or(bit, std::memory_order_acq_rel);
    }
    return launch_after(sort_small_kernel<ITEMS>, dim3(1 + fill_ctas(zeros)), kSortThreads, smem, stream, tokens, static_cast<int>(T), first,
                        rows, plan, keys, pos, zeros);
}

}  // namespace

lowbit_status embedding_launch(const Table& t, const int32_t* tokens, int64_t T, float multiplier, void* out, cudaStream_t stream) {
    const int K8 = static_cast<int>(t.K / 8), segs = (K8 + 32 * kPieces - 1) / (32 * kPieces);
    const int64_t units = T * segs;
    const dim3 grid(static_cast<unsigned>((units + kThreads / 32 - 1) / (kThreads / 32)));
    const __half *scales = static_cast<const __half*>(t.scales), *zeros = static_cast<const __half*>(t.zeros);
    const int gl = t.group_size == 64 ? 6 : 7;
    uint4* y = static_cast<uint4*>(out);
    auto run = [&](auto kernel) { return launch_after(kernel, grid, kThreads, 0, stream, t.rows, scales, zeros, tokens, units, segs, K8, t.N, gl, multiplier, y); };
    switch (t.bits) {
        case 1: return run(embedding_kernel<1>);
        case 2: return run(embedding_kernel<2>);
        case 4: return run(embedding_kernel<4>);
        default: return run(embedding_kernel<kDense>);
    }
}

size_t embedding_backward_bytes(int64_t T, int64_t rows, int64_t K) { return grad_layout(T, rows, K).total; }

lowbit_status embedding_backward_launch(const int32_t* tokens, const void* dy, int64_t T, int64_t K, int64_t first, int64_t rows,
                                        float multiplier, void* out, void* ws, cudaStream_t stream) {
    const GradLayout l = grad_layout(T, rows, K);
    uint8_t* base = static_cast<uint8_t*>(ws);
    auto at = [&](size_t o) { return reinterpret_cast<uint32_t*>(base + o); };
    const SortPlan plan = sort_plan(rows);
    const int K8 = static_cast<int>(K / 8);
    if (few_rows(T, rows, K))
        return launch_after(sum_few_rows_kernel, dim3(static_cast<unsigned>(rows), (K8 + 31) / 32), 32 * kJoinWarps, 0, stream, tokens,
                            static_cast<int>(T), first, static_cast<const uint4*>(dy), K8, multiplier, static_cast<uint4*>(out));
    uint4* dE = static_cast<uint4*>(out);
    if (few_tokens(T, rows, K))
        return launch_after(sum_few_tokens_kernel, dim3(static_cast<unsigned>((rows + 31) / 32), (K8 + 31) / 32), 32 * kJoinWarps, 0, stream,
                            tokens, static_cast<int>(T), first, rows, static_cast<const uint4*>(dy), K8, multiplier, dE);
    uint32_t *keys = at(l.keys), *pos = at(l.pos);
    lowbit_status st = LOWBIT_OK;
    if (T <= kSortMost) {
        const Zeros all{dE, 0, rows * K8};
        st = T <= kSortThreads ? sort_small<1>(tokens, T, first, rows, plan, keys, pos, all, stream)
                               : sort_small<2>(tokens, T, first, rows, plan, keys, pos, all, stream);
        if (st != LOWBIT_OK) return st;
    } else {
        uint32_t *k2 = at(l.keys2), *p2 = at(l.pos2), *counts = at(l.counts);
        const uint32_t *kin = nullptr, *pin = nullptr;
        // (zeros in equal parts beside the launches)
        const int64_t n = rows * K8, part = (n + 2 * plan.passes - 1) / (2 * plan.passes);
        auto zeros = [&](int i) {
            const int64_t from = i * part < n ? i * part : n, to = (i + 1) * part < n ? (i + 1) * part : n;
            return Zeros{dE, from, to};
        };
        for (int pass = 0; pass < plan.passes; ++pass) {
            // (the last pass ends in `keys`)
            uint32_t *ko = (plan.passes - pass) % 2 ? keys : k2, *po = (plan.passes - pass) % 2 ? pos : p2;
            const int32_t* tok = pass == 0 ? tokens : nullptr;
            const int shift = pass * plan.bits, tiles = static_cast<int>(l.tiles);
            const Zeros z0 = zeros(2 * pass), z1 = zeros(2 * pass + 1);
            st = launch_after(sort_count_kernel, dim3(tiles + fill_ctas(z0)), kSortThreads, 0, stream, tok, kin, T, first, rows, shift,
                              plan.bits, counts, tiles, z0);
            if (st != LOWBIT_OK) return st;
            if (tiles > kFewTiles) {
                st = launch_after(sort_scan_kernel, dim3(1), kSortThreads, 0, stream, counts, (int64_t(1) << plan.bits) * tiles);
                if (st != LOWBIT_OK) return st;
            }
            st = launch_after(sort_move_kernel, dim3(tiles + fill_ctas(z1)), kSortThreads, 0, stream, tok, kin, pin, T, first, rows, shift,
                              plan.bits, counts, tiles, ko, po, z1);
            if (st != LOWBIT_OK) return st;
            kin = ko;
            pin = po;
        }
    }
    const unsigned slabs = (K8 + kSumThreads - 1) / kSumThreads;
    float4* parts = reinterpret_cast<float4*>(base + l.parts);
    st = launch_after(sum_runs_kernel, dim3(static_cast<unsigned>(l.runs), slabs), kSumThreads, 0, stream, keys, pos, T,
                      static_cast<uint32_t>(rows), static_cast<const uint4*>(dy), K8, multiplier, dE, parts, l.runs);
    if (st != LOWBIT_OK) return st;
    const unsigned strips = (K8 + 31) / 32;
    return launch_after(join_runs_kernel, dim3(static_cast<unsigned>(l.runs), strips), 32 * kJoinWarps, 0,
                        stream, keys, T, static_cast<uint32_t>(rows), K8, multiplier, parts, l.runs, dE);
}

}  // namespace lowbit
