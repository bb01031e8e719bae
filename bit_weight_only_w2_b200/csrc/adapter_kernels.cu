// The stages around the fused adapter product: tokens sorted by adapter, the low-rank product
// ("shrink"), the fp16 copy of the input with the slots' P, and the adapters' gradients.
//
// For one product of M tokens, each with an adapter a(m) of rank R (or none):
//   p[m]  = scaling[a] * in[m] A_a^T            shrink, then summed and scaled by the copy pass
//   out   = in W^T + p B_a^T                    gemm_kernel.cuh (kExtAdapter / kExtGrad)
//   dA_a  = sum_{m in a} dp[m]^T x[m],  dB_a = sum_{m in a} dy[m]^T p[m]      wgrad
// Everything is summed in fp32 in a fixed order (no atomics on results), so results do not depend
// on timing.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cmath>
#include <cstdint>
#include <type_traits>

#include "adapter_internal.h"
#include "checkpoint.cuh"
#include "sm100_ptx.cuh"
#include "tcgen05_ptx.cuh"

namespace lowbit {
namespace {

constexpr int kSmsAssumed = 148;   // the workspace's size may not depend on the device

// ---------------------------------------------------------------------------------------------
// Plan: the tokens of each adapter, and the slots of each token tile
// ---------------------------------------------------------------------------------------------
// One CTA per adapter counts the tokens of lower adapters (its start in the sorted order) and its
// own, and writes its tokens in ascending order: every warp takes a contiguous range of the
// tokens, counts its matches, and after one exchange of the counts compacts them by ballots.
// Scanning all M indices once per adapter costs L * M * 4 bytes of L2 reads, little next to the
// products for the L and M of a batch, and needs neither atomics nor a second launch.
// One more CTA per token tile lists the distinct adapters of the tile in ascending order (its
// "slots") from a bitmap, and each token's slot.
//
// A tile's slots share products in which other adapters' entries of P are zero, and zero times an
// infinity or NaN in the weight side would spread to their tokens. So the adapters in use have their
// weight side looked over here, cut over gridDim.y (it is read by the product soon after, from L2
// then); the shrink kernel joins the parts. A `bad` one is multiplied as zeros with P = NaN, which
// gives its own tokens NaN and others nothing.
//
// Shrink blocks of T = kShrinkTokens: adapter a's tokens [seg[a], seg[a + 1]) get the block numbers
// seg[a] / T + a + i, i < ceil(count / T), which never collide: the next adapter starts at
// floor(seg[a + 1] / T) + a + 1, and ceil(count / T) <= floor(seg[a + 1] / T) -
// floor(seg[a] / T) + 1. Numbers in between stay empty (count 0).
//
// Without an index every token has adapter 0 and lies where it belongs: no plan is made, and the
// kernels below are given null pointers for its parts (perm, blocks, seg, token_slot).
constexpr int kPlanThreads = 512;
constexpr int kPlanWarps = kPlanThreads / 32;

__device__ __forceinline__ int adapter_of(const int* __restrict__ index, int m, int num) {
    const int a = index ? index[m] : 0;
    return a >= 0 && a < num ? a : -1;   // anything else: no adapter
}

__global__ void __launch_bounds__(kPlanThreads)
    plan_kernel(const int* __restrict__ index, int M, int num, int tile_tokens, int slot_pitch, int num_blocks,
                const uint4* __restrict__ side, int64_t side8, int* __restrict__ perm, int* __restrict__ seg,
                int4* __restrict__ blocks, int* __restrict__ tile_slots, int* __restrict__ slot_adapter,
                int* __restrict__ token_slot, int* __restrict__ odd_parts, unsigned* status) {
    grid_dependency_wait();
    grid_launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (blockIdx.x < static_cast<unsigned>(num)) {
        const int a = blockIdx.x;
        __shared__ int warp_eq[kPlanWarps], warp_lt[kPlanWarps];
        if (blockIdx.y > 0) {
            // look over this CTA's share of the weight side, if the adapter has tokens at all
            bool used = false;
            for (int m = threadIdx.x; m < M; m += kPlanThreads) used |= adapter_of(index, m, num) == a;
            if (!__syncthreads_or(used)) return;
            const uint4* mine = side + static_cast<size_t>(a) * side8;
            const int64_t stride = static_cast<int64_t>(gridDim.y - 1) * kPlanThreads;
            bool odd = false;
            auto look = [&](uint32_t w) { odd |= (w & 0x7F80u) == 0x7F80u || (w & 0x7F800000u) == 0x7F800000u; };
#pragma unroll 4
            for (int64_t i = static_cast<int64_t>(blockIdx.y - 1) * kPlanThreads + threadIdx.x; i < side8; i += stride) {
                const uint4 v = __ldg(mine + i);
                look(v.x);
                look(v.y);
                look(v.z);
                look(v.w);
            }
            const int any = __syncthreads_or(odd);
            if (threadIdx.x == 0) odd_parts[static_cast<size_t>(blockIdx.y - 1) * num + a] = any;
            return;
        }
        const int per = ((M + kPlanWarps - 1) / kPlanWarps + 31) / 32 * 32;
        const int m0 = min(M, warp * per), m1 = min(M, m0 + per);
        int eq = 0, lt = 0;
#pragma unroll 4
        for (int m = m0 + lane; m < m1; m += 32) {
            const int v = adapter_of(index, m, num);
            eq += v == a;
            lt += v >= 0 && v < a;
        }
        eq = __reduce_add_sync(0xffffffffu, eq);
        lt = __reduce_add_sync(0xffffffffu, lt);
        if (lane == 0) {
            warp_eq[warp] = eq;
            warp_lt[warp] = lt;
        }
        __syncthreads();
        int start = 0, count = 0, before = 0;
#pragma unroll
        for (int w = 0; w < kPlanWarps; ++w) {
            start += warp_lt[w];
            before += w < warp ? warp_eq[w] : 0;
            count += warp_eq[w];
        }
        int at = start + before;
        for (int mb = m0; mb < m1; mb += 32) {
            const int m = mb + lane;
            const bool mine = m < m1 && adapter_of(index, m, num) == a;
            const unsigned votes = __ballot_sync(0xffffffffu, mine);
            const int to = at + __popc(votes & ((1u << lane) - 1u));
            if (mine && dcheck(to >= 0 && to < M, status)) perm[to] = m;
            at += __popc(votes);
        }
        const int first = start / kShrinkTokens + a;
        const int last = a + 1 == num ? num_blocks : (start + count) / kShrinkTokens + a + 1;
        for (int i = threadIdx.x; first + i < last; i += kPlanThreads)
            if (dcheck(first + i < num_blocks, status))
                blocks[first + i] = make_int4(a, start + i * kShrinkTokens, min(kShrinkTokens, count - i * kShrinkTokens), i == 0);
        if (threadIdx.x == 0) {
            seg[a] = start;
            if (a + 1 == num) seg[num] = start + count;
        }
        return;
    }
    if (blockIdx.y > 0) return;
    // ---- slots of one tile
    const int tile = blockIdx.x - num;
    __shared__ unsigned bits[kMaxAdapters / 32];
    __shared__ int base[kMaxAdapters / 32 + 1];
    const int words = (num + 31) / 32;
    for (int i = threadIdx.x; i < words; i += kPlanThreads) bits[i] = 0;
    __syncthreads();
    const int m0 = tile * tile_tokens, m1 = min(M, m0 + tile_tokens);
    for (int m = m0 + static_cast<int>(threadIdx.x); m < m1; m += kPlanThreads) {
        const int v = adapter_of(index, m, num);
        if (v >= 0) atomicOr(&bits[v >> 5], 1u << (v & 31));
    }
    __syncthreads();
    for (int i = threadIdx.x; i <= words; i += kPlanThreads) {
        int n = 0;
        for (int j = 0; j < i; ++j) n += __popc(bits[j]);
        base[i] = n;
    }
    __syncthreads();
    if (threadIdx.x == 0) tile_slots[tile] = base[words];
    for (int i = threadIdx.x; i < words; i += kPlanThreads) {
        unsigned b = bits[i];
        int at = base[i];
        for (; b; b &= b - 1, ++at)
            if (dcheck(at < slot_pitch, status)) slot_adapter[static_cast<size_t>(tile) * slot_pitch + at] = i * 32 + __ffs(b) - 1;
    }
    for (int m = m0 + static_cast<int>(threadIdx.x); m < m1; m += kPlanThreads) {
        const int v = adapter_of(index, m, num);
        token_slot[m] = v < 0 ? -1 : base[v >> 5] + __popc(bits[v >> 5] & ((1u << (v & 31)) - 1u));
    }
}

// ---------------------------------------------------------------------------------------------
// Gathered products on tcgen05: the common part of shrink and wgrad
// ---------------------------------------------------------------------------------------------
// Both multiply 128 rows by Rp <= 128 columns over a long reduction whose rows are gathered (the
// tokens of one adapter), and read their wide operand once, so they are bound by that stream. One
// warp gathers: each four lanes hold sixteen rows of a stage and ask for them as one box where they
// follow one another (the tokens of one request do), else four rows a lane by tile::gather4; both
// arrive swizzled as the MMA reads them. One thread issues the MMAs (bf16 x bf16, fp32 in tensor
// memory) and frees stages by commits. Slower forms that came before: warp-level MMAs with ldmatrix,
// bound by shared-memory reads (90 us for the two gradients of 4173 tokens x 9216 at rank 64, floor
// 18), 16-byte cp.async by eight warps, bound by the instructions that form their addresses (55 us),
// and gather4 alone, which takes about 80 clocks per 512 bytes (130 us).
constexpr int kWideBytes = 128 * 128;                        // 128 x 64 bf16
__host__ __device__ constexpr int gather_stage(int rp) { return kWideBytes + rp * 128; }

__device__ __forceinline__ void* shared_ptr(uint32_t a) {
    return reinterpret_cast<void*>(__cvta_shared_to_generic(a));
}
// Sixteen bytes of shared memory, read where this stands: an ordinary load whose value is used only later may
// take effect later, behind an arrival that hands the bytes back (in the tensor-memory product such loads
// read a stage that had been refilled).
__device__ __forceinline__ uint4 shared_now(const void* from) {
    uint4 v;
    asm volatile("ld.volatile.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(smem_u32(from))
                 : "memory");
    return v;
}
// Four rows of a 2-D tensor map whose box is one row high, to consecutive rows of shared memory.
// Rows outside the tensor arrive as zeros.
__device__ __forceinline__ void tma_gather4(const CUtensorMap* map, uint64_t* bar, uint32_t dst, int x, const int (&r)[4]) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cta.global.tile::gather4.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5, %6, %7}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3])
        : "memory");
}

// This lane's four rows `r` of a stage, to `dst`: sixteen rows held by four neighbouring lanes come as
// one box (of `box`, 16 rows high) if they follow one another, which gather_plan finds out (`valid`:
// whether all four rows are in the stage), else each lane gathers its own (`one`, one row high).
__device__ __forceinline__ bool gather_plan(const int (&r)[4], bool valid) {
    const int lane = threadIdx.x & 31;
    const int first = __shfl_sync(0xffffffffu, r[0], lane & ~3) + 4 * (lane & 3);
    const bool run = valid && r[0] == first && r[1] == first + 1 && r[2] == first + 2 && r[3] == first + 3;
    return ((__ballot_sync(0xffffffffu, run) >> (lane & ~3)) & 0xFu) == 0xFu;
}
__device__ __forceinline__ void gather_rows(const CUtensorMap* box, const CUtensorMap* one, uint64_t* bar, uint32_t dst,
                                            int x, const int (&r)[4], bool as_box) {
    if (!as_box) tma_gather4(one, bar, dst, x, r);
    else if ((threadIdx.x & 3) == 0) tma_load_2d(box, bar, shared_ptr(dst), x, r[0]);
}

struct GatherPipe {
    uint64_t* full;            // a stage's copies have landed (one expecting arrival)
    uint64_t* empty;           // its products have read it
    uint64_t* done;
    volatile int* abort_flag;
    unsigned* status;
};
__device__ __forceinline__ void gather_init(const GatherPipe& g, int stages, int readers) {
    for (int i = 0; i < stages; ++i) {
        mbar_init(&g.full[i], 1);
        mbar_init(&g.empty[i], readers);
    }
    mbar_init(g.done, 1);
    *g.abort_flag = 0;
}
// Ends the issuing thread's products: no MMA may be in flight when tensor memory is freed, whatever
// ended its loop.
__device__ __forceinline__ void gather_drain_mma(const GatherPipe& g) {
    mma_commit(g.done);
    const long long t0 = clock64();
    while (!mbar_try_wait(g.done, 0)) {
        if (clock64() - t0 > kWaitLimitCycles) {
            atomicOr(g.status, kDevErrTimeout);
            *g.abort_flag = 1;
            break;
        }
    }
}
// Waits (bounded) for the copies of the stages [from, to) still in flight before the CTA may exit.
template <int S>
__device__ __forceinline__ void gather_drain_copies(const GatherPipe& g, int from, int to) {
    for (int i = from; i < to; ++i) {
        const long long t0 = clock64();
        while (!mbar_try_wait(&g.full[i % S], (i / S) & 1u) && clock64() - t0 < kWaitLimitCycles) {
        }
    }
}

// The narrow operand as MN-major [64 reduction rows][Rp]: rows of up to 128 bytes; Rp = 128 is two
// such tiles of 64 columns, 8 KB apart.
template <int RP>
__device__ __forceinline__ uint64_t narrow_mn_desc(uint32_t tile, int k16) {
    constexpr int rb = RP < 64 ? RP * 2 : 128;
    return smem_desc_mn(tile + k16 * 16 * rb, rb, 8192);
}
template <int RP>
constexpr int kNarrowCols = RP < 64 ? RP : 64;

// ---------------------------------------------------------------------------------------------
// Shrink: partial[s][m][0..Rp) = in[m][slice s] * side_a[slice s]^T for the tokens of each block
// ---------------------------------------------------------------------------------------------
// A block is up to 128 tokens of one adapter (the MMA's 128 rows); the reduction is cut into
// slices over gridDim.y so that a few blocks fill the GPU, and the slices' fp32 partials are added
// by the pass that writes the slots' P (side_row). KMAJOR: the adapter's side is [R][red] (A); otherwise
// [red][R] (B). Bound by the stream of the input and, beside it from L2, of the adapter's side, once a
// block: 22 us cold for 4173 tokens x 9216 at rank 64 (3.7 TB/s of DRAM, 5.4 TB/s with L2).
// A block of at most 32 tokens (a decode batch of many adapters) brings so few bytes a stage that its
// ring is cut into stages of 32 rows and made deeper instead; the MMA's other 96 rows then read
// whatever follows, which stays in rows of the product that nobody stores.
constexpr int kFewTokens = 32;
constexpr int kShrinkThreads = 160;   // four warps that store, one of them gathering; one issuing MMAs
template <int RP>
constexpr int kShrinkStages = RP == 128 ? 3 : 4;
template <int RP>
constexpr int kShrinkFewStages = RP == 128 ? 4 : RP == 64 ? 6 : 8;
template <int RP>
constexpr int kShrinkRing = kShrinkStages<RP> * gather_stage(RP);
template <int RP>
constexpr int kShrinkSmem = 1024 + kShrinkRing<RP>;

struct ShrinkArgs {
    CUtensorMap map_in;        // the input as (red, M), boxes of 64 x 16
    CUtensorMap map_in1;       // the same, boxes of 64 x 1
    CUtensorMap map_side;      // A as (red, R, L), boxes of 64 x Rp, or B as (R, red, L), boxes of up to 64 x 64
    int M, red, kslice;
    const int* perm;
    const int4* blocks;
    const int* odd_parts;      // [slices][num] of the plan kernel
    int slices, num;
    int* bad;                  // [num]
    float* partial;
    unsigned* status;
};

// The stages of one block: ROWS token rows each, S stages. The gathering warp is warp 0, the issuing
// thread the first of warp 4.
template <int RP, bool KMAJOR, int ROWS, int S>
__device__ __forceinline__ void shrink_stages(const ShrinkArgs& p, const GatherPipe& g, const int* tok, int count,
                                              int adapter, uint32_t s0, uint32_t tmem) {
    constexpr int kXBytes = ROWS * 128, kStage = kXBytes + RP * 128;
    static_assert((S - 1) * kStage + kWideBytes <= kShrinkRing<RP> && S * kStage <= kShrinkRing<RP>, "ring");
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int k_begin = blockIdx.y * p.kslice, k_end = min(p.red, k_begin + p.kslice);
    const int steps = (k_end - k_begin + 63) / 64;
    if (warp == 0) {
        // this lane's four token rows (past the block's tokens the last one again, or nothing: whatever
        // those rows hold stays in their own rows of the product, which are not stored)
        const int groups = (count + 3) / 4;
        int rows[4] = {tok[4 * lane], tok[4 * lane + 1], tok[4 * lane + 2], tok[4 * lane + 3]};
        // (rows past the block's tokens may be any: the next ones, to make up a box)
        const int lead = tok[4 * (lane & ~3)] + 4 * (lane & 3);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (4 * lane + i >= count) rows[i] = lead + i;
        const bool as_box = gather_plan(rows, true);
        const bool asks = ROWS == 128 || lane < ROWS / 4 ? lane < groups || (as_box && (lane & ~3) < groups) : false;
        const int bytes = __popc(__ballot_sync(0xffffffffu, asks)) * 512 + RP * 128;
        int step = 0;
        for (; step < steps; ++step) {
            const int s = step % S;
            if (!__all_sync(0xffffffffu, mbar_wait(&g.empty[s], ((step / S) & 1u) ^ 1u, g.abort_flag, g.status))) break;
            if (lane == 0) mbar_arrive_expect_tx(&g.full[s], bytes);
            __syncwarp();
            const uint32_t st = s0 + s * kStage;
            const int k0 = k_begin + step * 64;
            if (asks) gather_rows(&p.map_in, &p.map_in1, &g.full[s], st + lane * 512, k0, rows, as_box);
            if (lane == 0) {
                uint8_t* ws = static_cast<uint8_t*>(shared_ptr(st + kXBytes));
                if (KMAJOR) {
                    tma_load_3d(&p.map_side, &g.full[s], ws, k0, 0, adapter);
                } else {
                    tma_load_3d(&p.map_side, &g.full[s], ws, 0, k0, adapter);
                    if (RP == 128) tma_load_3d(&p.map_side, &g.full[s], ws + 8192, 64, k0, adapter);
                }
            }
        }
        if (step < steps) gather_drain_copies<S>(g, max(0, step - S), step);
    } else if (threadIdx.x == 128) {
        constexpr uint32_t idesc = idesc_bf16_f32(128, RP) | (KMAJOR ? 0u : kIdescTransposeB);
        int step = 0;
        for (; step < steps; ++step) {
            const int s = step % S;
            if (!mbar_wait(&g.full[s], (step / S) & 1u, g.abort_flag, g.status)) break;
            tc_fence_after();
            const uint32_t st = s0 + s * kStage, ws = st + kXBytes;
#pragma unroll
            for (int k16 = 0; k16 < 4; ++k16)
                mma_f16_ss(tmem, smem_desc_k_sw128(st + k16 * 32),
                           KMAJOR ? smem_desc_k_sw128(ws + k16 * 32) : narrow_mn_desc<RP>(ws, k16), idesc,
                           step > 0 || k16 > 0 ? 1u : 0u);
            mma_commit(&g.empty[s]);
        }
        if (step > 0) gather_drain_mma(g);
    }
}

template <int RP, bool KMAJOR>
__global__ void __launch_bounds__(kShrinkThreads, 2) shrink_kernel(const __grid_constant__ ShrinkArgs p) {
    constexpr int S = kShrinkStages<RP>, F = kShrinkFewStages<RP>, kBars = S > F ? S : F;
    constexpr uint32_t kCols = RP < 32 ? 32 : RP;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    __shared__ uint64_t bars[2 * kBars + 1];
    __shared__ uint32_t tmem_holder;
    __shared__ int abort_word;
    __shared__ int tok[kShrinkTokens];
    const GatherPipe g = {bars, bars + kBars, bars + 2 * kBars, &abort_word, p.status};
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 128) {
        tma_prefetch_desc(&p.map_in);
        tma_prefetch_desc(&p.map_in1);
        tma_prefetch_desc(&p.map_side);
    }
    grid_dependency_wait();
    grid_launch_dependents();
    const int at = static_cast<int>(blockIdx.x) * kShrinkTokens;
    const int4 blk = p.blocks ? p.blocks[blockIdx.x] : make_int4(0, at, min(kShrinkTokens, p.M - at), 0);
    const int count = blk.z;
    if (count <= 0) return;
    if (tid < kShrinkTokens) {
        const int t = blk.y + min(tid, count - 1);
        const int m = !dcheck(t >= 0 && t < p.M, p.status) ? 0 : p.perm ? p.perm[t] : t;
        tok[tid] = dcheck(m >= 0 && m < p.M, p.status) ? m : 0;
    }
    if (blk.w && blockIdx.y == 0) {   // the adapter's first block: join the parts of its weight side's look-over
        int odd = 0;
        for (int i = tid; i < p.slices; i += kShrinkThreads) odd |= p.odd_parts[static_cast<size_t>(i) * p.num + blk.x];
        odd = __syncthreads_or(odd);
        if (tid == 0 && dcheck(blk.x >= 0 && blk.x < p.num, p.status)) p.bad[blk.x] = odd;
    }
    if (tid == 0) {
        gather_init(g, kBars, 1);
        fence_mbar_init();
    }
    if (warp == 4) {
        tmem_alloc(&tmem_holder, kCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_holder, s0 = smem_u32(smem);
    if (count <= kFewTokens)
        shrink_stages<RP, KMAJOR, kFewTokens, F>(p, g, tok, count, blk.x, s0, tmem);
    else
        shrink_stages<RP, KMAJOR, kShrinkTokens, S>(p, g, tok, count, blk.x, s0, tmem);
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp < 4 && warp * 32 < count && !*g.abort_flag) {   // warp w reads tensor-memory lanes 32 w ..: its tokens
        const int row = warp * 32 + lane;
        float* dst = p.partial + (static_cast<size_t>(blockIdx.y) * p.M + tok[row]) * RP;
#pragma unroll
        for (int c = 0; c < RP; c += 16) {
            uint32_t v[16];
            tmem_ld16(tmem + (static_cast<uint32_t>(warp * 32) << 16) + c, v);
            tmem_wait_ld();
            if (row < count) {
#pragma unroll
                for (int i = 0; i < 16; i += 4)
                    *reinterpret_cast<uint4*>(dst + c + i) = make_uint4(v[i], v[i + 1], v[i + 2], v[i + 3]);
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 4) {
        tc_fence_after();
        tmem_dealloc(tmem, kCols);
    }
}

// Shrink for up to 16 tokens, which may all have adapters of their own: p[m][r] for two ranks of one
// token per CTA, each of the four warps a quarter of the reduction, lanes on 16-byte pieces. It is
// bound by the latency of its loads (A's rows come from memory once; 1 MB or so), so it has no
// stages: every load of a warp's quarter is in flight at once for the usual widths. The result is
// final (scaled fp32): the small-M kernel reads it directly.
constexpr int kShrinkSmallWarps = 4;

__global__ void __launch_bounds__(32 * kShrinkSmallWarps)
    shrink_small_kernel(const uint4* __restrict__ in, const uint4* __restrict__ A, int K8, int R, int num,
                        const float* __restrict__ scaling, const int* __restrict__ index, float* __restrict__ p,
                        __nv_bfloat16* __restrict__ p_out) {
    grid_dependency_wait();
    grid_launch_dependents();   // (only now: the small-M kernel that follows reads X without waiting)
    const int m = blockIdx.y, r = 2 * blockIdx.x;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int a = adapter_of(index, m, num);
    float s0 = 0.f, s1 = 0.f, sc = 0.f;
    if (a >= 0) {
        sc = scaling[a];
        const uint4* x = in + static_cast<size_t>(m) * K8;
        const uint4* a0 = A + (static_cast<size_t>(a) * R + r) * K8;
        const uint4* a1 = a0 + K8;
        auto dot = [](uint32_t u, uint32_t v, float s) {
            s = fmaf(__uint_as_float(u << 16), __uint_as_float(v << 16), s);
            return fmaf(__uint_as_float(u & 0xFFFF0000u), __uint_as_float(v & 0xFFFF0000u), s);
        };
#pragma unroll 4
        for (int i = warp * 32 + lane; i < K8; i += 32 * kShrinkSmallWarps) {
            const uint4 u = __ldg(x + i), v = __ldg(a0 + i), w = __ldg(a1 + i);
            s0 = dot(u.x, v.x, dot(u.y, v.y, dot(u.z, v.z, dot(u.w, v.w, s0))));
            s1 = dot(u.x, w.x, dot(u.y, w.y, dot(u.z, w.z, dot(u.w, w.w, s1))));
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        s0 += __shfl_xor_sync(0xffffffffu, s0, o);
        s1 += __shfl_xor_sync(0xffffffffu, s1, o);
    }
    __shared__ float2 part[kShrinkSmallWarps];
    if (lane == 0) part[warp] = make_float2(s0, s1);
    __syncthreads();
    if (threadIdx.x < 2) {
        float s = 0.f;
#pragma unroll
        for (int w = 0; w < kShrinkSmallWarps; ++w) s += threadIdx.x ? part[w].y : part[w].x;
        s *= sc;
        const size_t at = static_cast<size_t>(m) * R + r + threadIdx.x;
        p[at] = s;
        if (p_out) p_out[at] = __float2bfloat16_rn(s);
    }
}

// ---------------------------------------------------------------------------------------------
// Copy pass: fp16 copy of the input, the slots' P, the kept p and the 8-bit copy
// ---------------------------------------------------------------------------------------------
// One CTA per token row, as the plain GEMM's conversion (the row's power of two 2^e comes from its
// largest |value|). P is multiplied by 2^-e as well, since the epilogue multiplies the whole sum
// by 2^e; that is exact in bf16. p (in the backward dp) itself is rounded to bf16 once as the MMA's
// operand: 2^-8 of each entry at most, like the output's own rounding, and there beside the larger
// product with W (2.0e-3 off in the norm against 64 bits where adapters weigh most, 1.7e-3 with p in fp32 as
// up to 16 tokens have it; a second term would double the slots' columns). dA has nothing beside it, so it gets dp in two bf16 terms, the second for what the first
// leaves (2^-16): with the first alone it was 2.4e-3 off in the norm against 64 bits, and more where a few
// large channels of x rule it, with both 1.7e-3, which is the rounding of the result.
struct SideArgs {
    const float* partial;      // [ksplit][M][Rp]
    int ksplit;
    int rp_log2, rank, num;
    const float* scaling;
    const int* index;
    const int* token_slot;
    const int* tile_slots;
    const int* bad;            // [num], nullptr: no index, nothing was looked over
    const int* slot_adapter;   // [token tile][slot_pitch]
    int* slot_side;            // the same with `num` for a bad adapter, for the product
    int slot_pitch;
    int tile_log2;
    __nv_bfloat16* pslots;
    long long p_cols;
    __nv_bfloat16* p_out;      // nullptr: not kept
    __nv_bfloat16* p_rest;     // what p_out's rounding leaves, or nullptr
    uint8_t* codes;            // 8-bit copy
    uint8_t* exps;
    bool beside;               // a copy without the slots' P that runs beside the shrink kernel
    unsigned* status;          // the device status word
};

// P of one token: the sum of the slices' partials, times its adapter's scaling, in its slot's columns and
// zeros in the tile's others. By T threads (`tid`), which `sync` joins; `scale`: the row's 2^-e. The sum's
// order is fixed by T and the rank: slice after slice, or (T == 32) strided over groups of lanes and then
// across them, so p's last bits may differ between batches that the copy pass and side_kernel handle.
template <int T, class Sync>
__device__ __forceinline__ void side_row(const SideArgs& s, int row, int M, float scale, int tid, float* prow, Sync sync) {
    const int slot = s.token_slot ? s.token_slot[row] : 0;
    const int cols = (s.tile_slots ? s.tile_slots[row >> s.tile_log2] : 1) << s.rp_log2;   // the columns the MMA reads
    const int a = adapter_of(s.index, row, s.num);
    const bool odd = s.bad && a >= 0 && s.bad[a];
    const float* part = s.partial + (static_cast<size_t>(row) << s.rp_log2);
    const size_t step = static_cast<size_t>(M) << s.rp_log2;
    auto keep = [&](int r, float p) {
        p = a < 0 ? 0.f : p * s.scaling[a];                      // (no adapter: its partials are not written)
        if (s.p_out && r < s.rank) {
            const __nv_bfloat16 h = __float2bfloat16_rn(p);
            const size_t at = static_cast<size_t>(row) * s.rank + r;
            s.p_out[at] = h;
            if (s.p_rest) {
                const float rest = p - __bfloat162float(h);
                s.p_rest[at] = __float2bfloat16_rn(isfinite(rest) ? rest : 0.f);   // (an infinity is all in the first)
            }
        }
        prow[r] = odd ? __int_as_float(0x7FC00000) : p;          // NaN
    };
    if (T == 32) {
        // four ranks a lane, and as many slices at once as the warp's lanes then hold
        const int log2 = s.rp_log2 - 2, r = (tid & ((1 << log2) - 1)) * 4;
        float4 p = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
        for (int k = tid >> log2; k < s.ksplit; k += 32 >> log2) {
            const float4 v = *reinterpret_cast<const float4*>(part + k * step + r);
            p = make_float4(p.x + v.x, p.y + v.y, p.z + v.z, p.w + v.w);
        }
        for (int o = 1 << log2; o < 32; o <<= 1) {
            p.x += __shfl_xor_sync(0xffffffffu, p.x, o);
            p.y += __shfl_xor_sync(0xffffffffu, p.y, o);
            p.z += __shfl_xor_sync(0xffffffffu, p.z, o);
            p.w += __shfl_xor_sync(0xffffffffu, p.w, o);
        }
        if (tid < 1 << log2) {
            keep(r, p.x);
            keep(r + 1, p.y);
            keep(r + 2, p.z);
            keep(r + 3, p.w);
        }
    } else if (tid < (1 << s.rp_log2)) {
        float p = 0.f;
#pragma unroll 8
        for (int k = 0; k < s.ksplit; ++k) p += part[k * step + tid];
        keep(tid, p);
    }
    sync();
    if (s.bad && (row & ((1 << s.tile_log2) - 1)) == 0) {        // a tile's first row: its slots' weight sides
        const size_t at = static_cast<size_t>(row >> s.tile_log2) * s.slot_pitch;
        for (int i = tid; i < cols >> s.rp_log2; i += T) {
            if (!dcheck(i < s.slot_pitch, s.status)) break;
            const int b = s.slot_adapter[at + i];
            if (dcheck(b >= 0 && b < s.num, s.status)) s.slot_side[at + i] = s.bad[b] ? s.num : b;
        }
    }
    uint4* pd = reinterpret_cast<uint4*>(s.pslots + static_cast<size_t>(row) * s.p_cols);
    for (int c = tid; c < cols / 8; c += T) {
        uint4 o = make_uint4(0, 0, 0, 0);
        if ((c * 8) >> s.rp_log2 == slot) {
            const float* pr = prow + ((c * 8) & ((1 << s.rp_log2) - 1));
            uint32_t u[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                // round p first (what p_out holds), then the exact power of two
                const float lo = __bfloat162float(__float2bfloat16_rn(pr[2 * q])) * scale;
                const float hi = __bfloat162float(__float2bfloat16_rn(pr[2 * q + 1])) * scale;
                const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
                u[q] = *reinterpret_cast<const uint32_t*>(&h);
            }
            o = make_uint4(u[0], u[1], u[2], u[3]);
        }
        if (dcheck(c * 8 + 8 <= s.p_cols && slot < s.slot_pitch, s.status)) pd[c] = o;
    }
}

constexpr int kConvThreads = 256;

// With adapters the row itself is copied before the wait for the shrink kernel, which runs meanwhile:
// that kernel let this one start only after everything earlier in the stream was complete.
//
// PER: 16-byte pieces of the row that a thread holds (0: any width, the row is read twice). 512 threads
// of four pieces instead of 256 of eight took 50 us instead of 41 for 4173 x 9216 with the 8-bit copy.
// LR: with the slots' P; CK: with the 8-bit copy. (A kernel each, so that the plain copy keeps the
// registers, and so the resident rows, that its bandwidth needs.)
template <int PER, bool LR, bool CK>
__global__ void __launch_bounds__(kConvThreads, 4)
    convert_side_kernel(const uint4* __restrict__ in, int M, int K8, int K8p, uint4* __restrict__ xh,
                        float* __restrict__ rowmul, const SideArgs s) {
    if (!LR) {
        if (!s.beside) grid_dependency_wait();
        grid_launch_dependents();
    }
    const int row = blockIdx.x, tid = threadIdx.x;
    const uint4* src = in + static_cast<size_t>(row) * K8;
    uint4* dst = xh + static_cast<size_t>(row) * K8p;
    uint4 v[PER > 0 ? PER : 1];
    if (PER > 0) {
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            const int i = tid + j * kConvThreads;
            v[j] = i < K8 ? ldg_nc_v4(src + i) : make_uint4(0, 0, 0, 0);
        }
    }
    uint32_t mx = 0;   // two running maxima of |value| bits, one per half word
    auto amax = [](const uint4& a, uint32_t m) {
        constexpr uint32_t kAbs = 0x7FFF7FFFu;
        return __vmaxs2(__vmaxs2(__vmaxs2(a.x & kAbs, a.y & kAbs), __vmaxs2(a.z & kAbs, a.w & kAbs)), m);
    };
    if (PER > 0) {
#pragma unroll
        for (int j = 0; j < PER; ++j) mx = amax(v[j], mx);
    } else {
        for (int i = tid; i < K8; i += kConvThreads) mx = amax(src[i], mx);
    }
    auto copy8 = [&](int i, const uint4& a, bool valid) {
        // four neighbouring lanes hold a block of 32 values (K8 is a multiple of 4)
        uint8_t ex;
        const uint2 c = checkpoint_encode8(a, ex);
        if (valid) {
            const size_t at = static_cast<size_t>(row) * K8 + i;
            reinterpret_cast<uint2*>(s.codes)[at] = c;
            if ((i & 3) == 0) s.exps[at >> 2] = ex;
        }
    };
    if (CK && PER > 0) {   // (before the row's maximum is known: it does not need it)
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            const int i = tid + j * kConvThreads;
            if (j * kConvThreads < K8) copy8(i, v[j], i < K8);
        }
    }
    mx = __reduce_max_sync(0xffffffffu, max(mx & 0xFFFFu, mx >> 16));
    __shared__ uint32_t warp_max[kConvThreads / 32];
    if ((tid & 31) == 0) warp_max[tid >> 5] = mx;
    __syncthreads();
    mx = 0;
#pragma unroll
    for (int w = 0; w < kConvThreads / 32; ++w) mx = max(mx, warp_max[w]);
    const int E = static_cast<int>(mx >> 7);              // biased exponent of the largest |value|
    int e = (mx == 0 || E >= 255) ? 0 : E - 142;          // largest * 2^-e in [2^15, 2^16)
    e = max(-100, min(112, e));
    const float scale = __int_as_float((127 - e) << 23);  // 2^-e
    const __nv_bfloat162 scale2 = __float2bfloat162_rn(scale);
    auto cvt = [&](uint32_t w) {   // (the product with a power of two is exact in bf16, or below fp16's range)
        const __nv_bfloat162 y = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&w), scale2);
        const uint32_t u = *reinterpret_cast<const uint32_t*>(&y);
        return pack_f16x2(__uint_as_float(u << 16), __uint_as_float(u & 0xFFFF0000u));
    };
    if (PER > 0) {
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            const int i = tid + j * kConvThreads;
            if (i < K8p) dst[i] = make_uint4(cvt(v[j].x), cvt(v[j].y), cvt(v[j].z), cvt(v[j].w));
        }
    } else {
        // (whole warps take part in every round: the 8-bit copy exchanges between lanes)
        const int rounds = (K8p + kConvThreads - 1) / kConvThreads;
        for (int j = 0; j < rounds; ++j) {
            const int i = tid + j * kConvThreads;
            const uint4 a = i < K8 ? src[i] : make_uint4(0, 0, 0, 0);
            if (i < K8p) dst[i] = make_uint4(cvt(a.x), cvt(a.y), cvt(a.z), cvt(a.w));
            if (CK) copy8(i, a, i < K8);
        }
    }
    if (tid == 0) rowmul[row] = __int_as_float((127 + e) << 23);   // 2^e
    if (LR) {
        __shared__ float prow[kMaxRank];
        grid_dependency_wait();
        grid_launch_dependents();   // (not earlier: what follows takes tensor memory, which that kernel needs first)
        side_row<kConvThreads>(s, row, M, scale, tid, prow, [] { __syncthreads(); });
    } else if (s.beside && row == 0) {
        grid_dependency_wait();     // what waits for this kernel waits for the shrink kernel as well
    }
}

// The slots' P by itself, a warp per token, after the copy of more rows than the GPU holds at once (about
// five an SM, whose copies would all wait for the shrink kernel before the next ones start). From 770 to
// 1000 tokens both ways take the same within 4 %, the kernel of its own 1 % less on average; below 700 it
// costs up to 7 % (one launch more), and 4173 tokens x 9216 gain 9 us of 536.
constexpr int kSideWarps = 8;
constexpr int kSideRows = 5 * kSmsAssumed;

__global__ void __launch_bounds__(32 * kSideWarps)
    side_kernel(int M, const float* __restrict__ rowmul, const SideArgs s) {
    grid_dependency_wait();
    grid_launch_dependents();
    __shared__ float prow[kSideWarps][kMaxRank];
    const int warp = threadIdx.x >> 5, row = blockIdx.x * kSideWarps + warp;
    if (row >= M) return;
    const float scale = __int_as_float((254 << 23) - __float_as_int(rowmul[row]));   // of 2^e the inverse
    side_row<32>(s, row, M, scale, threadIdx.x & 31, prow[warp], [] { __syncwarp(); });
}

// ---------------------------------------------------------------------------------------------
// Adapter gradients: dA_a[r][k] = sum dp[m][r] x[m][k], dB_a[n][r] = sum dy[m][n] p[m][r]
// ---------------------------------------------------------------------------------------------
// Both are the same product G^T P over an adapter's tokens, G = x or dy: A = G^T (128 columns of G,
// MN-major), B = P (MN-major), reduction over the tokens in stages of 64. Persistent CTAs walk tiles of
// both gradients and all adapters through one ring, with two accumulators, so that a tile's start and
// its stores lie under its neighbours' products. dA multiplies dp's two terms into one accumulator. x may
// be the 8-bit copy: eight warps widen a stage's codes into the MMA's tile (exactly). Bound by the stream
// of x and dy: beyond a start of some 15 us, 30 us per 151 MB of bf16 (5.0 TB/s, 0.77 of the copy rate; P
// comes from L2 on top), 56 us cold for three adapters of 1391 tokens x (9216 + 9216) at rank 64 with x in
// 8 bits, dp's second term 6 of them. Cutting the tokens of few tiles into slices that meet in a workspace
// cost 12 us a slice and gained nothing, nor did more stages.
// With dX it comes after the product and runs beside it: the product lets it start once the copy pass
// (all that it depends on) is complete, and it ends only when the product has. (After one another, wgrad
// first: 28.1 instead of 20.3 us for 77 tokens x 2560 x 2560, 565 instead of 533 for the 4173 tokens.)
struct WgradPart {
    const uint8_t* exps;       // the 8-bit copy's exponents, nullptr for a bf16 G
    __nv_bfloat16* out;        // [a][R][C] (dA) or [a][C][R] (dB)
    int C;
    int tiles;                 // ceil(C / 128)
};
struct WgradArgs {
    // of dA and dB: G as (C, M), boxes of 64 bf16 or 128 codes, and P as (R, M), boxes of up to 64, by
    // 64 rows (a whole stage), 16 rows and 1 row
    CUtensorMap map_g[3][2], map_p[3][2], map_rest[3];   // (map_rest: dp's second term)
    WgradPart part[2];         // dA, dB
    int R, M, num;
    bool beside;               // the kernel before is the product, which this one runs beside
    const int* perm;
    const int* seg;
    unsigned* status;
};
constexpr int kWgradWideners = 8;
constexpr int kWgradThreads = 32 * (6 + kWgradWideners);   // warp 0 gathers, 1 issues MMAs, then widen, 4 store
template <int RP>
constexpr int kWgradCtas = RP == 128 ? 1 : 2;              // per SM
template <int RP>
constexpr int kWgradStages = RP == 16 ? 5 : RP == 64 ? 3 : 4;
constexpr int kRawBytes = 64 * 128;               // 64 tokens x 128 codes, in the second half of G's tile
__host__ __device__ constexpr int wgrad_stage(int rp) { return gather_stage(rp) + rp * 128; }
template <int RP>
constexpr int kWgradSmem = 1024 + kWgradStages<RP> * wgrad_stage(RP);

template <int RP>
__global__ void __launch_bounds__(kWgradThreads, kWgradCtas<RP>) wgrad_kernel(const __grid_constant__ WgradArgs w) {
    constexpr int S = kWgradStages<RP>, kStage = wgrad_stage(RP);
    constexpr uint32_t kAcc = RP, kCols = 2 * kAcc < 32 ? 32 : 2 * kAcc;
    static_assert(kWgradCtas<RP> * (kWgradSmem<RP> + 2048) <= 228 * 1024, "shared memory");
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    __shared__ uint64_t bars[2 * S + 1], taken[S], wide[S], accfull[2], accempty[2];
    __shared__ uint32_t tmem_holder;
    __shared__ int abort_word;
    const GatherPipe g = {bars, bars + S, bars + 2 * S, &abort_word, w.status};
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        gather_init(g, S, 1 + kWgradWideners);
        for (int i = 0; i < S; ++i) {
            mbar_init(&taken[i], kWgradWideners);
            mbar_init(&wide[i], kWgradWideners);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&accfull[i], 1);
            mbar_init(&accempty[i], 4);
            tma_prefetch_desc(&w.map_g[0][i]);
            tma_prefetch_desc(&w.map_p[0][i]);
        }
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc(&tmem_holder, kCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_holder, s0 = smem_u32(smem);
    if (!w.beside) grid_dependency_wait();
    grid_launch_dependents();
    const int tiles = w.part[0].tiles + w.part[1].tiles;
    const int64_t items = static_cast<int64_t>(tiles) * w.num, stride = gridDim.x;
    // Item -> 128 columns of one part for one adapter. Its segment's bounds are the only loads; they are
    // asked for an item ahead.
    struct Item {
        int a, part, c0, seg0, count;
        __device__ int steps() const { return (count + 63) / 64; }
    };
    auto item_of = [&](int64_t i) {
        Item it = {0, 0, 0, 0, 0};
        if (i < items) {
            const int y = static_cast<int>(i % tiles);
            it.a = static_cast<int>(i / tiles);
            it.part = y < w.part[0].tiles ? 0 : 1;
            it.c0 = (it.part ? y - w.part[0].tiles : y) * 128;
            it.seg0 = w.seg ? w.seg[it.a] : 0;
            it.count = (w.seg ? w.seg[it.a + 1] : it.a == 0 ? w.M : 0) - it.seg0;
        }
        return it;
    };
    auto token_of = [&](const Item& it, int t) {
        if (!dcheck(it.seg0 >= 0 && it.seg0 + t < w.M, w.status)) return 0;
        const int m = w.perm ? w.perm[it.seg0 + t] : t;
        return dcheck(m >= 0 && m < w.M, w.status) ? m : 0;
    };
    if (warp == 0) {
        // ---------------------------------------------------------------- gather
        // lane -> token rows 4 (lane % 16) .. + 3 of a stage, columns 64 (lane / 16) .. of G
        const int row = 4 * (lane & 15), half = lane >> 4;
        auto rows_of = [&](const Item& it, int step, int (&r)[4]) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int t = step * 64 + row + i;
                r[i] = t >= it.count ? w.M : token_of(it, t);   // (row M: zeros)
            }
        };
        // the stage whose rows are asked for next, two ahead of the one that is copied
        int64_t ai = blockIdx.x;
        int astep = -1;
        Item aitem = item_of(ai), anext = item_of(ai + stride);
        auto rows_ahead = [&](int (&r)[4]) {
            if (++astep >= aitem.steps()) {
                astep = 0;
                do {
                    ai += stride;
                    aitem = anext;
                    anext = item_of(ai + stride);
                } while (ai < items && aitem.steps() == 0);
            }
            rows_of(aitem, astep, r);
        };
        int it = 0, rows[4], rows1[4];
        bool ok = true;
        if (aitem.steps() == 0) astep = 0;   // (moves on to the first item with tokens)
        rows_ahead(rows);
        rows_ahead(rows1);
        Item next = item_of(blockIdx.x);
        for (int64_t i = blockIdx.x; ok && i < items; i += stride) {
            const Item cur = next;
            next = item_of(i + stride);
            const int steps = cur.steps();
            const bool q8 = w.part[cur.part].exps != nullptr, dA = cur.part == 0;
            for (int step = 0; step < steps; ++step, ++it) {
                int rows2[4];
                rows_ahead(rows2);
                const int s = it % S;
                const bool as_box = gather_plan(rows, step * 64 + row + 4 <= cur.count);
                // whether all 64 rows follow one another: one request for each 64 columns then
                const int first = __shfl_sync(0xffffffffu, rows[0], 0);
                const bool as_stage = __all_sync(0xffffffffu, as_box && rows[0] == first + row);
                if (!(ok = __all_sync(0xffffffffu, mbar_wait(&g.empty[s], ((it / S) & 1u) ^ 1u, g.abort_flag, g.status)))) break;
                if (lane == 0) mbar_arrive_expect_tx(&g.full[s], (q8 ? kRawBytes : kWideBytes) + (dA ? 2 : 1) * RP * 128);
                __syncwarp();
                const uint32_t st = s0 + s * kStage, rw = st + kWideBytes - kRawBytes, ps = st + kWideBytes;
                if (as_stage) {
                    if ((lane & 15) == 0) {
                        if (!q8) tma_load_2d(&w.map_g[0][cur.part], &g.full[s], shared_ptr(st + half * 8192), cur.c0 + half * 64, first);
                        else if (half == 0) tma_load_2d(&w.map_g[0][cur.part], &g.full[s], shared_ptr(rw), cur.c0, first);
                        if (half == 0 || RP == 128) {
                            tma_load_2d(&w.map_p[0][cur.part], &g.full[s], shared_ptr(ps + half * 8192), half * 64, first);
                            if (dA) tma_load_2d(&w.map_rest[0], &g.full[s], shared_ptr(ps + RP * 128 + half * 8192), half * 64, first);
                        }
                    }
                } else {
                    const CUtensorMap *mg = &w.map_g[1][cur.part], *mg1 = &w.map_g[2][cur.part];
                    if (!q8) gather_rows(mg, mg1, &g.full[s], st + half * 8192 + row * 128, cur.c0 + half * 64, rows, as_box);
                    else if (half == 0) gather_rows(mg, mg1, &g.full[s], rw + row * 128, cur.c0, rows, as_box);
                    // P: rows of kNarrowCols columns, a second tile of 64 for Rp = 128
                    if (half == 0 || RP == 128) {
                        const uint32_t to = ps + half * 8192 + row * kNarrowCols<RP> * 2;
                        gather_rows(&w.map_p[1][cur.part], &w.map_p[2][cur.part], &g.full[s], to, half * 64, rows, as_box);
                        if (dA) gather_rows(&w.map_rest[1], &w.map_rest[2], &g.full[s], to + RP * 128, half * 64, rows, as_box);
                    }
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    rows[j] = rows1[j];
                    rows1[j] = rows2[j];
                }
            }
        }
        if (!ok) gather_drain_copies<S>(g, max(0, it - S), it);
    } else if (warp == 1) {
        // ---------------------------------------------------------------- MMA issuer
        if (lane == 0) {
            constexpr uint32_t idesc = idesc_bf16_f32(128, RP) | kIdescTransposeA | kIdescTransposeB;
            int it = 0, n = 0;
            uint32_t wide_phase = 0;                 // bit s: the phase that slot s's widening completes next
            bool ok = true;
            Item next = item_of(blockIdx.x);
            for (int64_t i = blockIdx.x; ok && i < items; i += stride) {
                const int steps = next.steps();
                const bool q8 = w.part[next.part].exps != nullptr, dA = next.part == 0;
                next = item_of(i + stride);
                if (steps == 0) continue;
                const int b = n & 1;
                if (!(ok = mbar_wait(&accempty[b], ((n >> 1) & 1u) ^ 1u, g.abort_flag, g.status))) break;
                tc_fence_after();
                for (int step = 0; step < steps; ++step, ++it) {
                    const int s = it % S;
                    if (!(ok = mbar_wait(&g.full[s], (it / S) & 1u, g.abort_flag, g.status))) break;
                    if (q8) {
                        if (!(ok = mbar_wait(&wide[s], (wide_phase >> s) & 1u, g.abort_flag, g.status))) break;
                        wide_phase ^= 1u << s;
                    }
                    tc_fence_after();
                    const uint32_t st = s0 + s * kStage;
#pragma unroll
                    for (int k16 = 0; k16 < 4; ++k16)
                        mma_f16_ss(tmem + b * kAcc, smem_desc_mn(st + k16 * 2048, 128, 8192),
                                   narrow_mn_desc<RP>(st + kWideBytes, k16), idesc, step > 0 || k16 > 0 ? 1u : 0u);
                    if (dA) {
#pragma unroll
                        for (int k16 = 0; k16 < 4; ++k16)
                            mma_f16_ss(tmem + b * kAcc, smem_desc_mn(st + k16 * 2048, 128, 8192),
                                       narrow_mn_desc<RP>(st + kWideBytes + RP * 128, k16), idesc, 1u);
                    }
                    mma_commit(&g.empty[s]);
                }
                if (!ok) break;
                mma_commit(&accfull[b]);
                ++n;
            }
            if (it > 0) gather_drain_mma(g);
        }
    } else if (warp < 2 + kWgradWideners) {
        // ---------------------------------------------------------------- widen 8-bit stages
        // thread -> 16 columns (chunk tid % 8) of token rows tid / 8 + 32 i; row ids come two stages and
        // exponents one stage ahead
        constexpr int kRowsOf = 64 * 8 / (32 * kWgradWideners), kStep = 64 / kRowsOf;
        const int wt = tid - 64, ch = wt & 7, row0 = wt >> 3;
        int it = 0;
        uint32_t taken_phase = 0;                    // bit s: the phase that slot s's taking completes next
        Item next = item_of(blockIdx.x);
        bool ok = true;
        for (int64_t i = blockIdx.x; ok && i < items; i += stride) {
            const Item cur = next;
            next = item_of(i + stride);
            const int steps = cur.steps();
            const WgradPart& part = w.part[cur.part];
            if (part.exps == nullptr) {
                // nothing to do but to keep in step with the ring: a warp that fell behind or ran ahead by
                // two of a slot's fills would take one for the other
                for (int step = 0; step < steps; ++step, ++it) {
                    const int s = it % S;
                    if (!(ok = __all_sync(0xffffffffu, mbar_wait(&g.full[s], (it / S) & 1u, g.abort_flag, g.status)))) break;
                    if (lane == 0) mbar_arrive(&g.empty[s]);
                }
                continue;
            }
            const bool c_ok = cur.c0 + ch * 16 < part.C;
            auto ids_of = [&](int step, int (&id)[kRowsOf]) {
#pragma unroll
                for (int j = 0; j < kRowsOf; ++j) {
                    const int t = step * 64 + row0 + kStep * j;
                    id[j] = t < cur.count && c_ok ? token_of(cur, t) : -1;
                }
            };
            auto exps_of = [&](const int (&id)[kRowsOf], uint32_t (&e)[kRowsOf]) {
#pragma unroll
                for (int j = 0; j < kRowsOf; ++j)
                    e[j] = id[j] >= 0 ? part.exps[static_cast<size_t>(id[j]) * (part.C / 32) + (cur.c0 + ch * 16) / 32] : 0;
            };
            int id[kRowsOf];
            uint32_t e[kRowsOf];
            ids_of(0, id);
            exps_of(id, e);
            ids_of(1, id);
            for (int step = 0; step < steps; ++step, ++it) {
                const int s = it % S;
                uint32_t e_next[kRowsOf];
                exps_of(id, e_next);
                ids_of(step + 2, id);
                if (!(ok = __all_sync(0xffffffffu, mbar_wait(&g.full[s], (it / S) & 1u, g.abort_flag, g.status)))) break;
                uint8_t *tile = smem + s * kStage, *half = tile + (ch >> 2) * 8192;
                uint4 c[kRowsOf];
#pragma unroll
                for (int j = 0; j < kRowsOf; ++j)
                    c[j] = shared_now(tile + kWideBytes - kRawBytes + (row0 + kStep * j) * 128 + ch * 16);
                // the codes lie where their values go: every warp has to have taken its own
                __syncwarp();
                if (lane == 0) mbar_arrive(&taken[s]);
                if (!(ok = __all_sync(0xffffffffu, mbar_wait(&taken[s], (taken_phase >> s) & 1u, g.abort_flag, g.status)))) break;
                taken_phase ^= 1u << s;
#pragma unroll
                for (int j = 0; j < kRowsOf; ++j) {
                    const int row = row0 + kStep * j;
                    uint8_t* dst = half + row * 128;
                    *reinterpret_cast<uint4*>(dst + ((((2 * ch) & 7) ^ (row & 7)) << 4)) =
                        checkpoint_decode8(make_uint2(c[j].x, c[j].y), e[j]);
                    *reinterpret_cast<uint4*>(dst + ((((2 * ch + 1) & 7) ^ (row & 7)) << 4)) =
                        checkpoint_decode8(make_uint2(c[j].z, c[j].w), e[j]);
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&wide[s]);
                    mbar_arrive(&g.empty[s]);
                }
#pragma unroll
                for (int j = 0; j < kRowsOf; ++j) e[j] = e_next[j];
            }
        }
    } else {
        // ---------------------------------------------------------------- stores: lane = column of G
        const int quarter = warp & 3, R = w.R;
        int n = 0;
        Item next = item_of(blockIdx.x);
        for (int64_t i = blockIdx.x; i < items; i += stride) {
            const Item it = next;
            next = item_of(i + stride);
            const bool some = it.count > 0, first = it.part == 0;
            __nv_bfloat16* out = w.part[it.part].out;
            const int C = w.part[it.part].C, c = it.c0 + quarter * 32 + lane, b = n & 1;
            if (some) {
                if (!__all_sync(0xffffffffu, mbar_wait(&accfull[b], (n >> 1) & 1u, g.abort_flag, g.status))) break;
                tc_fence_after();
            }
#pragma unroll
            for (int r0 = 0; r0 < RP; r0 += 16) {
                if (r0 >= R) break;
                uint32_t v[16] = {};
                if (some) {
                    tmem_ld16(tmem + b * kAcc + (static_cast<uint32_t>(quarter * 32) << 16) + r0, v);
                    tmem_wait_ld();
                }
                uint32_t u[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const __nv_bfloat162 h = __floats2bfloat162_rn(__uint_as_float(v[2 * j]), __uint_as_float(v[2 * j + 1]));
                    u[j] = *reinterpret_cast<const uint32_t*>(&h);
                }
                if (first) {
                    // dA [a][R][C]: neighbouring lanes swap halves, so that each stores two columns of one rank
                    const bool even = (lane & 1) == 0;
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const uint32_t other = __shfl_xor_sync(0xffffffffu, u[j], 1);
                        const uint32_t word = even ? __byte_perm(u[j], other, 0x5410) : __byte_perm(other, u[j], 0x7632);
                        const int r = r0 + 2 * j + (even ? 0 : 1), ce = c & ~1;
                        if (r < R && ce < C && dcheck(it.a < w.num && ce >= 0 && ce + 1 < C, w.status))
                            *reinterpret_cast<uint32_t*>(out + (static_cast<size_t>(it.a) * R + r) * C + ce) = word;
                    }
                } else if (c < C && dcheck(it.a < w.num && c >= 0 && r0 + 8 <= R, w.status)) {
                    // dB [a][C][R]: eight ranks a store
                    uint4* dst = reinterpret_cast<uint4*>(out + (static_cast<size_t>(it.a) * C + c) * R + r0);
                    dst[0] = make_uint4(u[0], u[1], u[2], u[3]);
                    if (r0 + 8 < R) dst[1] = make_uint4(u[4], u[5], u[6], u[7]);
                }
            }
            if (some) {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&accempty[b]);
                ++n;
            }
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, kCols);
    }
    grid_dependency_wait();   // what waits for this kernel waits for the product before it as well
}

// ---------------------------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------------------------
template <class... Args, class... Given>
lowbit_status launch_pdl(void (*kernel)(Args...), dim3 grid, int threads, int smem, cudaStream_t stream, Given... args) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attrs[1];
    attrs[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attrs[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attrs;
    cfg.numAttrs = 1;
    if (take_injected_failure(kInjectLaunch)) return LOWBIT_ERR_CUDA;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<Args>(args)...) == cudaSuccess ? LOWBIT_OK : LOWBIT_ERR_CUDA;
}

// Allows `fn` its dynamic shared memory, once per device (`devices`: one bit per device that has it).
template <class F>
bool allow_smem(F fn, int bytes, std::atomic<uint64_t>& devices) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return false;
    const uint64_t bit = dev < 64 ? (uint64_t(1) << dev) : 0;
    if (bit && (devices.load(std::memory_order_acquire) & bit)) return true;
    if (cudaFuncSetAttribute(reinterpret_cast<const void*>(fn), cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) !=
        cudaSuccess)
        return false;
    devices.fetch_or(bit, std::memory_order_acq_rel);
    return true;
}

// Map of a [rows][cols] row-major tensor, boxes of `box` columns x `high` rows.
bool make_map_rows(CUtensorMap* map, CUtensorMapDataType type, int elem, const void* base, int64_t cols, int64_t rows, int box,
                   int high, CUtensorMapSwizzle swz) {
    return make_map_2d(map, type, elem, base, cols, rows, static_cast<uint64_t>(cols) * elem, box, high, swz);
}
CUtensorMapSwizzle swizzle_of(int bytes) {
    return bytes == 32 ? CU_TENSOR_MAP_SWIZZLE_32B : bytes == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B;
}

template <int RP, bool KMAJOR>
lowbit_status shrink_launch(const ExtProblem& e, const ExtBuffers& b, cudaStream_t stream) {
    const ExtWorkspace& w = b.w;
    auto fn = shrink_kernel<RP, KMAJOR>;
    static std::atomic<uint64_t> devices{0};
    ShrinkArgs p;
    p.status = device_status_address();
    if (!p.status || !allow_smem(fn, kShrinkSmem<RP>, devices)) return LOWBIT_ERR_CUDA;
    const uint64_t in = KMAJOR ? e.red : e.ad.rank, mid = KMAJOR ? e.ad.rank : e.red;
    const uint64_t dims[3] = {in, mid, static_cast<uint64_t>(e.ad.num)};
    const uint64_t strides[2] = {in * 2, in * mid * 2};
    constexpr uint32_t cols = KMAJOR ? 64 : kNarrowCols<RP>;
    const uint32_t box[3] = {cols, KMAJOR ? RP : 64, 1};
    const CUtensorMapDataType bf16 = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    if (!make_map_rows(&p.map_in, bf16, 2, e.in, e.red, e.M, 64, 16, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !make_map_rows(&p.map_in1, bf16, 2, e.in, e.red, e.M, 64, 1, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !make_map_3d(&p.map_side, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, e.grad ? e.ad.B : e.ad.A, dims, strides, box,
                     swizzle_of(cols * 2)))
        return LOWBIT_ERR_CUDA;
    p.M = static_cast<int>(e.M);
    p.red = static_cast<int>(e.red);
    p.kslice = static_cast<int>(w.kslice);
    p.perm = e.ad.index ? b.at<int>(w.perm) : nullptr;
    p.blocks = e.ad.index ? b.at<int4>(w.blocks) : nullptr;
    p.odd_parts = b.at<int>(w.odd_parts);
    p.slices = w.plan_slices;
    p.num = e.ad.num;
    p.bad = b.at<int>(w.bad);
    p.partial = b.at<float>(w.partial);
    const int64_t num_blocks = e.ad.index ? w.num_blocks : (e.M + kShrinkTokens - 1) / kShrinkTokens;
    return launch_pdl(fn, dim3(static_cast<unsigned>(num_blocks), static_cast<unsigned>(w.ksplit), 1), kShrinkThreads,
                      kShrinkSmem<RP>, stream, p);
}

template <int RP>
lowbit_status wgrad_launch(const WgradProblem& g, WgradArgs& a, cudaStream_t stream) {
    auto fn = wgrad_kernel<RP>;
    static std::atomic<uint64_t> devices{0};
    if (!allow_smem(fn, kWgradSmem<RP>, devices)) return LOWBIT_ERR_CUDA;
    constexpr int cols = kNarrowCols<RP>;
    const CUtensorMapDataType bf16 = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, u8 = CU_TENSOR_MAP_DATA_TYPE_UINT8;
    bool ok = true;
    for (int k = 0; k < 3; ++k) {
        const int high = k == 0 ? 64 : k == 1 ? 16 : 1;
        CUtensorMap *mg = a.map_g[k], *mp = a.map_p[k];
        ok = ok &&
             (g.x ? make_map_rows(&mg[0], bf16, 2, g.x, g.K, g.M, 64, high, CU_TENSOR_MAP_SWIZZLE_128B)
                  : make_map_rows(&mg[0], u8, 1, g.ck_codes, g.K, g.M, 128, high, CU_TENSOR_MAP_SWIZZLE_NONE)) &&
             make_map_rows(&mg[1], bf16, 2, g.dy, g.N, g.M, 64, high, CU_TENSOR_MAP_SWIZZLE_128B) &&
             make_map_rows(&mp[0], bf16, 2, g.dp, g.rank, g.M, cols, high, swizzle_of(cols * 2)) &&
             make_map_rows(&a.map_rest[k], bf16, 2, g.dp_rest, g.rank, g.M, cols, high, swizzle_of(cols * 2)) &&
             make_map_rows(&mp[1], bf16, 2, g.p, g.rank, g.M, cols, high, swizzle_of(cols * 2));
    }
    if (!ok) return LOWBIT_ERR_CUDA;
    const int64_t items = static_cast<int64_t>(a.part[0].tiles + a.part[1].tiles) * g.num, slots = kWgradCtas<RP> * num_sms();
    return launch_pdl(fn, dim3(static_cast<unsigned>(items < slots ? items : slots), 1, 1), kWgradThreads,
                      kWgradSmem<RP>, stream, a);
}

}  // namespace

namespace {

// Tokens per tile and K slices of the product. The time of a launch is modelled as
//   waves * blocks per slice * t(tile) + the slices' reduction s(tile),
// a block being 128 of the reduction (slot columns included: as many adapters as a tile's tokens
// would hold drawn at random), with t and s fitted to B200 sweeps over tiles, slices, M = 24 .. 1537
// and the text encoder's and square widths (in us: a tile of 32 / 64 / 128 / 256 tokens takes 0.42 /
// 0.5 / 0.68 / 0.82 per block and 1.5 / 2 / 3 / 9 for a reduction, 3 more where two split 64-token
// tiles share an SM). The model's choice is mostly within 10 % of the best of each sweep; a rule on
// M alone left 30-40 % at M = 100 .. 200 (4096 x 4096 at 203 tokens: 29.8 us unsplit, 21.1 as 128
// tokens x 2 slices).
constexpr int kTileTokens[4] = {32, 64, 128, 256};
void choose_tile(int64_t M, int64_t rows, int64_t red, int num, int rank, int* tile, int* split) {
    static constexpr double kBlockUs[4] = {0.42, 0.5, 0.68, 0.82}, kSplitUs[4] = {1.5, 2.0, 3.0, 9.0};
    static constexpr double kSharedUs[4] = {0.0, 3.0, 0.0, 0.0};
    // clusters of ks CTAs, one per SM, that the GPU's processing clusters hold at once (a B200 said 45, 33,
    // 26, 22, 15 and 15 from three CTAs on, others have their SMs spread differently; one too many here
    // costs a second wave: 53 instead of 40 us for 945 tokens x 7680 -> 384)
    static constexpr int kClusters[9] = {0, kSmsAssumed, 74, 44, 32, 24, 21, 15, 15};
    double best = 0;
    *tile = 0;
    for (int i = 0; i < 4; ++i) {
        const int bt = kTileTokens[i];
        if (bt < 256 && M > 16 * bt) continue;   // (small tiles of many tokens re-read W too often)
        const int64_t tiles = (M + bt - 1) / bt * ((rows + 127) / 128);
        double slots = 0;
        if (num > 0) {
            const double tokens = M < bt ? M : bt;
            slots = num * -std::expm1(-tokens / num);
        }
        const double blocks = static_cast<double>((red + 127) / 128) + slots * (1 << slot_log2(rank)) / 128;
        for (int ks = 1; ks <= 8; ++ks) {
            if (ks > 1 && blocks < 3 * ks) break;
            const int cap = kClusters[ks];
            double t = kBlockUs[i], waves;
            if (bt <= 64 && tiles > cap) {   // two CTAs per SM, which share its issue slots
                waves = static_cast<double>((tiles + 2 * cap - 1) / (2 * cap));
                t *= 1.5;
            } else {
                waves = static_cast<double>((tiles + cap - 1) / cap);
            }
            if (ks > 1 && waves > 1) continue;   // (a split grid is not persistent)
            const double us = waves * std::ceil(blocks / ks) * t + (ks > 1 ? kSplitUs[i] : 0.0) +
                              (ks > 1 && tiles > cap ? kSharedUs[i] : 0.0);
            if (!*tile || us < best) {
                best = us;
                *tile = bt;
                *split = ks;
            }
        }
    }
}

// K slices of the shrink kernel: one wave of two CTAs per SM over the blocks that hold tokens. (Slices down to
// 64 of K: at least 256 each took 28.9 us against 24.8 for 306 tokens of K = 512 that do not follow one
// another, 39.4 against 36.2 for the backward of 879 tokens, and nothing more anywhere but 1 us in 45.)
constexpr int kMaxSlices = 16;
int64_t shrink_slices(int64_t M, int64_t red64, int num) {
    const int64_t busy = M / kShrinkTokens + (num < M ? num : M);
    int64_t ks = 2 * kSmsAssumed / (busy > 0 ? busy : 1);
    if (ks > red64 / 64) ks = red64 / 64;
    if (ks > kMaxSlices) ks = kMaxSlices;
    return ks < 1 ? 1 : ks;
}

// The parts of the workspace one after another, of `slots` slots in all tiles and `partial_rows` rows of
// partials in all K slices.
void lay_out(ExtWorkspace& w, int64_t M, int64_t rows, int num, int rank, int64_t slots, int64_t partial_rows) {
    size_t at = 0;
    auto take = [&](size_t bytes) {
        const size_t o = at;
        at += (bytes + 255) / 256 * 256;
        return o;
    };
    w.xh = take(static_cast<size_t>(M) * w.red64 * 2);
    w.rowmul = take(static_cast<size_t>(M) * 4);
    if (num > 0) {
        const int rp = 1 << slot_log2(rank);
        w.num_blocks = M / kShrinkTokens + num + 1;
        w.p_cols = (w.slot_pitch * rp + 63) / 64 * 64;
        w.perm = take(static_cast<size_t>(M) * 4);
        w.seg = take((static_cast<size_t>(num) + 1) * 4);
        w.blocks = take(static_cast<size_t>(w.num_blocks) * 16);
        w.tile_slots = take(static_cast<size_t>(w.m_tiles) * 4);
        w.slot_adapter = take(static_cast<size_t>(slots) * 4);
        w.slot_side = take(static_cast<size_t>(slots) * 4);
        w.token_slot = take(static_cast<size_t>(M) * 4);
        // CTAs per adapter of the plan kernel: about four per SM in all, 32 KB of the weight side each
        const int64_t parts = (rows * rank / 8 + 2047) / 2048;
        w.plan_slices = static_cast<int>(4 * kSmsAssumed / num < parts ? 4 * kSmsAssumed / num : parts);
        if (w.plan_slices > 64) w.plan_slices = 64;
        if (w.plan_slices < 1) w.plan_slices = 1;
        w.odd_parts = take(static_cast<size_t>(w.plan_slices) * num * 4);
        w.bad = take(static_cast<size_t>(num) * 4);
        w.partial = take(static_cast<size_t>(partial_rows) * rp * 4);
        w.pslots = take(static_cast<size_t>(M) * w.p_cols * 2);
        w.p = take(static_cast<size_t>(M) * rank * 2);
        w.p_rest = take(static_cast<size_t>(M) * rank * 2);
    }
    w.total = at;
}

}  // namespace

ExtWorkspace ext_workspace(int64_t M, int64_t rows, int64_t red, int num, int rank) {
    ExtWorkspace w = {};
    w.red64 = (red + 63) / 64 * 64;
    choose_tile(M, rows, red, num, rank, &w.tile_tokens, &w.product_split);
    w.m_tiles = (M + w.tile_tokens - 1) / w.tile_tokens;
    if (num > 0) {
        w.slot_pitch = num < w.tile_tokens ? num : w.tile_tokens;
        const int64_t ks = shrink_slices(M, w.red64, num);
        w.kslice = ((w.red64 + ks - 1) / ks + 63) / 64 * 64;
        if (w.kslice < 64) w.kslice = 64;   // (an empty reduction)
        w.ksplit = static_cast<int>((w.red64 + w.kslice - 1) / w.kslice);
    }
    lay_out(w, M, rows, num, rank, w.m_tiles * w.slot_pitch, w.ksplit * M);
    return w;
}

// The largest workspace of up to M tokens. A longer batch may get narrower tiles (fewer slots of P each) or
// fewer K slices of the shrink kernel, so the size for M itself falls here and there as M grows; the bound
// takes each part that depends on them at its most, and the others grow with M.
size_t ext_workspace_bound(int64_t M, int64_t rows, int64_t red, int num, int rank) {
    ExtWorkspace w = {};
    w.red64 = (red + 63) / 64 * 64;
    w.m_tiles = (M + kTileTokens[0] - 1) / kTileTokens[0];
    int64_t slots = 0, partial_rows = M;
    for (int bt : kTileTokens) {
        w.slot_pitch = num < bt ? num : bt;   // (the last one, of the widest tile, stays)
        const int64_t n = (M + bt - 1) / bt * w.slot_pitch;
        if (n > slots) slots = n;
    }
    // k slices are taken up to the M where `busy` (see shrink_slices) passes 2 * kSmsAssumed / k
    for (int64_t k = 2; k <= kMaxSlices && k <= w.red64 / 64; ++k) {
        const int64_t busy = 2 * kSmsAssumed / k, past = (busy - num) * kShrinkTokens + kShrinkTokens - 1;
        int64_t m = past > busy ? past : busy;
        if (m > M) m = M;
        if (k * m > partial_rows) partial_rows = k * m;
    }
    lay_out(w, M, rows, num, rank, slots, partial_rows);
    return w.total;
}

lowbit_status launch_plan(const ExtProblem& e, const ExtBuffers& b, cudaStream_t stream) {
    const ExtWorkspace& w = b.w;
    unsigned* status = device_status_address();
    if (!status) return LOWBIT_ERR_CUDA;
    return launch_pdl(plan_kernel, dim3(static_cast<unsigned>(e.ad.num + w.m_tiles), 1 + w.plan_slices, 1), kPlanThreads, 0,
                      stream, e.ad.index, static_cast<int>(e.M), e.ad.num, w.tile_tokens, static_cast<int>(w.slot_pitch),
                      static_cast<int>(w.num_blocks), static_cast<const uint4*>(e.grad ? e.ad.A : e.ad.B),
                      e.rows * e.ad.rank / 8, b.at<int>(w.perm), b.at<int>(w.seg), b.at<int4>(w.blocks),
                      b.at<int>(w.tile_slots), b.at<int>(w.slot_adapter), b.at<int>(w.token_slot), b.at<int>(w.odd_parts),
                      status);
}

lowbit_status launch_shrink(const ExtProblem& e, const ExtBuffers& b, cudaStream_t stream) {
    switch (slot_log2(e.ad.rank)) {
        case 4: return e.grad ? shrink_launch<16, false>(e, b, stream) : shrink_launch<16, true>(e, b, stream);
        case 5: return e.grad ? shrink_launch<32, false>(e, b, stream) : shrink_launch<32, true>(e, b, stream);
        case 6: return e.grad ? shrink_launch<64, false>(e, b, stream) : shrink_launch<64, true>(e, b, stream);
        default: return e.grad ? shrink_launch<128, false>(e, b, stream) : shrink_launch<128, true>(e, b, stream);
    }
}

lowbit_status launch_shrink_small(const ExtProblem& e, float* p, cudaStream_t stream) {
    return launch_pdl(shrink_small_kernel, dim3(e.ad.rank / 2, static_cast<unsigned>(e.M), 1), 32 * kShrinkSmallWarps, 0,
                      stream, static_cast<const uint4*>(e.in), static_cast<const uint4*>(e.ad.A),
                      static_cast<int>(e.red / 8), e.ad.rank, e.ad.num, e.ad.scaling, e.ad.index, p,
                      static_cast<__nv_bfloat16*>(e.p_out));
}

lowbit_status launch_convert(const ExtProblem& e, const ExtBuffers& b, cudaStream_t stream) {
    const ExtWorkspace& w = b.w;
    SideArgs s = {};
    if (e.ad.num > 0) {
        s.status = device_status_address();
        if (!s.status) return LOWBIT_ERR_CUDA;
        s.partial = b.at<float>(w.partial);
        s.ksplit = w.ksplit;
        s.rp_log2 = slot_log2(e.ad.rank);
        s.rank = e.ad.rank;
        s.num = e.ad.num;
        s.scaling = e.ad.scaling;
        s.index = e.ad.index;
        s.token_slot = e.ad.index ? b.at<int>(w.token_slot) : nullptr;
        s.tile_slots = e.ad.index ? b.at<int>(w.tile_slots) : nullptr;
        s.bad = e.ad.index ? b.at<int>(w.bad) : nullptr;
        s.slot_adapter = b.at<int>(w.slot_adapter);
        s.slot_side = b.at<int>(w.slot_side);
        s.slot_pitch = static_cast<int>(w.slot_pitch);
        while ((1 << s.tile_log2) < w.tile_tokens) ++s.tile_log2;
        s.pslots = b.at<__nv_bfloat16>(w.pslots);
        s.p_cols = w.p_cols;
        s.p_out = static_cast<__nv_bfloat16*>(e.p_out);
        s.p_rest = e.grad ? b.at<__nv_bfloat16>(w.p_rest) : nullptr;
    }
    s.codes = e.ck_codes;
    s.exps = e.ck_exps;
    const int K8 = static_cast<int>(e.red / 8), K8p = static_cast<int>(w.red64 / 8);
    const dim3 grid(static_cast<unsigned>(e.M), 1, 1);
    const uint4* in = static_cast<const uint4*>(e.in);
    uint4* xh = b.at<uint4>(w.xh);
    float* rm = b.at<float>(w.rowmul);
    auto go = [&](auto fn) {
        return launch_pdl(fn, grid, kConvThreads, 0, stream, in, static_cast<int>(e.M), K8, K8p, xh, rm, s);
    };
    auto pick = [&](auto lr, auto ck) {
        constexpr bool LR = decltype(lr)::value, CK = decltype(ck)::value;
        if (K8p <= kConvThreads) return go(convert_side_kernel<1, LR, CK>);
        if (K8p <= 2 * kConvThreads) return go(convert_side_kernel<2, LR, CK>);
        if (K8p <= 4 * kConvThreads) return go(convert_side_kernel<4, LR, CK>);
        if (K8p <= 8 * kConvThreads) return go(convert_side_kernel<8, LR, CK>);
        return go(convert_side_kernel<0, LR, CK>);
    };
    if (e.ad.num == 0) return pick(std::false_type{}, std::false_type{});   // (the 8-bit copy comes with adapters only)
    if (e.M <= kSideRows) return s.codes ? pick(std::true_type{}, std::true_type{}) : pick(std::true_type{}, std::false_type{});
    s.beside = true;
    const lowbit_status st = s.codes ? pick(std::false_type{}, std::true_type{}) : pick(std::false_type{}, std::false_type{});
    if (st != LOWBIT_OK) return st;
    return launch_pdl(side_kernel, dim3(static_cast<unsigned>((e.M + kSideWarps - 1) / kSideWarps), 1, 1), 32 * kSideWarps, 0,
                      stream, static_cast<int>(e.M), rm, s);
}

lowbit_status launch_wgrad(const WgradProblem& g, const ExtBuffers& b, cudaStream_t stream) {
    WgradArgs a = {};
    a.part[0].exps = g.x ? nullptr : g.ck_exps;
    a.part[0].out = static_cast<__nv_bfloat16*>(g.dA);
    a.part[0].C = static_cast<int>(g.K);
    a.part[0].tiles = static_cast<int>((g.K + 127) / 128);
    a.part[1].out = static_cast<__nv_bfloat16*>(g.dB);
    a.part[1].C = static_cast<int>(g.N);
    a.part[1].tiles = static_cast<int>((g.N + 127) / 128);
    a.R = g.rank;
    a.M = static_cast<int>(g.M);
    a.num = g.num;
    a.beside = g.beside_product;
    a.perm = g.planned ? b.at<int>(b.w.perm) : nullptr;
    a.seg = g.planned ? b.at<int>(b.w.seg) : nullptr;
    a.status = device_status_address();
    if (!a.status) return LOWBIT_ERR_CUDA;
    switch (slot_log2(g.rank)) {
        case 4: return wgrad_launch<16>(g, a, stream);
        case 5: return wgrad_launch<32>(g, a, stream);
        case 6: return wgrad_launch<64>(g, a, stream);
        default: return wgrad_launch<128>(g, a, stream);
    }
}

}  // namespace lowbit
