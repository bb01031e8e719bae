// The logits' products of vocab_gemm.cuh for up to 128 tokens of a packed table, the other way round: a tile is 256 rows of
// the vocabulary (the lanes of tensor memory of a CTA pair, 128 each) by the tokens, so that the decoded weights go into
// tensor memory as the MMA's first operand and never through shared memory. With the tokens on the lanes a stage of 64
// columns moved 16 KB of decoded weights into shared memory and 32 KB out of it for the MMA, which took 700 clocks (ternary;
// uint4, of two terms, 1000) where the MMAs need 256. Here shared memory holds the tokens only, half of them in each CTA,
// and a stage takes 500 (840): 77 tokens against 32768 x 2560 uint4 in 45 us with all launches (53 before; 48 with the
// terms' sums apart), a sixth of what memory and tensor cores would allow. It is the decoding warps' chain of waits and
// latencies that is left, not the MMAs (one instead of four a stage: 450 clocks), the barriers (half as many: the same)
// nor the width of the loads of words (128 bytes of a row at a time: the same). Without the decoding's arithmetic a uint4
// stage takes 515.
//
//   * warp 8 (one lane): TMA of the CTA's half of the tokens, 64 columns a stage;
//   * warp 10 (one lane): TMA of the words and scales of its 128 rows x 128 columns;
//   * warps 11-18: decode, a row of 64 codes per lane, into tensor memory;
//   * warp 9 (one lane of the first CTA): tcgen05.mma, two accumulators;
//   * warps 0-7: the epilogue, 32 rows x 32 tokens at a time, a row per lane. What belongs to a token (its maximum, its
//     sum) is joined over the lanes by exchanging halves: 31 shuffles leave each lane one token's.
#pragma once

#include "vocab_gemm.cuh"

namespace lowbit {
namespace vocab {

constexpr int kFewTokens = 128;

template <int MODE, int BITS>
struct FewCfg {
    static_assert(MODE == kVocabStats || MODE == kVocabGrad, "the logits' products");
    static constexpr int kTerms = BITS == 4 ? 2 : 1;
    static constexpr int kThreads = 32 * (kEpiWarps + 3 + 8);
    static constexpr int kWRowBytes = 128 * BITS / 8;
    static constexpr int kWBytes = 128 * kWRowBytes;
    static constexpr int kSBytes = 2 * 128 * 2;                  // room for two groups
    static constexpr int kZBytes = BITS == 4 ? kSBytes : 0;
    static constexpr int kWStageBytes = (kWBytes + kSBytes + kZBytes + 1023) / 1024 * 1024;
    static constexpr int kWStages = BITS == 4 ? 8 : 12;          // some 50 KB of uint4 or ternary words under way
    static constexpr int kXStageBytes = kFewTokens / 2 * 128;
    static constexpr int kXStages = 8;
    static constexpr int kACol0 = 2 * kFewTokens, kACols = 32 * kTerms, kAStages = (512 - kACol0) / kACols;
    static constexpr int kStagingBytes = MODE == kVocabGrad ? kEpiWarps * 2048 : 0;   // fp16 [32 tokens][32 rows] a warp
    static constexpr int kWOff = kXStages * kXStageBytes;
    static constexpr int kStagingOff = kWOff + kWStages * kWStageBytes;
    static constexpr int kTokenOff = kStagingOff + kStagingBytes;                     // rl, shift, label by token; off by warp
    static constexpr int kBarOff = kTokenOff + 3 * kFewTokens * 4 + kEpiWarps * 32 * 4;
    static constexpr int kUsed = 1024 + kBarOff + 1024;
    static constexpr int kSmemBytes = kUsed > kSmemLimit / 2 + 1024 ? kUsed : kSmemLimit / 2 + 1024;
    static_assert(kSmemBytes <= kSmemLimit, "one CTA per SM (tensor memory)");
};

// x[j] of every lane joined over the lanes: lane j gets x[j]'s.
template <class Op>
__device__ __forceinline__ float across(float (&x)[32], int lane, Op op) {
#pragma unroll
    for (int o = 16; o > 0; o /= 2) {
        const bool up = lane & o;
#pragma unroll
        for (int i = 0; i < o; ++i) {
            const float got = __shfl_xor_sync(0xffffffffu, up ? x[i] : x[i + o], o);
            x[i] = op(up ? x[i + o] : x[i], got);
        }
    }
    return x[0];
}

template <int MODE, int BITS>
__global__ void __launch_bounds__(FewCfg<MODE, BITS>::kThreads, 1)
    vocab_few_kernel(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_w,
                     const __grid_constant__ CUtensorMap map_s, const __grid_constant__ CUtensorMap map_z,
                     const __grid_constant__ CUtensorMap map_out, const __grid_constant__ Params p) {
    using C = FewCfg<MODE, BITS>;
    constexpr int S = C::kXStages, SA = C::kAStages, SW = C::kWStages, T = C::kTerms;

    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kBarOff);
    uint64_t* empty = full + S;
    uint64_t* afull = empty + S;      // the decoded weights' ring
    uint64_t* aempty = afull + SA;
    uint64_t* wfull = aempty + SA;
    uint64_t* wempty = wfull + SW;
    uint64_t* accfull = wempty + SW;
    uint64_t* accempty = accfull + 2;
    uint64_t* drain = accempty + 2;
    uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(drain + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const bool issuer = rank == 0;
    auto on_issuer = [&](uint64_t* bar) { return map_shared_rank(smem_u32(bar), 0); };
    auto arrive_on_issuer = [&](uint64_t* bar) {
        if (!issuer)
            mbar_arrive_remote(on_issuer(bar));
        else
            mbar_arrive(bar);
    };

    if (threadIdx.x == 0) {
        for (int i = 0; i < S; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < SA; ++i) {
            mbar_init(&afull[i], 2 * 4);   // four decoding warps of either CTA
            mbar_init(&aempty[i], 1);
        }
        for (int i = 0; i < SW; ++i) {
            mbar_init(&wfull[i], 1);
            mbar_init(&wempty[i], 8);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&accfull[i], 1);
            mbar_init(&accempty[i], 2 * kEpiWarps);
        }
        mbar_init(drain, 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 8 && lane == 0) {
        tma_prefetch_desc(&map_x);
        tma_prefetch_desc(&map_w);
        tma_prefetch_desc(&map_s);
    }
    if (warp == 9) {
        tmem_alloc<true>(tmem_holder, 512);
        tmem_relinquish<true>();
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();   // both CTAs' barriers are initialised before either uses the other's
    tc_fence_after();
    const uint32_t tmem_base = *tmem_holder;
    grid_launch_dependents();
    grid_dependency_wait();

    const int tile0 = static_cast<int>(blockIdx.x >> 1), tile_step = static_cast<int>(gridDim.x >> 1);
    auto row0_of = [&](int t) { return 256 * t + static_cast<int>(rank) * 128; };   // this CTA's first row, within the piece
    const int half_tokens = p.a_rows;                                               // of the CTA's half: a multiple of 16
    // Two accumulators of 128 columns in turn; uint4 keeps the terms' sums apart (as vocab_kernel does), in two of 64
    // columns each, or for more tokens in one of 128.
    const bool wide = T == 2 && half_tokens > 32;
    const uint32_t bufs = wide ? 1 : 2, term = T == 1 ? 0 : wide ? kFewTokens : kFewTokens / 2;

    if (warp == 8) {
        // ------------------------------------------------------------ TMA of the tokens
        if (elect_one()) {
            uint32_t it = 0;
            bool ok = true;
            for (int t = tile0; t < p.num_tiles && ok; t += tile_step) {
                for (int j = 0; j < p.stages; ++j, ++it) {
                    const uint32_t s = it % S;
                    if (!mbar_wait(&empty[s], ((it / S) & 1u) ^ 1u, abort_flag, p.status)) { ok = false; break; }
                    if (issuer) mbar_arrive_expect_tx(&full[s], 2 * half_tokens * 128);
                    tma_load_2d_pair(&map_x, on_issuer(&full[s]), smem + s * C::kXStageBytes, j * 64,
                                     static_cast<int>(rank) * half_tokens);
                }
            }
            if (!ok) {
                // Wait (bounded) for the copies still in flight before the CTA exits. The second CTA of a pair cannot
                // wait on the issuer's barrier that its copies count on: it gives them a fixed time instead.
                if (!issuer) {
                    const long long t0 = clock64();
                    while (clock64() - t0 < kWaitLimitCycles / 64) {
                    }
                } else {
                    for (uint32_t j = it > static_cast<uint32_t>(S) ? it - S : 0u; j < it; ++j) {
                        const long long t0 = clock64();
                        while (!mbar_try_wait(&full[j % S], (j / S) & 1u) && clock64() - t0 < kWaitLimitCycles / 64) {
                        }
                    }
                }
            }
        }
    } else if (warp == 9) {
        // ------------------------------------------------------------ MMA issuer
        if (issuer && elect_one()) {
            const uint32_t idesc = idesc_f16_f32(256, 2 * half_tokens);
            uint32_t it = 0, n = 0;
            bool ok = true, issued = false;
            for (int t = tile0; t < p.num_tiles && ok; t += tile_step, ++n) {
                const uint32_t b = wide ? 0u : n & 1u;
                if (!mbar_wait(&accempty[b], ((n / bufs) & 1u) ^ 1u, abort_flag, p.status)) { ok = false; break; }
                tc_fence_after();
                const uint32_t d = tmem_base + b * kFewTokens;
                for (int j = 0; j < p.stages; ++j, ++it) {
                    const uint32_t s = it % S, a = it % SA;
                    if (!mbar_wait(&full[s], (it / S) & 1u, abort_flag, p.status) ||
                        !mbar_wait(&afull[a], (it / SA) & 1u, abort_flag, p.status)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t xs = smem_u32(smem + s * C::kXStageBytes), wa = tmem_base + C::kACol0 + a * C::kACols;
#pragma unroll
                    for (int i = 0; i < 4 * T; ++i)
                        mma_f16_ts_pair(d + (i >> 2) * term, wa + i * 8, smem_desc_k_sw128(xs + (i & 3) * 32), idesc,
                                        (j > 0 || (i & 3) > 0) ? 1u : 0u);
                    issued = true;
                    mma_commit_pair_mc(&empty[s], 0x3);
                    mma_commit_pair_mc(&aempty[a], 0x3);
                }
                if (!ok) break;
                mma_commit_pair_mc(&accfull[b], 0x3);
            }
            if (!ok && issued) {   // no MMA may still write tensor memory when it is freed
                mma_commit_pair(drain);
                const long long t0 = clock64();
                while (!mbar_try_wait(drain, 0) && clock64() - t0 < kWaitLimitCycles / 64) {
                }
            }
        }
    } else if (warp == 10) {
        // ------------------------------------------------------------ TMA of words and scales
        if (elect_one()) {
            uint32_t it = 0;
            bool ok = true;
            for (int t = tile0; t < p.num_tiles && ok; t += tile_step) {
                const int v = p.v0 + row0_of(t);
                for (int w = 0; w < p.stages / 2; ++w, ++it) {
                    const uint32_t s = it % SW;
                    if (!mbar_wait(&wempty[s], ((it / SW) & 1u) ^ 1u, abort_flag, p.status)) { ok = false; break; }
                    uint8_t* st = smem + C::kWOff + s * C::kWStageBytes;
                    mbar_arrive_expect_tx(&wfull[s], p.wtx);
                    tma_load_2d(&map_w, &wfull[s], st, w * (4 * BITS), v);
                    tma_load_2d(&map_s, &wfull[s], st + C::kWBytes, v, w * p.groups);
                    if (BITS == 4) tma_load_2d(&map_z, &wfull[s], st + C::kWBytes + C::kSBytes, v, w * p.groups);
                }
            }
            if (!ok) {
                for (uint32_t j = it > static_cast<uint32_t>(SW) ? it - SW : 0u; j < it; ++j) {
                    const long long t0 = clock64();
                    while (!mbar_try_wait(&wfull[j % SW], (j / SW) & 1u) && clock64() - t0 < kWaitLimitCycles / 64) {
                    }
                }
            }
        }
    } else if (warp >= 11) {
        // ------------------------------------------------------------ decoding warps
        const int half = (warp - 11) >> 2;               // which 64 of a row's 128 codes
        const int quarter = warp & 3, row = quarter * 32 + lane;   // (a warp reaches its own quarter of the lanes)
        const uint32_t lane_base = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) + C::kACol0;
        uint32_t wit = 0;
        bool ok = true;
        for (int t = tile0; t < p.num_tiles && ok; t += tile_step) {
            for (int w = 0; w < p.stages / 2; ++w, ++wit) {
                const uint32_t ws = wit % SW;
                if (!__all_sync(0xffffffffu, mbar_wait(&wfull[ws], (wit / SW) & 1u, abort_flag, p.status))) { ok = false; break; }
                const uint8_t* st = smem + C::kWOff + ws * C::kWStageBytes;
                const int at = (p.groups == 2 ? half : 0) * 128 + row;
                Row64<BITS, T> codes;
                codes.load(st + row * C::kWRowBytes, row, half, reinterpret_cast<const uint16_t*>(st + C::kWBytes)[at],
                           BITS == 4 ? reinterpret_cast<const uint16_t*>(st + C::kWBytes + C::kSBytes)[at] : uint16_t(0));
                const uint32_t i = 2 * wit + half, a = i % SA;
                if (!__all_sync(0xffffffffu, mbar_wait(&aempty[a], ((i / SA) & 1u) ^ 1u, abort_flag, p.status))) { ok = false; break; }
                tc_fence_after();
                uint32_t out[32], rest[32];
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    uint32_t hi[4], lo[4];
                    codes.piece(c, hi, lo);
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        out[4 * c + q] = hi[q];
                        if (T == 2) rest[4 * c + q] = lo[q];
                    }
                }
                tmem_st32(lane_base + a * C::kACols, out);
                if (T == 2) tmem_st32(lane_base + a * C::kACols + 32, rest);
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    arrive_on_issuer(&afull[a]);
                    mbar_arrive(&wempty[ws]);   // (freed behind the last use of what was read from it)
                }
            }
        }
    } else {
        // ------------------------------------------------------------ epilogue
        const int quarter = warp & 3;
        const uint32_t lane_base = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16);
        float* rl = reinterpret_cast<float*>(smem + C::kTokenOff);   // log2(e) times what a token's products are to be scaled by
        float* shift = rl + kFewTokens;                              // log2(e) lse
        int* label = reinterpret_cast<int*>(shift + kFewTokens);     // -1: none
        float* off = reinterpret_cast<float*>(label + kFewTokens) + warp * 32;
        for (int m = threadIdx.x; m < kFewTokens; m += 32 * kEpiWarps) {
            const bool in = m < p.M;
            const int l = in ? p.labels[m] : -1;
            label[m] = static_cast<unsigned>(l) < static_cast<unsigned>(p.vocab) ? l : -1;
            rl[m] = in ? p.rowmul[m] * p.evened * kLog2e : 0.f;
            if (MODE == kVocabGrad) shift[m] = in ? p.lse[m] * kLog2e : 0.f;
        }
        named_bar_sync(1, 32 * kEpiWarps);
        uint32_t n = 0;
        for (int t = tile0; t < p.num_tiles; t += tile_step, ++n) {
            const uint32_t b = wide ? 0u : n & 1u;
            const int first = row0_of(t) + quarter * 32;    // the warp's first row, within the piece
            const int row = p.v0 + first + lane;
            const bool live = row < p.vocab;
            if (!__all_sync(0xffffffffu, mbar_wait(&accfull[b], (n / bufs) & 1u, abort_flag, p.status))) break;
            tc_fence_after();
#pragma unroll 1
            for (int m0 = 32 * (warp >> 2); m0 < p.M; m0 += 64) {
                uint32_t v[32];
                tmem_ld32(lane_base + b * kFewTokens + m0, v);
                if constexpr (T == 2) {
                    uint32_t w[32];
                    tmem_ld32(lane_base + b * kFewTokens + term + m0, w);
                    tmem_wait_ld();
#pragma unroll
                    for (int j = 0; j < 32; ++j) v[j] = __float_as_uint(__uint_as_float(v[j]) + __uint_as_float(w[j]));
                } else {
                    tmem_wait_ld();
                }
                const float4* rl4 = reinterpret_cast<const float4*>(rl + m0);
                if constexpr (MODE == kVocabStats) {
                    const int m = m0 + lane;                 // the token that this lane ends up with
                    float x[32];
#pragma unroll
                    for (int j = 0; j < 32; ++j) x[j] = live ? __uint_as_float(v[j]) : -INFINITY;
                    const float top = across(x, lane, [](float a, float c) { return fmaxf(a, c); });
                    // An infinite maximum stands aside: with no row at all the sum is 0, with +inf it is +inf.
                    const bool inf = fabsf(top) == INFINITY;
                    off[lane] = inf ? 0.f : -top * rl[m];
                    const int at = label[m] - (p.v0 + first);
                    uint32_t hit = __ballot_sync(0xffffffffu, label[m] >= 0 && at >= 0 && at < 32);
                    while (hit) {                            // a token whose label is one of these rows
                        const int k = __ffs(hit) - 1;
                        hit &= hit - 1;
                        float l = 0.f;
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            if (j == k) l = __uint_as_float(v[j]);
                        l = __shfl_sync(0xffffffffu, l, __shfl_sync(0xffffffffu, at, k));
                        if (lane == 0) p.target[m0 + k] = l * (p.rowmul[m0 + k] * p.evened);
                    }
                    __syncwarp();
                    const float4* off4 = reinterpret_cast<const float4*>(off);
#pragma unroll
                    for (int q = 0; q < 8; ++q) {
                        const float4 r = rl4[q], o = off4[q];
                        x[4 * q] = ex2(fmaf(__uint_as_float(v[4 * q]), r.x, o.x));
                        x[4 * q + 1] = ex2(fmaf(__uint_as_float(v[4 * q + 1]), r.y, o.y));
                        x[4 * q + 2] = ex2(fmaf(__uint_as_float(v[4 * q + 2]), r.z, o.z));
                        x[4 * q + 3] = ex2(fmaf(__uint_as_float(v[4 * q + 3]), r.w, o.w));
                    }
                    if (!live) {
#pragma unroll
                        for (int j = 0; j < 32; ++j) x[j] = 0.f;
                    }
                    const float s = across(x, lane, [](float a, float c) { return a + c; });
                    if (m < p.M) {
                        const float r = inf ? (top > 0.f ? 3.4e38f : -INFINITY) : top * (p.rowmul[m] * p.evened);
                        p.part[static_cast<size_t>(first / 32) * p.M + m] = make_float2(r, s);
                    }
                    __syncwarp();
                } else {
                    __half* staging = reinterpret_cast<__half*>(smem + C::kStagingOff + warp * 2048);
                    const float4* shift4 = reinterpret_cast<const float4*>(shift + m0);
                    const int4* label4 = reinterpret_cast<const int4*>(label + m0);
                    if (lane == 0) bulk_wait_read_all();     // the previous store has read the staging rows
                    __syncwarp();
#pragma unroll
                    for (int q = 0; q < 8; ++q) {
                        const float4 r = rl4[q], o = shift4[q];
                        const int4 l = label4[q];
                        const float rs[4] = {r.x, r.y, r.z, r.w}, os[4] = {o.x, o.y, o.z, o.w};
                        const int ls[4] = {l.x, l.y, l.z, l.w};
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            float g = ex2(fmaf(__uint_as_float(v[4 * q + k]), rs[k], -os[k]));
                            if (ls[k] == row) g -= 1.f;
                            staging[(4 * q + k) * 32 + lane] = __float2half_rn(ls[k] >= 0 && live ? g * p.gscale : 0.f);
                        }
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        tma_store_2d(&map_out, staging, first, m0);
                        bulk_commit_group();
                    }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) arrive_on_issuer(&accempty[b]);
        }
        if (MODE == kVocabGrad && lane == 0) bulk_wait_read_all();
    }

    __syncwarp();
    tc_fence_before();
    __syncthreads();
    // a pair's tensor memory is freed by both CTAs together, once neither uses it (and no remote arrival or copy of
    // one CTA targets the other after it has exited)
    cluster_sync_all();
    if (warp == 9) {
        tc_fence_after();
        tmem_dealloc<true>(tmem_base, 512);
    }
}

template <int MODE, int BITS>
lowbit_status launch_few(const VocabProduct& v, cudaStream_t stream) {
    using C = FewCfg<MODE, BITS>;
    auto kernel = vocab_few_kernel<MODE, BITS>;
    const void* fn = reinterpret_cast<const void*>(kernel);
    if (!opt_in<MODE, BITS, true, true>(fn, C::kSmemBytes)) return LOWBIT_ERR_CUDA;
    const LossProblem& q = *v.p;
    const LossLayout& l = *v.l;
    const Table& w = q.table;
    const uint64_t M = q.M, K = w.K, vocab = q.vocab;
    const uint32_t half = static_cast<uint32_t>((M + 31) / 32 * 16), groups = 128 / w.group_size;
    const CUtensorMapDataType f16 = CU_TENSOR_MAP_DATA_TYPE_FLOAT16, u16 = CU_TENSOR_MAP_DATA_TYPE_UINT16;
    const CUtensorMapSwizzle none = CU_TENSOR_MAP_SWIZZLE_NONE;
    CUtensorMap mx, mw, ms, mz, mo;
    bool ok = make_map_2d(&mx, f16, 2, v.ws + l.xh, K, M, K * 2, 64, half, CU_TENSOR_MAP_SWIZZLE_128B);
    ok = ok && make_map_2d(&mw, CU_TENSOR_MAP_DATA_TYPE_UINT32, 4, w.rows, K * BITS / 32, vocab, K * BITS / 8, C::kWRowBytes / 4, 128,
                           word_swizzle(C::kWRowBytes));
    ok = ok && make_map_2d(&ms, u16, 2, w.scales, vocab, K / w.group_size, static_cast<uint64_t>(w.N) * 2, 128, groups, none);
    mz = ms;
    if (BITS == 4) ok = ok && make_map_2d(&mz, u16, 2, w.zeros, vocab, K / w.group_size, static_cast<uint64_t>(w.N) * 2, 128, groups, none);
    mo = mx;
    if (MODE == kVocabGrad) ok = ok && make_map_2d(&mo, f16, 2, v.ws + l.g, l.piece, M, l.piece * 2, 32, 32, none);
    Params p = {};
    p.status = device_status_address();
    if (!ok || !p.status) return LOWBIT_ERR_CUDA;
    p.M = static_cast<int>(M);
    p.vocab = static_cast<int>(vocab);
    p.v0 = static_cast<int>(v.v0);
    p.a_rows = static_cast<int>(half);
    p.groups = static_cast<int>(groups);
    p.wtx = static_cast<uint32_t>(C::kWBytes + (BITS == 4 ? 2 : 1) * p.groups * 256);
    p.stages = static_cast<int>((K + 127) / 128 * 2);
    p.num_tiles = static_cast<int>((v.cols + 255) / 256);
    p.evened = evened(p.stages);
    p.rowmul = reinterpret_cast<const float*>(v.ws + l.rowmul);
    p.labels = q.labels;
    p.lse = q.lse;
    p.part = reinterpret_cast<float2*>(v.ws + l.part);
    p.target = reinterpret_cast<float*>(v.ws + l.target);
    p.gscale = 32768.f;

    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attrs[2];
    attrs[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attrs[0].val.programmaticStreamSerializationAllowed = 1;
    attrs[1].id = cudaLaunchAttributeClusterDimension;
    attrs[1].val.clusterDim.x = 2;
    attrs[1].val.clusterDim.y = 1;
    attrs[1].val.clusterDim.z = 1;
    const int pairs = pair_slots(fn, C::kThreads, C::kSmemBytes);
    cfg.gridDim = dim3(2 * (p.num_tiles < pairs ? p.num_tiles : pairs), 1, 1);
    cfg.blockDim = dim3(C::kThreads, 1, 1);
    cfg.dynamicSmemBytes = C::kSmemBytes;
    cfg.stream = stream;
    cfg.attrs = attrs;
    cfg.numAttrs = 2;
    if (take_injected_failure(kInjectLaunch)) return LOWBIT_ERR_CUDA;
    return cudaLaunchKernelEx(&cfg, kernel, mx, mw, ms, mz, mo, p) == cudaSuccess ? LOWBIT_OK : LOWBIT_ERR_CUDA;
}

// The products over a packed table.
template <int BITS>
lowbit_status dispatch_packed(const VocabProduct& v, cudaStream_t s) {
    switch (v.mode) {
        case kVocabStats: return v.pair ? launch<kVocabStats, BITS, true>(v, s) : launch_few<kVocabStats, BITS>(v, s);
        case kVocabGrad: return v.pair ? launch<kVocabGrad, BITS, true>(v, s) : launch_few<kVocabGrad, BITS>(v, s);
        case kVocabDx: return v.pair ? launch<kVocabDx, BITS, true>(v, s) : launch<kVocabDx, BITS, false>(v, s);
        default: return LOWBIT_ERR_UNSUPPORTED;
    }
}

}  // namespace vocab
}  // namespace lowbit
