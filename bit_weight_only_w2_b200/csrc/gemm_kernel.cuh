// Weight-only low-bit GEMM for sm_100a:  Y[M][N] = X[M][K] * W^T,  W decoded from packed
// binary / ternary / uint4 codes and fp16 group scales (and zeros).
//
// The multiply behind the Bonsai Image (FLUX.2-Klein-4B) transformer linears: binary weights
// w = scale_g * b (bonsai-image-binary-4B-gemlite-1bit model card, "Binary Weight
// Representation: 1-bit g128"), ternary 2-bit weights (mlx-vlm Bonsai article, model
// overview) and the 4-bit group-64 text-encoder linears (same article, component
// architecture). After decoding it is a dense contraction, so it runs on the tcgen05 tensor
// cores.
//
// Precision: the tensor cores run in fp16 with fp32 accumulation. A pre-pass converts X from
// bf16 to fp16 (exact: every bf16 value in fp16's normal range is an fp16 value), with a
// per-row power-of-two scale so that rows whose magnitude exceeds fp16's range still convert
// exactly (the epilogue multiplies that row back). In fp16 a binary or ternary weight t * s is
// exactly +-s or 0 for the fp16 scale s, and a uint4 weight (q - z) * s is rounded once to fp16
// (2^-11 relative); rounding s to bf16 instead would cost up to 2^-8 per group, enough to
// break a 1e-2 tolerance in the tails.
//
// Kernel design ("swap AB", weights as the MMA's A operand):
//   * One CTA tile = up to 128 weight rows (MMA M) x BT tokens (MMA N), K in stages of 128.
//   * Warp 0 (one lane) is the TMA producer: per stage it loads two 64-wide, 128B-swizzled
//     boxes of the fp16 copy of X (the MMA's B operand, K-major), the packed code box of the
//     tile's rows and their group scales (and zeros) into a shared-memory ring. The first
//     stages' weight boxes are requested before waiting for the X conversion to finish.
//   * The dequant warps each own 32 weight rows (one per lane, matching the tensor-memory lane
//     quarter the warp may access): they read the row's packed words from shared memory,
//     decode codes x scale to fp16 pairs with a few integer / fp16x2 instructions per pair,
//     and store them straight into a tensor-memory ring with tcgen05.st. The decoded weights
//     never touch shared memory, which leaves its bandwidth to TMA and the MMA's B reads.
//   * Warp 1 (one lane) issues tcgen05.mma (kind::f16, A from tensor memory, B from shared
//     memory, fp32 accumulators in tensor memory) and frees ring slots with tcgen05.commit.
//   * Epilogue warps (8 for 128/256-token tiles) read the accumulators with tcgen05.ld, apply
//     the row's power-of-two factor, round to bf16 into registers and hand the accumulator
//     back before storing, so a tile's stores overlap the next tile's MMAs even with a single
//     accumulator buffer; neighbouring lanes swap halves so each store writes two outputs.
//   * Grids: persistent over 128-row tiles when there are many; for small M either "flat"
//     tiles of ceil(N / #SMs) rows with the whole K per CTA, or K split over the CTAs of a
//     thread-block cluster whose fp32 partial tiles are summed in rank order through
//     distributed shared memory.
//   * Every mbarrier wait is bounded (see sm100_ptx.cuh): a wait that gives up records
//     LOWBIT_ERR_TIMEOUT in the device status word and the CTA drains and exits.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

#include "lowbit_internal.h"
#include "sm100_ptx.cuh"
#include "tcgen05_ptx.cuh"

namespace lowbit {

constexpr int kBlockN = 128;        // weight rows per tile at most (MMA M)
constexpr int kBlockK = 128;        // K per pipeline stage
constexpr int kNumCtrlWarps = 2;    // warp 0: TMA producer, warp 1: MMA issuer + TMEM owner
constexpr int kSmemLimit = 232448;  // 227 KB opt-in dynamic shared memory per block

// PAIR: a tile of 256 weight rows x BT tokens computed by a CTA pair on cta_group::2 MMAs. Each
// CTA decodes its 128 weight rows into its own tensor memory and loads half of the X tile (BT/2
// tokens); the even CTA issues the MMAs, which read both halves of X, so every X element read
// into shared memory serves 256 weight rows instead of 128.
//
// Variants of the kernel that adapters and gradients run on (EXT).
//   kExtAdapter   Y = X W^T + P B: behind the K of the packed weights the reduction goes on over
//                 `slot` columns, Rp (a power of two >= 16) for each adapter that the token tile
//                 holds. The X side of a slot is P (bf16, zero in the rows of other adapters'
//                 tokens), the weight side the adapter's rows B[a][n][0..R). Both come through the X
//                 ring (a stage of each per block of columns) and are multiplied bf16 x bf16 out of
//                 shared memory onto the same fp32 accumulators, so Y is rounded once and the
//                 dequant warps have no part in it. (Rows of B moved through the tensor-memory ring
//                 by the dequant warps, from global memory or from 4 KB weight stages, cost 4-5 us
//                 per block of 128 columns against 0.8 for a block of packed weights.)
//   kExtGrad      dX = dY W (+ dP A): the packed words of W^T (rows k, codes along n). A group
//                 scale now belongs to a column pair of the reduction instead of to the row, so the
//                 stage's scales [group of the tile's rows][128 n] multiply fp16x2 pairs. The
//                 adapters' weight side is A[a][0..R)[k], which lies with its rows k contiguous: an
//                 MN-major operand.
constexpr int kExtNone = 0, kExtAdapter = 1, kExtGrad = 2;

template <int BITS, int GS, int BT, bool PAIR = false, int EXT = kExtNone>
struct Cfg {
    static_assert(BITS == 1 || BITS == 2 || BITS == 4, "bits");
    static_assert(GS == 64 || GS == 128, "group size");
    static_assert(BT % 16 == 0 && BT >= 16 && BT <= 256, "MMA N");
    static_assert(!PAIR || BT == 256, "pair tiles are 256 x 256");
    static constexpr int kCtasPerSm = (BT <= 64) ? 2 : 1;
    // Epilogue: warps e and e+4 cover the same 32 weight rows (TMEM lane quarter = warp % 4),
    // each half of the tile's token columns when there are 8.
    static constexpr int kNumEpiWarps = (BT >= 128) ? 8 : 4;
    static constexpr int kEpiParts = kNumEpiWarps / 4;
    static constexpr int kEpiCols = BT / kEpiParts;                 // accumulator columns per thread
    static constexpr int kNumDqWarps = (BITS == 4) ? 8 : 4;
    static constexpr int kParts = kNumDqWarps / 4;                  // dequant warps per row quarter
    static constexpr int kFirstEpiWarp = kNumCtrlWarps;
    static constexpr int kFirstDqWarp = kNumCtrlWarps + kNumEpiWarps;
    static constexpr int kThreads = 32 * (kNumCtrlWarps + kNumEpiWarps + kNumDqWarps);
    static constexpr int kNumAcc = (BT == 64 || BT == 256) ? 1 : 2;   // fit the tensor-memory budget
    static constexpr int kAccCols = kNumAcc * BT;
    static constexpr int kACol0 = (kAccCols + 31) / 32 * 32;
    static constexpr int kNumA = (kCtasPerSm == 2) ? 3 : 4;          // A ring stages (64 columns each)
    static constexpr int kColsUsed = kACol0 + kNumA * 64;
    static constexpr int kTmemCols = kColsUsed <= 32 ? 32 : kColsUsed <= 64 ? 64 : kColsUsed <= 128 ? 128
                                     : kColsUsed <= 256 ? 256 : 512;
    static_assert(kColsUsed <= 512 && kTmemCols * kCtasPerSm <= 512, "tensor memory");

    static constexpr int kWordsPerRow = kBlockK * BITS / 32;        // 4 / 8 / 16
    static constexpr int kWRowBytes = kWordsPerRow * 4;             // 16 / 32 / 64
    static constexpr int kXRows = PAIR ? BT / 2 : BT;               // token rows of X in this CTA
    static constexpr int kXHalfBytes = kXRows * 128;                // 64 fp16 per row
    static constexpr int kXBytes = 2 * kXHalfBytes;
    static constexpr int kWBytes = kBlockN * kWRowBytes;
    static constexpr int kGroupsPerStage = kBlockK / GS;            // 1 or 2
    static constexpr int kSBytes = kGroupsPerStage * kBlockN * 2;
    static constexpr int kZBytes = (BITS == 4) ? kSBytes : 0;
    // Two rings in shared memory: X stages (the MMA's B operand, freed by the MMA) and weight
    // stages (packed codes + scales + zeros, freed by the dequant warps). The weight ring runs
    // ahead of the X ring, so decoding never waits for X. One X stage is one 128-wide k-block,
    // fetched by a single TMA request (large requests stream from L2 faster than small ones).
    static constexpr int kXStageBytes = kXBytes;                    // a multiple of 2048
    static constexpr int kWOff = 0;
    static constexpr int kSOff = kWBytes;
    static constexpr int kZOff = kSOff + kSBytes;
    static constexpr int kWStageBytes = (kZOff + kZBytes + 1023) / 1024 * 1024;
    static constexpr int kWTxFixed = kSBytes + kZBytes;            // plus rows * kWRowBytes
    static constexpr int kBarBytes = 1024;
    static constexpr int kBudget = kSmemLimit / kCtasPerSm - 1024 /*align*/ - kBarBytes - 2048 /*reserve*/;
    static constexpr int kXStagesFit = (kBudget - 2 * kWStageBytes) / kXStageBytes;
    static constexpr int kXStages = kXStagesFit > 8 ? 8 : kXStagesFit;
    static constexpr int kWStagesFit = (kBudget - kXStages * kXStageBytes) / kWStageBytes;
    static constexpr int kWStages = kWStagesFit > 8 ? 8 : kWStagesFit;
    static_assert(kXStages >= 2 && kWStages >= 2, "shared memory");
    static constexpr int kWRingOff = kXStages * kXStageBytes;
    static constexpr int kBarOff = kWRingOff + kWStages * kWStageBytes;
    // Request enough shared memory that at most kCtasPerSm CTAs of these kernels share an SM:
    // tensor memory (512 columns per SM) is not a scheduling resource, so residency is capped
    // through shared memory instead (228 KB per SM).
    static constexpr int kSmemNeeded = 1024 + kBarOff + kBarBytes;
    static constexpr int kSmemFloor = (kCtasPerSm == 2) ? 80 * 1024 : 150 * 1024;
    static constexpr int kSmemBytes = kSmemNeeded > kSmemFloor ? kSmemNeeded : kSmemFloor;
    static_assert(kSmemBytes <= kSmemLimit, "shared memory");
    // split-K receive buffers (fp32 [ksplit][128 rows][odd number of 16-byte chunks]) reuse the
    // X ring: the largest over ksplit 2..8
    static constexpr int recv_bytes(int ks) {
        return ks * kBlockN * ((((BT + ks - 1) / ks + 3) / 4) | 1) * 16;
    }
    static constexpr int max_recv_bytes() {
        int m = 0;
        for (int ks = 2; ks <= 8; ++ks) m = recv_bytes(ks) > m ? recv_bytes(ks) : m;
        return m;
    }
    static_assert((PAIR && EXT == kExtNone) || max_recv_bytes() <= kXStages * kXStageBytes, "split-K receive buffer");
    static constexpr uint32_t kIdesc = idesc_f16_f32(PAIR ? 2 * kBlockN : kBlockN, BT);
    // Slot columns: a block of them is what fits one X stage as 128 rows of the weight side; P's box
    // of a block is one or two 64-wide halves.
    static constexpr int kSlotCols = kXStageBytes >= 256 * 128 ? 128 : kXStageBytes / 256;
    static constexpr int kPHalves = (kSlotCols + 63) / 64;
    static_assert(EXT == kExtNone || (kSlotCols >= 32 && kPHalves * kXHalfBytes <= kXStageBytes), "slot block");
    static constexpr uint32_t kIdescSlot =
        idesc_bf16_f32(PAIR ? 2 * kBlockN : kBlockN, BT) | (EXT == kExtGrad ? kIdescTransposeA : 0u);
    // the last tile's bf16 Y box [BT][128 rows] is staged at the start of the (idle) X ring
    static constexpr int kYStageBytes = BT * kBlockN * 2;
    static_assert(kYStageBytes <= kXStages * kXStageBytes, "Y staging");
};

struct KernelParams {
    int M, N, K;
    int num_kb;          // k-blocks of 128
    int kb_per_split;    // k-blocks per cluster rank (split-K), else num_kb
    int rows;            // weight rows per tile: 128, or fewer (multiple of 8) for small M
    int m_tiles, n_tiles, num_tiles;
    int ksplit;          // cluster size along z (1 = no split)
    uint32_t wtx_bytes;  // bytes delivered into one weight stage
    __nv_bfloat16* Y;
    const float* rowmul; // per-row power-of-two factor written by the X conversion pass
};

struct ExtParams : KernelParams {
    CUtensorMap map_p;       // P as (64, M, columns / 64) bf16, boxes of kPHalves halves
    CUtensorMap map_side;    // B as (R, N, L), boxes of `chunk` ranks x 128 rows, or A as (K, R, L),
                             // boxes of 64 rows x `chunk` ranks
    bool adapters;           // any at all
    const int* tile_slots;   // slots of each token tile (nullptr: one, adapter 0)
    const int* slot_side;    // [token tile][slot_pitch]: adapter, or L (read as zeros) if it is not finite
    int slot_pitch;
    int rank_log2;           // log2 of the slot width Rp
    int chunk_log2;          // log2 of the slot columns per box of the weight side
    unsigned* status;        // the device status word
};
// Slot columns per box: up to 64 for B (the widest swizzled row), whole slots for A, and no more
// than a block.
inline int side_chunk_log2(bool grad, int rank_log2, int slot_cols) {
    int c = rank_log2;
    while ((1 << c) > slot_cols || (!grad && c > 6)) --c;
    return c;
}
template <int EXT>
using ParamsOf = std::conditional_t<EXT == kExtNone, KernelParams, ExtParams>;

// The device status word, where it is defined (the plain kernel's translation unit).
__device__ unsigned* status_word();

// ---------------------------------------------------------------------------------------------
// Decoders: one 64-wide K half of one weight row -> 32 fp16x2 values (even k low, odd k high),
// out[i] holding columns 2i and 2i + 1 of the half. 2- and 4-bit words are in block order
// (word q of a four-word block holds, in pair p, columns 8p + 2q and 8p + 2q + 1 of the
// block), so pair p of word w lands in out[4p + q] of its block; binary words are in plain order.
// ---------------------------------------------------------------------------------------------

// Binary: bit 1 -> +s, 0 -> -s. Pair c of a word is (bit c, bit 16 + c); shifting the word
// left by 15 - c puts them on the two fp16 sign bits, and one LOP3 flips the sign of s where
// the bit is 0. Exact.
__device__ __forceinline__ void decode_half_b1(uint32_t w0, uint32_t w1, uint32_t s2, uint32_t (&out)[32]) {
#pragma unroll
    for (int c = 0; c < 16; ++c) out[c] = xor_andnot(s2, w0 << (15 - c), 0x80008000u);
#pragma unroll
    for (int c = 0; c < 16; ++c) out[16 + c] = xor_andnot(s2, w1 << (15 - c), 0x80008000u);
}

// Ternary: field f = t + 1 in {0,1,2}. OR-ing the two fields of a pair, left at bit 2j of each
// half, into the mantissas of fp16 1024.0 gives e = 1024 + f * 4^j exactly (j <= 4 keeps the
// field inside the 10-bit mantissa). One fp16x2 FMA computes e * 4^-j - (1024 * 4^-j + 1) =
// f - 1 = t exactly (the exact result is representable, so nothing rounds) and a multiply by
// s gives t * s exactly. Pairs 0..4 are decoded in place, pairs 5..7 after one shift by 10.
// Word q of the half's only block: pair c goes to out[4c + q].
__device__ __forceinline__ void decode_word_b2(uint32_t v, uint32_t s2, uint32_t* out, int q) {
    constexpr uint32_t kMagic = 0x64006400u;                                           // 1024.0
    constexpr uint32_t kMul[5] = {0x3C003C00u, 0x34003400u, 0x2C002C00u, 0x24002400u, 0x1C001C00u};  // 4^-j
    constexpr uint32_t kAdd[5] = {0xE401E401u, 0xDC04DC04u, 0xD410D410u, 0xCC40CC40u, 0xC500C500u};  // -(1024*4^-j+1)
#pragma unroll
    for (int c = 0; c < 8; ++c) {
        const int shift = (c < 5) ? 0 : 10;
        const int j = (c < 5) ? c : c - 5;
        const uint32_t e = and_or(v >> shift, 0x00030003u << (2 * j), kMagic);
        const uint32_t t = f16x2_fma(e, kMul[j], kAdd[j]);
        out[4 * c + q] = f16x2_mul(t, s2);
    }
}

// uint4: the nibbles of a pair, left at bit 4j of each half (j <= 1), OR-ed into fp16 1024.0
// give 1024 + q * 16^j exactly, and one fp16x2 FMA recovers q exactly. Each weight is then
// (q - z) * s = q * s + cz with cz = -z * s in fp32 (exact: the product of two fp16 values has
// at most 22 significant bits), formed by one mixed-precision FMA (q * s is exact as well, so
// the only fp32 rounding is below 2^-24 relative) and rounded to fp16 once. A code equal or
// next to its zero point thus keeps the full fp16 precision of the small difference (q - z) * s;
// rounding -z * s to fp16 first would cost up to 2^-11 |z * s| per weight, which is most of
// such a weight. Word w of the half (block w / 4, word q = w % 4 of it): pair c goes to
// out[16 * (w / 4) + 4c + q].
__device__ __forceinline__ void decode_word_b4(uint32_t v, uint16_t s, float cz, uint32_t* out, int w) {
    constexpr uint32_t kMagic = 0x64006400u;
    constexpr uint32_t kMul[2] = {0x3C003C00u, 0x2C002C00u};   // 1, 1/16
    constexpr uint32_t kAdd[2] = {0xE400E400u, 0xD400D400u};   // -1024, -64
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        const int shift = (c < 2) ? 0 : 8;
        const int j = c & 1;
        const uint32_t e = and_or(v >> shift, 0x000F000Fu << (4 * j), kMagic);
        const uint32_t q = f16x2_fma(e, kMul[j], kAdd[j]);
        float lo, hi;
        fma_f16x2_f32(q, s, cz, lo, hi);
        out[16 * (w >> 2) + 4 * c + (w & 3)] = pack_f16x2(lo, hi);
    }
}

// One 64-wide half of a reduction stage of W^T: the row's codes as above, but each pair of
// columns has scales (and zeros) of its own, read from shared memory (`s4`, `z4`) four pairs at a
// time. Binary and ternary weights are again exactly +-s or 0. uint4: q is exact, q - z and the
// product with s are each rounded to fp16 once (2^-11 relative each, no cancellation behind a
// rounding), which halves the instructions of an fp32 product per weight; both together stay below
// the 2^-8 of one bf16 rounding.
template <int BITS>
__device__ __forceinline__ void decode_half_grad(const uint32_t* words, const uint4* s4, const uint4* z4,
                                                 uint32_t (&out)[32]) {
    constexpr uint32_t kMagic = 0x64006400u;   // 1024.0, and the constants of the decoders above
    constexpr uint32_t kMul[5] = {0x3C003C00u, 0x34003400u, 0x2C002C00u, 0x24002400u, 0x1C001C00u};
    constexpr uint32_t kAdd2[5] = {0xE401E401u, 0xDC04DC04u, 0xD410D410u, 0xCC40CC40u, 0xC500C500u};
    constexpr uint32_t kAdd4[2] = {0xE400E400u, 0xD400D400u};
#pragma unroll
    for (int g = 0; g < 8; ++g) {              // pairs 4g .. 4g + 3 of the half
        const uint4 sv = s4[g];
        const uint32_t sp[4] = {sv.x, sv.y, sv.z, sv.w};
        uint32_t zp[4] = {0, 0, 0, 0};
        if (BITS == 4) {
            const uint4 zv = z4[g];
            zp[0] = zv.x; zp[1] = zv.y; zp[2] = zv.z; zp[3] = zv.w;
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            if (BITS == 1) {
                const int i = 4 * g + q;
                out[i] = xor_andnot(sp[q], words[i >> 4] << (15 - (i & 15)), 0x80008000u);
            } else if (BITS == 2) {            // pair g of word q
                const int j = g < 5 ? g : g - 5;
                const uint32_t e = and_or(words[q] >> (g < 5 ? 0 : 10), 0x00030003u << (2 * j), kMagic);
                out[4 * g + q] = f16x2_mul(f16x2_fma(e, kMul[j], kAdd2[j]), sp[q]);
            } else {                           // pair c of word q of block g / 4
                const int c = g & 3;
                const uint32_t e = and_or(words[4 * (g >> 2) + q] >> (c < 2 ? 0 : 8), 0x000F000Fu << (4 * (c & 1)), kMagic);
                const uint32_t v = f16x2_fma(e, kMul[2 * (c & 1)], kAdd4[c & 1]);
                out[4 * g + q] = f16x2_mul(f16x2_sub(v, zp[q]), sp[q]);
            }
        }
    }
}

// ---------------------------------------------------------------------------------------------
// The kernel
// ---------------------------------------------------------------------------------------------
template <int BITS, int GS, int BT, bool PAIR, int EXT = kExtNone>
__global__ void __launch_bounds__(Cfg<BITS, GS, BT, PAIR, EXT>::kThreads, Cfg<BITS, GS, BT, PAIR, EXT>::kCtasPerSm)
    lowbit_gemm_kernel(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_w,
                       const __grid_constant__ CUtensorMap map_s, const __grid_constant__ CUtensorMap map_z,
                       const __grid_constant__ CUtensorMap map_y, const __grid_constant__ ParamsOf<EXT> p) {
    using C = Cfg<BITS, GS, BT, PAIR, EXT>;
    constexpr int SX = C::kXStages;
    constexpr int SW = C::kWStages;
    constexpr int NA = C::kNumA;
    constexpr int NACC = C::kNumAcc;

    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* wring = smem + C::kWRingOff;
    uint64_t* xfull = reinterpret_cast<uint64_t*>(smem + C::kBarOff);
    uint64_t* xempty = xfull + SX;
    uint64_t* wfull = xempty + SX;
    uint64_t* wempty = wfull + SW;
    uint64_t* afull = wempty + SW;
    uint64_t* aempty = afull + NA;
    uint64_t* accfull = aempty + NA;
    uint64_t* accempty = accfull + NACC;
    uint64_t* drain = accempty + NACC;
    uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(drain + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    // Pair mode: the CTA of cluster rank 0 issues the MMAs. The other CTA's X copies complete on
    // the issuer's X barrier, its dequant and epilogue warps arrive on the issuer's A-ready and
    // accumulator-free barriers, and the issuer's commits arrive on the empty / ready barriers of
    // both CTAs (same offsets).
    // (The variants also split K over clusters of CTA pairs: ranks 2z and 2z + 1 are slice z's pair.)
    constexpr bool kPairSplit = PAIR && EXT != kExtNone;
    const uint32_t ctarank = PAIR ? cluster_ctarank() : 0u;
    const uint32_t pair_rank = kPairSplit ? ctarank & 1u : ctarank;
    const uint32_t lead = kPairSplit ? ctarank & ~1u : 0u;   // cluster rank of the pair's issuer
    const uint16_t pair_mask = static_cast<uint16_t>(kPairSplit ? 0x3u << lead : 0x3u);
    const bool issuer = pair_rank == 0;
    constexpr int kPairCtas = PAIR ? 2 : 1;
    auto on_issuer = [&](uint64_t* bar) { return map_shared_rank(smem_u32(bar), lead); };

    if (threadIdx.x == 0) {
        for (int i = 0; i < SX; ++i) {
            mbar_init(&xfull[i], 1);
            mbar_init(&xempty[i], 1);
        }
        for (int i = 0; i < SW; ++i) {
            mbar_init(&wfull[i], 1);
            mbar_init(&wempty[i], C::kNumDqWarps);
        }
        for (int i = 0; i < NA; ++i) {
            mbar_init(&afull[i], kPairCtas * C::kNumDqWarps);
            mbar_init(&aempty[i], 1);
        }
        for (int i = 0; i < NACC; ++i) {
            mbar_init(&accfull[i], 1);
            mbar_init(&accempty[i], kPairCtas * C::kNumEpiWarps);
        }
        mbar_init(drain, 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 0 && lane == 0) {
        tma_prefetch_desc(&map_x);
        tma_prefetch_desc(&map_w);
        tma_prefetch_desc(&map_s);
        if (BITS == 4) tma_prefetch_desc(&map_z);
        tma_prefetch_desc(&map_y);
    }
    if (warp == 1) {
        tmem_alloc<PAIR>(tmem_holder, C::kTmemCols);
        tmem_relinquish<PAIR>();
    }
    tc_fence_before();
    __syncthreads();
    if (PAIR) cluster_sync_all();   // both CTAs' barriers are initialised before either uses the other's
    tc_fence_after();
    const uint32_t tmem_base = *tmem_holder;

    // Programmatic dependent launch: the next kernel in the stream may start its prologue now.
    // Threads that touch global memory wait for the previous kernel (the X conversion) first. (kExtGrad:
    // not before that has completed, since the kernel that may follow, the adapters' gradients, reads
    // what it wrote without waiting for this one.)
    if constexpr (EXT != kExtGrad) grid_launch_dependents();

    const bool split = p.ksplit > 1;
    const int kb_begin = split ? static_cast<int>(blockIdx.z) * p.kb_per_split : 0;
    const int kb_end = split ? min(p.num_kb, kb_begin + p.kb_per_split) : p.num_kb;
    const int nkb = kb_end - kb_begin;
    // first tile and tile stride of this CTA (a pair's two CTAs, adjacent along x, share both)
    const int tile0 = PAIR ? static_cast<int>(blockIdx.x >> 1) : static_cast<int>(blockIdx.x);
    const int tile_step = split ? p.num_tiles : static_cast<int>(PAIR ? gridDim.x >> 1 : gridDim.x);
    const int my_tiles = tile0 < p.num_tiles ? (p.num_tiles - 1 - tile0) / tile_step + 1 : 0;
    // first weight row of this CTA in tile t: pair tiles cover 2 * p.rows rows, this CTA's half
    // starting at pair_rank * p.rows
    const int n_stride = PAIR ? 2 * p.rows : p.rows;
    const int n_off = PAIR ? static_cast<int>(pair_rank) * p.rows : 0;
    // The slot columns that the adapters of tile t's tokens add behind this CTA's K slice: columns
    // [x0, x1) of the tile's, multiples of 16, in blocks of kSlotCols shared out over the K slices.
    // Read after grid_dependency_wait().
    struct Extra {
        int x0, x1;
        __device__ int blocks() const { return (x1 - x0 + C::kSlotCols - 1) / C::kSlotCols; }
    };
    // Split in a load and the arithmetic on it, so that a tile's count can be asked for a tile ahead
    // without the asking thread waiting for it.
    auto slots_of = [&](int t) -> int {
        if constexpr (EXT == kExtNone) return 0;
        else if (!p.adapters || t >= my_tiles) return 0;
        else return p.tile_slots ? __ldg(p.tile_slots + (tile0 + t * tile_step) / p.n_tiles) : 1;
    };
    auto extra_of = [&](int slots) -> Extra {
        if constexpr (EXT == kExtNone) {
            return Extra{0, 0};
        } else {
            const int cols = slots << p.rank_log2;
            if (!split) return Extra{0, cols};
            const int per = ((cols + C::kSlotCols - 1) / C::kSlotCols + p.ksplit - 1) / p.ksplit * C::kSlotCols;
            const int x0 = min(cols, static_cast<int>(blockIdx.z) * per);
            return Extra{x0, min(cols, x0 + per)};
        }
    };
    unsigned* status;
    if constexpr (EXT == kExtNone)
        status = status_word();
    else
        status = p.status;

    if (warp == 0) {
        // ---------------------------------------------------------------- TMA producer
        if (lane == 0) {
            const uint32_t total = static_cast<uint32_t>(my_tiles * nkb);   // (slot columns not counted)
            auto coords = [&](uint32_t it, int& m0, int& n0, int& kb) {
                const int tile = tile0 + static_cast<int>(it / nkb) * tile_step;
                kb = kb_begin + static_cast<int>(it % nkb);
                m0 = (tile / p.n_tiles) * BT;
                n0 = (tile % p.n_tiles) * n_stride + n_off;
            };
            // The variants keep the next stages' coordinates at hand instead of deriving them from `it`:
            // the X ring's refill latency bounds the kernel (divisions between a slot's release and its
            // next request cost 4.5 % on 4173 x 9216 x 9216).
            int wt = 0, wk = kb_begin, wn0 = (tile0 % p.n_tiles) * n_stride + n_off;
            auto issue_w = [&](uint32_t it) {
                int m0, n0, kb;
                if constexpr (EXT == kExtNone) {
                    coords(it, m0, n0, kb);
                } else {
                    n0 = wn0;
                    kb = wk;
                }
                const uint32_t s = it % SW;
                uint8_t* st = wring + s * C::kWStageBytes;
                mbar_arrive_expect_tx(&wfull[s], p.wtx_bytes);
                tma_load_2d(&map_w, &wfull[s], st + C::kWOff, kb * C::kWordsPerRow, n0);
                // (W^T: the groups of the tile's rows, the stage's 128 columns)
                const int sx = EXT == kExtGrad ? kb * kBlockK : n0;
                const int sy = EXT == kExtGrad ? n0 / GS : kb * C::kGroupsPerStage;
                tma_load_2d(&map_s, &wfull[s], st + C::kSOff, sx, sy);
                if (BITS == 4) tma_load_2d(&map_z, &wfull[s], st + C::kZOff, sx, sy);
                if (EXT != kExtNone && ++wk == kb_end) {
                    wk = kb_begin;
                    wn0 = ((tile0 + ++wt * tile_step) % p.n_tiles) * n_stride + n_off;
                }
            };
            // With slot columns a tile has more X stages than nkb: behind the K blocks, P and the weight
            // side of each block of columns. xj: the next stage of tile xt (of nkb + 2 * blocks).
            int xt = 0, xj = 0, xn = nkb, xm0 = (tile0 / p.n_tiles) * BT + static_cast<int>(pair_rank) * C::kXRows;
            int next_slots = 0;
            Extra xe{0, 0};
            auto start_tile = [&](int slots) {
                xe = extra_of(slots);
                xn = nkb + 2 * xe.blocks();
                next_slots = slots_of(xt + 1);
            };
            auto next_x = [&] {
                if (++xj == xn) {
                    xj = 0;
                    xm0 = ((tile0 + ++xt * tile_step) / p.n_tiles) * BT + static_cast<int>(pair_rank) * C::kXRows;
                    start_tile(next_slots);
                }
            };
            auto issue_slots = [&](uint32_t s) {
                if constexpr (EXT != kExtNone) {
                    const int tile = tile0 + xt * tile_step;
                    const int n0 = tile % p.n_tiles * n_stride + n_off;
                    const int c0 = xe.x0 + (xj - nkb) / 2 * C::kSlotCols;
                    const int c1 = min(xe.x1, c0 + C::kSlotCols);
                    uint8_t* st = smem + s * C::kXStageBytes;
                    auto load = [&](const CUtensorMap* map, uint8_t* dst, int x, int y, int z) {
                        if (PAIR)
                            tma_load_3d_pair(map, on_issuer(&xfull[s]), dst, x, y, z);
                        else
                            tma_load_3d(map, &xfull[s], dst, x, y, z);
                    };
                    if (((xj - nkb) & 1) == 0) {
                        if (issuer) mbar_arrive_expect_tx(&xfull[s], kPairCtas * C::kPHalves * C::kXHalfBytes);
                        load(&p.map_p, st, 0, xm0, c0 / 64);
                    } else {
                        const int chunk = 1 << p.chunk_log2, chunks = (c1 - c0) >> p.chunk_log2;
                        const int* slots = p.slot_side + static_cast<size_t>(tile / p.n_tiles) * p.slot_pitch;
                        if (issuer) mbar_arrive_expect_tx(&xfull[s], kPairCtas * (chunks << (p.chunk_log2 + 8)));
                        for (int i = 0; i < chunks; ++i) {
                            const int c = c0 + i * chunk, r = c & ((1 << p.rank_log2) - 1);
                            const int a = p.tile_slots ? __ldg(slots + (c >> p.rank_log2)) : 0;
                            uint8_t* dst = st + i * chunk * 256;
                            if (EXT == kExtAdapter) {
                                load(&p.map_side, dst, r, n0, a);
                            } else {
                                load(&p.map_side, dst, n0, r, a);
                                load(&p.map_side, dst + chunk * 128, n0 + 64, r, a);
                            }
                        }
                    }
                    next_x();
                }
            };
            auto issue_x = [&](uint32_t it) {
                const uint32_t s = it % SX;
                int m, kb;   // first token row of this CTA's box, k-block
                if constexpr (EXT == kExtNone) {
                    int m0, n0;
                    coords(it, m0, n0, kb);
                    m = m0 + static_cast<int>(pair_rank) * C::kXRows;
                } else {
                    if (xj >= nkb) return issue_slots(s);
                    m = xm0;
                    kb = kb_begin + xj;
                }
                uint8_t* st = smem + s * C::kXStageBytes;
                // box (64 k, kXRows tokens, 2 halves) = both 128-byte-swizzled K halves in one request
                if (!PAIR) {
                    mbar_arrive_expect_tx(&xfull[s], C::kXBytes);
                    tma_load_3d(&map_x, &xfull[s], st, 0, m, kb * 2);
                } else {
                    // both halves complete on the issuer's barrier, which expects both
                    if (issuer) mbar_arrive_expect_tx(&xfull[s], 2 * C::kXBytes);
                    tma_load_3d_pair(&map_x, on_issuer(&xfull[s]), st, 0, m, kb * 2);
                }
                if (EXT != kExtNone) next_x();
            };
            // The packed weights and scales are not written by the kernel just before this one
            // (the X conversion, which itself starts only once everything earlier in the stream
            // has completed), so the first weight stages are requested before waiting for it.
            uint32_t itw = 0, itx = 0;
            const uint32_t wpre = total < static_cast<uint32_t>(SW) ? total : static_cast<uint32_t>(SW);
            for (; itw < wpre; ++itw) issue_w(itw);
            grid_dependency_wait();
            if constexpr (EXT == kExtGrad) grid_launch_dependents();
            if constexpr (EXT != kExtNone) {
                start_tile(slots_of(0));
            }
            auto x_left = [&] { return EXT == kExtNone ? itx < total : xt < my_tiles; };
            // Fill both rings as their slots free up, without blocking on either.
            bool ok = true;
            long long t_last = clock64();
            uint32_t idle = 0;
            while (x_left() || itw < total) {
                bool progress = false;
                if (x_left() && mbar_test_wait(&xempty[itx % SX], ((itx / SX) & 1u) ^ 1u)) {
                    issue_x(itx++);
                    progress = true;
                }
                if (itw < total && mbar_test_wait(&wempty[itw % SW], ((itw / SW) & 1u) ^ 1u)) {
                    issue_w(itw++);
                    progress = true;
                }
                if (progress) {
                    idle = 0;
                    t_last = clock64();
                } else if ((++idle & 63u) == 0) {
                    if (*abort_flag) { ok = false; break; }
                    if (clock64() - t_last > kWaitLimitCycles) {
                        atomicOr(status, kDevErrTimeout);
                        *abort_flag = 1;
                        ok = false;
                        break;
                    }
                }
            }
            if (!ok) {
                // Drain: wait (bounded) for the copies still in flight before the CTA exits. The
                // second CTA of a pair cannot wait on the issuer's barrier its X copies count on:
                // it gives them a fixed time instead (both CTAs meet again before either exits).
                if (PAIR && !issuer) {
                    const long long t0 = clock64();
                    while (clock64() - t0 < kWaitLimitCycles / 64) {
                    }
                } else {
                    for (uint32_t j = (itx > static_cast<uint32_t>(SX) ? itx - SX : 0u); j < itx; ++j) {
                        const long long t0 = clock64();
                        while (!mbar_try_wait(&xfull[j % SX], (j / SX) & 1u) && clock64() - t0 < kWaitLimitCycles) {
                        }
                    }
                }
                for (uint32_t j = (itw > static_cast<uint32_t>(SW) ? itw - SW : 0u); j < itw; ++j) {
                    const long long t0 = clock64();
                    while (!mbar_try_wait(&wfull[j % SW], (j / SW) & 1u) && clock64() - t0 < kWaitLimitCycles) {
                    }
                }
            }
        }
    } else if (warp == 1) {
        // ---------------------------------------------------------------- MMA issuer
        if (lane == 0 && issuer) {
            uint32_t it = 0, ait = 0, tcount = 0;
            bool ok = true;
            bool issued = false;
            Extra xe{0, 0};
            if constexpr (EXT != kExtNone) {
                grid_dependency_wait();   // before the tiles' slot counts
                xe = extra_of(slots_of(0));
            }
            for (int t = 0; t < my_tiles && ok; ++t, ++tcount) {
                const uint32_t b = tcount % NACC, acc_ph = (tcount / NACC) & 1u;
                if (!mbar_wait(&accempty[b], acc_ph ^ 1u, abort_flag, status)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t d_tmem = tmem_base + b * BT;
                const int next_slots = slots_of(t + 1);
                for (int kb = kb_begin; kb < kb_end; ++kb, ++it, ++ait) {
                    const uint32_t s = it % SX, ph = (it / SX) & 1u;
                    const uint32_t a = ait % NA, aph = (ait / NA) & 1u;
                    if (!mbar_wait(&xfull[s], ph, abort_flag, status)) { ok = false; break; }
                    if (!mbar_wait(&afull[a], aph, abort_flag, status)) { ok = false; break; }
                    tc_fence_after();
                    const uint32_t xs = smem_u32(smem + s * C::kXStageBytes);
#pragma unroll
                    for (int kk = 0; kk < kBlockK / 16; ++kk) {
                        const uint32_t a_tmem = tmem_base + C::kACol0 + a * 64 + kk * 8;
                        const uint64_t bdesc =
                            smem_desc_k_sw128(xs + (kk >> 2) * C::kXHalfBytes + (kk & 3) * 32);
                        if (PAIR)
                            mma_f16_ts_pair(d_tmem, a_tmem, bdesc, C::kIdesc, (kb > kb_begin || kk > 0) ? 1u : 0u);
                        else
                            mma_f16_ts(d_tmem, a_tmem, bdesc, C::kIdesc, (kb > kb_begin || kk > 0) ? 1u : 0u);
                    }
                    issued = true;
                    if (PAIR) {
                        mma_commit_pair_mc(&xempty[s], pair_mask);
                        mma_commit_pair_mc(&aempty[a], pair_mask);
                    } else {
                        mma_commit(&xempty[s]);
                        mma_commit(&aempty[a]);
                    }
                }
                if constexpr (EXT != kExtNone) {
                    // slot columns: P in one stage (the MMA's B operand), the weight side in the next (A)
                    for (int c0 = xe.x0; ok && c0 < xe.x1; c0 += C::kSlotCols, it += 2) {
                        const uint32_t sp = it % SX, ss = (it + 1) % SX;
                        if (!mbar_wait(&xfull[sp], (it / SX) & 1u, abort_flag, status) ||
                            !mbar_wait(&xfull[ss], ((it + 1) / SX) & 1u, abort_flag, status)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        const uint32_t ps = smem_u32(smem + sp * C::kXStageBytes);
                        const uint32_t as = smem_u32(smem + ss * C::kXStageBytes);
                        const int cols = min(C::kSlotCols, xe.x1 - c0);
#pragma unroll 1
                        for (int c = 0; c < cols; c += 16) {
                            // P's box starts at a multiple of 64 columns
                            const int pc = (c0 & 63) + c;
                            const uint64_t bdesc =
                                smem_desc_k_sw128(ps + (pc >> 6) * C::kXHalfBytes + (pc & 63) * 2);
                            const uint32_t box = as + ((c >> p.chunk_log2) << (p.chunk_log2 + 8));
                            const int in = c & ((1 << p.chunk_log2) - 1);
                            const uint64_t adesc = EXT == kExtAdapter
                                                       ? smem_desc_k(box + in * 2, 2 << p.chunk_log2)
                                                       : smem_desc_mn(box + in * 128, 128, 128 << p.chunk_log2);
                            if (PAIR)
                                mma_f16_ss_pair(d_tmem, adesc, bdesc, C::kIdescSlot, 1u);
                            else
                                mma_f16_ss(d_tmem, adesc, bdesc, C::kIdescSlot, 1u);
                        }
                        if (PAIR) {
                            mma_commit_pair_mc(&xempty[sp], pair_mask);
                            mma_commit_pair_mc(&xempty[ss], pair_mask);
                        } else {
                            mma_commit(&xempty[sp]);
                            mma_commit(&xempty[ss]);
                        }
                    }
                    xe = extra_of(next_slots);
                }
                if (!ok) break;
                if (PAIR)
                    mma_commit_pair_mc(&accfull[b], pair_mask);
                else
                    mma_commit(&accfull[b]);
            }
            if (!ok && issued) {
                // Drain: make sure no MMA is still writing tensor memory before it is freed.
                if (PAIR)
                    mma_commit_pair(drain);
                else
                    mma_commit(drain);
                const long long t0 = clock64();
                while (!mbar_try_wait(drain, 0) && clock64() - t0 < kWaitLimitCycles) {
                }
            }
        }
    } else if (warp >= C::kFirstDqWarp) {
        // ---------------------------------------------------------------- dequant warps
        const int dq = warp - C::kFirstDqWarp;
        const int quarter = warp & 3;
        const int part = dq >> 2;                    // which K part of the stage this warp decodes
        const int row = quarter * 32 + lane;         // weight row within the tile = TMEM lane
        const bool row_ok = row < p.rows;
        const uint32_t lane_base = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16);
        constexpr int kHalvesPerPart = 2 / C::kParts;   // 64-wide K halves decoded by this warp
        uint32_t it = 0, ait = 0;
        bool ok = true;
        for (int t = 0; t < my_tiles && ok; ++t) {
            for (int kb = kb_begin; kb < kb_end; ++kb, ++it, ++ait) {
                const uint32_t s = it % SW, ph = (it / SW) & 1u;
                const uint32_t a = ait % NA, aph = (ait / NA) & 1u;
                if (!__all_sync(0xffffffffu, mbar_wait(&wfull[s], ph, abort_flag, status))) { ok = false; break; }
                const uint8_t* st = wring + s * C::kWStageBytes;
                // --- this row's packed words and scales (rows past the tile decode to zero)
                uint32_t words[kHalvesPerPart][C::kWordsPerRow / 2];
                uint32_t s2[kHalvesPerPart];
                float cz[kHalvesPerPart];
                const uint8_t* wrow = st + C::kWOff + row * C::kWRowBytes;
#pragma unroll
                for (int hh = 0; hh < kHalvesPerPart; ++hh) {
                    const int h = part * kHalvesPerPart + hh;
                    const int gi = (GS == 64) ? h : 0;
#pragma unroll
                    for (int w = 0; w < C::kWordsPerRow / 2; ++w) words[hh][w] = 0;
                    s2[hh] = 0;
                    cz[hh] = 0.f;
                    if (row_ok) {
                        if (BITS == 1) {
                            const uint2 v = *reinterpret_cast<const uint2*>(wrow + h * 8);
                            words[hh][0] = v.x;
                            words[hh][1] = v.y;
                        } else if (BITS == 2) {
                            const int chunk = h ^ ((row >> 2) & 1);           // 32-byte swizzle
                            const uint4 v = *reinterpret_cast<const uint4*>(wrow + chunk * 16);
                            words[hh][0] = v.x; words[hh][1] = v.y; words[hh][2] = v.z; words[hh][3] = v.w;
                        } else {
#pragma unroll
                            for (int q = 0; q < 2; ++q) {
                                const int chunk = (2 * h + q) ^ ((row >> 1) & 3);  // 64-byte swizzle
                                const uint4 v = *reinterpret_cast<const uint4*>(wrow + chunk * 16);
                                words[hh][4 * q + 0] = v.x; words[hh][4 * q + 1] = v.y;
                                words[hh][4 * q + 2] = v.z; words[hh][4 * q + 3] = v.w;
                            }
                        }
                        const uint16_t* srow = reinterpret_cast<const uint16_t*>(st + C::kSOff) + gi * kBlockN;
                        const uint32_t sb = EXT == kExtGrad ? 0u : srow[row];
                        s2[hh] = sb | (sb << 16);
                        if (BITS == 4 && EXT != kExtGrad) {   // -z * s, exact in fp32
                            const __half* zrow = reinterpret_cast<const __half*>(st + C::kZOff) + gi * kBlockN;
                            cz[hh] = -__half2float(zrow[row]) *
                                     __half2float(__ushort_as_half(static_cast<unsigned short>(sb)));
                        }
                    }
                }
                // --- decode into the tensor-memory A ring
                if (!__all_sync(0xffffffffu, mbar_wait(&aempty[a], aph ^ 1u, abort_flag, status))) {
                    ok = false;
                    break;
                }
                tc_fence_after();
#pragma unroll
                for (int hh = 0; hh < kHalvesPerPart; ++hh) {
                    const int h = part * kHalvesPerPart + hh;
                    uint32_t out[32];
                    if constexpr (EXT == kExtGrad) {
                        // scales (zeros) of the half's 64 columns for this row's group: the same
                        // words for the whole warp (a group holds at least 64 rows)
                        const int gr = (GS == 64) ? (row >> 6) : 0;
                        const uint8_t* sz = st + gr * kBlockN * 2 + h * 128;
                        decode_half_grad<BITS>(words[hh], reinterpret_cast<const uint4*>(sz + C::kSOff),
                                               reinterpret_cast<const uint4*>(sz + C::kZOff), out);
                    } else if (BITS == 1) {
                        decode_half_b1(words[hh][0], words[hh][1], s2[hh], out);
                    } else if (BITS == 2) {
#pragma unroll
                        for (int w = 0; w < 4; ++w) decode_word_b2(words[hh][w], s2[hh], out, w);
                    } else {
#pragma unroll
                        for (int w = 0; w < 8; ++w)
                            decode_word_b4(words[hh][w], static_cast<uint16_t>(s2[hh]), cz[hh], out, w);
                    }
                    if (dcheck(C::kACol0 + a * 64 + h * 32 + 32 <= C::kTmemCols, status))
                        tmem_st32(lane_base + C::kACol0 + a * 64 + h * 32, out);
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    // The weight stage is freed only here, when everything read from it has been used. Freed
                    // right behind the loads of the words, it was refilled under them: with several streams on
                    // the GPU a warp of the uint4 variant of 64 tokens (72 registers, spills) waits long for
                    // its A slot, and its loads took effect after the arrival (some rows of a tile were decoded
                    // from the next stage, once in some thousand calls). The later release costs nothing: 160.8
                    // against 162.9 us for 4096 x 3072 x 9216, 20.4 against 20.8 for 64 x 2560 x 9728 uint4, and
                    // within 3 % either way on 19 shapes.
                    mbar_arrive(&wempty[s]);
                    if (PAIR && !issuer)
                        mbar_arrive_remote(on_issuer(&afull[a]));
                    else
                        mbar_arrive(&afull[a]);
                }
            }
        }
    } else {
        // ---------------------------------------------------------------- epilogue warps
        const int e = warp - C::kFirstEpiWarp;
        const int quarter = warp & 3;
        const int epart = e >> 2;                    // which slice of the token columns
        const int col0 = epart * C::kEpiCols;
        const int row = quarter * 32 + lane;
        const bool row_ok = row < p.rows;
        const uint32_t lane_base = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16);
        grid_dependency_wait();                      // before the first global access
        constexpr int kChunk = (C::kEpiCols >= 32) ? 32 : 16;
        uint32_t tcount = 0;
        constexpr int kChunks = C::kEpiCols / kChunk;
        for (int t = 0; t < my_tiles; ++t, ++tcount) {
            const int tile = tile0 + t * tile_step;
            const uint32_t b = tcount % NACC, acc_ph = (tcount / NACC) & 1u;
            const int m0 = (tile / p.n_tiles) * BT + col0;   // first token of this thread's columns
            const int n = (tile % p.n_tiles) * n_stride + n_off + row;
            // Lane j of the warp holds the row factor of token m0 + c0 + j of every chunk c0,
            // requested before waiting for the accumulator so the loads overlap the MMAs.
            float mul[kChunks];
#pragma unroll
            for (int ci = 0; ci < kChunks; ++ci) {
                const int mj = m0 + ci * kChunk + lane;
                mul[ci] = (!split && lane < kChunk && mj < p.M && dcheck(mj >= 0, status)) ? p.rowmul[mj] : 1.0f;
            }
            if (!__all_sync(0xffffffffu, mbar_wait(&accfull[b], acc_ph, abort_flag, status))) break;
            tc_fence_after();
            if (!split && t + 1 == my_tiles) {
                // The CTA's last tile has nothing to overlap its stores with, and its X ring is
                // idle (the MMAs just completed consumed every stage, and no copy is in flight):
                // the tile goes, chunk by chunk, to the start of the X ring as the Y box [BT
                // tokens][p.rows rows] (one X stage, or two of a CTA pair's half-size stages) and
                // leaves in one TMA store, which clips the parts past M or N.
                uint32_t* stg = reinterpret_cast<uint32_t*>(smem);
                const bool even = (lane & 1) == 0;
                const int r_pair = row - (even ? 0 : 1);   // the pair's even row within the tile
#pragma unroll 1
                for (int c0 = 0; c0 < C::kEpiCols; c0 += kChunk) {
                    uint32_t v[32];
                    if (kChunk == 32) {
                        tmem_ld32(lane_base + b * BT + col0 + c0, v);
                    } else {
                        tmem_ld16(lane_base + b * BT + col0 + c0, *reinterpret_cast<uint32_t(*)[16]>(v));
                    }
                    float mul_j = mul[0];
#pragma unroll
                    for (int ci = 1; ci < kChunks; ++ci)
                        if (ci == c0 / kChunk) mul_j = mul[ci];   // keeps mul[] in registers
                    tmem_wait_ld();
#pragma unroll
                    for (int j = 0; j < kChunk; j += 2) {
                        const float f0 = __uint_as_float(v[j]) * __shfl_sync(0xffffffffu, mul_j, j);
                        const float f1 = __uint_as_float(v[j + 1]) * __shfl_sync(0xffffffffu, mul_j, j + 1);
                        const __nv_bfloat162 h2 = __floats2bfloat162_rn(f0, f1);   // (token j, token j+1)
                        const uint32_t mine = *reinterpret_cast<const uint32_t*>(&h2);
                        // lanes 2i, 2i+1 (rows n, n+1) swap halves: (row n, row n+1) at one token
                        const uint32_t other = __shfl_xor_sync(0xffffffffu, mine, 1);
                        const uint32_t outw =
                            even ? __byte_perm(mine, other, 0x5410) : __byte_perm(other, mine, 0x7632);
                        const int ml = col0 + c0 + j + (even ? 0 : 1);   // token within the tile
                        if (r_pair < p.rows && dcheck((ml * p.rows + r_pair) * 2 + 4 <= C::kYStageBytes, status))
                            stg[(ml * p.rows + r_pair) >> 1] = outw;
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    if (PAIR && !issuer)
                        mbar_arrive_remote(on_issuer(&accempty[b]));
                    else
                        mbar_arrive(&accempty[b]);
                }
                fence_proxy_async_smem();
                named_bar_sync(1, 32 * C::kNumEpiWarps);
                if (e == 0 && lane == 0) {
                    tma_store_2d(&map_y, smem, (tile % p.n_tiles) * n_stride + n_off, (tile / p.n_tiles) * BT);
                    bulk_commit_group();
                    bulk_wait_read_all();   // the shared memory may not be released before this
                }
            } else if (!split) {
                // Read the whole slice into registers (scaled, rounded to bf16), hand the
                // accumulator back to the MMA issuer, then store: the stores of this tile
                // overlap the next tile's MMAs.
                uint32_t packed[C::kEpiCols / 2];
#pragma unroll
                for (int c0 = 0; c0 < C::kEpiCols; c0 += kChunk) {
                    uint32_t v[32];
                    if (kChunk == 32) {
                        tmem_ld32(lane_base + b * BT + col0 + c0, v);
                    } else {
                        tmem_ld16(lane_base + b * BT + col0 + c0, *reinterpret_cast<uint32_t(*)[16]>(v));
                    }
                    const float mul_j = mul[c0 / kChunk];
                    tmem_wait_ld();
#pragma unroll
                    for (int j = 0; j < kChunk; j += 2) {
                        const float f0 = __uint_as_float(v[j]) * __shfl_sync(0xffffffffu, mul_j, j);
                        const float f1 = __uint_as_float(v[j + 1]) * __shfl_sync(0xffffffffu, mul_j, j + 1);
                        const __nv_bfloat162 h2 = __floats2bfloat162_rn(f0, f1);   // (token j, token j+1)
                        packed[(c0 + j) / 2] = *reinterpret_cast<const uint32_t*>(&h2);
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    if (PAIR && !issuer)
                        mbar_arrive_remote(on_issuer(&accempty[b]));
                    else
                        mbar_arrive(&accempty[b]);
                }
                // Lanes 2i and 2i+1 hold rows n and n+1: one shuffle turns each lane's
                // (token m, token m+1) pair into a 4-byte (row n, row n+1) store at one token.
                const bool even = (lane & 1) == 0;
                const int n_pair = even ? n : n - 1;
                const bool pair_ok = row_ok && (n_pair + 1 < p.N + 1) && n_pair < p.N;
#pragma unroll
                for (int j = 0; j < C::kEpiCols; j += 2) {
                    const uint32_t mine = packed[j / 2];
                    const uint32_t other = __shfl_xor_sync(0xffffffffu, mine, 1);
                    const uint32_t outw = even ? __byte_perm(mine, other, 0x5410) : __byte_perm(other, mine, 0x7632);
                    const int m = m0 + j + (even ? 0 : 1);
                    if (pair_ok && m < p.M &&
                        dcheck(m >= 0 && n_pair >= 0 && n_pair + 1 < p.N && (n_pair & 1) == 0, status))
                        *reinterpret_cast<uint32_t*>(p.Y + static_cast<size_t>(m) * p.N + n_pair) = outw;
                }
            } else {
                // split-K (one tile per CTA): the accumulator stays in tensor memory until every
                // rank of the cluster has finished its K slice, when it is pushed to the ranks
                // that reduce it (below). The row factors of the tile's tokens go to the weight
                // ring (every stage has been decoded by now), for the reduction to read from
                // shared memory instead of waiting on a global load behind each store.
                const int te = (warp - C::kFirstEpiWarp) * 32 + lane;
                const int mt = (tile / p.n_tiles) * BT;
                if (te < BT) reinterpret_cast<float*>(wring)[te] = (mt + te < p.M) ? p.rowmul[mt + te] : 1.0f;
            }
        }
    }

    __syncwarp();
    if (split) {
        // Sum the K slices of the cluster in rank order. Rank r owns a contiguous range of the
        // tile's token columns (a multiple of 4 wide). Once every rank has finished its slice
        // (barrier 1; their X rings are free), each rank pushes its fp32 partial of every range
        // into the owner's shared memory with remote stores, which do not wait for a reply;
        // after barrier 2 every owner adds the ranks' partials from its own shared memory,
        // scales them by the row factors and stores the bf16 result.
        // Receive buffer of an owner: [source rank][128 rows][P 16-byte chunks], P = its column
        // count / 4 made odd, so that 32 rows' chunks at one column fall in distinct banks.
        const int ks = p.ksplit;
        const int rank = static_cast<int>(kPairSplit ? ctarank >> 1 : cluster_ctarank());
        const int per_rank = ((BT + ks - 1) / ks + 3) / 4 * 4;
        const int chunks = per_rank / 4;
        const int P = chunks | 1;
        const uint32_t recv0 = smem_u32(smem);
        cluster_sync_all();   // barrier 1
        const bool epi = warp >= C::kFirstEpiWarp && warp < C::kFirstDqWarp;
        if (epi && !*abort_flag) {
            tc_fence_after();
            const int e = warp - C::kFirstEpiWarp;
            const int quarter = warp & 3;
            const int row = quarter * 32 + lane;
            const int col0 = (e >> 2) * C::kEpiCols;
            const uint32_t lane_base = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16);
            constexpr int kChunk = (C::kEpiCols >= 32) ? 32 : 16;
#pragma unroll
            for (int c0 = 0; c0 < C::kEpiCols; c0 += kChunk) {
                uint32_t v[32];
                if (kChunk == 32) {
                    tmem_ld32(lane_base + col0 + c0, v);
                } else {
                    tmem_ld16(lane_base + col0 + c0, *reinterpret_cast<uint32_t(*)[16]>(v));
                }
                tmem_wait_ld();
#pragma unroll
                for (int j = 0; j < kChunk; j += 4) {
                    const int col = col0 + c0 + j;
                    const int owner = col / per_rank;
                    const int cl = (col - owner * per_rank) >> 2;
                    const uint32_t off = static_cast<uint32_t>(((rank * kBlockN + row) * P + cl) * 16);
                    if (dcheck(owner < ks && off + 16 <= static_cast<uint32_t>(C::kXStages * C::kXStageBytes), status))
                        st_shared_cluster_v4(map_shared_rank(recv0 + off, static_cast<uint32_t>(kPairSplit ? 2 * owner + pair_rank : owner)),
                                             make_float4(__uint_as_float(v[j]), __uint_as_float(v[j + 1]),
                                                         __uint_as_float(v[j + 2]), __uint_as_float(v[j + 3])));
                }
            }
        }
        cluster_sync_all();   // barrier 2: every push has landed
        if (epi && !*abort_flag) {
            const int e = warp - C::kFirstEpiWarp;
            const int quarter = warp & 3;
            const int epart = e >> 2;
            const int row = quarter * 32 + lane;
            const int tile = tile0;
            const int m0 = (tile / p.n_tiles) * BT;
            const int n = (tile % p.n_tiles) * n_stride + n_off + row;
            const int cb = rank * per_rank;
            const int cend = min(min(BT, cb + per_rank), p.M - m0);
            const float* fac = reinterpret_cast<const float*>(wring);
            const float4* recv = reinterpret_cast<const float4*>(smem);
            if (row < p.rows && n < p.N) {
                constexpr int kStep = 4 * C::kEpiParts;
                for (int c = cb + 4 * epart; c < cend; c += kStep) {
                    const int cl = (c - cb) >> 2;
                    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
                    for (int q = 0; q < ks; ++q) {
                        const float4 v = recv[(q * kBlockN + row) * P + cl];
                        acc.x += v.x;
                        acc.y += v.y;
                        acc.z += v.z;
                        acc.w += v.w;
                    }
                    const float a4[4] = {acc.x, acc.y, acc.z, acc.w};
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int m = m0 + c + j;
                        if (m < p.M && dcheck(m >= 0 && n >= 0 && n < p.N && c + j < BT, status))
                            p.Y[static_cast<size_t>(m) * p.N + n] = __float2bfloat16_rn(a4[j] * fac[c + j]);
                    }
                }
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    // a pair's tensor memory is freed by both CTAs together, once neither uses it (and no
    // remote arrival or copy of one CTA targets the other after it has exited)
    if (PAIR) cluster_sync_all();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc<PAIR>(tmem_base, C::kTmemCols);
    }
}

}  // namespace lowbit
