// The products of the softmax cross entropy over a vocabulary, one kernel for sm_100a:
//
//   kVocabStats  l = X W^T, kept in tensor memory only: each tile leaves, per token, the maximum r of its
//                columns and s = sum exp(l - r), and the logit of the token's label
//   kVocabGrad   l again, and G = f (exp(l - lse) - [column = label]) in 16 bits, a piece of the columns at a time
//   kVocabDx     dX += G W over a piece (fp32 sums in the workspace)
//   kVocabDw     dW = G^T X, the rows of a piece, with G as two bf16 values, whose products are reduced one after the other:
//                of few tokens everywhere, of more where a label makes a block of 64 tokens by 256 rows (vocab_loss.cu)
//
// W is bf16, or decoded from packed binary, ternary or uint4 words inside the kernel. Precision: bf16 tables
// multiply bf16 x bf16; packed ones fp16 x fp16 on an exact fp16 copy of X (a power of two per row taken out),
// binary and ternary weights being exact in fp16. A uint4 weight (q - z) s is not: one rounding to fp16 (2^-11)
// moves a logit by some 2^-12 of |x||w|, which an fp32 loss shows, so the logits take it as the sum of two fp16
// values (2^-22, twice the MMAs); dX, rounded to bf16, takes the first of them. Sums are fp32 throughout.
//
// Design. A CTA's tile is 128 rows (tokens; vocabulary rows for dW) on the lanes of tensor memory, so that a
// softmax over columns stays inside a thread, by 128 columns, or 256 for a CTA pair (cta_group::2), each of whose
// CTAs holds half of the columns' operand. Both operands come through one shared-memory ring of 64-wide stages:
//   * warp 8 (one lane): TMA of the rows' operand, and of a bf16 table's rows;
//   * warp 10 (packed tables): TMA of the words and scales of 128 rows x 128 columns; warps 11-18 decode them, a row
//     of 64 codes per lane, into the swizzled layout the MMA reads;
//   * warp 9 (one lane): tcgen05.mma, two accumulators in tensor memory;
//   * warps 0-7: the epilogue of one tile, beside the MMAs of the next.
// Persistent grids; the logits' tiles go through the tokens first, so that a table's rows are read from memory once.
// Operands are K-major for the logits; for the gradients the table [v][k] (dX: reduced over v), G [m][v] and X [m][k]
// (dW: reduced over m) are read as they lie, as MN-major operands, so nothing is transposed.
// The narrow tiles serve up to 128 tokens: logits of bf16 tables, and dX; logits of packed ones are vocab_few.cuh's.
#pragma once

#include <atomic>

#include "gemm_kernel.cuh"
#include "vocab_internal.h"

namespace lowbit {
namespace vocab {

constexpr int kOperandBytes = 16384;    // 128 x 64 of the rows' operand, or of the columns' (of each of its terms)
constexpr int kEpiWarps = 8;

template <int MODE, int BITS, bool PAIR>
struct Cfg {
    static constexpr bool kPacked = BITS != kDense && MODE != kVocabDw;
    static_assert(MODE != kVocabDw || (BITS == kDense && PAIR), "dW: bf16 tables, CTA pairs");
    static constexpr bool kLogits = MODE == kVocabStats || MODE == kVocabGrad;
    static constexpr int kTerms = kLogits && BITS == 4 ? 2 : 1;   // fp16 values per weight
    static constexpr int kDqWarps = kPacked ? 8 : 0;
    static constexpr int kThreads = 32 * (kEpiWarps + (kPacked ? 3 : 2) + kDqWarps);
    static constexpr int kCols = PAIR ? 256 : 128;                // of a tile
    static constexpr int kRows = PAIR ? 256 : 128;
    // Two accumulators in turn; or one, of each term apart: the second term's sums are 2^-11 of the first's, and adding
    // them to those would cut twice as much off (the loss of 509 tokens against 100003 x 2560 uint4: 1.0e-6 off in the
    // norm, apart 5.8e-7, at 411 us instead of 382).
    static constexpr int kBufs = kTerms == 2 ? 1 : 2;
    static constexpr int kTmemCols = 2 * kCols;
    static_assert(kTerms == 1 || PAIR, "few tokens of uint4 tables: vocab_few.cuh");
    // Stages of words: kLogits 128 rows, kVocabDx 64 (one stage of the reduction), 128 codes of each
    static constexpr int kWRows = kLogits ? 128 : 64;
    static constexpr int kWRowBytes = kPacked ? 128 * BITS / 8 : 0;
    static constexpr int kWBytes = kWRows * kWRowBytes;
    static constexpr int kSBytes = kPacked ? 2 * kWRows * 2 : 0;  // room for two groups
    static constexpr int kZBytes = BITS == 4 ? kSBytes : 0;
    static constexpr int kWStageBytes = (kWBytes + kSBytes + kZBytes + 1023) / 1024 * 1024;
    // Rings: one of both operands (bf16 tables), or one of the rows' operand, which comes from L2 with some 1500 clocks
    // of latency, and a shorter one of the decoded columns' (in one ring the gradient of 77 tokens against uint4 rows
    // would wait for its rows).
    static constexpr int kAStageBytes = kPacked ? kOperandBytes : 2 * kOperandBytes;
    static constexpr int kBStageBytes = kPacked ? kTerms * kOperandBytes : 0;
    // (kVocabDx: 12, since a stage of its ring takes a stage of words, which come from memory: with 4 the gradient of 77
    // tokens waited for them, 37 us against 28)
    static constexpr int kWStages = !kPacked ? 0 : !kLogits ? 12 : kTerms == 2 ? 3 : 4;
    static constexpr int kStagingBytes = (MODE == kVocabGrad || MODE == kVocabDw) ? kEpiWarps * 4096 : 0;
    static constexpr int kRoom = kSmemLimit - 2048 - kStagingBytes - kWStages * kWStageBytes;
    static constexpr int kAStages = !kPacked ? kRoom / kAStageBytes : kTerms == 2 && kStagingBytes > 0 ? 4 : 6;
    static constexpr int kBFit = kPacked ? (kRoom - kAStages * kAStageBytes) / (kPacked ? kBStageBytes : 1) : 0;
    static constexpr int kBStages = kBFit > 6 ? 6 : kBFit;
    static_assert(kAStages >= 4 && (!kPacked || kBStages >= 3), "shared memory");
    static constexpr int kBOff = kAStages * kAStageBytes;
    static constexpr int kWOff = kBOff + kBStages * kBStageBytes;
    static constexpr int kStagingOff = kWOff + kWStages * kWStageBytes;
    static constexpr int kBarOff = kStagingOff + kStagingBytes;
    static constexpr int kSmemBytes = 1024 + kBarOff + 1024;
    static_assert(kSmemBytes <= kSmemLimit && kSmemBytes > kSmemLimit / 2, "one CTA per SM (tensor memory)");
    static constexpr bool kAMn = MODE == kVocabDw, kBMn = !kLogits;   // MN-major operands
    static constexpr uint32_t kIdesc = (BITS == kDense ? idesc_bf16_f32(kRows, kCols) : idesc_f16_f32(kRows, kCols)) |
                                       (kAMn ? kIdescTransposeA : 0u) | (kBMn ? kIdescTransposeB : 0u);
    // arrivals of decoding warps per stage: 128 rows (or 64 rows x two halves), 32 a warp
    static constexpr int kDqArrivals = 4 * (PAIR ? 2 : 1);
    static constexpr int kWReaders = kLogits ? 8 : 4;             // decoding warps that read a stage of words
};

struct Params {
    int M;                  // tokens
    int vocab;
    int stages;             // of a tile's whole reduction
    int per_slice;          // of a slice of it (kVocabDx), else `stages`
    int m_tiles, n_tiles, num_tiles;
    int v0;                 // first column (vocabulary row) of the piece
    int a_rows;             // rows of the rows' operand per stage (a tile of fewer tokens leaves the rest as it is)
    int groups;             // scale groups per 128 codes: 1 or 2
    uint32_t wtx;           // bytes of a stage of words
    float evened;           // kLogits: makes up for the sums' truncation
    const float* rowmul;    // packed: the power of two taken out of each token's row
    const int32_t* labels;
    const float* lse;
    const float* grad;
    float2* part;           // kVocabStats: [2 * n_tiles][M]
    float* target;          // [M]
    float* rest;            // kVocabGrad, bf16 tables: what rounding took from G's value at each token's label
    float4* acc;            // kVocabDx: [tile][CTA of the pair][warp][column / 4][lane]
    int accumulate;         // add to what acc holds
    float gscale;           // packed: the power of two in G
    int out_rows, out_cols; // kVocabGrad, kVocabDw: of what map_out covers
    int g_terms;            // bf16 tables: 2 where G is kept as two bf16 values for dW (map_s covers the second)
    int of_term;            // kVocabDw: stages of G's first term
    const uint32_t* marks;  // [rows / 256][mark_words]: a bit per 64 tokens whose second term is kept; nullptr: all
    int mark_words;
    unsigned* status;
};

constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float ex2(float x) {   // 2^x, within 2 ulp; 0 below fp32's normal range
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// True in one lane of the (converged) warp. The compiler knows it for one lane, and forms the operands of tcgen05.mma and
// TMA instructions in uniform registers at once: behind `lane == 0` an MMA took 90 clocks to issue, which held the tensor
// pipe at 53 % of its cycles for ternary tables (1537 tokens, gradient: 1375 us, with this 1143) and at 85 % for bf16.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}
__device__ __forceinline__ void tma_load_2d_pair(const CUtensorMap* map, uint32_t cluster_bar, void* dst, int c0, int c1) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4}], [%2];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(cluster_bar), "r"(c0), "r"(c1)
        : "memory");
}
__device__ __forceinline__ void st_shared_v4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
    uint32_t d;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
}

// One row's 64 codes of a stage of words, and their group's scale (and zero). piece(c) decodes columns 8c .. 8c + 7,
// one 16-byte piece of the operand's row, into `hi` and, for uint4 logits, what is left into `lo`, with packed fp16
// arithmetic only (conversions between fp32 and fp16 run at a fraction of its rate: forming (q - z) s in fp32 took
// 4600 clocks for 128 x 128 codes, this 1/5 of it). In block order pair p of a block's four words is one such piece.
template <int BITS, int TERMS>
struct Row64 {
    uint32_t words[2 * BITS];
    uint32_t s2, zh2, zl2;   // scale; zero, and what was left of it, in both halves

    __device__ __forceinline__ void load(const uint8_t* wrow, int row, int half, uint16_t s, uint16_t z) {
        if (BITS == 1) {
            const uint2 v = *reinterpret_cast<const uint2*>(wrow + half * 8);
            words[0] = v.x;
            words[1] = v.y;
        } else {
#pragma unroll
            for (int q = 0; q < BITS / 2; ++q) {
                // (TMA's 32- and 64-byte swizzles)
                const int chunk = BITS == 2 ? half ^ ((row >> 2) & 1) : (2 * half + q) ^ ((row >> 1) & 3);
                const uint4 v = *reinterpret_cast<const uint4*>(wrow + chunk * 16);
                words[4 * q] = v.x; words[4 * q + 1] = v.y; words[4 * q + 2] = v.z; words[4 * q + 3] = v.w;
            }
        }
        s2 = s | (static_cast<uint32_t>(s) << 16);
        if (BITS == 4) {
            zh2 = z | (static_cast<uint32_t>(z) << 16);
            if (TERMS == 2) {
                // z = zh + zl, both exact, with zh of the step that fp16 has at |z| + 24 (2^-6 up to |z| = 8), so that
                // q - zh, at most |z| + 15.5, is exact in fp16 as long as that step is at most 1 (|z| <= 2000): adding 24 of
                // z's own sign and taking it off again rounds z to it. (With 24 of one sign a z below -8 kept its finer
                // step, and q - z was rounded: 2^-7 of the scale at -9.0078.) From 2^14 on zh = z.
                const uint32_t k24 = 0x4E004E00u | (zh2 & 0x80008000u);
                const uint32_t zr = f16x2_sub(f16x2_fma(zh2, 0x3C003C00u, k24), k24);
                const uint32_t rest = f16x2_sub(zr, zh2);   // -zl
                const bool coarse = (z & 0x7FFFu) < 0x7400u;
                zl2 = coarse ? rest : 0u;
                zh2 = coarse ? zr : zh2;
            }
        }
    }
    __device__ __forceinline__ void piece(int c, uint32_t (&hi)[4], uint32_t (&lo)[4]) const {
        constexpr uint32_t kMagic = 0x64006400u;   // 1024.0, and the constants of decode_word_b2 / _b4
        constexpr uint32_t kMul[5] = {0x3C003C00u, 0x34003400u, 0x2C002C00u, 0x24002400u, 0x1C001C00u};
        constexpr uint32_t kAdd2[5] = {0xE401E401u, 0xDC04DC04u, 0xD410D410u, 0xCC40CC40u, 0xC500C500u};
        constexpr uint32_t kAdd4[2] = {0xE400E400u, 0xD400D400u};
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            if (BITS == 1) {            // plain order: pairs 4 (c % 4) .. + 3 of word c / 4
                hi[q] = xor_andnot(s2, words[c >> 2] << (15 - (4 * (c & 3) + q)), 0x80008000u);
            } else if (BITS == 2) {     // pair c of word q: f - 1 exactly, times s exactly
                const int j = c < 5 ? c : c - 5;
                const uint32_t e = and_or(words[q] >> (c < 5 ? 0 : 10), 0x00030003u << (2 * j), kMagic);
                hi[q] = f16x2_mul(f16x2_fma(e, kMul[j], kAdd2[j]), s2);
            } else {                    // pair c % 4 of word q of block c / 4
                const int k = c & 3;
                const uint32_t e = and_or(words[4 * (c >> 2) + q] >> (k < 2 ? 0 : 8), 0x000F000Fu << (4 * (k & 1)), kMagic);
                const uint32_t d = f16x2_sub(f16x2_fma(e, kMul[2 * (k & 1)], kAdd4[k & 1]), zh2);
                hi[q] = f16x2_mul(d, s2);
                // d s = hi + (d s - hi), the second exact in fp16 (above its smallest step), and (q - z) s = d s - zl s:
                // |lo| <= 2^-11 (|d| + |z| + 24) s, rounded once (its parts below fp16's normal range: 2^-24)
                if (TERMS == 2) lo[q] = f16x2_fma(zl2, s2, f16x2_fma(d, s2, hi[q] ^ 0x80008000u));
            }
        }
    }
};

// The stages of a tile of dW behind those of G's first term: of its second, 64 tokens each, where `marks` has a bit.
struct MarkedStages {
    const uint32_t* marks = nullptr;   // of the tile's 256 rows
    int words = 0, next_word = 0;
    uint32_t left = 0;
    __device__ __forceinline__ int next() {   // the next one's tokens / 64, or -1
        while (!left) {
            if (next_word == words) return -1;
            left = marks[next_word++];
        }
        const int bit = __ffs(left) - 1;
        left &= left - 1;
        return 32 * (next_word - 1) + bit;
    }
};

template <int MODE, int BITS, bool PAIR>
__global__ void __launch_bounds__(Cfg<MODE, BITS, PAIR>::kThreads, 1)
    vocab_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
                 const __grid_constant__ CUtensorMap map_s, const __grid_constant__ CUtensorMap map_z,
                 const __grid_constant__ CUtensorMap map_out, const __grid_constant__ Params p) {
    using C = Cfg<MODE, BITS, PAIR>;
    constexpr int S = C::kAStages, SB = C::kBStages > 0 ? C::kBStages : 1, SW = C::kWStages > 0 ? C::kWStages : 1, T = C::kTerms;
    constexpr int kCtas = PAIR ? 2 : 1;

    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kBarOff);
    uint64_t* empty = full + S;
    uint64_t* bfull = empty + S;      // packed: the decoded operand's ring
    uint64_t* bempty = bfull + SB;
    uint64_t* wfull = bempty + SB;
    uint64_t* wempty = wfull + SW;
    uint64_t* accfull = wempty + SW;
    uint64_t* accempty = accfull + 2;
    uint64_t* drain = accempty + 2;
    uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(drain + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = PAIR ? cluster_ctarank() : 0u;
    const bool issuer = rank == 0;
    auto on_issuer = [&](uint64_t* bar) { return map_shared_rank(smem_u32(bar), 0); };
    auto arrive_on_issuer = [&](uint64_t* bar) {
        if (PAIR && !issuer)
            mbar_arrive_remote(on_issuer(bar));
        else
            mbar_arrive(bar);
    };

    if (threadIdx.x == 0) {
        for (int i = 0; i < S; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < SB; ++i) {
            mbar_init(&bfull[i], C::kDqArrivals);
            mbar_init(&bempty[i], 1);
        }
        for (int i = 0; i < SW; ++i) {
            mbar_init(&wfull[i], 1);
            mbar_init(&wempty[i], C::kWReaders);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&accfull[i], 1);
            mbar_init(&accempty[i], kCtas * kEpiWarps);
        }
        mbar_init(drain, 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 8 && lane == 0) {
        tma_prefetch_desc(&map_a);
        tma_prefetch_desc(&map_b);
        if (C::kPacked) tma_prefetch_desc(&map_s);
    }
    if (warp == 9) {
        tmem_alloc<PAIR>(tmem_holder, C::kTmemCols);
        tmem_relinquish<PAIR>();
    }
    tc_fence_before();
    __syncthreads();
    if (PAIR) cluster_sync_all();   // both CTAs' barriers are initialised before either uses the other's
    tc_fence_after();
    const uint32_t tmem_base = *tmem_holder;
    grid_launch_dependents();
    grid_dependency_wait();

    const int tile0 = static_cast<int>(PAIR ? blockIdx.x >> 1 : blockIdx.x);
    const int tile_step = static_cast<int>(PAIR ? gridDim.x >> 1 : gridDim.x);
    const int per_mn = p.m_tiles * p.n_tiles;
    // Tile t of the grid: rows [m0, ..) and columns [n0, ..) of this CTA's, stages [j0, j1) of the reduction.
    struct Tile {
        int m0, n0, j0, j1;
    };
    auto tile_of = [&](int t) {
        const int slice = t / per_mn, mn = t - slice * per_mn;
        // (dW: through the columns first, so that G, the larger operand, is read from memory once: a third of the time
        // was spent on it otherwise)
        const int n = MODE == kVocabDw ? mn % p.n_tiles : mn / p.m_tiles, m = MODE == kVocabDw ? mn / p.n_tiles : mn - n * p.m_tiles;
        Tile r;
        r.m0 = m * C::kRows + static_cast<int>(rank) * 128;
        r.n0 = n * C::kCols;
        r.j0 = slice * p.per_slice;
        r.j1 = min(p.stages, r.j0 + p.per_slice);
        return r;
    };
    auto marked_of = [&](const Tile& tl) {
        MarkedStages w;
        if (MODE == kVocabDw && p.marks) {
            w.marks = p.marks + static_cast<size_t>((p.v0 + tl.m0) / 256) * p.mark_words;
            w.words = p.mark_words;
        }
        return w;
    };
    // The stage after j of a tile (those of G's second term count on behind the first's), or -1.
    auto stage_after = [&](int j, const Tile& tl, MarkedStages& marked) {
        if (j + 1 < tl.j1) return j + 1;
        if (MODE != kVocabDw) return -1;
        const int s = marked.next();
        return s < 0 ? -1 : p.of_term + s;
    };

    if (warp == 8) {
        // ------------------------------------------------------------ TMA of the rows' operand, and of a bf16 table
        if (elect_one()) {
            uint32_t it = 0;
            bool ok = true;
            const uint32_t bytes = MODE == kVocabDw ? C::kAStageBytes : (C::kPacked ? 0 : kOperandBytes) + p.a_rows * 128;
            for (int t = tile0; t < p.num_tiles && ok; t += tile_step) {
                const Tile tl = tile_of(t);
                const int nb = tl.n0 + static_cast<int>(rank) * 128;   // first of this CTA's half of the columns
                MarkedStages marked = marked_of(tl);
                for (int j = tl.j0; j >= 0; j = stage_after(j, tl, marked), ++it) {
                    const uint32_t s = it % S;
                    if (!mbar_wait(&empty[s], ((it / S) & 1u) ^ 1u, abort_flag, p.status)) { ok = false; break; }
                    uint8_t* a = smem + s * C::kAStageBytes;
                    uint8_t* b = a + kOperandBytes;
                    if (issuer) mbar_arrive_expect_tx(&full[s], kCtas * bytes);
                    auto load = [&](const CUtensorMap* map, uint8_t* dst, int x, int y) {
                        if (PAIR)
                            tma_load_2d_pair(map, on_issuer(&full[s]), dst, x, y);
                        else
                            tma_load_2d(map, &full[s], dst, x, y);
                    };
                    if (MODE == kVocabDw) {          // G [m][v], X [m][k]: 64 tokens, two boxes of 64 columns each
                        const int y = (j < p.of_term ? j : j - p.of_term) * 64;
                        const CUtensorMap* map_g = j < p.of_term ? &map_a : &map_s;
                        load(map_g, a, tl.m0, y);
                        load(map_g, a + 8192, tl.m0 + 64, y);
                        load(&map_b, b, nb, y);
                        load(&map_b, b + 8192, nb + 64, y);
                    } else {
                        load(&map_a, a, j * 64, tl.m0);
                        if (MODE == kVocabDx && !C::kPacked) {   // W [v][k]: 64 rows
                            load(&map_b, b, nb, p.v0 + j * 64);
                            load(&map_b, b + 8192, nb + 64, p.v0 + j * 64);
                        } else if (!C::kPacked) {
                            load(&map_b, b, j * 64, p.v0 + nb);
                        }
                    }
                }
            }
            if (!ok) {
                // Wait (bounded) for the copies still in flight before the CTA exits. The second CTA of a pair cannot
                // wait on the issuer's barrier that its copies count on: it gives them a fixed time instead.
                if (PAIR && !issuer) {
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
            uint32_t it = 0, n = 0;
            bool ok = true, issued = false;
            for (int t = tile0; t < p.num_tiles && ok; t += tile_step, ++n) {
                const Tile tl = tile_of(t);
                const uint32_t b = n % C::kBufs;
                if (!mbar_wait(&accempty[b], ((n / C::kBufs) & 1u) ^ 1u, abort_flag, p.status)) { ok = false; break; }
                tc_fence_after();
                MarkedStages marked = marked_of(tl);
                for (int j = tl.j0; j >= 0; j = stage_after(j, tl, marked), ++it) {
                    const uint32_t s = it % S, sb = it % SB;
                    if (!mbar_wait(&full[s], (it / S) & 1u, abort_flag, p.status) ||
                        (C::kPacked && !mbar_wait(&bfull[sb], (it / SB) & 1u, abort_flag, p.status))) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t as = smem_u32(smem + s * C::kAStageBytes);
                    const uint32_t b0 = C::kPacked ? smem_u32(smem + C::kBOff + sb * C::kBStageBytes) : as + kOperandBytes;
#pragma unroll
                    for (int i = 0; i < 4 * T; ++i) {
                        const int kk = i & 3;
                        const uint32_t bs = b0 + (i >> 2) * kOperandBytes;
                        const uint64_t ad = C::kAMn ? smem_desc_mn(as + kk * 2048, 128, 8192) : smem_desc_k_sw128(as + kk * 32);
                        const uint64_t bd = C::kBMn ? smem_desc_mn(bs + kk * 2048, 128, 8192) : smem_desc_k_sw128(bs + kk * 32);
                        const uint32_t d = tmem_base + (T == 2 ? i >> 2 : b) * C::kCols;
                        const uint32_t more = (j > tl.j0 || kk > 0) ? 1u : 0u;
                        if (PAIR)
                            mma_f16_ss_pair(d, ad, bd, C::kIdesc, more);
                        else
                            mma_f16_ss(d, ad, bd, C::kIdesc, more);
                    }
                    issued = true;
                    auto release = [&](uint64_t* bar) {
                        if (PAIR)
                            mma_commit_pair_mc(bar, 0x3);
                        else
                            mma_commit(bar);
                    };
                    release(&empty[s]);
                    if (C::kPacked) release(&bempty[sb]);
                }
                if (!ok) break;
                if (PAIR)
                    mma_commit_pair_mc(&accfull[b], 0x3);
                else
                    mma_commit(&accfull[b]);
            }
            if (!ok && issued) {   // no MMA may still write tensor memory when it is freed
                if (PAIR)
                    mma_commit_pair(drain);
                else
                    mma_commit(drain);
                const long long t0 = clock64();
                while (!mbar_try_wait(drain, 0) && clock64() - t0 < kWaitLimitCycles / 64) {
                }
            }
        }
    } else if (C::kPacked && warp == 10) {
        // ------------------------------------------------------------ TMA of words and scales
        if constexpr (C::kPacked) {
            if (elect_one()) {
                uint32_t it = 0;
                bool ok = true;
                for (int t = tile0; t < p.num_tiles && ok; t += tile_step) {
                    const Tile tl = tile_of(t);
                    const int nb = tl.n0 + static_cast<int>(rank) * 128;
                    // (kLogits: a stage of words is two stages of the ring, and a tile has them all)
                    const int w1 = C::kLogits ? p.stages / 2 : tl.j1;
                    for (int w = C::kLogits ? 0 : tl.j0; w < w1; ++w, ++it) {
                        const uint32_t s = it % SW;
                        if (!mbar_wait(&wempty[s], ((it / SW) & 1u) ^ 1u, abort_flag, p.status)) { ok = false; break; }
                        uint8_t* st = smem + C::kWOff + s * C::kWStageBytes;
                        mbar_arrive_expect_tx(&wfull[s], p.wtx);
                        const int wx = C::kLogits ? w * (4 * BITS) : nb * BITS / 32, v = p.v0 + (C::kLogits ? nb : w * 64);
                        const int sy = (C::kLogits ? w : nb / 128) * p.groups;
                        tma_load_2d(&map_b, &wfull[s], st, wx, v);
                        tma_load_2d(&map_s, &wfull[s], st + C::kWBytes, v, sy);
                        if (BITS == 4) tma_load_2d(&map_z, &wfull[s], st + C::kWBytes + C::kSBytes, v, sy);
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
        }
    } else if (C::kPacked && warp >= 11) {
        // ------------------------------------------------------------ decoding warps
        if constexpr (C::kPacked) {
            const int dq = warp - 11;
            const int row = (C::kLogits ? (dq & 3) : (dq & 1)) * 32 + lane;
            const int half = C::kLogits ? dq >> 2 : (dq >> 1) & 1;   // which 64 of a row's 128 codes
            uint32_t wit = 0;   // stages of words seen
            uint32_t it = 0;    // stages of the ring before the present stage of words
            bool ok = true;
            for (int t = tile0; t < p.num_tiles && ok; t += tile_step) {
                const Tile tl = tile_of(t);
                const int count = C::kLogits ? p.stages / 2 : tl.j1 - tl.j0;
                for (int w = 0; w < count; ++w, ++wit, it += C::kLogits ? 2 : 1) {
                    if (!C::kLogits && (it & 1u) != static_cast<uint32_t>(dq >> 2)) continue;   // the other four warps'
                    const uint32_t ws = wit % SW;
                    if (!__all_sync(0xffffffffu, mbar_wait(&wfull[ws], (wit / SW) & 1u, abort_flag, p.status))) { ok = false; break; }
                    const uint8_t* st = smem + C::kWOff + ws * C::kWStageBytes;
                    const uint8_t* wrow = st + row * C::kWRowBytes;
                    const int at = (p.groups == 2 ? half : 0) * C::kWRows + row;
                    Row64<BITS, T> codes;
                    codes.load(wrow, row, half, reinterpret_cast<const uint16_t*>(st + C::kWBytes)[at],
                               BITS == 4 ? reinterpret_cast<const uint16_t*>(st + C::kWBytes + C::kSBytes)[at] : uint16_t(0));
                    const uint32_t i = it + (C::kLogits ? half : 0), s = i % SB;   // the stage of the ring that it fills
                    if (!__all_sync(0xffffffffu, mbar_wait(&bempty[s], ((i / SB) & 1u) ^ 1u, abort_flag, p.status))) { ok = false; break; }
                    // kLogits: 128 rows of 64 columns; kVocabDx: two halves of 64 rows
                    const uint32_t dst = smem_u32(smem + C::kBOff + s * C::kBStageBytes) + (C::kLogits ? 0 : half * 8192) + row * 128;
#pragma unroll
                    for (int c = 0; c < 8; ++c) {
                        uint32_t hi[4], lo[4];
                        codes.piece(c, hi, lo);
                        const uint32_t to = (c ^ (row & 7)) << 4;
                        st_shared_v4(dst + to, hi[0], hi[1], hi[2], hi[3]);
                        if (T == 2) st_shared_v4(dst + kOperandBytes + to, lo[0], lo[1], lo[2], lo[3]);
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) arrive_on_issuer(&bfull[s]);
                    // (freed behind the last use of what was read from it)
                    if (lane == 0) mbar_arrive(&wempty[ws]);
                }
            }
        }
    } else if (warp < kEpiWarps) {
        // ------------------------------------------------------------ epilogue
        const int quarter = warp & 3, part = warp >> 2;
        constexpr int kCols = C::kCols / 2;                  // this warp's half of the tile's columns
        const uint32_t lane_base = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16);
        [[maybe_unused]] const uint32_t staging = smem_u32(smem + C::kStagingOff + warp * 4096);
        uint32_t n = 0;
        for (int t = tile0; t < p.num_tiles; t += tile_step, ++n) {
            const Tile tl = tile_of(t);
            const uint32_t b = n % C::kBufs;
            const int r0 = tl.m0 + quarter * 32, row = r0 + lane;
            const int c0 = tl.n0 + part * kCols;             // first column, within the piece
            const int left = p.vocab - (p.v0 + c0);          // columns of the vocabulary from there on
            // what the token needs, requested before the accumulator is waited for
            [[maybe_unused]] int label = -1;
            [[maybe_unused]] float mul = 1.f, shift = 0.f, f = 0.f;
            [[maybe_unused]] uint32_t marks = 0xffffffffu;   // (a tile's columns are 256 rows of dW)
            if (MODE == kVocabGrad && BITS == kDense && PAIR && p.marks && r0 < p.M)
                marks = p.marks[static_cast<size_t>((p.v0 + tl.n0) / 256) * p.mark_words + r0 / 2048];
            if (C::kLogits && row < p.M) {
                label = p.labels[row];
                if (static_cast<unsigned>(label) >= static_cast<unsigned>(p.vocab)) label = -1;
                mul = C::kPacked ? p.rowmul[row] * p.evened : p.evened;
                if (MODE == kVocabGrad) {
                    shift = p.lse[row] * kLog2e;
                    f = C::kPacked ? p.gscale : p.grad[row];
                }
            }
            const uint32_t acc = lane_base + b * C::kCols + part * kCols;
            if (!__all_sync(0xffffffffu, mbar_wait(&accfull[b], (n / C::kBufs) & 1u, abort_flag, p.status))) break;
            tc_fence_after();
            // 32 columns of the accumulator (both terms' sums)
            auto load32 = [&](int c, uint32_t (&v)[32]) {
                tmem_ld32(acc + c, v);
                if constexpr (T == 2) {
                    uint32_t w[32];
                    tmem_ld32(acc + C::kCols + c, w);
                    tmem_wait_ld();
#pragma unroll
                    for (int j = 0; j < 32; ++j) v[j] = __float_as_uint(__uint_as_float(v[j]) + __uint_as_float(w[j]));
                } else {
                    tmem_wait_ld();
                }
            };
            if constexpr (MODE == kVocabStats) {
                if (r0 < p.M) {
                    const float rl = mul * kLog2e;
                    const int want = label >= 0 ? label - (p.v0 + c0) : -1;   // the label's place in this warp's columns
                    float top = -INFINITY;
#pragma unroll 1
                    for (int c = 0; c < kCols; c += 32) {
                        uint32_t v[32];
                        load32(c, v);
                        if (left < c + 32) {
#pragma unroll
                            for (int j = 0; j < 32; ++j)
                                if (c + j < left) top = fmaxf(top, __uint_as_float(v[j]));
                        } else {
                            float m4[4] = {top, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                            for (int j = 0; j < 32; ++j) m4[j & 3] = fmaxf(m4[j & 3], __uint_as_float(v[j]));
                            top = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
                        }
                        if (static_cast<unsigned>(want - c) < 32u) {
                            float l = 0.f;
#pragma unroll
                            for (int j = 0; j < 32; ++j)
                                if (j == want - c) l = __uint_as_float(v[j]);
                            p.target[row] = l * mul;
                        }
                    }
                    // An infinite maximum stands aside: with no column at all s is 0, with +inf s is +inf.
                    const bool inf = fabsf(top) == INFINITY;
                    const float off = inf ? 0.f : -top * rl;
                    float s4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
                    for (int c = 0; c < kCols; c += 32) {
                        uint32_t v[32];
                        load32(c, v);
                        if (left < c + 32) {
#pragma unroll
                            for (int j = 0; j < 32; ++j)
                                if (c + j < left) s4[0] += ex2(fmaf(__uint_as_float(v[j]), rl, off));
                        } else {
#pragma unroll
                            for (int j = 0; j < 32; ++j) s4[j & 3] += ex2(fmaf(__uint_as_float(v[j]), rl, off));
                        }
                    }
                    const float s = (s4[0] + s4[1]) + (s4[2] + s4[3]);
                    const float r = inf ? (top > 0.f ? 3.4e38f : -INFINITY) : top * mul;
                    if (row < p.M) p.part[static_cast<size_t>(2 * (tl.n0 / C::kCols) + part) * p.M + row] = make_float2(r, s);
                }
            } else if constexpr (MODE == kVocabGrad || MODE == kVocabDw) {
                const float rl = mul * kLog2e;
                const int want = label >= 0 ? label - (p.v0 + c0) : -1;
                // (64 columns at a time; G's second term, where it is kept, behind the first)
                const int terms = MODE == kVocabGrad && BITS == kDense ? (((marks >> (r0 / 64 % 32)) & 1u) ? p.g_terms : 1) : 1;
#pragma unroll 1
                for (int i = 0; i < kCols / 64 * terms; ++i) {
                    const int c = (terms == 1 ? i : i >> 1) * 64;
                    const bool second = terms == 2 && (i & 1);
                    // the staging rows are read out by the previous store
                    if (lane == 0) bulk_wait_read_all();
                    __syncwarp();
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        uint32_t v[32];
                        load32(c + h * 32, v);
                        uint32_t o[16];
#pragma unroll
                        for (int j = 0; j < 32; j += 2) {
                            float e[2];
#pragma unroll
                            for (int k = 0; k < 2; ++k) {
                                const int col = c + h * 32 + j + k;
                                e[k] = __uint_as_float(v[j + k]);
                                if constexpr (MODE == kVocabGrad) {
                                    float g = ex2(fmaf(e[k], rl, -shift));
                                    if (col == want) g -= 1.f;
                                    e[k] = label >= 0 && col < left ? g * f : 0.f;
                                    if (BITS == kDense && (second || col == want)) {
                                        const float left_over = e[k] - __bfloat162float(__float2bfloat16_rn(e[k]));
                                        if (col == want) p.rest[row] = left_over;
                                        if (second) e[k] = fabsf(e[k]) < INFINITY ? left_over : 0.f;
                                    }
                                }
                            }
                            o[j / 2] = BITS == kDense ? pack_bf16x2(e[0], e[1]) : pack_f16x2(e[0], e[1]);
                        }
#pragma unroll
                        for (int q = 0; q < 4; ++q)
                            st_shared_v4(staging + lane * 128 + (((h * 4 + q) ^ (lane & 7)) << 4), o[4 * q], o[4 * q + 1],
                                         o[4 * q + 2], o[4 * q + 3]);
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0 && r0 < p.out_rows && c0 + c < p.out_cols) {
                        tma_store_2d(second ? &map_s : &map_out, smem + C::kStagingOff + warp * 4096, c0 + c, r0);
                        bulk_commit_group();
                    }
                }
            } else {
                float4* dst = p.acc + ((static_cast<size_t>(t) * kCtas + rank) * kEpiWarps + warp) * (kCols / 4) * 32 + lane;
                if (r0 < p.M) {
#pragma unroll 1
                    for (int c = 0; c < kCols; c += 32) {
                        uint32_t v[32];
                        tmem_ld32(acc + c, v);
                        float4 old[8];
                        if (p.accumulate) {
#pragma unroll
                            for (int q = 0; q < 8; ++q) old[q] = dst[(c / 4 + q) * 32];
                        } else {
#pragma unroll
                            for (int q = 0; q < 8; ++q) old[q] = make_float4(0.f, 0.f, 0.f, 0.f);
                        }
                        tmem_wait_ld();
#pragma unroll
                        for (int q = 0; q < 8; ++q)
                            dst[(c / 4 + q) * 32] =
                                make_float4(old[q].x + __uint_as_float(v[4 * q]), old[q].y + __uint_as_float(v[4 * q + 1]),
                                            old[q].z + __uint_as_float(v[4 * q + 2]), old[q].w + __uint_as_float(v[4 * q + 3]));
                    }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) arrive_on_issuer(&accempty[b]);
        }
        if (C::kStagingBytes > 0 && lane == 0) bulk_wait_read_all();
    }

    __syncwarp();
    tc_fence_before();
    __syncthreads();
    // a pair's tensor memory is freed by both CTAs together, once neither uses it (and no remote arrival or copy of
    // one CTA targets the other after it has exited)
    if (PAIR) cluster_sync_all();
    if (warp == 9) {
        tc_fence_after();
        tmem_dealloc<PAIR>(tmem_base, C::kTmemCols);
    }
}

// The shared-memory opt-in, once per kernel and device.
template <int MODE, int BITS, bool PAIR, bool FEW>
bool opt_in(const void* fn, int bytes) {
    static std::atomic<uint64_t> devices{0};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return false;
    const uint64_t bit = dev < 64 ? (uint64_t(1) << dev) : 0;
    if (!bit || !(devices.load(std::memory_order_acquire) & bit)) {
        if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess) return false;
        devices.fetch_or(bit, std::memory_order_acq_rel);
    }
    return true;
}
inline CUtensorMapSwizzle word_swizzle(int row_bytes) {
    return row_bytes == 16 ? CU_TENSOR_MAP_SWIZZLE_NONE : row_bytes == 32 ? CU_TENSOR_MAP_SWIZZLE_32B : CU_TENSOR_MAP_SWIZZLE_64B;
}
// The tensor cores cut what they add to an accumulator off below its last bit, towards zero. A logit that counts in a softmax
// is a sum of products of both signs that grows to it, on average over the columns' order in proportion: over n MMA steps it
// loses 0.26 n 2^-24 of itself, always to the same side, with a spread of a fifth of that, and is scaled up by as much.
// 509 tokens of normal values against 8000 rows, all formats, off in the norm: K = 2560 lse 5 to 9e-8 and loss 2.5 to 2.9e-7
// (unscaled 9e-7 and 1.0 to 1.1e-6); K = 8192 1 to 2e-7 and 8 to 10e-7 (3e-6 and 3.5e-6); with four columns fifty times the
// others, K = 2560, loss 1.2 to 1.6e-6 (3.1 to 3.7e-6). Sums that grow otherwise lose otherwise: where a few large products come
// last nothing, so that the factor stays (2.5e-6 of the logit at K = 2560), where they come first up to 4.4 x 2^-24 a step, and
// of one sign throughout 0.4 to 1.6. Measured up to 4096 steps; more are scaled as those.
inline float evened(int stages) { return 1.f + 0.26f * 5.9604645e-8f * 4.f * static_cast<float>(stages < 1024 ? stages : 1024); }
// CTA pairs that the GPU holds at once.
inline int pair_slots(const void* fn, int threads, int smem_bytes) {
    int pairs = cluster_capacity(fn, 2, threads, smem_bytes, true);
    if (pairs > num_sms() / 2) pairs = num_sms() / 2;
    return pairs < 1 ? 1 : pairs;
}

template <int MODE, int BITS, bool PAIR>
lowbit_status launch(const VocabProduct& v, cudaStream_t stream) {
    using C = Cfg<MODE, BITS, PAIR>;
    auto kernel = vocab_kernel<MODE, BITS, PAIR>;
    const void* fn = reinterpret_cast<const void*>(kernel);
    if (!opt_in<MODE, BITS, PAIR, false>(fn, C::kSmemBytes)) return LOWBIT_ERR_CUDA;
    const LossProblem& q = *v.p;
    const LossLayout& l = *v.l;
    const Table& w = q.table;
    const uint64_t M = q.M, K = w.K, vocab = q.vocab, ld = l.piece;
    const CUtensorMapDataType half =
        BITS == kDense ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    const CUtensorMapSwizzle sw = CU_TENSOR_MAP_SWIZZLE_128B;
    CUtensorMap ma, mb, ms, mz, mo;
    bool ok = true;
    uint64_t rows = M;
    const uint32_t a_rows = M >= 128 ? 128 : (static_cast<uint32_t>(M) + 7) / 8 * 8;
    void* g = v.ws + l.g;
    if (MODE == kVocabDw) {
        ok = ok && make_map_2d(&ma, half, 2, g, ld, M, ld * 2, 64, 64, sw);
        ok = ok && make_map_2d(&mb, half, 2, v.ws + l.xz, K, M, K * 2, 64, 64, sw);
        rows = v.cols;
        ok = ok && make_map_2d(&mo, half, 2, static_cast<uint8_t*>(q.dW) + static_cast<size_t>(v.v0) * K * 2, K, rows, K * 2, 64, 32, sw);
    } else {
        const void* x = BITS == kDense ? q.X : v.ws + l.xh;
        ok = ok && (C::kLogits ? make_map_2d(&ma, half, 2, x, K, M, K * 2, 64, a_rows, sw)
                               : make_map_2d(&ma, half, 2, g, ld, M, ld * 2, 64, a_rows, sw));
        if (!C::kPacked) {
            ok = ok && make_map_2d(&mb, half, 2, w.rows, K, vocab, K * 2, 64, C::kLogits ? 128 : 64, sw);
        } else {
            ok = ok && make_map_2d(&mb, CU_TENSOR_MAP_DATA_TYPE_UINT32, 4, w.rows, K * BITS / 32, vocab, K * BITS / 8,
                                   C::kWRowBytes / 4, C::kWRows, word_swizzle(C::kWRowBytes));
            const uint32_t groups = 128 / w.group_size;
            ok = ok && make_map_2d(&ms, CU_TENSOR_MAP_DATA_TYPE_UINT16, 2, w.scales, vocab, K / w.group_size,
                                   static_cast<uint64_t>(w.N) * 2, C::kWRows, groups, CU_TENSOR_MAP_SWIZZLE_NONE);
            if (BITS == 4)
                ok = ok && make_map_2d(&mz, CU_TENSOR_MAP_DATA_TYPE_UINT16, 2, w.zeros, vocab, K / w.group_size,
                                       static_cast<uint64_t>(w.N) * 2, C::kWRows, groups, CU_TENSOR_MAP_SWIZZLE_NONE);
        }
        mo = ma;
        if (MODE == kVocabGrad) ok = ok && make_map_2d(&mo, half, 2, g, ld, M, ld * 2, 64, 32, sw);
    }
    if (!C::kPacked) ms = mb;
    if (BITS == kDense && l.g_terms == 2 && (MODE == kVocabGrad || MODE == kVocabDw))
        ok = ok && make_map_2d(&ms, half, 2, v.ws + l.g + M * ld * 2, ld, M, ld * 2, 64, MODE == kVocabDw ? 64 : 32, sw);
    if (BITS != 4) mz = ms;
    Params p = {};
    p.status = device_status_address();
    if (!ok || !p.status) return LOWBIT_ERR_CUDA;
    p.M = static_cast<int>(M);
    p.vocab = static_cast<int>(vocab);
    p.v0 = static_cast<int>(v.v0);
    p.a_rows = static_cast<int>(a_rows);
    if (C::kPacked) {
        p.groups = 128 / w.group_size;
        p.wtx = static_cast<uint32_t>(C::kWBytes + (BITS == 4 ? 2 : 1) * p.groups * C::kWRows * 2);
    }
    const int64_t cols = v.cols;
    if (C::kLogits) {
        p.stages = static_cast<int>(C::kPacked ? (K + 127) / 128 * 2 : (K + 63) / 64);
        p.m_tiles = static_cast<int>(l.m_tiles);
        p.n_tiles = static_cast<int>((cols + C::kCols - 1) / C::kCols);
    } else if (MODE == kVocabDx) {
        p.stages = static_cast<int>((cols + 63) / 64);
        p.m_tiles = static_cast<int>(l.m_tiles);
        p.n_tiles = static_cast<int>(l.dx_tiles);
    } else {
        p.of_term = static_cast<int>((M + 63) / 64);
        p.stages = p.of_term * (l.mark_words ? 1 : l.g_terms);
        p.m_tiles = static_cast<int>((cols + C::kRows - 1) / C::kRows);
        p.n_tiles = static_cast<int>((K + C::kCols - 1) / C::kCols);
    }
    p.evened = evened(p.stages);
    int slices = 1;
    if (MODE == kVocabDx) {
        slices = l.slices < p.stages ? l.slices : p.stages;
        p.per_slice = (p.stages + slices - 1) / slices;
        slices = (p.stages + p.per_slice - 1) / p.per_slice;
    } else {
        p.per_slice = p.stages;
    }
    p.num_tiles = p.m_tiles * p.n_tiles * slices;
    p.rowmul = reinterpret_cast<const float*>(v.ws + l.rowmul);
    p.labels = q.labels;
    p.lse = q.lse;
    p.grad = q.grad;
    p.part = reinterpret_cast<float2*>(v.ws + l.part);
    p.target = reinterpret_cast<float*>(v.ws + l.target);
    p.rest = reinterpret_cast<float*>(v.ws + l.rest);
    p.acc = reinterpret_cast<float4*>(v.ws + l.acc);
    p.accumulate = v.first ? 0 : 1;
    p.gscale = 32768.f;
    p.g_terms = l.g_terms;
    p.marks = l.mark_words ? reinterpret_cast<const uint32_t*>(v.ws + l.marks) : nullptr;
    p.mark_words = static_cast<int>(l.mark_words);
    p.out_rows = static_cast<int>(rows);
    p.out_cols = static_cast<int>(MODE == kVocabDw ? K : ld);

    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attrs[2];
    int na = 0;
    attrs[na].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attrs[na].val.programmaticStreamSerializationAllowed = 1;
    ++na;
    if (PAIR) {
        const int pairs = pair_slots(fn, C::kThreads, C::kSmemBytes);
        cfg.gridDim = dim3(2 * (p.num_tiles < pairs ? p.num_tiles : pairs), 1, 1);
        attrs[na].id = cudaLaunchAttributeClusterDimension;
        attrs[na].val.clusterDim.x = 2;
        attrs[na].val.clusterDim.y = 1;
        attrs[na].val.clusterDim.z = 1;
        ++na;
    } else {
        const int slots = num_sms();
        cfg.gridDim = dim3(p.num_tiles < slots ? p.num_tiles : slots, 1, 1);
    }
    cfg.blockDim = dim3(C::kThreads, 1, 1);
    cfg.dynamicSmemBytes = C::kSmemBytes;
    cfg.stream = stream;
    cfg.attrs = attrs;
    cfg.numAttrs = na;
    if (take_injected_failure(kInjectLaunch)) return LOWBIT_ERR_CUDA;
    return cudaLaunchKernelEx(&cfg, kernel, ma, mb, ms, mz, mo, p) == cudaSuccess ? LOWBIT_OK : LOWBIT_ERR_CUDA;
}

// The products over a bf16 table.
inline lowbit_status dispatch_dense(const VocabProduct& v, cudaStream_t s) {
    switch (v.mode) {
        case kVocabStats: return v.pair ? launch<kVocabStats, kDense, true>(v, s) : launch<kVocabStats, kDense, false>(v, s);
        case kVocabGrad: return v.pair ? launch<kVocabGrad, kDense, true>(v, s) : launch<kVocabGrad, kDense, false>(v, s);
        case kVocabDx: return v.pair ? launch<kVocabDx, kDense, true>(v, s) : launch<kVocabDx, kDense, false>(v, s);
        case kVocabDw: return launch<kVocabDw, kDense, true>(v, s);
        default: return LOWBIT_ERR_UNSUPPORTED;
    }
}

}  // namespace vocab
}  // namespace lowbit
