// Host-side declarations shared by the adapter translation units: problem descriptions, the
// workspace layout and the launches of each stage.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "lowbit_internal.h"

namespace lowbit {

constexpr int kMaxAdapters = 4096;
constexpr int kMaxRank = 128;
constexpr int kShrinkTokens = 128;  // tokens of one adapter per block of the shrink kernel

// Slot width: the rank rounded up to a power of two >= 16 (one MMA K step).
inline int slot_log2(int rank) { return rank <= 16 ? 4 : rank <= 32 ? 5 : rank <= 64 ? 6 : 7; }

struct AdapterSet {
    int num = 0, rank = 0;        // L adapters of rank R; num == 0: none
    const void* A = nullptr;      // [L][R][K] bf16
    const void* B = nullptr;      // [L][N][R] bf16
    const float* scaling = nullptr;
    const int32_t* index = nullptr;   // [M], nullptr: every token takes adapter 0
};

// One product with the fused adapter term, on the tensor-memory kernel: out[M][rows] =
// in[M][red] * W'^T, W' [rows][red] decoded from packed words (W itself, or W^T when `grad`).
struct ExtProblem {
    bool grad = false;
    int64_t M = 0, rows = 0, red = 0;
    int64_t N = 0, K = 0;             // the linear's own sizes (the scales' layout is [K/g][N])
    int bits = 0, group_size = 0;
    const void* in = nullptr;         // bf16 [M][red]
    const uint32_t* words = nullptr;
    const void* scales = nullptr;
    const void* zeros = nullptr;
    void* out = nullptr;              // bf16 [M][rows]
    AdapterSet ad;
    void* p_out = nullptr;            // bf16 [M][R] or nullptr: the scaled low-rank product of `in`
    uint8_t* ck_codes = nullptr;      // 8-bit copy of `in` or nullptr
    uint8_t* ck_exps = nullptr;
};

// Workspace of one such product, offsets in bytes (each part 256-byte aligned):
//   xh       fp16 copy of the input, rows of red64 (red rounded up to 64) elements
//   rowmul   fp32 per token
//   and with adapters: perm (tokens sorted by adapter), seg (start of each adapter's tokens, L + 1
//   entries), blocks (int4 per shrink block), tile_slots, slot_adapter, slot_side, token_slot, odd_parts and bad (which
//   adapters' weight sides are not finite), partial (fp32 [ksplit][M][Rp]), pslots (bf16 [M][slot columns])
//   p        bf16 [M][R] (backward: dp), and p_rest, what its rounding left
struct ExtWorkspace {
    int64_t red64;
    int tile_tokens;         // tokens per tile and K slices of the product, chosen from the sizes
    int product_split;
    int64_t m_tiles;
    int64_t num_blocks;      // shrink blocks, at most
    int ksplit;              // K slices of the shrink kernel
    int64_t kslice;
    int plan_slices;         // CTAs per adapter of the plan kernel
    int64_t slot_pitch;      // slots of a tile, at most
    int64_t p_cols;          // columns of pslots
    size_t xh, rowmul, perm, seg, blocks, tile_slots, slot_adapter, slot_side, token_slot, odd_parts, bad, partial, pslots, p, p_rest, total;
};
ExtWorkspace ext_workspace(int64_t M, int64_t rows, int64_t red, int num, int rank);
// Bytes that hold the workspace of M tokens or fewer: grows with M, which `total` does not everywhere.
size_t ext_workspace_bound(int64_t M, int64_t rows, int64_t red, int num, int rank);

struct ExtBuffers {
    ExtWorkspace w;
    uint8_t* base;
    template <class T>
    T* at(size_t offset) const {
        return reinterpret_cast<T*>(base + offset);
    }
};

// The stages (adapter_kernels.cu), each one launch on `stream`, programmatic dependents of one
// another: sort the tokens by adapter and list each tile's slots; low-rank product; copy to fp16
// with the slots' P (and the 8-bit copy); gradients of the adapters.
lowbit_status launch_plan(const ExtProblem& e, const ExtBuffers& b, cudaStream_t stream);
lowbit_status launch_shrink(const ExtProblem& e, const ExtBuffers& b, cudaStream_t stream);
lowbit_status launch_convert(const ExtProblem& e, const ExtBuffers& b, cudaStream_t stream);
// Up to 16 tokens: p fp32 [M][R], scaled, for the small-M kernel's low-rank term.
lowbit_status launch_shrink_small(const ExtProblem& e, float* p, cudaStream_t stream);

struct WgradProblem {
    const void* dy;            // bf16 [M][N]
    const void* x;             // bf16 [M][K], or nullptr:
    const uint8_t* ck_codes;   // the 8-bit copy
    const uint8_t* ck_exps;
    const void* p;             // bf16 [M][R]
    const void* dp;            // bf16 [M][R], and
    const void* dp_rest;       // what its rounding left
    void* dA;                  // bf16 [L][R][K]
    void* dB;                  // bf16 [L][N][R]
    int64_t M, N, K;
    int num, rank;
    bool planned;              // false: no index, every token has adapter 0
    bool beside_product;       // launched right after the product, beside which it runs
};
lowbit_status launch_wgrad(const WgradProblem& g, const ExtBuffers& b, cudaStream_t stream);

// The fused product (gemm_ext_*.cu), one translation unit per code width and direction.
lowbit_status ext_gemm_b1(const ExtProblem& e, const ExtBuffers& b, cudaStream_t stream);
lowbit_status ext_gemm_b2(const ExtProblem& e, const ExtBuffers& b, cudaStream_t stream);
lowbit_status ext_gemm_b4(const ExtProblem& e, const ExtBuffers& b, cudaStream_t stream);
lowbit_status ext_grad_b1(const ExtProblem& e, const ExtBuffers& b, cudaStream_t stream);
lowbit_status ext_grad_b2(const ExtProblem& e, const ExtBuffers& b, cudaStream_t stream);
lowbit_status ext_grad_b4(const ExtProblem& e, const ExtBuffers& b, cudaStream_t stream);

// Clusters of `ks` CTAs of `kernel` that fit on the current device at once (gemm_sm100.cu).
int cluster_capacity(const void* kernel, int ks, int threads, int smem_bytes, bool along_x = false);

// 8-bit copies and W^T (checkpoint.cu, pack_sm100.cu).
lowbit_status checkpoint_store_launch(const void* x, int64_t count, uint8_t* codes, uint8_t* exps, cudaStream_t s);
lowbit_status checkpoint_load_launch(const uint8_t* codes, const uint8_t* exps, int64_t count, void* x, cudaStream_t s);
lowbit_status transpose_launch(const uint32_t* packed, int64_t N, int64_t K, int bits, uint32_t* out, cudaStream_t s);

}  // namespace lowbit
