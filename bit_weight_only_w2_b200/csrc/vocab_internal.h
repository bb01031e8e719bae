// Host-side declarations of the vocabulary operators: the softmax cross entropy over a table of
// vocabulary rows with its gradients, and the lookup of rows with its gradient.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "lowbit_internal.h"

namespace lowbit {

constexpr int kDense = 16;   // `bits` of a bf16 table

// A table of rows [N][K]: bf16, or packed words with group scales (and zeros).
struct Table {
    int64_t N = 0, K = 0;
    int bits = 0, group_size = 0;
    const void* rows = nullptr;    // bf16 [N][K], or words [N][K*bits/32]
    const void* scales = nullptr;  // fp16 [K/group_size][N]
    const void* zeros = nullptr;
};

struct LossProblem {
    int64_t M = 0, vocab = 0;      // tokens; rows of the table that take part (the first `vocab`)
    Table table;
    const void* X = nullptr;       // bf16 [M][K]
    const int32_t* labels = nullptr;
    float* loss = nullptr;         // forward: [M], and
    float* lse_out = nullptr;      // [M]
    const float* lse = nullptr;    // backward: [M]
    const float* grad = nullptr;   // [M]
    void* dX = nullptr;            // bf16 [M][K]
    void* dW = nullptr;            // bf16 [N][K] or nullptr
};

// Workspace of the loss, offsets in bytes (each part 256-byte aligned), and the choices made with it:
//   forward   xh (with rowmul behind it, packed tables only), target [M], part [parts][M] (float2);
//             small: logits [M][N] fp32
//   backward  xh, xz (the tokens with a label, dW only), marks [rows / 256][M / 2048] (dW of many tokens), rest [M] (bf16
//             tables), g [g_terms][M][piece], acc (fp32 tiles of dX)
struct LossLayout {
    bool small;              // up to 16 tokens, packed: fp32 logits by the small-M kernel
    bool pair;               // tiles of 256 tokens x 256 columns on CTA pairs, else 128 x 128 (logits of a packed table:
                             // 256 rows of it x the tokens, on CTA pairs, vocab_few.cuh)
    int64_t m_tiles, n_tiles;
    int64_t parts;           // forward: (maximum, sum) of each token that the tiles leave
    int64_t piece;           // columns of G formed at a time
    int64_t dx_tiles;        // tiles of dX in the columns' direction
    int g_terms;             // bf16 values that G is kept as
    int slices;              // slices of a piece whose products are summed apart
    int64_t mark_words;      // words of marks per 256 rows of the table; 0: G's second term is taken everywhere
    size_t xh, rowmul, logits, target, part, xz, marks, rest, g, acc, total;
};
constexpr int64_t kSmallTokens = 16;
LossLayout loss_layout(int64_t M, int64_t vocab, int64_t K, int bits, bool backward, bool need_dw);

lowbit_status loss_forward(const LossProblem& p, const LossLayout& l, uint8_t* ws, cudaStream_t stream);
lowbit_status loss_backward(const LossProblem& p, const LossLayout& l, uint8_t* ws, cudaStream_t stream);

// One product over the vocabulary (vocab_gemm*.cu), of the kinds listed there.
struct VocabProduct {
    int mode = 0;
    bool pair = false;
    const LossProblem* p = nullptr;
    const LossLayout* l = nullptr;
    uint8_t* ws = nullptr;
    int64_t v0 = 0, cols = 0;      // the piece: first column, columns
    bool first = false;            // kVocabDx: the first piece (the sums start from zero)
};
constexpr int kVocabStats = 0, kVocabGrad = 1, kVocabDx = 2, kVocabDw = 3;
lowbit_status vocab_product_dense(const VocabProduct& v, cudaStream_t stream);
lowbit_status vocab_product_b1(const VocabProduct& v, cudaStream_t stream);
lowbit_status vocab_product_b2(const VocabProduct& v, cudaStream_t stream);
lowbit_status vocab_product_b4(const VocabProduct& v, cudaStream_t stream);

int cluster_capacity(const void* kernel, int ks, int threads, int smem_bytes, bool along_x);

// Lookup (embedding.cu).
lowbit_status embedding_launch(const Table& t, const int32_t* tokens, int64_t T, float multiplier, void* out,
                               cudaStream_t stream);
size_t embedding_backward_bytes(int64_t T, int64_t rows, int64_t K);
lowbit_status embedding_backward_launch(const int32_t* tokens, const void* dy, int64_t T, int64_t K, int64_t first,
                                        int64_t rows, float multiplier, void* out, void* ws, cudaStream_t stream);

}  // namespace lowbit
