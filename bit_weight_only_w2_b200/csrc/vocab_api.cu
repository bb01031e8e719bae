// C entry points of the vocabulary operators (declared in include/lowbit.h): argument checks and dispatch. Every check
// runs before any launch.
#include <cuda_runtime.h>

#include <cstdint>

#include "vocab_internal.h"

#define LOWBIT_API extern "C" __attribute__((visibility("default")))

namespace lowbit {
namespace {

bool aligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

constexpr int64_t kMaxSize = int64_t(1) << 31;

// A table's description; its pointers are looked at where `used`.
lowbit_status check_table(const Table& t, bool used) {
    const bool dense = t.bits == kDense;
    if (!dense && t.bits != 1 && t.bits != 2 && t.bits != 4) return LOWBIT_ERR_INVALID_ARG;
    if (t.N < 0 || t.K <= 0) return LOWBIT_ERR_INVALID_ARG;
    if (dense) {
        if (t.scales || t.zeros) return LOWBIT_ERR_INVALID_ARG;
    } else {
        if (t.group_size <= 0 || t.K % t.group_size != 0 || t.group_size % (32 / t.bits) != 0) return LOWBIT_ERR_INVALID_ARG;
        if ((t.bits == 4) != (t.zeros != nullptr)) return LOWBIT_ERR_INVALID_ARG;
    }
    if (used) {
        if (!t.rows || (!dense && !t.scales)) return LOWBIT_ERR_INVALID_ARG;
        if (!aligned(t.rows, 16) || !aligned(t.scales, 16) || !aligned(t.zeros, 16)) return LOWBIT_ERR_ALIGNMENT;
    }
    if (t.N >= kMaxSize || t.K >= kMaxSize || t.K % 8 != 0) return LOWBIT_ERR_UNSUPPORTED;
    if (!dense) {
        if (t.group_size != 64 && t.group_size != 128) return LOWBIT_ERR_UNSUPPORTED;
        if ((t.bits == 1 && t.K % 128 != 0) || t.N % 8 != 0) return LOWBIT_ERR_UNSUPPORTED;
    }
    return LOWBIT_OK;
}

Table table(int64_t N, int64_t K, int bits, int group_size, const void* rows, const void* scales, const void* zeros) {
    Table t;
    t.N = N;
    t.K = K;
    t.bits = bits;
    t.group_size = group_size;
    t.rows = rows;
    t.scales = scales;
    t.zeros = zeros;
    return t;
}

lowbit_status check_loss(const LossProblem& p) {
    if (p.M < 0 || p.vocab < 1 || p.vocab > p.table.N) return LOWBIT_ERR_INVALID_ARG;
    const lowbit_status st = check_table(p.table, p.M > 0);
    if (st != LOWBIT_OK) return st;
    if (p.M > 0) {
        if (!p.X || !p.labels) return LOWBIT_ERR_INVALID_ARG;
        if (!aligned(p.X, 16) || !aligned(p.labels, 4)) return LOWBIT_ERR_ALIGNMENT;
    }
    // (tiles of the products are counted in 32 bits, and so are their rows and columns)
    if (p.M > kMaxExtent || p.vocab > kMaxExtent || p.table.K > kMaxExtent || (p.M + 255) / 256 * ((p.table.K + 255) / 256) >= int64_t(1) << 24) return LOWBIT_ERR_UNSUPPORTED;
    return LOWBIT_OK;
}

lowbit_status check_workspace(const void* ws, size_t have, size_t need) {
    return ws && aligned(ws, 256) && have >= need ? LOWBIT_OK : LOWBIT_ERR_WORKSPACE;
}

}  // namespace
}  // namespace lowbit

using namespace lowbit;

LOWBIT_API size_t lowbit_cross_entropy_workspace_size(int64_t M, int64_t vocab, int64_t K, int bits, int backward) {
    if (M < 0 || vocab < 1 || K < 1 || (bits != 1 && bits != 2 && bits != 4 && bits != kDense) || backward < 0 || backward > 2) return 0;
    if (M > kMaxExtent || vocab > kMaxExtent || K > kMaxExtent) return 0;
    return loss_layout(M, vocab, K, bits, backward > 0, backward == 2).total;
}

LOWBIT_API lowbit_status lowbit_cross_entropy(int64_t M, int64_t vocab, int64_t N, int64_t K, int bits, int group_size, const void* X,
                                              const void* W, const void* scales, const void* zeros, const int32_t* labels, float* loss,
                                              float* lse, void* workspace, size_t workspace_bytes, void* stream) {
    LossProblem p;
    p.M = M;
    p.vocab = vocab;
    p.table = table(N, K, bits, group_size, W, scales, zeros);
    p.X = X;
    p.labels = labels;
    p.loss = loss;
    p.lse_out = lse;
    lowbit_status st = check_loss(p);
    if (st != LOWBIT_OK || M == 0) return st;
    if (!loss || !lse) return LOWBIT_ERR_INVALID_ARG;
    if (!aligned(loss, 4) || !aligned(lse, 4)) return LOWBIT_ERR_ALIGNMENT;
    const LossLayout l = loss_layout(M, vocab, K, bits, false, false);
    if ((st = check_workspace(workspace, workspace_bytes, l.total)) != LOWBIT_OK) return st;
    if ((st = check_device()) != LOWBIT_OK) return st;
    return loss_forward(p, l, static_cast<uint8_t*>(workspace), static_cast<cudaStream_t>(stream));
}

LOWBIT_API lowbit_status lowbit_cross_entropy_backward(int64_t M, int64_t vocab, int64_t N, int64_t K, int bits, int group_size,
                                                       const void* X, const void* W, const void* scales, const void* zeros,
                                                       const int32_t* labels, const float* lse, const float* grad, void* dX, void* dW,
                                                       void* workspace, size_t workspace_bytes, void* stream) {
    LossProblem p;
    p.M = M;
    p.vocab = vocab;
    p.table = table(N, K, bits, group_size, W, scales, zeros);
    p.X = X;
    p.labels = labels;
    p.lse = lse;
    p.grad = grad;
    p.dX = dX;
    p.dW = dW;
    lowbit_status st = check_loss(p);
    if (st != LOWBIT_OK) return st;
    if (dW && bits != kDense) return LOWBIT_ERR_UNSUPPORTED;   // packed rows are frozen
    if (!aligned(dW, 16)) return LOWBIT_ERR_ALIGNMENT;
    if (M == 0) {   // a sum over nothing
        if (!dW) return LOWBIT_OK;
        if ((st = check_device()) != LOWBIT_OK) return st;
        return cudaMemsetAsync(dW, 0, static_cast<size_t>(N) * K * 2, static_cast<cudaStream_t>(stream)) == cudaSuccess ? LOWBIT_OK
                                                                                                                  : LOWBIT_ERR_CUDA;
    }
    if (!lse || !grad || !dX) return LOWBIT_ERR_INVALID_ARG;
    if (!aligned(lse, 4) || !aligned(grad, 4) || !aligned(dX, 16)) return LOWBIT_ERR_ALIGNMENT;
    const LossLayout l = loss_layout(M, vocab, K, bits, true, dW != nullptr);
    if ((st = check_workspace(workspace, workspace_bytes, l.total)) != LOWBIT_OK) return st;
    if ((st = check_device()) != LOWBIT_OK) return st;
    return loss_backward(p, l, static_cast<uint8_t*>(workspace), static_cast<cudaStream_t>(stream));
}

LOWBIT_API lowbit_status lowbit_embedding(int64_t T, int64_t N, int64_t K, int bits, int group_size, const int32_t* tokens, const void* W,
                                          const void* scales, const void* zeros, float multiplier, void* Y, void* stream) {
    const Table t = table(N, K, bits, group_size, W, scales, zeros);
    if (T < 0) return LOWBIT_ERR_INVALID_ARG;
    lowbit_status st = check_table(t, T > 0 && N > 0);
    if (st != LOWBIT_OK || T == 0) return st;
    if (!tokens || !Y) return LOWBIT_ERR_INVALID_ARG;
    if (!aligned(tokens, 4) || !aligned(Y, 16)) return LOWBIT_ERR_ALIGNMENT;
    if (T >= kMaxSize || T * ((K + 1023) / 1024) >= int64_t(1) << 33) return LOWBIT_ERR_UNSUPPORTED;   // grid
    if ((st = check_device()) != LOWBIT_OK) return st;
    return embedding_launch(t, tokens, T, multiplier, Y, static_cast<cudaStream_t>(stream));
}

LOWBIT_API size_t lowbit_embedding_workspace_size(int64_t T, int64_t rows, int64_t K) {
    if (T < 0 || rows < 0 || K < 0 || T >= kMaxSize || rows >= kMaxSize || K >= kMaxSize) return 0;
    return embedding_backward_bytes(T, rows, K);
}

LOWBIT_API lowbit_status lowbit_embedding_backward(int64_t T, int64_t K, int64_t first, int64_t rows, const int32_t* tokens,
                                                   const void* dY, float multiplier, void* dE, void* workspace, size_t workspace_bytes,
                                                   void* stream) {
    if (T < 0 || K <= 0 || first < 0 || rows < 0) return LOWBIT_ERR_INVALID_ARG;
    if (rows == 0) return LOWBIT_OK;
    if (!dE || (T > 0 && (!tokens || !dY))) return LOWBIT_ERR_INVALID_ARG;
    if (!aligned(tokens, 4) || !aligned(dY, 16) || !aligned(dE, 16)) return LOWBIT_ERR_ALIGNMENT;
    if (K % 8 != 0 || T >= kMaxSize || K >= int64_t(1) << 23 || first >= kMaxSize || rows >= kMaxSize) return LOWBIT_ERR_UNSUPPORTED;
    lowbit_status st;
    if (T == 0) {   // sums over nothing
        if ((st = check_device()) != LOWBIT_OK) return st;
        return cudaMemsetAsync(dE, 0, static_cast<size_t>(rows) * K * 2, static_cast<cudaStream_t>(stream)) == cudaSuccess ? LOWBIT_OK
                                                                                                                     : LOWBIT_ERR_CUDA;
    }
    if ((st = check_workspace(workspace, workspace_bytes, embedding_backward_bytes(T, rows, K))) != LOWBIT_OK) return st;
    if ((st = check_device()) != LOWBIT_OK) return st;
    return embedding_backward_launch(tokens, dY, T, K, first, rows, multiplier, dE, workspace, static_cast<cudaStream_t>(stream));
}
