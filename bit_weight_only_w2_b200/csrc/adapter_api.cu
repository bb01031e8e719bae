// C entry points of the adapters, the gradients and the 8-bit activation copies (declared in
// include/lowbit.h): argument checks, the workspace, and the order of the stages. Every check runs
// before any launch.
#include <cuda_runtime.h>

#include <cstdint>

#include "adapter_internal.h"

#define LOWBIT_API extern "C" __attribute__((visibility("default")))

namespace lowbit {
namespace {

bool aligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

constexpr int64_t kMaxSize = int64_t(1) << 31;

// The linear by lowbit_gemm's description (the workspace is checked separately).
GemmProblem linear_problem(int64_t M, int64_t N, int64_t K, int bits, int gs, const void* in, const uint32_t* W,
                           const void* scales, const void* zeros, const void* out) {
    GemmProblem g;
    g.M = M;
    g.N = N;
    g.K = K;
    g.bits = bits;
    g.group_size = gs;
    g.X = in;
    g.Wp = W;
    g.scales = scales;
    g.zeros = zeros;
    g.Y = const_cast<void*>(out);
    g.workspace = reinterpret_cast<void*>(uintptr_t(256));
    g.workspace_bytes = SIZE_MAX;
    return g;
}

lowbit_status check_linear(int64_t M, int64_t N, int64_t K, int bits, int gs, const void* in, const uint32_t* W,
                           const void* scales, const void* zeros, const void* out) {
    return validate_gemm(linear_problem(M, N, K, bits, gs, in, W, scales, zeros, out));
}

lowbit_status check_adapters(const lowbit_adapters* a, int64_t N) {
    if (!a || a->num < 1 || a->rank < 1) return LOWBIT_ERR_INVALID_ARG;
    if (!a->A || (N > 0 && !a->B) || !a->scaling) return LOWBIT_ERR_INVALID_ARG;
    if (!aligned(a->A, 16) || !aligned(a->B, 16) || !aligned(a->scaling, 4) || !aligned(a->index, 4))
        return LOWBIT_ERR_ALIGNMENT;
    if (a->num > kMaxAdapters || a->rank > kMaxRank || a->rank % 8 != 0) return LOWBIT_ERR_UNSUPPORTED;
    return LOWBIT_OK;
}

lowbit_status check_copy(const uint8_t* codes, const uint8_t* exps) {
    if ((codes == nullptr) != (exps == nullptr)) return LOWBIT_ERR_INVALID_ARG;
    return aligned(codes, 16) ? LOWBIT_OK : LOWBIT_ERR_ALIGNMENT;
}

lowbit_status check_workspace(const void* ws, size_t have, size_t need) {
    return ws && aligned(ws, 256) && have >= need ? LOWBIT_OK : LOWBIT_ERR_WORKSPACE;
}

AdapterSet adapter_set(const lowbit_adapters* a) {
    AdapterSet s;
    s.num = a->num;
    s.rank = a->rank;
    s.A = a->A;
    s.B = a->B;
    s.scaling = a->scaling;
    s.index = a->index;
    return s;
}

lowbit_status product(const ExtProblem& e, const ExtBuffers& b, cudaStream_t stream) {
    if (e.grad) return e.bits == 1 ? ext_grad_b1(e, b, stream) : e.bits == 2 ? ext_grad_b2(e, b, stream) : ext_grad_b4(e, b, stream);
    return e.bits == 1 ? ext_gemm_b1(e, b, stream) : e.bits == 2 ? ext_gemm_b2(e, b, stream) : ext_gemm_b4(e, b, stream);
}

// The stages before the product: the tokens' order, the low-rank product, the fp16 copy.
lowbit_status prepare(const ExtProblem& e, const ExtBuffers& b, cudaStream_t stream) {
    lowbit_status st = LOWBIT_OK;
    if (e.ad.num > 0) {
        if (e.ad.index && (st = launch_plan(e, b, stream)) != LOWBIT_OK) return st;
        if ((st = launch_shrink(e, b, stream)) != LOWBIT_OK) return st;
    }
    return launch_convert(e, b, stream);
}

}  // namespace
}  // namespace lowbit

using namespace lowbit;

LOWBIT_API size_t lowbit_transposed_words(int64_t N, int64_t K, int bits) {
    if ((bits != 1 && bits != 2 && bits != 4) || N < 0 || K < 0 || K % (32 / bits) != 0) return 0;
    return static_cast<size_t>(K) * static_cast<size_t>((N + 127) / 128 * 128) * bits / 32;
}

LOWBIT_API lowbit_status lowbit_transpose(const uint32_t* packed, int64_t N, int64_t K, int bits, uint32_t* packed_t,
                                          void* stream) {
    if ((bits != 1 && bits != 2 && bits != 4) || N < 0 || K < 0 || K % (32 / bits) != 0) return LOWBIT_ERR_INVALID_ARG;
    if (N == 0 || K == 0) return LOWBIT_OK;
    if (!packed || !packed_t) return LOWBIT_ERR_INVALID_ARG;
    if (!aligned(packed, 16) || !aligned(packed_t, 16)) return LOWBIT_ERR_ALIGNMENT;
    if (N >= kMaxSize || K >= kMaxSize) return LOWBIT_ERR_UNSUPPORTED;
    const lowbit_status st = check_device();
    if (st != LOWBIT_OK) return st;
    return transpose_launch(packed, N, K, bits, packed_t, static_cast<cudaStream_t>(stream));
}

LOWBIT_API size_t lowbit_adapter_workspace_size(int64_t M, int64_t N, int64_t K, int num, int rank) {
    if (M < 0 || N < 0 || K < 0 || num < 0 || num > kMaxAdapters || rank < 0 || rank > kMaxRank) return 0;
    if (num > 0 && rank == 0) return 0;
    // (without an index the product is laid out for one adapter; whichever needs more)
    size_t most = 0;
    for (int n : {num, num > 1 ? 1 : num})
        for (size_t t : {ext_workspace_bound(M, N, K, n, rank), ext_workspace_bound(M, K, N, n, rank)})
            if (t > most) most = t;
    return most;
}

LOWBIT_API lowbit_status lowbit_adapter_gemm(int64_t M, int64_t N, int64_t K, int bits, int group_size, const void* X,
                                             const uint32_t* Wp, const void* scales, const void* zeros,
                                             const lowbit_adapters* adapters, void* Y, void* P, uint8_t* ck_codes,
                                             uint8_t* ck_exps, void* workspace, size_t workspace_bytes, void* stream) {
    lowbit_status st = check_linear(M, N, K, bits, group_size, X, Wp, scales, zeros, Y);
    if (st != LOWBIT_OK) return st;
    if ((st = check_adapters(adapters, N)) != LOWBIT_OK || (st = check_copy(ck_codes, ck_exps)) != LOWBIT_OK) return st;
    if (!aligned(P, 16)) return LOWBIT_ERR_ALIGNMENT;
    if (M == 0) return LOWBIT_OK;
    if (N == 0) return P || ck_codes ? LOWBIT_ERR_UNSUPPORTED : LOWBIT_OK;   // (neither P nor the copy is empty)
    ExtProblem e;
    e.M = M;
    e.rows = e.N = N;
    e.red = e.K = K;
    e.bits = bits;
    e.group_size = group_size;
    e.in = X;
    e.words = Wp;
    e.scales = scales;
    e.zeros = zeros;
    e.out = Y;
    e.ad = adapter_set(adapters);
    e.p_out = P;
    e.ck_codes = ck_codes;
    e.ck_exps = ck_exps;
    ExtBuffers b{ext_workspace(M, N, K, e.ad.index ? e.ad.num : 1, e.ad.rank), static_cast<uint8_t*>(workspace)};
    if ((st = check_workspace(workspace, workspace_bytes, b.w.total)) != LOWBIT_OK) return st;
    if ((st = check_device()) != LOWBIT_OK) return st;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const GemmProblem g = linear_problem(M, N, K, bits, group_size, X, Wp, scales, zeros, Y);
    if (smallm_supported(g)) {
        // up to 16 tokens: the small-M kernel, which reads X directly and adds the low-rank terms itself
        if (ck_codes && (st = checkpoint_store_launch(X, M * K, ck_codes, ck_exps, s)) != LOWBIT_OK) return st;
        float* p = b.at<float>(b.w.partial);
        if ((st = launch_shrink_small(e, p, s)) != LOWBIT_OK) return st;
        const LowRank lr = {p, e.ad.B, e.ad.index, e.ad.num, e.ad.rank};
        return smallm_launch(g, 0, 0, M <= 8, s, &lr);
    }
    if ((st = prepare(e, b, s)) != LOWBIT_OK) return st;
    return product(e, b, s);
}

LOWBIT_API lowbit_status lowbit_gemm_dx(int64_t M, int64_t N, int64_t K, int bits, int group_size, const void* dY,
                                        const uint32_t* Wt, const void* scales, const void* zeros, void* dX,
                                        void* workspace, size_t workspace_bytes, void* stream) {
    lowbit_status st = check_linear(M, N, K, bits, group_size, dY, Wt, scales, zeros, dX);
    if (st != LOWBIT_OK || M == 0) return st;
    ExtProblem e;
    e.grad = true;
    e.M = M;
    e.rows = e.K = K;
    e.red = e.N = N;
    e.bits = bits;
    e.group_size = group_size;
    e.in = dY;
    e.words = Wt;
    e.scales = scales;
    e.zeros = zeros;
    e.out = dX;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (N == 0) {   // a sum over nothing
        if (!dX) return LOWBIT_ERR_INVALID_ARG;
        if ((st = check_device()) != LOWBIT_OK) return st;
        return cudaMemsetAsync(dX, 0, static_cast<size_t>(M) * K * 2, s) == cudaSuccess ? LOWBIT_OK : LOWBIT_ERR_CUDA;
    }
    ExtBuffers b{ext_workspace(M, K, N, 0, 0), static_cast<uint8_t*>(workspace)};
    if ((st = check_workspace(workspace, workspace_bytes, b.w.total)) != LOWBIT_OK) return st;
    if ((st = check_device()) != LOWBIT_OK) return st;
    if ((st = prepare(e, b, s)) != LOWBIT_OK) return st;
    return product(e, b, s);
}

LOWBIT_API lowbit_status lowbit_adapter_backward(int64_t M, int64_t N, int64_t K, int bits, int group_size,
                                                 const void* dY, const uint32_t* Wt, const void* scales,
                                                 const void* zeros, const lowbit_adapters* adapters, const void* X,
                                                 const uint8_t* ck_codes, const uint8_t* ck_exps, const void* P,
                                                 void* dX, void* dA, void* dB, void* workspace, size_t workspace_bytes,
                                                 void* stream) {
    // (dX may be absent; the linear's checks want an output, so dA stands in)
    lowbit_status st = check_linear(M, N, K, bits, group_size, dY, Wt, scales, zeros, dX ? dX : dA);
    if (st != LOWBIT_OK) return st;
    if ((st = check_adapters(adapters, N)) != LOWBIT_OK || (st = check_copy(ck_codes, ck_exps)) != LOWBIT_OK) return st;
    if (!dA || (N > 0 && !dB)) return LOWBIT_ERR_INVALID_ARG;
    if (M > 0 && (!P || (X == nullptr) == (ck_codes == nullptr))) return LOWBIT_ERR_INVALID_ARG;
    if (N == 0) return LOWBIT_ERR_UNSUPPORTED;
    if (!aligned(X, 16) || !aligned(P, 16) || !aligned(dA, 16) || !aligned(dB, 16)) return LOWBIT_ERR_ALIGNMENT;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (M == 0) {   // sums over nothing
        if ((st = check_device()) != LOWBIT_OK) return st;
        const size_t rows = static_cast<size_t>(adapters->num) * adapters->rank * 2;
        return cudaMemsetAsync(dA, 0, rows * K, s) == cudaSuccess && cudaMemsetAsync(dB, 0, rows * N, s) == cudaSuccess
                   ? LOWBIT_OK : LOWBIT_ERR_CUDA;
    }
    ExtProblem e;
    e.grad = true;
    e.M = M;
    e.rows = e.K = K;
    e.red = e.N = N;
    e.bits = bits;
    e.group_size = group_size;
    e.in = dY;
    e.words = Wt;
    e.scales = scales;
    e.zeros = zeros;
    e.out = dX;
    e.ad = adapter_set(adapters);
    ExtBuffers b{ext_workspace(M, K, N, e.ad.index ? e.ad.num : 1, e.ad.rank), static_cast<uint8_t*>(workspace)};
    if ((st = check_workspace(workspace, workspace_bytes, b.w.total)) != LOWBIT_OK) return st;
    e.p_out = b.at<void>(b.w.p);
    if ((st = check_device()) != LOWBIT_OK) return st;
    if ((st = prepare(e, b, s)) != LOWBIT_OK) return st;
    if (dX && (st = product(e, b, s)) != LOWBIT_OK) return st;
    const WgradProblem g = {dY, X, ck_codes, ck_exps, P, e.p_out, b.at<void>(b.w.p_rest), dA, dB, M, N, K, e.ad.num, e.ad.rank,
                            e.ad.index != nullptr, dX != nullptr};
    return launch_wgrad(g, b, s);
}

static lowbit_status check_checkpoint(const void* x, int64_t M, int64_t K, const uint8_t* codes, const uint8_t* exps) {
    if (M < 0 || K < 0 || K % 32 != 0) return LOWBIT_ERR_INVALID_ARG;
    if (M == 0 || K == 0) return LOWBIT_OK;
    if (!x || !codes || !exps) return LOWBIT_ERR_INVALID_ARG;
    if (!aligned(x, 16) || !aligned(codes, 16)) return LOWBIT_ERR_ALIGNMENT;
    if (M >= kMaxSize || K >= kMaxSize || M * (K / 32) >= int64_t(1) << 37) return LOWBIT_ERR_UNSUPPORTED;   // grid
    return check_device();
}

LOWBIT_API lowbit_status lowbit_checkpoint_store(const void* X, int64_t M, int64_t K, uint8_t* codes, uint8_t* exps,
                                                 void* stream) {
    const lowbit_status st = check_checkpoint(X, M, K, codes, exps);
    if (st != LOWBIT_OK || M == 0 || K == 0) return st;
    return checkpoint_store_launch(X, M * K, codes, exps, static_cast<cudaStream_t>(stream));
}

LOWBIT_API lowbit_status lowbit_checkpoint_load(const uint8_t* codes, const uint8_t* exps, int64_t M, int64_t K,
                                                void* X, void* stream) {
    const lowbit_status st = check_checkpoint(X, M, K, codes, exps);
    if (st != LOWBIT_OK || M == 0 || K == 0) return st;
    return checkpoint_load_launch(codes, exps, M * K, X, static_cast<cudaStream_t>(stream));
}
