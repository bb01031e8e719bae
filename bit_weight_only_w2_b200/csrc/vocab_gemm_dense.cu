// The products of the cross entropy over a vocabulary of bf16 rows.
#include "vocab_gemm.cuh"

namespace lowbit {
lowbit_status vocab_product_dense(const VocabProduct& v, cudaStream_t stream) { return vocab::dispatch_dense(v, stream); }
}  // namespace lowbit
