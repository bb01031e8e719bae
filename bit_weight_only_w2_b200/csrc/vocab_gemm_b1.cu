// The products of the cross entropy over a vocabulary of packed binary rows.
#include "vocab_few.cuh"

namespace lowbit {
lowbit_status vocab_product_b1(const VocabProduct& v, cudaStream_t stream) { return vocab::dispatch_packed<1>(v, stream); }
}  // namespace lowbit
