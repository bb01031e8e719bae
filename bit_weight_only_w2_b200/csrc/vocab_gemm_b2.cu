// The products of the cross entropy over a vocabulary of packed ternary rows.
#include "vocab_few.cuh"

namespace lowbit {
lowbit_status vocab_product_b2(const VocabProduct& v, cudaStream_t stream) { return vocab::dispatch_packed<2>(v, stream); }
}  // namespace lowbit
