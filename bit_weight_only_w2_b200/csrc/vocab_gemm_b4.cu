// The products of the cross entropy over a vocabulary of packed uint4 rows.
#include "vocab_few.cuh"

namespace lowbit {
lowbit_status vocab_product_b4(const VocabProduct& v, cudaStream_t stream) { return vocab::dispatch_packed<4>(v, stream); }
}  // namespace lowbit
