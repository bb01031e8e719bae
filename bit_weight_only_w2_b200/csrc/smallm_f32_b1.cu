// Instantiations of the small-M kernel with Y in fp32 for 1-bit codes (both group sizes, 1..16 octets per tile).
#include <utility>

#include "smallm_kernel.cuh"

LOWBIT_SMALLM_TABLE_OF(kernel_f32_b1, 1, false, true)
