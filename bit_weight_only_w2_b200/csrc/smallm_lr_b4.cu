// Instantiations of the small-M kernel with the adapters' low-rank term for 4-bit codes (both group sizes, 1..16 octets per tile).
#include <utility>

#include "smallm_kernel.cuh"

LOWBIT_SMALLM_TABLE(kernel_lr_b4, 4, true)
