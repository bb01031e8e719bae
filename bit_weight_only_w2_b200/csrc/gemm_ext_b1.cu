// The adapter product on binary weights (both group sizes, every token tile).
#include "gemm_ext.cuh"

LOWBIT_EXT_ENTRY(ext_gemm_b1, 1, kExtAdapter)
