// The adapter product on uint4 weights (both group sizes, every token tile).
#include "gemm_ext.cuh"

LOWBIT_EXT_ENTRY(ext_gemm_b4, 4, kExtAdapter)
