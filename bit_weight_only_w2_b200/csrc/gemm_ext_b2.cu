// The adapter product on ternary weights (both group sizes, every token tile).
#include "gemm_ext.cuh"

LOWBIT_EXT_ENTRY(ext_gemm_b2, 2, kExtAdapter)
