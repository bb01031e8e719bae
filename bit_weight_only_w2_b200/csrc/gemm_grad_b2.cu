// The input gradient on ternary weights (W^T words, both group sizes, every token tile).
#include "gemm_ext.cuh"

LOWBIT_EXT_ENTRY(ext_grad_b2, 2, kExtGrad)
