// The input gradient on uint4 weights (W^T words, both group sizes, every token tile).
#include "gemm_ext.cuh"

LOWBIT_EXT_ENTRY(ext_grad_b4, 4, kExtGrad)
