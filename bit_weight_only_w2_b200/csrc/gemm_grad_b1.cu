// The input gradient on binary weights (W^T words, both group sizes, every token tile).
#include "gemm_ext.cuh"

LOWBIT_EXT_ENTRY(ext_grad_b1, 1, kExtGrad)
