// dense.h - launches of the dense layer's matrix products (dense_gemm.cu).
#pragma once
#include <cuda_runtime.h>

#include "dense_gemm.cuh"

namespace c2d {

// dt: CONV2D_BF16 or CONV2D_FP16, the type T of the epilogue; mode: kDenseForward, kDenseDx or kDenseDw, for the pair
// kernel also kDenseDwAdd; fp8: e4m3 operands (kDenseForward).
cudaError_t launch_dense_pair(const DenseGemmParams& p, int dt, int mode, bool fp8, int grid, size_t smem,
                              cudaStream_t st);
cudaError_t launch_dense_cluster(const DenseGemmParams& p, int dt, int mode, bool fp8, int grid, size_t smem,
                                 cudaStream_t st);

}  // namespace c2d
