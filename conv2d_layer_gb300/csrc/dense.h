// dense.h - launches of the dense layer's matrix products (dense_gemm.cu).
#pragma once
#include <cuda_runtime.h>

#include "dense_gemm.cuh"

namespace c2d {

// dt: CONV2D_BF16 or CONV2D_FP16, the type T of the epilogue; mode: kDenseForward, kDenseDx or kDenseDw, for the pair
// kernel also kDenseDwAdd; q: how the operands are held (kRowScaled: kDenseForward, kBlockScaled: that or kDenseDx).
cudaError_t launch_dense_pair(const DenseGemmParams& p, int dt, int mode, int q, int grid, size_t smem,
                              cudaStream_t st);
cudaError_t launch_dense_cluster(const DenseGemmParams& p, int dt, int mode, int q, int grid, size_t smem,
                                 cudaStream_t st);

// Shared with the mixture-of-experts layer (dense.cu).
bool encode_operand(CUtensorMap* m, const void* base, int type, long rows, long cols, long ld, bool mn, int box_rows);
DenseScales block_scales(const uint8_t* scale, int group, long rows, long cols, bool down);

}  // namespace c2d
