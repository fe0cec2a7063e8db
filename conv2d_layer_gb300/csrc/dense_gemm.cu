// dense_gemm.cu - instantiation and launch of the dense layer's GEMM kernels.
#include "dense.h"

#include "conv2d.h"
#include "host.h"
#include "kernels.h"

namespace c2d {

namespace {

template <typename T, int EPI>
cudaError_t pair(const DenseGemmParams& p, int grid, size_t smem, cudaStream_t st) {
  const cudaError_t e = cudaFuncSetAttribute(dense_pair_kernel<T, EPI>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             static_cast<int>(smem));
  return e != cudaSuccess ? e : launch_k(dense_pair_kernel<T, EPI>, dim3(grid), dim3(kDenseThreads), smem, st, 2, p);
}

template <typename T, int EPI>
cudaError_t cluster(const DenseGemmParams& p, int grid, size_t smem, cudaStream_t st) {
  const cudaError_t e = cudaFuncSetAttribute(dense_cluster_kernel<T, EPI>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             static_cast<int>(smem));
  return e != cudaSuccess
             ? e
             : launch_k(dense_cluster_kernel<T, EPI>, dim3(grid), dim3(kDenseThreads), smem, st, p.cluster, p);
}

}  // namespace

cudaError_t launch_dense_pair(const DenseGemmParams& p, int dt, int epi, int grid, size_t smem, cudaStream_t st) {
  if (dt == CONV2D_BF16)
    return epi == kDenseForward ? pair<__nv_bfloat16, kDenseForward>(p, grid, smem, st)
                                : pair<__nv_bfloat16, kDenseStore>(p, grid, smem, st);
  return epi == kDenseForward ? pair<__half, kDenseForward>(p, grid, smem, st)
                              : pair<__half, kDenseStore>(p, grid, smem, st);
}

cudaError_t launch_dense_cluster(const DenseGemmParams& p, int dt, int epi, int grid, size_t smem, cudaStream_t st) {
  if (dt == CONV2D_BF16)
    return epi == kDenseForward ? cluster<__nv_bfloat16, kDenseForward>(p, grid, smem, st)
                                : cluster<__nv_bfloat16, kDenseStore>(p, grid, smem, st);
  return epi == kDenseForward ? cluster<__half, kDenseForward>(p, grid, smem, st)
                              : cluster<__half, kDenseStore>(p, grid, smem, st);
}

}  // namespace c2d
