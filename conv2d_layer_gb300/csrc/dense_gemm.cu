// dense_gemm.cu - instantiation and launch of the dense layer's GEMM kernels.
#include "dense.h"

#include <atomic>
#include <type_traits>

#include "conv2d.h"
#include "host.h"
#include "kernels.h"

namespace c2d {

namespace {

// Lets a kernel take up to the block's opt-in limit of shared memory, once for each device.
template <typename K>
cudaError_t opt_in(K kernel, std::atomic<uint64_t>& done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess || (done.load(std::memory_order_relaxed) >> dev & 1)) return e;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kMaxDynSmem));
  if (e == cudaSuccess) done.fetch_or(uint64_t(1) << dev);
  return e;
}

template <typename T, int MODE, int Q>
cudaError_t pair(const DenseGemmParams& p, int grid, size_t smem, cudaStream_t st) {
  const auto k = dense_pair_kernel<T, MODE, Q>;
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = opt_in(k, done);
  return e != cudaSuccess ? e : launch_k(k, dim3(grid), dim3(kPairThreads + dense_scale_threads(Q)), smem, st, 2, p);
}

template <typename T, int MODE, int Q>
cudaError_t cluster(const DenseGemmParams& p, int grid, size_t smem, cudaStream_t st) {
  const auto k = dense_cluster_kernel<T, MODE, Q>;
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = opt_in(k, done);
  return e != cudaSuccess ? e : launch_k(k, dim3(grid), dim3(kClusterThreads + dense_scale_threads(Q)), smem, st, p.cluster, p);
}

// Calls f(T{}, mode, q) with the type and constants of the instantiation.
template <typename T, typename F>
cudaError_t launch_t(int mode, int q, F&& f) {
  using std::integral_constant;
  if (mode == kDenseDw) return f(T{}, integral_constant<int, kDenseDw>{}, integral_constant<int, kHalves>{});
  if (mode == kDenseDx) {
    if (q == kBlockScaled) return f(T{}, integral_constant<int, kDenseDx>{}, integral_constant<int, kBlockScaled>{});
    return f(T{}, integral_constant<int, kDenseDx>{}, integral_constant<int, kHalves>{});
  }
  if (q == kBlockScaled) return f(T{}, integral_constant<int, kDenseForward>{}, integral_constant<int, kBlockScaled>{});
  if (q == kRowScaled) return f(T{}, integral_constant<int, kDenseForward>{}, integral_constant<int, kRowScaled>{});
  return f(T{}, integral_constant<int, kDenseForward>{}, integral_constant<int, kHalves>{});
}
template <typename F>
cudaError_t launch(int dt, int mode, int q, F&& f) {
  return dt == CONV2D_BF16 ? launch_t<__nv_bfloat16>(mode, q, f) : launch_t<__half>(mode, q, f);
}

}  // namespace

cudaError_t launch_dense_pair(const DenseGemmParams& p, int dt, int mode, int q, int grid, size_t smem,
                              cudaStream_t st) {
  if (mode == kDenseDwAdd)
    return dt == CONV2D_BF16 ? pair<__nv_bfloat16, kDenseDwAdd, kHalves>(p, grid, smem, st)
                             : pair<__half, kDenseDwAdd, kHalves>(p, grid, smem, st);
  return launch(dt, mode, q, [&](auto t, auto m, auto f) {
    return pair<decltype(t), decltype(m)::value, decltype(f)::value>(p, grid, smem, st);
  });
}

cudaError_t launch_dense_cluster(const DenseGemmParams& p, int dt, int mode, int q, int grid, size_t smem,
                                 cudaStream_t st) {
  return launch(dt, mode, q, [&](auto t, auto m, auto f) {
    return cluster<decltype(t), decltype(m)::value, decltype(f)::value>(p, grid, smem, st);
  });
}

}  // namespace c2d
