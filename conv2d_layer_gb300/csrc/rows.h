// rows.h - kernels over rows of features (rows.cu) used by the dense layer's calls.
#pragma once
#include <cuda_runtime.h>
#include <cstdint>

#include "conv2d.h"

namespace c2d {

// late: the kernel before this one in the call writes nothing that this one reads or writes, and has waited for what
// came before the call: the two run side by side (see pdl_entry).

// x as type `dt` into a dense-layout copy of row length ldo (a multiple of 8): decoded (E4M3) or moved.
cudaError_t launch_to_rows(const conv2d_mat& x, long rows, int cols, int dt, void* out, long ldo, int late, cudaStream_t st);

// The same for 8-bit elements taken as they are.
cudaError_t launch_move_bytes(const void* x, long ldx, long rows, int cols, void* out, long ldo, int late, cudaStream_t st);

// Backward through the activation: dz = dy act'(z) (z null: act is the identity; dz null: not written) and
// column partials part[strips][cols] of the unrounded dz (null: none). dt: type of dy and dz.
struct DactPlan {
  int strips;          // row strips = rows of the partials
  long rows_per_strip;
};
DactPlan plan_dact(long rows, int cols, int sms);
cudaError_t launch_dact(const conv2d_mat* z, const conv2d_mat& dy, long rows, int cols, int dt, int act, void* dz,
                        long lddz, float* part, const DactPlan& pl, int late, cudaStream_t st);
// out[c] = (accumulate ? out[c] : 0) + sum over g of part[g][c], in the order of g; out2 (null: none) from part2.
cudaError_t launch_column_sum(const float* part, int G, int cols, float* out, int accumulate, int late, cudaStream_t st,
                              const float* part2 = nullptr, float* out2 = nullptr);
// Joins the splits of a weight gradient: out[r][c] (fp32 or dt, row length ldo) = (accumulate ? out : 0) +
// sum over s of part[s][r][c], in the order of s.
cudaError_t launch_split_join(const float* part, int splits, long rows, int cols, int type, void* out, long ldo,
                              int accumulate, cudaStream_t st);
// Zeroes rows x cols elements of a matrix (row length ld).
cudaError_t launch_zero_rows(long rows, int cols, int type, void* out, long ld, int late, cudaStream_t st);

}  // namespace c2d
