// rms_norm.cu - RMS norm's C entry points (kernels in rows_norm.cuh).
#include "rows.h"
#include "rows_norm.cuh"

using namespace c2d;

extern "C" {

int conv2d_rms_norm_fwd(int64_t rows, int32_t cols, float eps, const conv2d_mat* x, const conv2d_mat* residual,
                        const float* gamma, const conv2d_mat* h, const conv2d_mat* y, const conv2d_mat* q8,
                        float* inv_rms, void* stream) {
  int rc = check_rows(rows, cols);
  if (rc) return rc;
  if (!(eps > 0.f) || !std::isfinite(eps) || !gamma || !aligned16(gamma) || !aligned16(inv_rms))
    return CONV2D_ERR_INVALID_ARG;
  if ((residual == nullptr) != (h == nullptr) || (!y && !q8)) return CONV2D_ERR_INVALID_ARG;
  if (rows == 0) return CONV2D_OK;
  if ((rc = check_mat(x, cols))) return rc;
  if (!is_float(x->type)) return CONV2D_ERR_INVALID_ARG;
  for (const conv2d_mat* m : {residual, h, y})
    if (m && ((rc = check_mat(m, cols)) || m->type != x->type)) return CONV2D_ERR_INVALID_ARG;
  if (q8 && (check_mat(q8, cols) || q8->type != CONV2D_E4M3 || q8->group == kQ8Tile)) return CONV2D_ERR_INVALID_ARG;
  DevInfo* dev = nullptr;
  if ((rc = device_info(&dev))) return rc;
  NormArgs a = {};
  a.x = x->data;
  a.ldx = ld_of(x, cols);
  if (residual) {
    a.r = residual->data;
    a.ldr = ld_of(residual, cols);
    a.h = h->data;
    a.ldh = ld_of(h, cols);
  }
  a.gamma = gamma;
  if (y) {
    a.y = y->data;
    a.ldy = ld_of(y, cols);
  }
  if (q8) set_q8(a, q8, cols);
  a.inv = inv_rms;
  a.rows = rows;
  a.cols = cols;
  a.eps = eps;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  LAUNCH("rms_norm_fwd", st, rows_fwd_any<kRms>(a, x->type, st));
  return CONV2D_OK;
}

size_t conv2d_rms_norm_bwd_workspace_size(int64_t rows, int32_t cols) {
  if (check_rows(rows, cols)) return 0;
  return std::max<size_t>(256, static_cast<size_t>(norm_bwd_blocks(rows, cols, sms_for_sizing())) * cols * 4);
}

int conv2d_rms_norm_bwd(int64_t rows, int32_t cols, const conv2d_mat* h, const float* gamma, const float* inv_rms,
                        const conv2d_mat* dy, const conv2d_mat* dh, const conv2d_mat* dx, float* dgamma,
                        int accumulate, void* ws, size_t ws_bytes, void* stream) {
  int rc = check_rows(rows, cols);
  if (rc) return rc;
  if ((!dx && !dgamma) || !gamma || !aligned16(gamma) || !aligned16(dgamma)) return CONV2D_ERR_INVALID_ARG;
  DevInfo* dev = nullptr;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (rows == 0) {
    if (!dgamma || accumulate) return CONV2D_OK;
    if ((rc = device_info(&dev))) return rc;
    LAUNCH("zero", st, launch_zero_rows(1, cols, CONV2D_FP32, dgamma, cols, 0, st));
    return CONV2D_OK;
  }
  if (!inv_rms || !aligned16(inv_rms)) return CONV2D_ERR_INVALID_ARG;
  if ((rc = check_mat(h, cols)) || (rc = check_mat(dy, cols))) return rc;
  if (!is_float(h->type) || dy->type != h->type) return CONV2D_ERR_INVALID_ARG;
  for (const conv2d_mat* m : {dh, dx})
    if (m && (check_mat(m, cols) || m->type != h->type)) return CONV2D_ERR_INVALID_ARG;
  if ((rc = device_info(&dev))) return rc;
  const size_t need = conv2d_rms_norm_bwd_workspace_size(rows, cols);
  if (dgamma && (!ws || ws_bytes < need || (reinterpret_cast<uintptr_t>(ws) & 255u))) return CONV2D_ERR_WORKSPACE;
  NormBwdArgs a = {};
  a.h = h->data;
  a.ldh = ld_of(h, cols);
  a.dy = dy->data;
  a.lddy = ld_of(dy, cols);
  if (dx) {
    a.dx = dx->data;
    a.lddx = ld_of(dx, cols);
  }
  if (dh) {
    a.dh = dh->data;
    a.lddh = ld_of(dh, cols);
  }
  a.gamma = gamma;
  a.inv = inv_rms;
  a.part = dgamma ? static_cast<float*>(ws) : nullptr;
  a.rows = rows;
  a.cols = cols;
  int grid = 0;
  auto run = [&]() -> cudaError_t {
    if (h->type == CONV2D_BF16) return norm_bwd_vec<__nv_bfloat16, false>(a, dev->sms, &grid, st);
    if (h->type == CONV2D_FP16) return norm_bwd_vec<__half, false>(a, dev->sms, &grid, st);
    return norm_bwd_vec<float, false>(a, dev->sms, &grid, st);
  };
  LAUNCH("rms_norm_bwd", st, run());
  if (dgamma) LAUNCH("column_sum", st, launch_column_sum(a.part, grid, cols, dgamma, accumulate, 0, st));
  return CONV2D_OK;
}

}  // extern "C"
