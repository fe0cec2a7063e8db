// rows.cu - kernels over rows of features: RMS norm with the residual's
// addition and its backward, 8-bit checkpoints (encode, decode), the backward
// through a dense layer's activation, and the column sums and joins behind
// them. All are bound by memory: each reads its inputs once and writes its
// outputs once, in accesses of 32 bytes (a sector) a thread where the rows
// start on such boundaries, of 16 bytes where they start on those, element by
// element (V = 1) otherwise.
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <cmath>

#include "host.h"
#include "kernels.h"
#include "q8.cuh"
#include "rows.h"

namespace c2d {
namespace {

constexpr long kMaxGridX = 0x7fffffffL;

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Sum (or maximum of magnitude bits) over the TPR threads of a row; red: one word per warp. Every thread
// of the row gets the result, formed in the same order by all.
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float* red) {
  v = warp_sum(v);
  if constexpr (TPR > 32) {
    const int warp = threadIdx.x >> 5;
    __syncthreads();  // the last use of red is over
    if ((threadIdx.x & 31) == 0) red[warp] = v;
    __syncthreads();
    v = 0.f;
#pragma unroll
    for (int i = 0; i < TPR / 32; ++i) v += red[i];
  }
  return v;
}
template <int TPR>
__device__ __forceinline__ uint32_t row_max(uint32_t v, uint32_t* red) {
  v = __reduce_max_sync(0xffffffffu, v);
  if constexpr (TPR > 32) {
    const int warp = threadIdx.x >> 5;
    __syncthreads();
    if ((threadIdx.x & 31) == 0) red[warp] = v;
    __syncthreads();
    v = 0u;
#pragma unroll
    for (int i = 0; i < TPR / 32; ++i) v = max(v, red[i]);
  }
  return v;
}

struct NormArgs {
  const void *x, *r;
  const float* gamma;
  void *h, *y;
  uint8_t *q, *qs;
  float* inv;
  long ldx, ldr, ldh, ldy, ldq;
  long rows;
  int cols, ng;  // ng: scale bytes a row
  int group;     // 32 or 0 (whole row)
  float eps;
};

// RMS norm forward (NORM) or 8-bit encode (!NORM): TPR threads a row, a block of them or (TPR = 32) eight warps. Rows are
// held in registers between their sum of squares and their output, U vectors a thread, so memory is passed once;
// U = 0 is the form for rows longer than that, which reads the row again for each phase (from L2, mostly). NR
// rows are in flight at once where a row is a vector or two a thread (one row of 512 bytes a warp left a
// 200704 x 256 encode at 41 us). Threads hold neighbouring vectors, so a group of 32 columns lies in 32 / V
// neighbouring lanes and its maximum is found by shuffles. Bound by memory: 8192 x 4096 bf16 with the residual, y
// and its 8-bit form moves 303 MB in 47 us, 0.95 of the measured copy rate.
template <typename T, int V, int TPR, int U, int NR, bool NORM>
__global__ void __launch_bounds__(TPR == 32 ? 256 : TPR) rows_fwd_kernel(const NormArgs a) {
  pdl_entry();
  constexpr int RPB = TPR == 32 ? 8 : 1;  // groups of NR rows per block
  static_assert(U > 0 || NR == 1, "one row at a time where it is read again");
  constexpr int UC = U > 0 ? U : 1;
  __shared__ float red[32];
  const int t = RPB > 1 ? static_cast<int>(threadIdx.x) & 31 : static_cast<int>(threadIdx.x);
  const long row0 = (static_cast<long>(blockIdx.x) * RPB + (RPB > 1 ? threadIdx.x >> 5 : 0)) * NR;
  if (row0 >= a.rows) return;  // whole warps; rows that use block barriers are whole blocks
  const int nr = static_cast<int>(min(a.rows - row0, static_cast<long>(NR)));
  const int nv = (a.cols + V - 1) / V;
  const int nu = U > 0 ? U : (nv + TPR - 1) / TPR;  // vectors a thread
  const T* xb = static_cast<const T*>(a.x) + row0 * a.ldx;
  const T* rb = static_cast<const T*>(a.r) + row0 * a.ldr;
  T* hb = static_cast<T*>(a.h) + row0 * a.ldh;

  float v[NR][UC][V];
  auto widen = [](const T (&e)[V], float (&o)[V]) {
#pragma unroll
    for (int k = 0; k < V; ++k) o[k] = to_f(e[k]);
  };
  // x + r as stored (h is written); zeros past the end
  auto load_all = [&](int u0, int n) {
    T e[NR][UC][V], f[NR][UC][V];
#pragma unroll
    for (int i = 0; i < NR; ++i)
#pragma unroll
      for (int u = 0; u < UC; ++u) {
        const int c = ((u0 + u) * TPR + t);
        if (i < nr && c < nv && u < n) {
          ld_vec<T, V>(xb + i * a.ldx + static_cast<long>(c) * V, e[i][u]);
          if (a.r) ld_vec<T, V>(rb + i * a.ldr + static_cast<long>(c) * V, f[i][u]);
        } else {
#pragma unroll
          for (int k = 0; k < V; ++k) e[i][u][k] = f[i][u][k] = from_f<T>(0.f);
        }
      }
#pragma unroll
    for (int i = 0; i < NR; ++i)
#pragma unroll
      for (int u = 0; u < UC; ++u) {
        const int c = ((u0 + u) * TPR + t);
        if (a.r) {
#pragma unroll
          for (int k = 0; k < V; ++k) e[i][u][k] = from_f<T>(to_f(e[i][u][k]) + to_f(f[i][u][k]));
          if (i < nr && c < nv && u < n) st_vec<T, V>(hb + i * a.ldh + static_cast<long>(c) * V, e[i][u]);
        }
        widen(e[i][u], v[i][u]);
      }
  };
  auto reload = [&](int u) {  // U = 0: this thread's own h (or x) again
    const int c = u * TPR + t;
    if (c < nv) {
      T e[V];
      ld_vec<T, V>((a.r ? static_cast<const T*>(hb) : xb) + static_cast<long>(c) * V, e);
      widen(e, v[0][0]);
    } else {
#pragma unroll
      for (int k = 0; k < V; ++k) v[0][0][k] = 0.f;
    }
  };

  float inv[NR];
#pragma unroll
  for (int i = 0; i < NR; ++i) inv[i] = 1.f;
  if constexpr (U > 0) load_all(0, UC);
  if constexpr (NORM) {
    float ss[NR];
#pragma unroll
    for (int i = 0; i < NR; ++i) ss[i] = 0.f;
    if constexpr (U > 0) {
#pragma unroll
      for (int i = 0; i < NR; ++i)
#pragma unroll
        for (int u = 0; u < UC; ++u)
#pragma unroll
          for (int k = 0; k < V; ++k) ss[i] = fmaf(v[i][u][k], v[i][u][k], ss[i]);
    } else {
      for (int u = 0; u < nu; ++u) {
        load_all(u, 1);
#pragma unroll
        for (int k = 0; k < V; ++k) ss[0] = fmaf(v[0][0][k], v[0][0][k], ss[0]);
      }
    }
#pragma unroll
    for (int i = 0; i < NR; ++i) {
      inv[i] = 1.f / sqrtf(row_sum<TPR>(ss[i], red) / static_cast<float>(a.cols) + a.eps);
      if (t == 0 && i < nr && a.inv) a.inv[row0 + i] = inv[i];
    }
  }
  pdl_release();
  // y = gamma h s of vector u, in place, for all NR rows (U = 0: of the one vector at hand)
  auto scale = [&](int u, int slot) {
    const int c = u * TPR + t;
    if (!NORM || c >= nv) return;
    const float* gp = a.gamma + static_cast<long>(c) * V;
    float g[V];
    if constexpr (V >= 4) {
#pragma unroll
      for (int k = 0; k < V; k += 4) *reinterpret_cast<float4*>(g + k) = *reinterpret_cast<const float4*>(gp + k);
    } else {
      g[0] = gp[0];
    }
#pragma unroll
    for (int i = 0; i < NR; ++i)
#pragma unroll
      for (int k = 0; k < V; ++k) v[i][slot][k] = v[i][slot][k] * inv[i] * g[k];
  };
  // Largest magnitude's bits; fmaxf passes NaN over, and infinities are looked for only where one shows.
  auto absmax = [&](const float (&o)[V]) {
    float m = 0.f;
#pragma unroll
    for (int k = 0; k < V; ++k) m = fmaxf(m, fabsf(o[k]));
    return __float_as_uint(m);
  };
  auto absmax_finite = [&](const float (&o)[V]) {
    uint32_t m = 0u;
#pragma unroll
    for (int k = 0; k < V; ++k) m = max(m, finite_bits(o[k]));
    return m;
  };
  constexpr uint32_t kInf = 0x7f800000u;
  uint32_t rowbyte[NR];
  bool rowfinite[NR];
  if (a.q && a.group == 0) {
    if constexpr (U > 0) {
#pragma unroll
      for (int u = 0; u < UC; ++u) scale(u, u);
    }
#pragma unroll
    for (int i = 0; i < NR; ++i) {
      uint32_t m = 0u;
      if constexpr (U > 0) {
#pragma unroll
        for (int u = 0; u < UC; ++u) m = max(m, absmax(v[i][u]));
      } else {
        for (int u = 0; u < nu; ++u) {
          reload(u);
          scale(u, 0);
          m = max(m, absmax(v[0][0]));
        }
      }
      m = row_max<TPR>(m, reinterpret_cast<uint32_t*>(red));
      rowfinite[i] = m != kInf;
      if (m == kInf) {  // the same for the whole row
        m = 0u;
        if constexpr (U > 0) {
#pragma unroll
          for (int u = 0; u < UC; ++u) m = max(m, absmax_finite(v[i][u]));
        } else {
          for (int u = 0; u < nu; ++u) {
            reload(u);
            scale(u, 0);
            m = max(m, absmax_finite(v[0][0]));
          }
        }
        m = row_max<TPR>(m, reinterpret_cast<uint32_t*>(red));
      }
      rowbyte[i] = q8_scale_byte(m);
      if (t == 0 && i < nr) a.qs[(row0 + i) * a.ng] = static_cast<uint8_t>(rowbyte[i]);
    }
  }
  auto finish = [&](int u, int slot) {
    const int c = u * TPR + t;
#pragma unroll
    for (int i = 0; i < NR; ++i) {
      const bool on = i < nr && c < nv;
      float(&o)[V] = v[i][slot];
      if (a.y && on) {
        T e[V];
#pragma unroll
        for (int k = 0; k < V; ++k) e[k] = from_f<T>(o[k]);
        st_vec<T, V>(static_cast<T*>(a.y) + (row0 + i) * a.ldy + static_cast<long>(c) * V, e);
      }
      if (a.q) {
        uint32_t byte = rowbyte[i];
        bool finite = rowfinite[i];
        if (a.group != 0) {
          auto group_max = [](uint32_t m) {
            if constexpr (V == 1) {  // the group is the warp
              return __reduce_max_sync(0xffffffffu, m);
            } else {
#pragma unroll
              for (int s = 1; s < kQ8Group / V; s <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, s));
              return m;
            }
          };
          uint32_t m = group_max(absmax(o));
          finite = true;
          if (__any_sync(0xffffffffu, m == kInf)) {
            finite = false;
            m = group_max(absmax_finite(o));
          }
          byte = q8_scale_byte(m);
          if (on && (t & (kQ8Group / V - 1)) == 0)
            a.qs[(row0 + i) * a.ng + c / (kQ8Group / V)] = static_cast<uint8_t>(byte);
        }
        if (on) q8_store<V>(a.q + (row0 + i) * a.ldq + static_cast<long>(c) * V, o, q8_inv_scale(byte), finite);
      }
    }
  };
  if constexpr (U > 0) {
#pragma unroll
    for (int u = 0; u < UC; ++u) {
      if (!(a.q && a.group == 0)) scale(u, u);
      finish(u, u);
    }
  } else {
    for (int u = 0; u < nu; ++u) {
      if constexpr (NORM) {
        reload(u);
        scale(u, 0);
      } else {
        reload(u);
      }
      finish(u, 0);
    }
  }
}

template <typename T, int V, bool NORM>
cudaError_t rows_fwd(const NormArgs& a, cudaStream_t st) {
  const int nv = (a.cols + V - 1) / V;
#define ROWS_FWD(TPR, U, NR)                                                                                        \
  do {                                                                                                              \
    constexpr int nt = (TPR) == 32 ? 256 : (TPR), rpb = nt / (TPR) * (NR);                                         \
    return launch_k(rows_fwd_kernel<T, V, TPR, U, NR, NORM>, dim3(static_cast<unsigned>((a.rows + rpb - 1) / rpb)), \
                    dim3(nt), 0, st, 1, a);                                                                         \
  } while (0)
  // 16 to 32 values a thread where a warp takes a row (8 to 16 when they are loaded one by one); long rows are
  // spread over 256 or 512 threads
  if (nv <= 32) ROWS_FWD(32, 1, (V == 16 ? 2 : V == 1 ? 8 : 4));
  if (nv <= 64) ROWS_FWD(32, 2, (V == 16 ? 1 : V == 1 ? 4 : 2));
  if constexpr (V < 16)
    if (nv <= 128) ROWS_FWD(32, 4, (V == 1 ? 4 : 1));
  // vectors: no more threads than a row has of them, two each (16384 x 2048 bf16 51 us with 256 threads, 42 with 64; 1536
  // columns 46 and 32; 4096 x 5120 33 and 29); rows of single elements take 256 threads from 129 elements on
  if constexpr (V > 1) {
    if constexpr (V == 16)
      if (nv <= 128) ROWS_FWD(64, 2, 1);
    if (nv <= 192) ROWS_FWD(96, 2, 1);
  }
  if (nv <= 256) ROWS_FWD(256, 1, 1);
  if constexpr (V > 1) {
    if (nv <= 320) ROWS_FWD(160, 2, 1);
    if (nv <= 384) ROWS_FWD(192, 2, 1);
  }
  if (nv <= 512) ROWS_FWD(256, 2, 1);
  if constexpr (V == 16) {
    if (nv <= 1024) ROWS_FWD(512, 2, 1);
  } else {
    if (nv <= 1024) ROWS_FWD(256, 4, 1);
    if (nv <= 2048) ROWS_FWD(512, 4, 1);
  }
  if constexpr (V == 1) {  // single elements take few registers
    if (nv <= 4096) ROWS_FWD(512, 8, 1);
    if (nv <= 8192) ROWS_FWD(1024, 8, 1);
    if (nv <= 16384) ROWS_FWD(1024, 16, 1);
  }
  ROWS_FWD(1024, 0, 1);
#undef ROWS_FWD
}

// ------------------------------------------------------------------ RMS norm backward
struct NormBwdArgs {
  const void *h, *dy, *dh;
  void* dx;
  const float *gamma, *inv;
  float* part;  // [gridDim.x][cols], null: no dgamma
  long ldh, lddy, lddh, lddx;
  long rows;
  int cols;
};

// Blocks that an SM holds and is given, by the threads of a row (32: blocks of 256): about 512 threads of up to 128
// registers. A second wave of larger blocks only adds partial sums (8192 x 8192 bf16: 100 us, 91 without).
constexpr int norm_bwd_resident(int tpr) {
  return tpr > 256 ? 1 : tpr == 64 ? 8 : tpr == 128 ? 4 : tpr == 192 ? 3 : 2;
}

// Blocks walk the rows (row = block, block + grid, ...), TPR threads a row, and keep the sums of dgamma for their
// columns in registers. AHEAD: gamma too, and the vectors of the next row are in flight while this one is reduced;
// without it (rows whose values take the registers) gamma and dh are read where they are needed. U = 0: rows
// longer than the registers hold; each row is read twice and dgamma's sums live in this block's row of `part`.
// Bound by memory: 8192 x 4096 bf16 with dh moves 268 MB in 46 us, 0.85 of the copy rate (64 us with one block of
// 136 registers a thread an SM, before the registers were held to two).
template <typename T, int V, int TPR, int U, bool AHEAD>
__global__ void __launch_bounds__(TPR == 32 ? 256 : TPR, norm_bwd_resident(TPR)) norm_bwd_kernel(const NormBwdArgs a) {
  pdl_entry();
  constexpr int RPB = TPR == 32 ? 8 : 1;
  constexpr int UC = U > 0 ? U : 1;
  extern __shared__ float sums[];  // RPB > 1 with dgamma: [RPB][cols]
  __shared__ float red[32];
  const int t = RPB > 1 ? static_cast<int>(threadIdx.x) & 31 : static_cast<int>(threadIdx.x);
  const int wr = RPB > 1 ? static_cast<int>(threadIdx.x >> 5) : 0;
  const int nv = (a.cols + V - 1) / V;
  const float invD = 1.f / static_cast<float>(a.cols);
  const T* hb = static_cast<const T*>(a.h);
  const T* db = static_cast<const T*>(a.dy);
  const T* sb = static_cast<const T*>(a.dh);
  T* xb = static_cast<T*>(a.dx);
  const long step = static_cast<long>(gridDim.x) * RPB;
  const long row0 = static_cast<long>(blockIdx.x) * RPB + wr;

  if constexpr (U > 0) {
    float g[AHEAD ? UC : 1][V], acc[UC][V];
    auto load_gamma = [&](int u, float (&o)[V]) {
      const int c = (u * TPR + t) * V;
#pragma unroll
      for (int k = 0; k < V; ++k) o[k] = 0.f;
      if (c >= a.cols) return;
      if constexpr (V >= 4) {
#pragma unroll
        for (int k = 0; k < V; k += 4) *reinterpret_cast<float4*>(o + k) = *reinterpret_cast<const float4*>(a.gamma + c + k);
      } else {
        o[0] = a.gamma[c];
      }
    };
#pragma unroll
    for (int u = 0; u < UC; ++u) {
      if constexpr (AHEAD) load_gamma(u, g[u]);
#pragma unroll
      for (int k = 0; k < V; ++k) acc[u][k] = 0.f;
    }
    T h[UC][V], d[UC][V], s[AHEAD ? UC : 1][V];
    float inv = 0.f;
    auto fetch = [&](long row) {
      if (row < a.rows) inv = a.inv[row];
#pragma unroll
      for (int u = 0; u < UC; ++u) {
        const int i = u * TPR + t;
        if (row < a.rows && i < nv) {
          ld_vec<T, V>(hb + row * a.ldh + static_cast<long>(i) * V, h[u]);
          ld_vec<T, V>(db + row * a.lddy + static_cast<long>(i) * V, d[u]);
          if constexpr (AHEAD)
            if (sb && xb) ld_vec<T, V>(sb + row * a.lddh + static_cast<long>(i) * V, s[u]);
        } else {
#pragma unroll
          for (int k = 0; k < V; ++k) h[u][k] = d[u][k] = from_f<T>(0.f);
        }
      }
    };
    if constexpr (AHEAD) fetch(row0);
    for (long row = row0; row < a.rows; row += step) {
      if constexpr (!AHEAD) fetch(row);
      float hf[UC][V], df[UC][V];
      T sk[AHEAD ? UC : 1][V];
      const float iv = inv;
      float dot = 0.f;
#pragma unroll
      for (int u = 0; u < UC; ++u) {
        float gu[V];
        if constexpr (!AHEAD) load_gamma(u, gu);
#pragma unroll
        for (int k = 0; k < V; ++k) {
          hf[u][k] = to_f(h[u][k]) * iv;  // the normalised value
          df[u][k] = to_f(d[u][k]);
          if constexpr (AHEAD) sk[u][k] = s[u][k];
          acc[u][k] = fmaf(df[u][k], hf[u][k], acc[u][k]);
          df[u][k] *= AHEAD ? g[AHEAD ? u : 0][k] : gu[k];
          dot = fmaf(df[u][k], hf[u][k], dot);
        }
      }
      if constexpr (AHEAD) fetch(row + step);
      if (xb) {
        dot = row_sum<TPR>(dot, red) * invD;
#pragma unroll
        for (int u = 0; u < UC; ++u) {
          const int i = u * TPR + t;
          if (i < nv) {
            T o[V], sv[V];
            if constexpr (!AHEAD)
              if (sb) ld_vec<T, V>(sb + row * a.lddh + static_cast<long>(i) * V, sv);
#pragma unroll
            for (int k = 0; k < V; ++k) {
              float v = iv * fmaf(-hf[u][k], dot, df[u][k]);
              if (sb) v += to_f(AHEAD ? sk[AHEAD ? u : 0][k] : sv[k]);
              o[k] = from_f<T>(v);
            }
            st_vec<T, V>(xb + row * a.lddx + static_cast<long>(i) * V, o);
          }
        }
      }
    }
    pdl_release();
    if (!a.part) return;
    float* part = a.part + static_cast<long>(blockIdx.x) * a.cols;
    if constexpr (RPB > 1) {
#pragma unroll
      for (int u = 0; u < UC; ++u)
#pragma unroll
        for (int k = 0; k < V; ++k) {
          const int c = (u * TPR + t) * V + k;
          if (c < a.cols) sums[wr * a.cols + c] = acc[u][k];
        }
      __syncthreads();
      for (int c = threadIdx.x; c < a.cols; c += 256) {
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < RPB; ++w) v += sums[w * a.cols + c];
        part[c] = v;
      }
    } else {
#pragma unroll
      for (int u = 0; u < UC; ++u)
#pragma unroll
        for (int k = 0; k < V; ++k) {
          const int c = (u * TPR + t) * V + k;
          if (c < a.cols) part[c] = acc[u][k];
        }
    }
  } else {
    float* part = a.part ? a.part + static_cast<long>(blockIdx.x) * a.cols : nullptr;
    if (part)
      for (int i = t; i < nv; i += TPR)
        for (int k = 0; k < V; ++k) part[static_cast<long>(i) * V + k] = 0.f;
    for (long row = row0; row < a.rows; row += step) {
      const float iv = a.inv[row];
      float dot = 0.f;
      for (int i = t; i < nv; i += TPR) {
        T h[V], d[V];
        ld_vec<T, V>(hb + row * a.ldh + static_cast<long>(i) * V, h);
        ld_vec<T, V>(db + row * a.lddy + static_cast<long>(i) * V, d);
#pragma unroll
        for (int k = 0; k < V; ++k) {
          const long c = static_cast<long>(i) * V + k;
          const float hn = to_f(h[k]) * iv, dv = to_f(d[k]);
          if (part) part[c] = fmaf(dv, hn, part[c]);
          dot = fmaf(dv * a.gamma[c], hn, dot);
        }
      }
      if (!xb) continue;
      dot = row_sum<TPR>(dot, red) * invD;
      for (int i = t; i < nv; i += TPR) {
        T h[V], d[V], s[V], o[V];
        ld_vec<T, V>(hb + row * a.ldh + static_cast<long>(i) * V, h);
        ld_vec<T, V>(db + row * a.lddy + static_cast<long>(i) * V, d);
        if (sb) ld_vec<T, V>(sb + row * a.lddh + static_cast<long>(i) * V, s);
#pragma unroll
        for (int k = 0; k < V; ++k) {
          const long c = static_cast<long>(i) * V + k;
          float v = iv * fmaf(-to_f(h[k]) * iv, dot, to_f(d[k]) * a.gamma[c]);
          if (sb) v += to_f(s[k]);
          o[k] = from_f<T>(v);
        }
        st_vec<T, V>(xb + row * a.lddx + static_cast<long>(i) * V, o);
      }
    }
  }
}

// The most blocks that the backward of rows of this length is launched with (norm_bwd's choices below).
long norm_bwd_blocks(int64_t rows, int cols, int sms) {
  return std::min<long>(rows, static_cast<long>(sms) * (cols <= 64 * 16 ? 8 : cols <= 128 * 16 ? 4 : cols <= 192 * 16 ? 3 : 2));
}

// grid: blocks launched, one row of partial sums each.
template <typename T, int V>
cudaError_t norm_bwd(const NormBwdArgs& a, int sms, int* grid, cudaStream_t st) {
  const int nv = (a.cols + V - 1) / V;
#define NORM_BWD(TPR, U, AHEAD)                                                                   \
  do {                                                                                            \
    constexpr int nt = (TPR) == 32 ? 256 : (TPR);                                                 \
    const size_t smem = nt > (TPR) && a.part ? static_cast<size_t>(nt / (TPR)) * a.cols * 4 : 0;  \
    *grid = static_cast<int>(std::min<long>(a.rows, static_cast<long>(sms) * norm_bwd_resident(TPR))); \
    return launch_k(norm_bwd_kernel<T, V, TPR, U, AHEAD>, dim3(*grid), dim3(nt), smem, st, 1, a); \
  } while (0)
  // Vectors: as many threads as the row has of them (two a thread where a vector is 16 bytes), so that an SM's threads
  // all have loads in flight: 32768 x 1024 bf16 91 us with 256 threads, 50 with 64; 16384 x 1000 48 and 28. Rows of
  // single elements take 256 threads from 65 elements on, of which short rows leave most idle.
  if (nv <= 32) NORM_BWD(32, 1, true);
  if constexpr (V == 16) {
    if (nv <= 64) NORM_BWD(64, 1, true);
    if (nv <= 128) NORM_BWD(128, 1, true);
    if (nv <= 256) NORM_BWD(256, 1, true);
    if (nv <= 320) NORM_BWD(320, 1, true);
    if (nv <= 512) NORM_BWD(512, 1, true);
    if (nv <= 1024) NORM_BWD(512, 2, false);
  } else if constexpr (V > 1) {
    if (nv <= 64) NORM_BWD(32, 2, true);
    if (nv <= 128) NORM_BWD(64, 2, true);
    if (nv <= 256) NORM_BWD(128, 2, true);
    if (nv <= 384) NORM_BWD(192, 2, true);
    if (nv <= 512) NORM_BWD(256, 2, true);
    if (nv <= 768) NORM_BWD(384, 2, true);
    if (nv <= 1024) NORM_BWD(512, 2, true);
    if (nv <= 2048) NORM_BWD(512, 4, false);
  } else {
    if (nv <= 64) NORM_BWD(32, 2, true);
    if (nv <= 256) NORM_BWD(256, 1, true);
    if (nv <= 512) NORM_BWD(256, 2, true);
    if (nv <= 1024) NORM_BWD(512, 2, true);
    if (nv <= 2048) NORM_BWD(512, 4, true);
    if (nv <= 4096) NORM_BWD(1024, 4, true);
    if (nv <= 8192) NORM_BWD(1024, 8, true);
    if (nv <= 16384) NORM_BWD(1024, 16, false);
  }
  NORM_BWD(1024, 0, false);
#undef NORM_BWD
}

// ------------------------------------------------------------------ 8 bits, 16-bit types in whole groups
// Encode (ENC) or decode of rows of whole 32-column groups: two threads a group, 16 values each, two groups of a
// thread in flight (200704 x 256 there and back: 46.5 us, 0.99 of the copy rate; 59 us with 16-byte accesses).
// total = rows * cols / 16 < 2^31; x rows on 32-byte, q rows on 16-byte boundaries.
template <typename T, bool ENC, bool LATE>
__global__ void __launch_bounds__(256) q8_flat_kernel(T* x, long ldx, uint8_t* q, long ldq, uint8_t* scale,
                                                      uint32_t total, FastDiv div_nv) {
  if (!LATE) pdl_entry();
  pdl_release();
  constexpr int N = 2;
  const uint32_t step = gridDim.x * 256u;
  const int ng = static_cast<int>(div_nv.d / 2);
  for (uint32_t j0 = blockIdx.x * 256u + threadIdx.x; j0 < total; j0 += N * step) {
    uint32_t w[N][8];
    uint4 raw[N];
    uint32_t sb[N];
    long row[N];
    int v[N];  // 16-value vector of the row
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const uint32_t j = j0 + i * step;
      if (j >= total) break;
      const uint32_t r = fdiv(j, div_nv);
      row[i] = r;
      v[i] = static_cast<int>(j - r * div_nv.d);
      if constexpr (ENC) {
        ld_32b(x + row[i] * ldx + v[i] * 16, w[i]);
      } else {
        raw[i] = *reinterpret_cast<const uint4*>(q + row[i] * ldq + v[i] * 16);
        sb[i] = scale[row[i] * ng + (v[i] >> 1)];
      }
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (j0 + i * step >= total) break;  // the two threads of a group go on together (total is even)
      float f[16];
      if constexpr (ENC) {
        const T* e = reinterpret_cast<const T*>(w[i]);
        float m = 0.f;
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          f[k] = to_f(e[k]);
          m = fmaxf(m, fabsf(f[k]));
        }
        const uint32_t pair = 3u << (threadIdx.x & 30u);
        uint32_t top = __float_as_uint(m);
        top = max(top, __shfl_xor_sync(pair, top, 1));
        bool finite = true;
        if (top == 0x7f800000u) {
          finite = false;
          top = 0u;
#pragma unroll
          for (int k = 0; k < 16; ++k) top = max(top, finite_bits(f[k]));
          top = max(top, __shfl_xor_sync(pair, top, 1));
        }
        const uint32_t byte = q8_scale_byte(top);
        const float inv = q8_inv_scale(byte);
        *reinterpret_cast<uint4*>(q + row[i] * ldq + v[i] * 16) =
            make_uint4(q8_pack4(f, inv, finite), q8_pack4(f + 4, inv, finite), q8_pack4(f + 8, inv, finite),
                       q8_pack4(f + 12, inv, finite));
        if ((v[i] & 1) == 0) scale[row[i] * ng + (v[i] >> 1)] = static_cast<uint8_t>(byte);
      } else {
        const Q8Raw<16> rw = {{raw[i].x, raw[i].y, raw[i].z, raw[i].w}};
        const float sc = q8_scale(sb[i]);
        q8_values<16>(rw, f, sc);
        T* e = reinterpret_cast<T*>(w[i]);
        if (sc > q8_safe_scale<T>()) {
#pragma unroll
          for (int k = 0; k < 16; ++k) e[k] = from_q8<T>(f[k]);
        } else {
#pragma unroll
          for (int k = 0; k < 16; ++k) e[k] = from_f<T>(f[k]);
        }
        st_32b(x + row[i] * ldx + v[i] * 16, w[i]);
      }
    }
  }
  if (LATE) pdl_entry();
}
int stream_grid(long items) { return static_cast<int>(std::max<long>(1, std::min<long>((items + 255) / 256, 152L * 64))); }

// Whether the flat kernel takes it, and its launch.
template <typename T, bool ENC>
bool q8_flat(const void* x, long ldx, const void* q, long ldq, uint8_t* scale, int group, long rows, int cols, int late,
             cudaStream_t st, cudaError_t* e) {
  if (group != kQ8Group || cols % kQ8Group != 0 || ldx % 16 != 0 || ldq % 16 != 0 ||
      reinterpret_cast<uintptr_t>(x) % 32 != 0 || rows * (cols / 16) > 0x7fffffffL)
    return false;
  const long total = rows * (cols / 16);
  auto go = [&](auto kernel) {
    return launch_k(kernel, dim3(stream_grid((total + 1) / 2)), dim3(256), 0, st, 1,
                    static_cast<T*>(const_cast<void*>(x)), ldx, static_cast<uint8_t*>(const_cast<void*>(q)), ldq, scale,
                    static_cast<uint32_t>(total), make_fastdiv(static_cast<uint32_t>(cols / 16)));
  };
  if constexpr (!ENC)
    if (late) {
      *e = go(q8_flat_kernel<T, ENC, true>);
      return true;
    }
  *e = go(q8_flat_kernel<T, ENC, false>);
  return true;
}

// ------------------------------------------------------------------ decode / move
// V elements a thread and step of a [rows][cols] matrix, dense steps of the grid (E4M3 source: V bytes and
// their scale, two output vectors). rows * ceil(cols / V) below 2^31 (see to_rows).
template <typename T, int V, bool Q, bool LATE>
__global__ void __launch_bounds__(256) to_rows_kernel(const void* x, long ldx, const uint8_t* scale, int group, int ng,
                                                      uint32_t total, int cols, FastDiv div_nv, T* out, long ldo) {
  if (!LATE) pdl_entry();
  pdl_release();
  constexpr int VO = V * sizeof(T) > 16 ? 16 / static_cast<int>(sizeof(T)) : V;  // elements a store
  constexpr int N = 2;                                                          // steps in flight
  const uint32_t step = gridDim.x * 256u;
  for (uint32_t j0 = blockIdx.x * 256u + threadIdx.x; j0 < total; j0 += N * step) {
    Q8Raw<V> raw[N];
    T e[N][V];
    float sc[N];
    long row[N];
    int c[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const uint32_t j = j0 + i * step;
      if (j >= total) break;
      const uint32_t r = fdiv(j, div_nv);
      row[i] = r;
      c[i] = static_cast<int>(j - r * div_nv.d) * V;
      if constexpr (Q) {
        raw[i] = q8_load<V>(static_cast<const uint8_t*>(x) + row[i] * ldx + c[i]);
        sc[i] = q8_scale(scale[row[i] * ng + (group ? c[i] / kQ8Group : 0)]);
      } else {
        ld_vec<T, V>(static_cast<const T*>(x) + row[i] * ldx + c[i], e[i]);
      }
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (j0 + i * step >= total) break;
      if constexpr (Q) {
        float v[V];
        q8_values<V>(raw[i], v, sc[i]);
        if (sc[i] > q8_safe_scale<T>()) {
#pragma unroll
          for (int k = 0; k < V; ++k) e[i][k] = from_q8<T>(v[k]);
        } else {
#pragma unroll
          for (int k = 0; k < V; ++k) e[i][k] = from_f<T>(v[k]);
        }
      }
      T* o = out + row[i] * ldo + c[i];
#pragma unroll
      for (int k = 0; k < V; k += VO) st_vec<T, VO>(o + k, *reinterpret_cast<const T(*)[VO]>(&e[i][k]));
    }
  }
  if (LATE) pdl_entry();
}

// The same for rows that do not start on vector boundaries, or end within a vector: a warp takes 32 N W neighbouring
// elements of a row, W neighbours a lane (output rows start on boundaries of W elements). With W = 4 the neighbours
// come out of the aligned words that hold them: two for E4M3, three for 16-bit elements.
__host__ __device__ constexpr int ragged_chunk(int W) { return W == 4 ? 512 : 256; }
template <typename T, bool Q, int W, bool LATE>
__global__ void __launch_bounds__(256) to_rows_ragged_kernel(const void* x, long ldx, const uint8_t* scale, int group,
                                                             int ng, uint32_t total, FastDiv div_chunks, int cols, T* out,
                                                             long ldo) {
  if (!LATE) pdl_entry();
  pdl_release();
  constexpr int N = ragged_chunk(W) / (32 * W);
  const int lane = threadIdx.x & 31;
  for (uint32_t j = blockIdx.x * 8u + (threadIdx.x >> 5); j < total; j += gridDim.x * 8u) {
    const uint32_t r = fdiv(j, div_chunks);
    const long row = r;
    const int c0 = static_cast<int>(j - r * div_chunks.d) * ragged_chunk(W) + lane * W;
    alignas(8) T e[N][W];
    uint32_t raw[N], sb[N];
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const int c = c0 + 32 * W * k;
      if (c >= cols) continue;
      if constexpr (Q) {
        const uint8_t* p = static_cast<const uint8_t*>(x) + row * ldx + c;
        if (W == 4 && c + 8 <= cols) {  // both words lie within the row's end (and after the 16-byte aligned base)
          const uint32_t off = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p) & 3u);
          const uint32_t* w = reinterpret_cast<const uint32_t*>(p - off);
          raw[k] = __funnelshift_r(w[0], w[1], off * 8u);
        } else {
          raw[k] = p[0];
#pragma unroll
          for (int i = 1; i < W; ++i)
            if (c + i < cols) raw[k] |= static_cast<uint32_t>(p[i]) << (8 * i);
        }
        sb[k] = scale[row * ng + (group ? c / kQ8Group : 0)];  // W divides c and a group: one scale for the neighbours
      } else {
        const T* p = static_cast<const T*>(x) + row * ldx + c;
        if constexpr (W == 4) {
          if (c + 6 <= cols) {  // the words lie within the row's end
            const uint32_t off = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p) & 2u);
            const uint32_t* w = reinterpret_cast<const uint32_t*>(reinterpret_cast<const char*>(p) - off);
            uint32_t* o = reinterpret_cast<uint32_t*>(e[k]);
            const uint32_t a = w[0], b = w[1], d = off ? w[2] : 0u;
            o[0] = __funnelshift_r(a, b, off * 8u);
            o[1] = __funnelshift_r(b, d, off * 8u);
            continue;
          }
        }
#pragma unroll
        for (int w = 0; w < W; ++w)
          if (w == 0 || c + w < cols) e[k][w] = p[w];
      }
    }
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const int c = c0 + 32 * W * k;
      if (c >= cols) continue;
      if constexpr (Q) {
        const float sc = q8_scale(sb[k]);
#pragma unroll
        for (int i = 0; i < W; i += 2) {
          const float2 f = q8_unpack2(raw[k] >> (8 * i));
          e[k][i] = from_q8<T>(f.x * sc);
          if constexpr (W > 1) e[k][i + 1] = from_q8<T>(f.y * sc);
        }
      }
      T* o = out + row * ldo + c;
      if (W * sizeof(T) == 8 && c + W <= cols) {
        *reinterpret_cast<uint2*>(o) = *reinterpret_cast<const uint2*>(e[k]);
      } else if (W * sizeof(T) == 4 && c + W <= cols) {
        *reinterpret_cast<uint32_t*>(o) = *reinterpret_cast<const uint32_t*>(e[k]);
      } else {
#pragma unroll
        for (int w = 0; w < W; ++w)
          if (c + w < cols) o[w] = e[k][w];
      }
    }
  }
  if (LATE) pdl_entry();
}

// Rows that start on boundaries of a vector of V elements of es bytes (the base at least on 16 bytes by contract).
bool vec_ok(const void* p, long ld, int es, int V) {
  return reinterpret_cast<uintptr_t>(p) % (V * es > 16 ? 32 : 16) == 0 && ld % V == 0;
}

template <typename T, bool Q, int W>
cudaError_t to_rows_ragged(const void* x, long ldx, const uint8_t* scale, int group, int ng, long rows, int cols,
                           void* out, long ldo, int late, cudaStream_t st) {
  const int chunks = (cols + ragged_chunk(W) - 1) / ragged_chunk(W);
  const long slab = std::max<long>(1, 0x7fffffffL / chunks);  // rows a launch indexes in 31 bits
  const FastDiv div = make_fastdiv(static_cast<uint32_t>(chunks));
  for (long r0 = 0; r0 < rows; r0 += slab) {
    const long n = std::min(slab, rows - r0);
    const uint32_t total = static_cast<uint32_t>(n * chunks);
    const dim3 grid(static_cast<unsigned>(std::min<long>((n * chunks + 7) / 8, 152L * 64)));
    const void* src = static_cast<const char*>(x) + r0 * ldx * (Q ? 1 : static_cast<long>(sizeof(T)));
    const uint8_t* sc = Q ? scale + r0 * ng : nullptr;
    T* o = static_cast<T*>(out) + r0 * ldo;
    const cudaError_t e =
        late ? launch_k(to_rows_ragged_kernel<T, Q, W, true>, grid, dim3(256), 0, st, 1, src, ldx, sc, group, ng, total,
                        div, cols, o, ldo)
             : launch_k(to_rows_ragged_kernel<T, Q, W, false>, grid, dim3(256), 0, st, 1, src, ldx, sc, group, ng, total,
                        div, cols, o, ldo);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

template <typename T>
cudaError_t to_rows(const conv2d_mat& x, long rows, int cols, void* out, long ldo, int late, cudaStream_t st) {
  constexpr int VV = 16 / sizeof(T), VQ = 16;
  const bool q = x.type == CONV2D_E4M3;
  const long ldx = x.ld ? x.ld : cols, ld = ldo ? ldo : cols;
  const int ng = x.group ? (cols + kQ8Group - 1) / kQ8Group : 1;
  // whole vectors only: cols a multiple of the vector, and both rows' starts aligned to theirs
  if constexpr (sizeof(T) == 2) {
    cudaError_t e;
    if (q && q8_flat<T, false>(out, ld, x.data, ldx, x.scale, x.group, rows, cols, late, st, &e)) return e;
  }
  const int V = q ? VQ : VV;
  const bool vec = cols % V == 0 && vec_ok(out, ld, sizeof(T), VV) && vec_ok(x.data, ldx, q ? 1 : sizeof(T), V);
  if (!vec) {
    if constexpr (sizeof(T) == 2) {
      if (ld % 4 == 0)
        return q ? to_rows_ragged<T, true, 4>(x.data, ldx, x.scale, x.group, ng, rows, cols, out, ld, late, st)
                 : to_rows_ragged<T, false, 4>(x.data, ldx, nullptr, 0, 1, rows, cols, out, ld, late, st);
      if (ld % 2 == 0)
        return q ? to_rows_ragged<T, true, 2>(x.data, ldx, x.scale, x.group, ng, rows, cols, out, ld, late, st)
                 : to_rows_ragged<T, false, 2>(x.data, ldx, nullptr, 0, 1, rows, cols, out, ld, late, st);
    }
    return q ? to_rows_ragged<T, true, 1>(x.data, ldx, x.scale, x.group, ng, rows, cols, out, ld, late, st)
             : to_rows_ragged<T, false, 1>(x.data, ldx, nullptr, 0, 1, rows, cols, out, ld, late, st);
  }
  const int nv = cols / V;
  const long slab = std::max<long>(1, 0x7fffffffL / nv);  // rows a launch indexes in 31 bits
  for (long r0 = 0; r0 < rows; r0 += slab) {
    const long n = std::min(slab, rows - r0);
    const uint32_t total = static_cast<uint32_t>(n * nv);
    const dim3 grid(stream_grid((n * nv + 1) / 2));
    const char* src = static_cast<const char*>(x.data) + r0 * ldx * (q ? 1 : static_cast<long>(sizeof(T)));
    const uint8_t* sc = q ? x.scale + r0 * ng : nullptr;
    T* o = static_cast<T*>(out) + r0 * ld;
    const FastDiv div = make_fastdiv(static_cast<uint32_t>(nv));
#define TO_ROWS(V, Q)                                                                                                  \
  (late ? launch_k(to_rows_kernel<T, V, Q, true>, grid, dim3(256), 0, st, 1, static_cast<const void*>(src), ldx, sc,  \
                   x.group, ng, total, cols, div, o, ld)                                                               \
        : launch_k(to_rows_kernel<T, V, Q, false>, grid, dim3(256), 0, st, 1, static_cast<const void*>(src), ldx, sc, \
                   x.group, ng, total, cols, div, o, ld))
    const cudaError_t e = q ? TO_ROWS(VQ, true) : TO_ROWS(VV, false);
#undef TO_ROWS
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

// ------------------------------------------------------------------ backward through the activation
struct DactArgs {
  const void *dy, *z;
  const uint8_t* zs;
  void* dz;
  float* part;
  long lddy, ldz, lddz;
  long rows, rows_per_strip;
  int cols, group, ng, act;
};

// A block is 32 lanes of V columns by 8 rows; it walks the rows of its strip and keeps the column sums of
// the unrounded dz in registers, joined over the 8 row lanes at the end. ZK: 0 no activation, 1 z in T,
// 2 z as E4M3. Memory bounds it, with two special-function operations a value close behind (gelu): 4096 x 8192
// from 8-bit z moves 169 MB in 34 us, 0.74 of the copy rate (16 columns a lane; 70 against 63 us with 8 at twice the rows).
template <typename T, int V, int ZK, bool LATE>
__global__ void __launch_bounds__(256, V == 16 ? 2 : 3) dact_kernel(const DactArgs a) {
  if (!LATE) pdl_entry();
  constexpr int N = V == 1 ? 6 : V == 16 ? 2 : 3;  // rows in flight
  __shared__ float sums[8][32 * V];
  const int lane = threadIdx.x & 31, rl = threadIdx.x >> 5;
  const int c = (static_cast<int>(blockIdx.x) * 32 + lane) * V;
  const long r1 = min(a.rows, (static_cast<long>(blockIdx.y) + 1) * a.rows_per_strip);
  float acc[V];
#pragma unroll
  for (int k = 0; k < V; ++k) acc[k] = 0.f;
  if (c < a.cols) {
    const T* dy = static_cast<const T*>(a.dy) + c;
    const T* zt = static_cast<const T*>(a.z) + c;
    const uint8_t* zq = static_cast<const uint8_t*>(a.z) + c;
    const uint8_t* zs = a.zs + (a.group ? c / kQ8Group : 0);
    T* dz = a.dz ? static_cast<T*>(a.dz) + c : nullptr;
    with_dense_act(ZK ? a.act : 0, [&](auto act) {
#pragma unroll 1
      for (long r = blockIdx.y * a.rows_per_strip + rl; r < r1; r += 8 * N) {
        T d[N][V];
        [[maybe_unused]] T e[N][V];
        [[maybe_unused]] Q8Raw<V> q[N];
        [[maybe_unused]] uint32_t sb[N];
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const long ri = r + 8 * i;
          if (ri >= r1) break;
          ld_vec<T, V>(dy + ri * a.lddy, d[i]);
          if constexpr (ZK == 1) ld_vec<T, V>(zt + ri * a.ldz, e[i]);
          if constexpr (ZK == 2) {
            q[i] = q8_load<V>(zq + ri * a.ldz);
            sb[i] = zs[ri * a.ng];
          }
        }
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const long ri = r + 8 * i;
          if (ri >= r1) break;
          [[maybe_unused]] float f[V];
          if constexpr (ZK == 1) {
#pragma unroll
            for (int k = 0; k < V; ++k) f[k] = to_f(e[i][k]);
          }
          if constexpr (ZK == 2) q8_values<V>(q[i], f, q8_scale(sb[i]));
          T o[V];
          // products are not contracted into the sums: the column sums are the same whether dz is written or not
          if constexpr (V == 1) {
            float v = to_f(d[i][0]);
            if constexpr (ZK) v = __fmul_rn(v, dense_dact<decltype(act)::value>(make_float2(f[0], 0.f)).x);
            acc[0] += v;
            o[0] = from_f<T>(v);
          } else {
#pragma unroll
            for (int k = 0; k < V; k += 2) {
              float2 v = make_float2(to_f(d[i][k]), to_f(d[i][k + 1]));
              if constexpr (ZK) v = __fmul2_rn(v, dense_dact<decltype(act)::value>(make_float2(f[k], f[k + 1])));
              const float2 sum = __fadd2_rn(make_float2(acc[k], acc[k + 1]), v);
              acc[k] = sum.x;
              acc[k + 1] = sum.y;
              o[k] = from_f<T>(v.x);
              o[k + 1] = from_f<T>(v.y);
            }
          }
          if (dz) st_vec<T, V>(dz + ri * a.lddz, o);
        }
      }
    });
  }
  pdl_release();
  if (a.part) {
#pragma unroll
    for (int k = 0; k < V; ++k) sums[rl][lane * V + k] = acc[k];
    __syncthreads();
    for (int i = threadIdx.x; i < 32 * V; i += 256) {
      const int col = static_cast<int>(blockIdx.x) * 32 * V + i;
      if (col >= a.cols) continue;
      float v = 0.f;
#pragma unroll
      for (int w = 0; w < 8; ++w) v += sums[w][i];
      a.part[static_cast<long>(blockIdx.y) * a.cols + col] = v;
    }
  }
  if (LATE) pdl_entry();
}

template <typename T, int V, bool LATE>
cudaError_t dact_v(const DactArgs& a, int zk, int strips, cudaStream_t st) {
  const dim3 grid(static_cast<unsigned>((a.cols + 32 * V - 1) / (32 * V)), static_cast<unsigned>(strips));
  if (zk == 0) return launch_k(dact_kernel<T, V, 0, LATE>, grid, dim3(256), 0, st, 1, a);
  if (zk == 1) return launch_k(dact_kernel<T, V, 1, LATE>, grid, dim3(256), 0, st, 1, a);
  return launch_k(dact_kernel<T, V, 2, LATE>, grid, dim3(256), 0, st, 1, a);
}
template <typename T, int V>
cudaError_t dact_late(const DactArgs& a, int zk, int strips, int late, cudaStream_t st) {
  return late ? dact_v<T, V, true>(a, zk, strips, st) : dact_v<T, V, false>(a, zk, strips, st);
}
template <typename T>
cudaError_t dact(const DactArgs& a, int zk, int strips, int late, cudaStream_t st) {
  auto ok = [&](int V) {
    return a.cols % V == 0 && vec_ok(a.dy, a.lddy, sizeof(T), V) && (!a.dz || vec_ok(a.dz, a.lddz, sizeof(T), V)) &&
           (zk == 0 || vec_ok(a.z, a.ldz, zk == 2 ? 1 : sizeof(T), V));
  };
  // 16 columns a lane only where a warp's 512 are there
  if (a.cols >= 512 && ok(16)) return dact_late<T, 16>(a, zk, strips, late, st);
  return ok(8) ? dact_late<T, 8>(a, zk, strips, late, st) : dact_late<T, 1>(a, zk, strips, late, st);
}

// ------------------------------------------------------------------ column sums, joins, zeroes
// 32 columns a block, W warps over the partials (32 where there are many: a warp's loads come in rounds), then their
// sums in order.
template <int W>
__global__ void __launch_bounds__(W * 32) column_sum_kernel(const float* part, int G, int cols, float* out,
                                                         int accumulate, int late) {
  if (!late) pdl_entry();
  pdl_release();
  __shared__ float s[W][33];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int c = static_cast<int>(blockIdx.x) * 32 + lane;
  float v = 0.f;
  if (c < cols) {
#pragma unroll 10
    for (int g = w; g < G; g += W) v += part[static_cast<long>(g) * cols + c];
  }
  s[w][lane] = v;
  __syncthreads();
  if (w == 0 && c < cols) {
    float o = accumulate ? out[c] : 0.f;
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < W; ++i) sum += s[i][lane];
    out[c] = o + sum;
  }
  if (late) pdl_entry();
}

template <typename T, int V>
__global__ void __launch_bounds__(256) split_join_kernel(const float* part, int splits, long rows, int cols, T* out,
                                                         long ldo, int accumulate) {
  pdl_entry();
  pdl_release();
  const int nv = cols / V;
  const long total = rows * nv, plane = rows * cols;
  for (long j = static_cast<long>(blockIdx.x) * 256 + threadIdx.x; j < total; j += static_cast<long>(gridDim.x) * 256) {
    const long row = j / nv;
    const int c = static_cast<int>(j - row * nv) * V;
    const float* p = part + row * cols + c;
    float v[V];
#pragma unroll
    for (int k = 0; k < V; ++k) v[k] = 0.f;
#pragma unroll 4
    for (int s = 0; s < splits; ++s) {
      float e[V];
      if constexpr (V == 4) *reinterpret_cast<float4*>(e) = *reinterpret_cast<const float4*>(p + s * plane);
      else e[0] = p[s * plane];
#pragma unroll
      for (int k = 0; k < V; ++k) v[k] += e[k];
    }
    T* o = out + row * ldo + c;
#pragma unroll
    for (int k = 0; k < V; ++k) o[k] = from_f<T>(accumulate ? to_f(o[k]) + v[k] : v[k]);
  }
}

template <typename T>
__global__ void __launch_bounds__(256) zero_rows_kernel(long rows, int cols, T* out, long ld, int late) {
  if (!late) pdl_entry();
  pdl_release();
  const long total = rows * cols;
  for (long j = static_cast<long>(blockIdx.x) * 256 + threadIdx.x; j < total; j += static_cast<long>(gridDim.x) * 256) {
    const long row = j / cols;
    out[row * ld + (j - row * cols)] = from_f<T>(0.f);
  }
  if (late) pdl_entry();
}

}  // namespace

cudaError_t launch_to_rows(const conv2d_mat& x, long rows, int cols, int dt, void* out, long ldo, int late,
                           cudaStream_t st) {
  if (dt == CONV2D_BF16) return to_rows<__nv_bfloat16>(x, rows, cols, out, ldo, late, st);
  if (dt == CONV2D_FP16) return to_rows<__half>(x, rows, cols, out, ldo, late, st);
  return to_rows<float>(x, rows, cols, out, ldo, late, st);
}

cudaError_t launch_move_bytes(const void* x, long ldx, long rows, int cols, void* out, long ldo, int late,
                              cudaStream_t st) {
  return to_rows_ragged<uint8_t, false, 1>(x, ldx, nullptr, 0, 1, rows, cols, out, ldo, late, st);
}

DactPlan plan_dact(long rows, int cols, int sms) {
  // about eight blocks an SM, of 64 rows at least (eight passes, so that the joining at the end is small); a block
  // is 256 columns wide, or 32 where the columns do not divide into vectors
  const long chunks = cols % 8 == 0 ? (cols + 255) / 256 : (cols + 31) / 32;
  long strips = std::max<long>(1, 8L * sms / chunks);
  strips = std::min(strips, (rows + 63) / 64);
  strips = std::max<long>(1, std::min<long>(strips, 65535));
  DactPlan p;
  p.rows_per_strip = (rows + strips - 1) / strips;
  p.strips = static_cast<int>((rows + p.rows_per_strip - 1) / p.rows_per_strip);
  return p;
}

cudaError_t launch_dact(const conv2d_mat* z, const conv2d_mat& dy, long rows, int cols, int dt, int act, void* dz,
                        long lddz, float* part, const DactPlan& pl, int late, cudaStream_t st) {
  DactArgs a = {};
  a.dy = dy.data;
  a.lddy = dy.ld ? dy.ld : cols;
  int zk = 0;
  if (z) {
    zk = z->type == CONV2D_E4M3 ? 2 : 1;
    a.z = z->data;
    a.zs = z->scale;
    a.ldz = z->ld ? z->ld : cols;
    a.group = z->group;
    a.ng = z->group ? (cols + kQ8Group - 1) / kQ8Group : 1;
  }
  a.dz = dz;
  a.lddz = lddz;
  a.part = part;
  a.rows = rows;
  a.rows_per_strip = pl.rows_per_strip;
  a.cols = cols;
  a.act = act;
  return dt == CONV2D_BF16 ? dact<__nv_bfloat16>(a, zk, pl.strips, late, st) : dact<__half>(a, zk, pl.strips, late, st);
}

cudaError_t launch_column_sum(const float* part, int G, int cols, float* out, int accumulate, int late,
                              cudaStream_t st) {
  const dim3 grid((cols + 31) / 32);
  if (G > 320) return launch_k(column_sum_kernel<32>, grid, dim3(1024), 0, st, 1, part, G, cols, out, accumulate, late);
  return launch_k(column_sum_kernel<16>, grid, dim3(512), 0, st, 1, part, G, cols, out, accumulate, late);
}

template <typename T>
static cudaError_t split_join(const float* part, int splits, long rows, int cols, T* out, long ldo, int accumulate,
                              cudaStream_t st) {
  if (cols % 4 == 0)  // the partials are dense, so every row of them starts on a 16-byte boundary
    return launch_k(split_join_kernel<T, 4>, dim3(stream_grid(rows * (cols / 4))), dim3(256), 0, st, 1, part, splits,
                    rows, cols, out, ldo, accumulate);
  return launch_k(split_join_kernel<T, 1>, dim3(stream_grid(rows * cols)), dim3(256), 0, st, 1, part, splits, rows,
                  cols, out, ldo, accumulate);
}
cudaError_t launch_split_join(const float* part, int splits, long rows, int cols, int type, void* out, long ldo,
                              int accumulate, cudaStream_t st) {
  if (type == CONV2D_FP32) return split_join(part, splits, rows, cols, static_cast<float*>(out), ldo, accumulate, st);
  if (type == CONV2D_BF16)
    return split_join(part, splits, rows, cols, static_cast<__nv_bfloat16*>(out), ldo, accumulate, st);
  return split_join(part, splits, rows, cols, static_cast<__half*>(out), ldo, accumulate, st);
}

template <typename T>
static cudaError_t zero_rows(long rows, int cols, T* out, long ld, int late, cudaStream_t st) {
  return launch_k(zero_rows_kernel<T>, dim3(stream_grid(rows * cols)), dim3(256), 0, st, 1, rows, cols, out, ld, late);
}
cudaError_t launch_zero_rows(long rows, int cols, int type, void* out, long ld, int late, cudaStream_t st) {
  if (type == CONV2D_FP32) return zero_rows(rows, cols, static_cast<float*>(out), ld, late, st);
  if (type == CONV2D_BF16) return zero_rows(rows, cols, static_cast<__nv_bfloat16*>(out), ld, late, st);
  return zero_rows(rows, cols, static_cast<__half*>(out), ld, late, st);
}

}  // namespace c2d

// ------------------------------------------------------------------ C entry points
using namespace c2d;

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool is_float(int type) { return type == CONV2D_FP32 || type == CONV2D_BF16 || type == CONV2D_FP16; }

// A matrix argument: data present and aligned, ld at least cols, E4M3 with a known group and scales.
int check_mat(const conv2d_mat* m, int cols) {
  if (!m || !m->data || !aligned16(m->data)) return CONV2D_ERR_INVALID_ARG;
  if (m->ld != 0 && m->ld < cols) return CONV2D_ERR_INVALID_ARG;
  if (m->type == CONV2D_E4M3) {
    if (!m->scale || (m->group != 0 && m->group != kQ8Group)) return CONV2D_ERR_INVALID_ARG;
  } else if (!is_float(m->type)) {
    return CONV2D_ERR_INVALID_ARG;
  }
  return CONV2D_OK;
}
long ld_of(const conv2d_mat* m, int cols) { return m->ld ? m->ld : cols; }

// rows x cols within what the kernels index: 2^31 - 1 rows (one block each), byte offsets in 62 bits.
int check_rows(int64_t rows, int32_t cols) {
  if (rows < 0 || cols < 1) return CONV2D_ERR_INVALID_ARG;
  if (rows > kMaxGridX || cols > (1 << 28)) return CONV2D_ERR_UNSUPPORTED;
  return CONV2D_OK;
}

template <bool NORM>
bool rows_fwd_ok(const NormArgs& a, int es, int V) {
  return a.cols % V == 0 && vec_ok(a.x, a.ldx, es, V) && (!a.r || (vec_ok(a.r, a.ldr, es, V) && vec_ok(a.h, a.ldh, es, V))) &&
         (!a.y || vec_ok(a.y, a.ldy, es, V)) && (!a.q || vec_ok(a.q, a.ldq, 1, V));
}
template <typename T, bool NORM>
cudaError_t rows_fwd_vec(const NormArgs& a, cudaStream_t st) {
  constexpr int es = sizeof(T);
  // at 16 vectors of 32 bytes and fewer half of the lanes would idle (200704 x 256 to 8 bits too: 93 us, now 88)
  if (a.cols > 16 * 32 / es && rows_fwd_ok<NORM>(a, es, 32 / es)) return rows_fwd<T, 32 / es, NORM>(a, st);
  if (rows_fwd_ok<NORM>(a, es, 16 / es)) return rows_fwd<T, 16 / es, NORM>(a, st);
  return rows_fwd<T, 1, NORM>(a, st);
}
template <bool NORM>
cudaError_t rows_fwd_any(const NormArgs& a, int type, cudaStream_t st) {
  if (type == CONV2D_BF16) return rows_fwd_vec<__nv_bfloat16, NORM>(a, st);
  if (type == CONV2D_FP16) return rows_fwd_vec<__half, NORM>(a, st);
  return rows_fwd_vec<float, NORM>(a, st);
}

template <typename T>
cudaError_t norm_bwd_vec(const NormBwdArgs& a, int sms, int* grid, cudaStream_t st) {
  constexpr int es = sizeof(T);
  auto ok = [&](int V) {
    return a.cols % V == 0 && vec_ok(a.h, a.ldh, es, V) && vec_ok(a.dy, a.lddy, es, V) &&
           (!a.dx || vec_ok(a.dx, a.lddx, es, V)) && (!a.dh || vec_ok(a.dh, a.lddh, es, V));
  };
  if constexpr (es == 2)  // fp32 rows of 32-byte vectors take more registers than they win
    if (a.cols > 16 * 32 / es && ok(32 / es)) return norm_bwd<T, 32 / es>(a, sms, grid, st);
  if (ok(16 / es)) return norm_bwd<T, 16 / es>(a, sms, grid, st);
  return norm_bwd<T, 1>(a, sms, grid, st);
}

}  // namespace

extern "C" {

int conv2d_q8_encode(int64_t rows, int32_t cols, const conv2d_mat* x, const conv2d_mat* q8, void* stream) {
  int rc = check_rows(rows, cols);
  if (rc) return rc;
  if (rows == 0) return CONV2D_OK;
  if ((rc = check_mat(x, cols)) || (rc = check_mat(q8, cols))) return rc;
  if (!is_float(x->type) || q8->type != CONV2D_E4M3) return CONV2D_ERR_INVALID_ARG;
  DevInfo* dev = nullptr;
  if ((rc = device_info(&dev))) return rc;
  NormArgs a = {};
  a.x = x->data;
  a.ldx = ld_of(x, cols);
  a.q = static_cast<uint8_t*>(q8->data);
  a.qs = q8->scale;
  a.ldq = ld_of(q8, cols);
  a.rows = rows;
  a.cols = cols;
  a.group = q8->group;
  a.ng = q8->group ? (cols + kQ8Group - 1) / kQ8Group : 1;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  auto run = [&]() -> cudaError_t {
    cudaError_t e = cudaSuccess;
    if (x->type == CONV2D_BF16 && q8_flat<__nv_bfloat16, true>(a.x, a.ldx, a.q, a.ldq, a.qs, a.group, rows, cols, 0, st, &e))
      return e;
    if (x->type == CONV2D_FP16 && q8_flat<__half, true>(a.x, a.ldx, a.q, a.ldq, a.qs, a.group, rows, cols, 0, st, &e))
      return e;
    return rows_fwd_any<false>(a, x->type, st);
  };
  LAUNCH("q8_encode", st, run());
  return CONV2D_OK;
}

int conv2d_q8_decode(int64_t rows, int32_t cols, const conv2d_mat* q8, const conv2d_mat* x, void* stream) {
  int rc = check_rows(rows, cols);
  if (rc) return rc;
  if (rows == 0) return CONV2D_OK;
  if ((rc = check_mat(x, cols)) || (rc = check_mat(q8, cols))) return rc;
  if (!is_float(x->type) || q8->type != CONV2D_E4M3) return CONV2D_ERR_INVALID_ARG;
  DevInfo* dev = nullptr;
  if ((rc = device_info(&dev))) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  LAUNCH("q8_decode", st, launch_to_rows(*q8, rows, cols, x->type, x->data, x->ld, 0, st));
  return CONV2D_OK;
}

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
  if (q8 && (check_mat(q8, cols) || q8->type != CONV2D_E4M3)) return CONV2D_ERR_INVALID_ARG;
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
  if (q8) {
    a.q = static_cast<uint8_t*>(q8->data);
    a.qs = q8->scale;
    a.ldq = ld_of(q8, cols);
    a.group = q8->group;
    a.ng = q8->group ? (cols + kQ8Group - 1) / kQ8Group : 1;
  }
  a.inv = inv_rms;
  a.rows = rows;
  a.cols = cols;
  a.eps = eps;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  LAUNCH("rms_norm_fwd", st, rows_fwd_any<true>(a, x->type, st));
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
    if (h->type == CONV2D_BF16) return norm_bwd_vec<__nv_bfloat16>(a, dev->sms, &grid, st);
    if (h->type == CONV2D_FP16) return norm_bwd_vec<__half>(a, dev->sms, &grid, st);
    return norm_bwd_vec<float>(a, dev->sms, &grid, st);
  };
  LAUNCH("rms_norm_bwd", st, run());
  if (dgamma) LAUNCH("column_sum", st, launch_column_sum(a.part, grid, cols, dgamma, accumulate, 0, st));
  return CONV2D_OK;
}

}  // extern "C"
