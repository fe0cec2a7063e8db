// rows_norm.cuh - the kernels that hold rows of features in registers (norms
// and the 8-bit encoder, forward and backward), the choice of their shapes, and
// the checks of the entry points that launch them.
#pragma once
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "conv2d.h"
#include "host.h"
#include "kernels.h"
#include "q8.cuh"

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
// Two sums at once; red: two words per warp.
template <int TPR>
__device__ __forceinline__ float2 row_sum2(float2 v, float* red) {
  v.x = warp_sum(v.x);
  v.y = warp_sum(v.y);
  if constexpr (TPR > 32) {
    const int warp = threadIdx.x >> 5;
    __syncthreads();
    if ((threadIdx.x & 31) == 0) {
      red[2 * warp] = v.x;
      red[2 * warp + 1] = v.y;
    }
    __syncthreads();
    v = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < TPR / 32; ++i) {
      v.x += red[2 * i];
      v.y += red[2 * i + 1];
    }
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

// Largest magnitude's bits; fmaxf passes NaN over, and infinities are looked for only where one shows.
constexpr uint32_t kInf = 0x7f800000u;
template <int V>
__device__ __forceinline__ uint32_t absmax(const float (&o)[V]) {
  float m = 0.f;
#pragma unroll
  for (int k = 0; k < V; ++k) m = fmaxf(m, fabsf(o[k]));
  return __float_as_uint(m);
}
template <int V>
__device__ __forceinline__ uint32_t absmax_finite(const float (&o)[V]) {
  uint32_t m = 0u;
#pragma unroll
  for (int k = 0; k < V; ++k) m = max(m, finite_bits(o[k]));
  return m;
}
// Largest finite magnitude's bits over the warp's threads that share a group of 32 or 128 columns (V = 1: of 32);
// finite: no infinity among the warp's values. Warp-collective.
template <int V>
__device__ __forceinline__ uint32_t q8_group_max(int group, const float (&o)[V], bool& finite) {
  auto join = [&](uint32_t m) {
    if constexpr (V == 1) {  // the group is the warp
      return __reduce_max_sync(0xffffffffu, m);
    } else {
#pragma unroll
      for (int s = 1; s < kQ8Group / V; s <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, s));
      if (group == kQ8Wide) {
#pragma unroll
        for (int s = kQ8Group / V; s < kQ8Wide / V; s <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, s));
      }
      return m;
    }
  };
  uint32_t m = join(absmax(o));
  finite = true;
  if (__any_sync(0xffffffffu, m == kInf)) {
    finite = false;
    m = join(absmax_finite(o));
  }
  return m;
}

struct NormArgs {
  const void *x, *r;
  const float *gamma, *beta;  // beta: layer norm, may be null
  void *h, *y;
  uint8_t *q, *qs;
  float *inv, *mean;
  long ldx, ldr, ldh, ldy, ldq;
  long rows;
  int cols, ng;  // ng: scale bytes a row
  int group;     // 32, 128 or 0 (whole row)
  int wide;      // gamma and beta start on 32-byte boundaries
  float eps;
};
enum : int { kEncode = 0, kRms = 1, kLayer = 2 };  // what rows_fwd_kernel computes

// f over the pairs of U vectors, folded into one number: from zero, even and odd elements apart, then the two.
template <int U, int V, typename F>
__device__ __forceinline__ float row_fold(const float (&v)[U][V], F&& f) {
  float2 s = make_float2(0.f, 0.f);
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if constexpr (V == 1) {
      s = f(s, make_float2(v[u][0], 0.f));
    } else {
#pragma unroll
      for (int k = 0; k < V; k += 2) s = f(s, make_float2(v[u][k], v[u][k + 1]));
    }
  }
  return V == 1 ? s.x : s.x + s.y;
}

// RMS norm or layer norm forward, or 8-bit encode (KIND): TPR threads a row, a block of them or (TPR = 32) eight warps. Rows are
// held in registers between their sum of squares and their output, U vectors a thread, so memory is passed once;
// U = 0 is the form for rows longer than that, which reads the row again for each phase (from L2, mostly). NR
// rows are in flight at once where a row is a vector or two a thread (one row of 512 bytes a warp left a
// 200704 x 256 encode at 41 us). Threads hold neighbouring vectors, so a group of 32 columns lies in 32 / V
// neighbouring lanes and its maximum is found by shuffles. Bound by memory: 8192 x 4096 bf16 with the residual, y
// and its 8-bit form moves 303 MB in 47 us, 0.95 of the measured copy rate.
template <typename T, int V, int TPR, int U, int NR, int KIND>
__global__ void __launch_bounds__(TPR == 32 ? 256 : TPR) rows_fwd_kernel(const NormArgs a) {
  pdl_entry();
  constexpr int RPB = TPR == 32 ? 8 : 1;  // groups of NR rows per block
  static_assert(U > 0 || NR == 1, "one row at a time where it is read again");
  constexpr int UC = U > 0 ? U : 1;
  __shared__ float red[32];
  [[maybe_unused]] __shared__ uint32_t wide[2][32];
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
  [[maybe_unused]] float mean[NR];
  auto reload = [&](int u) {  // U = 0: this thread's own h (or x) again; layer norm: its distance from the mean
    const int c = u * TPR + t;
    if (c < nv) {
      T e[V];
      ld_vec<T, V>((a.r ? static_cast<const T*>(hb) : xb) + static_cast<long>(c) * V, e);
      widen(e, v[0][0]);
      if constexpr (KIND == kLayer) {
#pragma unroll
        for (int k = 0; k < V; ++k) v[0][0][k] -= mean[0];
      }
    } else {
#pragma unroll
      for (int k = 0; k < V; ++k) v[0][0][k] = 0.f;
    }
  };

  float inv[NR];
#pragma unroll
  for (int i = 0; i < NR; ++i) inv[i] = 1.f;
  if constexpr (U > 0) load_all(0, UC);
  if constexpr (KIND == kLayer && U > 0) {
    // Each warp takes the mean of its values and the squares of their distances from it, and the row's are joined from
    // those: sum of squares = sum over warps of (theirs + count (their mean - the row's mean)^2). So nothing is lost where
    // the mean is large against the deviation, and the block meets once.
    const int warp = TPR > 32 ? t >> 5 : 0;
    int count = 0;  // of this warp's values
#pragma unroll
    for (int u = 0; u < UC; ++u) count += V * min(max(nv - u * TPR - warp * 32, 0), 32);
    const float n = static_cast<float>(count), over = count > 0 ? 1.f / n : 0.f;
    float ss[NR];
    [[maybe_unused]] __shared__ float4 part[NR][TPR / 32];
#pragma unroll
    for (int i = 0; i < NR; ++i) {
      float sum = row_fold<UC, V>(v[i], [](float2 s, float2 e) { return __fadd2_rn(s, e); });
      sum = warp_sum(sum);
      mean[i] = TPR > 32 ? sum * over : sum / n;
      const float2 shift = make_float2(-mean[i], -mean[i]);
      ss[i] = 0.f;
#pragma unroll
      for (int u = 0; u < UC; ++u)
        if (u * TPR + t < nv)  // zeros past the end count in neither
          ss[i] += row_fold<1, V>(reinterpret_cast<float(&)[1][V]>(v[i][u]), [&](float2 s, float2 e) {
            const float2 d = __fadd2_rn(e, shift);
            return __ffma2_rn(d, d, s);
          });
      ss[i] = warp_sum(ss[i]);
      if (TPR > 32 && (t & 31) == 0) part[i][warp] = make_float4(sum, ss[i], mean[i], n);
    }
    if constexpr (TPR > 32) {
      __syncthreads();
#pragma unroll
      for (int i = 0; i < NR; ++i) {
        float sum = 0.f;
        ss[i] = 0.f;
#pragma unroll
        for (int w = 0; w < TPR / 32; ++w) sum += part[i][w].x;
        mean[i] = sum / static_cast<float>(a.cols);
#pragma unroll
        for (int w = 0; w < TPR / 32; ++w) {
          const float4 p = part[i][w];
          const float d = p.z - mean[i];
          ss[i] += fmaf(p.w * d, d, p.y);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < NR; ++i) {
      inv[i] = 1.f / sqrtf(ss[i] / static_cast<float>(a.cols) + a.eps);
      if (t == 0 && i < nr) {
        if (a.mean) a.mean[row0 + i] = mean[i];
        if (a.inv) a.inv[row0 + i] = inv[i];
      }
    }
  } else if constexpr (KIND == kLayer) {  // long rows, read again: the mean, then the squares of the distances from it
    float sum = 0.f, ss = 0.f;
    for (int u = 0; u < nu; ++u) {
      load_all(u, 1);
#pragma unroll
      for (int k = 0; k < V; ++k) sum += v[0][0][k];
    }
    mean[0] = row_sum<TPR>(sum, red) / static_cast<float>(a.cols);
    for (int u = 0; u < nu; ++u) {
      reload(u);
#pragma unroll
      for (int k = 0; k < V; ++k) ss = fmaf(v[0][0][k], v[0][0][k], ss);
    }
    inv[0] = 1.f / sqrtf(row_sum<TPR>(ss, red) / static_cast<float>(a.cols) + a.eps);
    if (t == 0) {
      if (a.mean) a.mean[row0] = mean[0];
      if (a.inv) a.inv[row0] = inv[0];
    }
  } else if constexpr (KIND == kRms) {
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
  // y = gamma h s (layer norm: gamma (h - mean) s + beta) of vector u, in place, for all NR rows (U = 0: of the one
  // vector at hand)
  auto scale = [&](int u, int slot) {
    const int c = u * TPR + t;
    if (KIND == kEncode || c >= nv) return;
    auto feature = [&](const float* p, float (&g)[V]) {
      p += static_cast<long>(c) * V;
      if constexpr (V >= 4) {
#pragma unroll
        for (int k = 0; k < V; k += 4) *reinterpret_cast<float4*>(g + k) = *reinterpret_cast<const float4*>(p + k);
      } else {
        g[0] = p[0];
      }
    };
    float g[V];
    if constexpr (KIND == kRms) {
      feature(a.gamma, g);
#pragma unroll
      for (int i = 0; i < NR; ++i)
#pragma unroll
        for (int k = 0; k < V; ++k) v[i][slot][k] = v[i][slot][k] * inv[i] * g[k];
    } else {
      // in sectors where the vectors start on them: neighbouring threads' 16-byte pieces of 16 features lie 64 bytes
      // apart, so that each such load passes four times the lines
      if (V >= 8 && a.wide) {
#pragma unroll
        for (int k = 0; k < V; k += 8) ld_32b(a.gamma + static_cast<long>(c) * V + k, reinterpret_cast<uint32_t(&)[8]>(g[k]));
      } else {
        feature(a.gamma, g);
      }
      float b[V];
      if (!a.beta) {
#pragma unroll
        for (int k = 0; k < V; ++k) b[k] = 0.f;
      } else if (V >= 8 && a.wide) {
#pragma unroll
        for (int k = 0; k < V; k += 8) ld_32b(a.beta + static_cast<long>(c) * V + k, reinterpret_cast<uint32_t(&)[8]>(b[k]));
      } else {
        feature(a.beta, b);
      }
#pragma unroll
      for (int i = 0; i < NR; ++i) {
        const float m = U > 0 ? mean[i] : 0.f;  // U = 0: taken off where the row is read again
        if constexpr (V == 1) {
          v[i][slot][0] = fmaf((v[i][slot][0] - m) * inv[i], g[0], b[0]);
        } else {
#pragma unroll
          for (int k = 0; k < V; k += 2) {
            float2 e = __fadd2_rn(make_float2(v[i][slot][k], v[i][slot][k + 1]), make_float2(-m, -m));
            e = __fmul2_rn(e, make_float2(inv[i], inv[i]));
            e = __ffma2_rn(e, make_float2(g[k], g[k + 1]), make_float2(b[k], b[k + 1]));
            v[i][slot][k] = e.x;
            v[i][slot][k + 1] = e.y;
          }
        }
      }
    }
  };
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
          uint32_t m;
          if (V == 1 && TPR > 32 && a.group == kQ8Wide) {
            // the group is four warps of the block, all of which are here
            m = __reduce_max_sync(0xffffffffu, absmax_finite(o));
            const int warp = threadIdx.x >> 5;
            if ((threadIdx.x & 31) == 0) wide[u & 1][warp] = m;
            __syncthreads();
#pragma unroll
            for (int w = 0; w < 4; ++w) m = max(m, wide[u & 1][(warp & ~3) + w]);
            finite = false;
          } else {
            m = q8_group_max(a.group, o, finite);
          }
          byte = q8_scale_byte(m);
          const int per = a.group / V;  // threads a group
          if (on && (t & (per - 1)) == 0) a.qs[(row0 + i) * a.ng + c / per] = static_cast<uint8_t>(byte);
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
      reload(u);
      scale(u, 0);
      finish(u, 0);
    }
  }
}

template <typename T, int V, int KIND>
cudaError_t rows_fwd(const NormArgs& a, cudaStream_t st) {
  const int nv = (a.cols + V - 1) / V;
#define ROWS_FWD(TPR, U, NR)                                                                                        \
  do {                                                                                                              \
    constexpr int nt = (TPR) == 32 ? 256 : (TPR), rpb = nt / (TPR) * (NR);                                         \
    return launch_k(rows_fwd_kernel<T, V, TPR, U, NR, KIND>, dim3(static_cast<unsigned>((a.rows + rpb - 1) / rpb)), \
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

// ------------------------------------------------------------------ norms, backward
struct NormBwdArgs {
  const void *h, *dy, *dh;
  void* dx;
  const float *gamma, *inv, *mean;  // mean: layer norm
  float *part, *partb;  // [gridDim.x][cols] of dgamma and (layer norm) dbeta; null: not asked for
  long ldh, lddy, lddh, lddx;
  long rows;
  int cols;
  int* err;  // layer norm: device error word for bounded waits
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
template <typename T, int V, int TPR, int U, bool AHEAD, bool LAYER>
__global__ void __launch_bounds__(TPR == 32 ? 256 : TPR, norm_bwd_resident(TPR)) norm_bwd_kernel(const NormBwdArgs a) {
  pdl_entry();
  constexpr int RPB = TPR == 32 ? 8 : 1;
  constexpr int UC = U > 0 ? U : 1;
  extern __shared__ float sums[];  // RPB > 1 with dgamma: [RPB][cols]
  __shared__ float red[LAYER ? 64 : 32];
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
    [[maybe_unused]] float accb[LAYER ? UC : 1][V];
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
      for (int k = 0; k < V; ++k) {
        acc[u][k] = 0.f;
        if constexpr (LAYER) accb[u][k] = 0.f;
      }
    }
    T h[UC][V], d[UC][V], s[AHEAD ? UC : 1][V];
    float inv = 0.f;
    [[maybe_unused]] float mean = 0.f;
    auto fetch = [&](long row) {
      if (row < a.rows) {
        inv = a.inv[row];
        if constexpr (LAYER) mean = a.mean[row];
      }
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
      [[maybe_unused]] const float mu = mean;
      float dot = 0.f;
      [[maybe_unused]] float sum = 0.f;
#pragma unroll
      for (int u = 0; u < UC; ++u) {
        float gu[V];
        if constexpr (!AHEAD) load_gamma(u, gu);
#pragma unroll
        for (int k = 0; k < V; ++k) {
          // the normalised value; past the row's end dy is zero, so it counts in no sum
          hf[u][k] = (LAYER ? to_f(h[u][k]) - mu : to_f(h[u][k])) * iv;
          df[u][k] = to_f(d[u][k]);
          if constexpr (LAYER) accb[u][k] += df[u][k];
          if constexpr (AHEAD) sk[u][k] = s[u][k];
          acc[u][k] = fmaf(df[u][k], hf[u][k], acc[u][k]);
          df[u][k] *= AHEAD ? g[AHEAD ? u : 0][k] : gu[k];
          dot = fmaf(df[u][k], hf[u][k], dot);
          if constexpr (LAYER) sum += df[u][k];
        }
      }
      if constexpr (AHEAD) fetch(row + step);
      if (xb) {
        if constexpr (LAYER) {
          const float2 both = row_sum2<TPR>(make_float2(dot, sum), red);
          dot = both.x * invD;
          sum = both.y * invD;
        } else {
          dot = row_sum<TPR>(dot, red) * invD;
        }
#pragma unroll
        for (int u = 0; u < UC; ++u) {
          const int i = u * TPR + t;
          if (i < nv) {
            T o[V], sv[V];
            if constexpr (!AHEAD)
              if (sb) ld_vec<T, V>(sb + row * a.lddh + static_cast<long>(i) * V, sv);
#pragma unroll
            for (int k = 0; k < V; ++k) {
              float v = iv * fmaf(-hf[u][k], dot, LAYER ? df[u][k] - sum : df[u][k]);
              if (sb) v += to_f(AHEAD ? sk[AHEAD ? u : 0][k] : sv[k]);
              o[k] = from_f<T>(v);
            }
            st_vec<T, V>(xb + row * a.lddx + static_cast<long>(i) * V, o);
          }
        }
      }
    }
    pdl_release();
    // this block's row of the partial sums
    auto partials = [&](float* base, const float (&v)[UC][V]) {
      if (!base) return;
      float* part = base + static_cast<long>(blockIdx.x) * a.cols;
      if constexpr (RPB > 1) {
        __syncthreads();  // the last use of sums is over
#pragma unroll
        for (int u = 0; u < UC; ++u)
#pragma unroll
          for (int k = 0; k < V; ++k) {
            const int c = (u * TPR + t) * V + k;
            if (c < a.cols) sums[wr * a.cols + c] = v[u][k];
          }
        __syncthreads();
        for (int c = threadIdx.x; c < a.cols; c += 256) {
          float s = 0.f;
#pragma unroll
          for (int w = 0; w < RPB; ++w) s += sums[w * a.cols + c];
          part[c] = s;
        }
      } else {
#pragma unroll
        for (int u = 0; u < UC; ++u)
#pragma unroll
          for (int k = 0; k < V; ++k) {
            const int c = (u * TPR + t) * V + k;
            if (c < a.cols) part[c] = v[u][k];
          }
      }
    };
    partials(a.part, acc);
    if constexpr (LAYER) partials(a.partb, accb);
  } else {
    float* part = a.part ? a.part + static_cast<long>(blockIdx.x) * a.cols : nullptr;
    [[maybe_unused]] float* partb = LAYER && a.partb ? a.partb + static_cast<long>(blockIdx.x) * a.cols : nullptr;
    for (int i = t; i < nv; i += TPR)
      for (int k = 0; k < V; ++k) {
        if (part) part[static_cast<long>(i) * V + k] = 0.f;
        if (LAYER && partb) partb[static_cast<long>(i) * V + k] = 0.f;
      }
    for (long row = row0; row < a.rows; row += step) {
      const float iv = a.inv[row], mu = LAYER ? a.mean[row] : 0.f;
      float dot = 0.f;
      [[maybe_unused]] float sum = 0.f;
      for (int i = t; i < nv; i += TPR) {
        T h[V], d[V];
        ld_vec<T, V>(hb + row * a.ldh + static_cast<long>(i) * V, h);
        ld_vec<T, V>(db + row * a.lddy + static_cast<long>(i) * V, d);
#pragma unroll
        for (int k = 0; k < V; ++k) {
          const long c = static_cast<long>(i) * V + k;
          const float hn = (LAYER ? to_f(h[k]) - mu : to_f(h[k])) * iv, dv = to_f(d[k]);
          if (part) part[c] = fmaf(dv, hn, part[c]);
          dot = fmaf(dv * a.gamma[c], hn, dot);
          if constexpr (LAYER) {
            if (partb) partb[c] += dv;
            sum = fmaf(dv, a.gamma[c], sum);
          }
        }
      }
      if (!xb) continue;
      if constexpr (LAYER) {
        const float2 both = row_sum2<TPR>(make_float2(dot, sum), red);
        dot = both.x * invD;
        sum = both.y * invD;
      } else {
        dot = row_sum<TPR>(dot, red) * invD;
      }
      for (int i = t; i < nv; i += TPR) {
        T h[V], d[V], s[V], o[V];
        ld_vec<T, V>(hb + row * a.ldh + static_cast<long>(i) * V, h);
        ld_vec<T, V>(db + row * a.lddy + static_cast<long>(i) * V, d);
        if (sb) ld_vec<T, V>(sb + row * a.lddh + static_cast<long>(i) * V, s);
#pragma unroll
        for (int k = 0; k < V; ++k) {
          const long c = static_cast<long>(i) * V + k;
          float v = LAYER ? iv * fmaf((mu - to_f(h[k])) * iv, dot, fmaf(to_f(d[k]), a.gamma[c], -sum))
                          : iv * fmaf(-to_f(h[k]) * iv, dot, to_f(d[k]) * a.gamma[c]);
          if (sb) v += to_f(s[k]);
          o[k] = from_f<T>(v);
        }
        st_vec<T, V>(xb + row * a.lddx + static_cast<long>(i) * V, o);
      }
    }
  }
}

// The most blocks that the backward of rows of this length is launched with (norm_bwd's choices below).
inline long norm_bwd_blocks(int64_t rows, int cols, int sms) {
  return std::min<long>(rows, static_cast<long>(sms) * (cols <= 64 * 16 ? 8 : cols <= 128 * 16 ? 4 : cols <= 192 * 16 ? 3 : 2));
}

// grid: blocks launched, one row of partial sums each.
template <typename T, int V, bool LAYER>
cudaError_t norm_bwd(const NormBwdArgs& a, int sms, int* grid, cudaStream_t st) {
  const int nv = (a.cols + V - 1) / V;
#define NORM_BWD(TPR, U, AHEAD)                                                                   \
  do {                                                                                            \
    constexpr int nt = (TPR) == 32 ? 256 : (TPR);                                                 \
    const size_t smem = nt > (TPR) && (a.part || a.partb) ? static_cast<size_t>(nt / (TPR)) * a.cols * 4 : 0;  \
    *grid = static_cast<int>(std::min<long>(a.rows, static_cast<long>(sms) * norm_bwd_resident(TPR))); \
    return launch_k(norm_bwd_kernel<T, V, TPR, U, AHEAD, LAYER>, dim3(*grid), dim3(nt), smem, st, 1, a); \
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
// Rows that start on boundaries of a vector of V elements of es bytes (the base at least on 16 bytes by contract).
inline bool vec_ok(const void* p, long ld, int es, int V) {
  return reinterpret_cast<uintptr_t>(p) % (V * es > 16 ? 32 : 16) == 0 && ld % V == 0;
}

// ------------------------------------------------------------------ arguments of the entry points
inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool is_float(int type) { return type == CONV2D_FP32 || type == CONV2D_BF16 || type == CONV2D_FP16; }

// A matrix argument: data present and aligned, ld at least cols, E4M3 with a known group and scales.
inline int check_mat(const conv2d_mat* m, int cols) {
  if (!m || !m->data || !aligned16(m->data)) return CONV2D_ERR_INVALID_ARG;
  if (m->ld != 0 && m->ld < cols) return CONV2D_ERR_INVALID_ARG;
  if (m->type == CONV2D_E4M3) {
    if (!m->scale || !q8_known(m->group)) return CONV2D_ERR_INVALID_ARG;
  } else if (!is_float(m->type)) {
    return CONV2D_ERR_INVALID_ARG;
  }
  return CONV2D_OK;
}
inline long ld_of(const conv2d_mat* m, int cols) { return m->ld ? m->ld : cols; }

// rows x cols within what the kernels index: 2^31 - 1 rows (one block each), byte offsets in 62 bits.
inline int check_rows(int64_t rows, int32_t cols) {
  if (rows < 0 || cols < 1) return CONV2D_ERR_INVALID_ARG;
  if (rows > kMaxGridX || cols > (1 << 28)) return CONV2D_ERR_UNSUPPORTED;
  return CONV2D_OK;
}

// The 8-bit output. A group of 128 in rows no longer than that is the row.
inline void set_q8(NormArgs& a, const conv2d_mat* q8, int cols) {
  a.q = static_cast<uint8_t*>(q8->data);
  a.qs = q8->scale;
  a.ldq = ld_of(q8, cols);
  a.group = q8->group == kQ8Wide && cols <= kQ8Wide ? 0 : q8->group;
  a.ng = q8_layout(a.group, cols).ng;
}

inline bool rows_fwd_ok(const NormArgs& a, int es, int V) {
  return a.cols % V == 0 && vec_ok(a.x, a.ldx, es, V) && (!a.r || (vec_ok(a.r, a.ldr, es, V) && vec_ok(a.h, a.ldh, es, V))) &&
         (!a.y || vec_ok(a.y, a.ldy, es, V)) && (!a.q || vec_ok(a.q, a.ldq, 1, V));
}
template <typename T, int KIND>
cudaError_t rows_fwd_vec(const NormArgs& a, cudaStream_t st) {
  constexpr int es = sizeof(T);
  // at 16 vectors of 32 bytes and fewer half of the lanes would idle (200704 x 256 to 8 bits too: 93 us, now 88)
  if (a.cols > 16 * 32 / es && rows_fwd_ok(a, es, 32 / es)) return rows_fwd<T, 32 / es, KIND>(a, st);
  if (rows_fwd_ok(a, es, 16 / es)) return rows_fwd<T, 16 / es, KIND>(a, st);
  return rows_fwd<T, 1, KIND>(a, st);
}
template <int KIND>
cudaError_t rows_fwd_any(const NormArgs& a, int type, cudaStream_t st) {
  if (type == CONV2D_BF16) return rows_fwd_vec<__nv_bfloat16, KIND>(a, st);
  if (type == CONV2D_FP16) return rows_fwd_vec<__half, KIND>(a, st);
  return rows_fwd_vec<float, KIND>(a, st);
}

template <typename T, bool LAYER>
cudaError_t norm_bwd_vec(const NormBwdArgs& a, int sms, int* grid, cudaStream_t st) {
  constexpr int es = sizeof(T);
  auto ok = [&](int V) {
    return a.cols % V == 0 && vec_ok(a.h, a.ldh, es, V) && vec_ok(a.dy, a.lddy, es, V) &&
           (!a.dx || vec_ok(a.dx, a.lddx, es, V)) && (!a.dh || vec_ok(a.dh, a.lddh, es, V));
  };
  if constexpr (es == 2)  // fp32 rows of 32-byte vectors take more registers than they win
    if (a.cols > 16 * 32 / es && ok(32 / es)) return norm_bwd<T, 32 / es, LAYER>(a, sms, grid, st);
  if (ok(16 / es)) return norm_bwd<T, 16 / es, LAYER>(a, sms, grid, st);
  return norm_bwd<T, 1, LAYER>(a, sms, grid, st);
}

}  // namespace
}  // namespace c2d
