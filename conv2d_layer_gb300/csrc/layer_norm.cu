// layer_norm.cu - layer norm's C entry points (kernels in rows_norm.cuh).
#include <atomic>

#include "rows.h"
#include "rows_norm.cuh"
#include "schedule.h"

namespace c2d {
namespace {

// Layer norm forward in one stream of rows: a block (WARP: a warp) walks the rows, NR at a time, with gamma and beta in
// its registers (KEEP) and the next rows' vectors in flight while these are reduced and written; U vectors of V elements a
// thread, as many threads as the row has vectors. The statistics are joined as in rows_fwd_kernel. Bound by memory: 8192 x
// 4096 bf16 with the residual moves 268 MB in 45 us, 0.88 of the copy rate (in rows_fwd_kernel, a row a block with gamma
// and beta read for each, 49).
template <typename T, int V, int U, int NR, bool WARP, bool KEEP, int MT, int MB>
__global__ void __launch_bounds__(MT, MB) layer_stream_kernel(const NormArgs a) {
  pdl_entry();
  __shared__ float4 part[2][NR][32];
  __shared__ uint32_t red[32];
  const int tpr = WARP ? 32 : static_cast<int>(blockDim.x), nw = tpr / 32;
  const int t = WARP ? static_cast<int>(threadIdx.x) & 31 : static_cast<int>(threadIdx.x);
  const int warp = WARP ? 0 : t >> 5, lane = t & 31;
  const int nv = a.cols / V;
  const long per = (WARP ? blockDim.x / 32 : 1) * NR;  // rows a block takes at a time
  const long row0 = blockIdx.x * per + (WARP ? (threadIdx.x >> 5) * NR : 0);
  const long step = gridDim.x * per;
  const float cols = static_cast<float>(a.cols);

  auto feature = [&](const float* p, int u, float (&g)[V]) {
    const int c = u * tpr + t;
#pragma unroll
    for (int k = 0; k < V; ++k) g[k] = 0.f;
    if (!p || c >= nv) return;
    p += static_cast<long>(c) * V;
    if (V >= 8 && a.wide) {
#pragma unroll
      for (int k = 0; k < V; k += 8) ld_32b(p + k, reinterpret_cast<uint32_t(&)[8]>(g[k]));
    } else {
#pragma unroll
      for (int k = 0; k < V; k += 4) *reinterpret_cast<float4*>(g + k) = *reinterpret_cast<const float4*>(p + k);
    }
  };
  float g[KEEP ? U : 1][V], b[KEEP ? U : 1][V];
  if constexpr (KEEP) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      feature(a.gamma, u, g[u]);
      feature(a.beta, u, b[u]);
    }
  }
  int count = 0;  // of this warp's values
#pragma unroll
  for (int u = 0; u < U; ++u) count += V * min(max(nv - u * tpr - warp * 32, 0), 32);
  const float n = static_cast<float>(count), over = count > 0 ? 1.f / n : 0.f;

  T e[NR][U][V], f[NR][U][V];
  auto fetch = [&](long row) {
#pragma unroll
    for (int i = 0; i < NR; ++i)
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int c = u * tpr + t;
        if (row + i < a.rows && c < nv) {
          ld_vec<T, V>(static_cast<const T*>(a.x) + (row + i) * a.ldx + static_cast<long>(c) * V, e[i][u]);
          if (a.r) ld_vec<T, V>(static_cast<const T*>(a.r) + (row + i) * a.ldr + static_cast<long>(c) * V, f[i][u]);
        } else {
#pragma unroll
          for (int k = 0; k < V; ++k) e[i][u][k] = f[i][u][k] = from_f<T>(0.f);
        }
      }
  };
  fetch(row0);
  int par = 0;
  for (long row = row0; row < a.rows; row += step, par ^= 1) {
    float v[NR][U][V];
#pragma unroll
    for (int i = 0; i < NR; ++i)
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int c = u * tpr + t;
        if (a.r) {
#pragma unroll
          for (int k = 0; k < V; ++k) e[i][u][k] = from_f<T>(to_f(e[i][u][k]) + to_f(f[i][u][k]));
          if (row + i < a.rows && c < nv)
            st_vec<T, V>(static_cast<T*>(a.h) + (row + i) * a.ldh + static_cast<long>(c) * V, e[i][u]);
        }
#pragma unroll
        for (int k = 0; k < V; ++k) v[i][u][k] = to_f(e[i][u][k]);
      }
    if (row + step < a.rows) fetch(row + step);
    else pdl_release();
    float mean[NR], ss[NR];
#pragma unroll
    for (int i = 0; i < NR; ++i) {
      const float sum = warp_sum(row_fold<U, V>(v[i], [](float2 s, float2 x) { return __fadd2_rn(s, x); }));
      mean[i] = WARP ? sum / n : sum * over;
      const float2 shift = make_float2(-mean[i], -mean[i]);
      ss[i] = 0.f;
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (u * tpr + t < nv)  // zeros past the end count in neither
          ss[i] += row_fold<1, V>(reinterpret_cast<float(&)[1][V]>(v[i][u]), [&](float2 s, float2 x) {
            const float2 d = __fadd2_rn(x, shift);
            return __ffma2_rn(d, d, s);
          });
      ss[i] = warp_sum(ss[i]);
      if (!WARP && lane == 0) part[par][i][warp] = make_float4(sum, ss[i], mean[i], n);
    }
    if constexpr (!WARP) {
      __syncthreads();  // once a row: the next one writes the other half of part
#pragma unroll
      for (int i = 0; i < NR; ++i) {
        float sum = 0.f;
        ss[i] = 0.f;
#pragma unroll 8
        for (int w = 0; w < nw; ++w) sum += part[par][i][w].x;
        mean[i] = sum / cols;
#pragma unroll 8
        for (int w = 0; w < nw; ++w) {
          const float4 p = part[par][i][w];
          const float d = p.z - mean[i];
          ss[i] += fmaf(p.w * d, d, p.y);
        }
      }
    }
    float inv[NR];
#pragma unroll
    for (int i = 0; i < NR; ++i) {
      inv[i] = 1.f / sqrtf(ss[i] / cols + a.eps);
      if (t == 0 && row + i < a.rows) {
        if (a.mean) a.mean[row + i] = mean[i];
        if (a.inv) a.inv[row + i] = inv[i];
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if constexpr (!KEEP) {
        feature(a.gamma, u, g[0]);
        feature(a.beta, u, b[0]);
      }
      const int c = u * tpr + t;
      if (c >= nv) continue;
#pragma unroll
      for (int i = 0; i < NR; ++i)
#pragma unroll
        for (int k = 0; k < V; k += 2) {
          float2 x = __fadd2_rn(make_float2(v[i][u][k], v[i][u][k + 1]), make_float2(-mean[i], -mean[i]));
          x = __fmul2_rn(x, make_float2(inv[i], inv[i]));
          x = __ffma2_rn(x, make_float2(g[KEEP ? u : 0][k], g[KEEP ? u : 0][k + 1]),
                         make_float2(b[KEEP ? u : 0][k], b[KEEP ? u : 0][k + 1]));
          v[i][u][k] = x.x;
          v[i][u][k + 1] = x.y;
        }
    }
#pragma unroll
    for (int i = 0; i < NR; ++i) {
      uint32_t byte = 0u;
      bool finite = true;
      if (a.q && a.group == 0) {
        auto whole = [&](auto&& top) {
          uint32_t m = 0u;
#pragma unroll
          for (int u = 0; u < U; ++u) m = max(m, top(v[i][u]));
          m = __reduce_max_sync(0xffffffffu, m);
          if constexpr (!WARP) {
            __syncthreads();  // the last use of red is over
            if (lane == 0) red[warp] = m;
            __syncthreads();
            m = 0u;
#pragma unroll 8
            for (int w = 0; w < nw; ++w) m = max(m, red[w]);
          }
          return m;
        };
        uint32_t m = whole([](const float (&o)[V]) { return absmax(o); });
        if (m == kInf) {  // the same for the whole row
          finite = false;
          m = whole([](const float (&o)[V]) { return absmax_finite(o); });
        }
        byte = q8_scale_byte(m);
        if (t == 0 && row + i < a.rows) a.qs[(row + i) * a.ng] = static_cast<uint8_t>(byte);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int c = u * tpr + t;
        const bool on = row + i < a.rows && c < nv;
        float(&o)[V] = v[i][u];
        if (a.y && on) {
          T w[V];
#pragma unroll
          for (int k = 0; k < V; ++k) w[k] = from_f<T>(o[k]);
          st_vec<T, V>(static_cast<T*>(a.y) + (row + i) * a.ldy + static_cast<long>(c) * V, w);
        }
        if (a.q) {
          if (a.group != 0) {
            byte = q8_scale_byte(q8_group_max(a.group, o, finite));
            const int share = a.group / V;  // threads a group
            if (on && (t & (share - 1)) == 0) a.qs[(row + i) * a.ng + c / share] = static_cast<uint8_t>(byte);
          }
          if (on) q8_store<V>(a.q + (row + i) * a.ldq + static_cast<long>(c) * V, o, q8_inv_scale(byte), finite);
        }
      }
    }
  }
}

template <typename T, int V, int U, int NR, bool WARP, bool KEEP, int MT, int MB>
cudaError_t layer_stream(const NormArgs& a, int threads, int sms, cudaStream_t st) {
  const long per = (WARP ? threads / 32 : 1) * NR;
  const long blocks = std::min<long>((a.rows + per - 1) / per, static_cast<long>(sms) * std::max(1, MT * MB / threads));
  return launch_k(layer_stream_kernel<T, V, U, NR, WARP, KEEP, MT, MB>, dim3(static_cast<unsigned>(blocks)), dim3(threads),
                  0, st, 1, a);
}

template <typename T, int V>
cudaError_t layer_vec(const NormArgs& a, int sms, cudaStream_t st) {
  // The stream for 16-bit rows: in 32-byte vectors, or of up to a warp's vectors. Elsewhere a row has too few or too many
  // threads for it (8192 x 1000 bf16 14.7 us, 11.0 in rows_fwd_kernel; fp32 8192 x 4096 92 and 79).
  if constexpr (sizeof(T) == 2) {
    const int nv = a.cols / V, threads = (nv + 31) / 32 * 32;
    if (nv <= 32) return layer_stream<T, V, 1, (V == 16 ? 2 : 4), true, true, 256, 2>(a, 256, sms, st);
    if constexpr (V == 16) {
      if (threads <= 256) return layer_stream<T, V, 1, 1, false, true, 256, 3>(a, threads, sms, st);
      if (threads <= 384) return layer_stream<T, V, 1, 1, false, true, 384, 2>(a, threads, sms, st);
      if (threads <= 512) return layer_stream<T, V, 1, 1, false, true, 512, 1>(a, threads, sms, st);
      if (nv <= 1024) return layer_stream<T, V, 2, 1, false, false, 512, 1>(a, (nv + 63) / 64 * 32, sms, st);
    }
  }
  return rows_fwd<T, V, kLayer>(a, st);
}
// Rows that start off 16-byte boundaries, without an 8-bit output: the stream's rows are a multiple of eight apart, so that all
// of a thread's rows start `m` features behind a boundary and its features stay the same. Vectors of 16 bytes in the middle
// of a row, single features at its ends. With the residual, feature by feature in rows_fwd_kernel and here: bf16 8192 x 1021
// 30 and 24 us, 8192 x 2047 137 and 52, 4096 x 7001 370 and 92 (floors 10, 20, 34), 300 x 4095 8.0 and 6.1; fp32 37312 x 399
// 105 and 51 (35), 100 x 1021 bf16 3.5 and 3.7. Rows of 77, whose warps are half idle, stay there: 31 and 92.
template <typename T, int U, bool WARP, int MT, int MB>
__global__ void __launch_bounds__(MT, MB) layer_shift_kernel(const NormArgs a) {
  constexpr int V = 16 / static_cast<int>(sizeof(T));
  constexpr uint32_t kWhole = (1u << V) - 1u;
  pdl_entry();
  __shared__ float4 part[2][32];
  const int tpr = WARP ? 32 : static_cast<int>(blockDim.x), nw = tpr / 32;
  const int t = WARP ? static_cast<int>(threadIdx.x) & 31 : static_cast<int>(threadIdx.x);
  const int warp = WARP ? 0 : t >> 5, lane = t & 31, per = WARP ? static_cast<int>(blockDim.x) / 32 : 1;
  const long row0 = static_cast<long>(blockIdx.x) * per + (WARP ? threadIdx.x >> 5 : 0);
  const long step = static_cast<long>(gridDim.x) * per;
  const float cols = static_cast<float>(a.cols);
  const int m = static_cast<int>(row0 * a.ldx % V);
  int c[U], count = 0;   // the vectors' first columns; this warp's features
  uint32_t there[U];     // a bit for each feature of a vector that is in the row
  float g[U][V], b[U][V];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    c[u] = (u * tpr + t) * V - m;
    there[u] = 0u;
#pragma unroll
    for (int k = 0; k < V; ++k) {
      const bool on = c[u] + k >= 0 && c[u] + k < a.cols;
      there[u] |= on ? 1u << k : 0u;
      g[u][k] = on ? a.gamma[c[u] + k] : 0.f;
      b[u][k] = on && a.beta ? a.beta[c[u] + k] : 0.f;
    }
    count += __popc(there[u]);
  }
  const float n = static_cast<float>(__reduce_add_sync(0xffffffffu, count)), over = n > 0.f ? 1.f / n : 0.f;
  auto read = [&](const void* from, long ld, long row, T (&e)[U][V]) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const T* x = static_cast<const T*>(from) + row * ld + c[u];
      if (there[u] == kWhole) {
        ld_vec<T, V>(x, e[u]);
      } else {
#pragma unroll
        for (int k = 0; k < V; ++k) e[u][k] = there[u] >> k & 1u ? x[k] : from_f<T>(0.f);
      }
    }
  };
  auto write = [&](void* to, long ld, long row, int u, const T (&e)[V]) {
    T* x = static_cast<T*>(to) + row * ld + c[u];
    if (there[u] == kWhole) {
      st_vec<T, V>(x, e);
    } else {
#pragma unroll
      for (int k = 0; k < V; ++k)
        if (there[u] >> k & 1u) x[k] = e[k];
    }
  };
  T e[U][V], f[U][V];
  auto fetch = [&](long row) {
    read(a.x, a.ldx, row, e);
    if (a.r) read(a.r, a.ldr, row, f);
  };
  if (row0 < a.rows) fetch(row0);
  int par = 0;
  for (long row = row0; row < a.rows; row += step, par ^= 1) {
    float v[U][V];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (a.r) {
#pragma unroll
        for (int k = 0; k < V; ++k) e[u][k] = from_f<T>(to_f(e[u][k]) + to_f(f[u][k]));
        write(a.h, a.ldh, row, u, e[u]);
      }
#pragma unroll
      for (int k = 0; k < V; ++k) v[u][k] = to_f(e[u][k]);
    }
    if (row + step < a.rows) fetch(row + step);
    else pdl_release();
    float sum = warp_sum(row_fold<U, V>(v, [](float2 s, float2 x) { return __fadd2_rn(s, x); }));  // zeros beside the row
    float mean = WARP ? sum / n : sum * over, ss = 0.f;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (there[u] == kWhole) {
        ss += row_fold<1, V>(reinterpret_cast<float(&)[1][V]>(v[u]), [&](float2 s, float2 x) {
          const float2 d = __fadd2_rn(x, make_float2(-mean, -mean));
          return __ffma2_rn(d, d, s);
        });
      } else {
#pragma unroll
        for (int k = 0; k < V; ++k) {
          const float d = there[u] >> k & 1u ? v[u][k] - mean : 0.f;
          ss = fmaf(d, d, ss);
        }
      }
    }
    ss = warp_sum(ss);
    if constexpr (!WARP) {
      if (lane == 0) part[par][warp] = make_float4(sum, ss, mean, n);
      __syncthreads();  // once a row: the next one writes the other half of part
      sum = ss = 0.f;
#pragma unroll 8
      for (int w = 0; w < nw; ++w) sum += part[par][w].x;
      mean = sum / cols;
#pragma unroll 8
      for (int w = 0; w < nw; ++w) {
        const float4 p = part[par][w];
        const float d = p.z - mean;
        ss += fmaf(p.w * d, d, p.y);
      }
    }
    const float inv = 1.f / sqrtf(ss / cols + a.eps);
    if (t == 0) {
      if (a.mean) a.mean[row] = mean;
      if (a.inv) a.inv[row] = inv;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      T w[V];
#pragma unroll
      for (int k = 0; k < V; k += 2) {
        float2 x = __fadd2_rn(make_float2(v[u][k], v[u][k + 1]), make_float2(-mean, -mean));
        x = __fmul2_rn(x, make_float2(inv, inv));
        x = __ffma2_rn(x, make_float2(g[u][k], g[u][k + 1]), make_float2(b[u][k], b[u][k + 1]));
        w[k] = from_f<T>(x.x);
        w[k + 1] = from_f<T>(x.y);
      }
      write(a.y, a.ldy, row, u, w);
    }
  }
}
template <typename T, int U, bool WARP, int MT, int MB>
cudaError_t layer_shift(const NormArgs& a, int threads, int sms, cudaStream_t st) {
  const long per = WARP ? threads / 32 : 1, need = (a.rows + per - 1) / per;
  long blocks = std::min<long>(need, static_cast<long>(sms) * std::max(1, MT * MB / threads));
  if (!WARP && blocks < need) blocks = std::max<long>(8, blocks / 8 * 8);  // a warp's rows are eight apart anyway
  return launch_k(layer_shift_kernel<T, U, WARP, MT, MB>, dim3(static_cast<unsigned>(blocks)), dim3(threads), 0, st, 1, a);
}
template <typename T>
cudaError_t layer_any(const NormArgs& a, int sms, cudaStream_t st) {
  constexpr int es = sizeof(T), V = 16 / es;
  if (a.cols > 16 * 32 / es && rows_fwd_ok(a, es, 32 / es)) return layer_vec<T, 32 / es>(a, sms, st);
  if (rows_fwd_ok(a, es, 16 / es)) return layer_vec<T, 16 / es>(a, sms, st);
  auto alike = [&](const void* p, long ld) { return !p || ld % V == a.ldx % V; };
  if (!a.q && a.cols > 256 && alike(a.r, a.ldr) && alike(a.h, a.ldh) && alike(a.y, a.ldy)) {
    const int nv = (a.cols + 2 * V - 2) / V, threads = (nv + 31) / 32 * 32;
    constexpr int UW = es == 2 ? 2 : 4;
    if (nv <= 32 * UW) return layer_shift<T, UW, true, 256, 2>(a, 256, sms, st);
    if (threads <= 512) return layer_shift<T, 1, false, 512, 2>(a, threads, sms, st);
    if (threads <= 1024) return layer_shift<T, 2, false, 512, 1>(a, threads / 2 + threads / 2 % 32, sms, st);
  }
  return rows_fwd<T, 1, kLayer>(a, st);
}

// Layer norm backward of 16-bit rows: as norm_bwd_kernel, with the arithmetic in packed pairs and one meeting of the block
// a row. A row's h, dy and dh come by bulk copies into one of kRing places in shared memory, four rows ahead (192 KB an SM):
// the sums of dgamma and dbeta leave no registers for that (512 threads an SM of 126 each, with one row ahead in registers:
// 8192 x 4096 bf16 54 us, 48 KB in flight). A thread has eight features in each half of the row, so that its 16-byte
// accesses meet no bank twice. Bound by memory: 8192 x 4096 bf16 with dh moves 268 MB in 44 us, 0.90 of the copy rate, then
// the column sums in 5. Rows of more than 8,192 features are shared by a cluster of two CTAs, or four (up to 32,768): a
// thread has no registers for more than 16 features, and norm_bwd_kernel leaves the row in L2 in between. 2048 x 16384 bf16
// 113 us there, 55 here; 3000 x 10240 129 and 60; 1024 x 32768 560 and 66; 32 x 16384 28 and 10.
constexpr int kRing = 4;
constexpr int kSiteLayerBwd = 20;
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "l"(src),
               "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}
__device__ __forceinline__ void send_pair(uint32_t to, float2 v, uint32_t bar) {  // both in one CTA of the cluster
  asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v2.b32 [%0], {%1, %2}, [%3];" ::"r"(to),
               "r"(__float_as_uint(v.x)), "r"(__float_as_uint(v.y)), "r"(bar)
               : "memory");
}
// CL: CTAs of a cluster, which share a row.
template <typename T, int MT, int MB, int CL>
__global__ void __launch_bounds__(MT, MB) layer_bwd_kernel(const NormBwdArgs a) {
  extern __shared__ uint4 ring[];  // [kRing][h, dy, dh][cols]
  __shared__ uint64_t full[kRing], met[2];
  __shared__ float2 part[2][CL * MT / 32];
  const int t = static_cast<int>(threadIdx.x), nw = static_cast<int>(blockDim.x) >> 5;
  const int rank = CL > 1 ? static_cast<int>(cluster_ctarank()) : 0, cols = a.cols / CL, from_col = rank * cols;
  const int half = cols / 2, c = t * 8;
  const bool on = c < half, skip = a.dh && a.dx;
  const float over = 1.f / static_cast<float>(a.cols);
  const uint32_t bytes = static_cast<uint32_t>(cols) * 2u, place = 3u * bytes, base = smem_u32(ring);
  const uint32_t sent = static_cast<uint32_t>(CL * nw) * 8u;  // bytes of all warps' sums of a row
  if (t == 0) {
    for (int i = 0; i < kRing; ++i) mbar_init(&full[i], 1);
    if (CL > 1)
      for (int i = 0; i < 2; ++i) mbar_init(&met[i], 1 + static_cast<uint32_t>(nw));  // the bytes' count, and this CTA's warps
    fence_mbar_init();
    if (CL > 1)
      for (int i = 0; i < 2; ++i) mbar_arrive_expect_tx(&met[i], sent);
  }
  pdl_entry();
  if (CL > 1)
    cluster_sync();
  else
    __syncthreads();
  const long step = gridDim.x / CL, first = blockIdx.x / CL;
  auto request = [&](long row, int i) {  // one thread
    if (row >= a.rows) return;
    mbar_arrive_expect_tx(&full[i], (skip ? 3u : 2u) * bytes);
    const uint32_t to = base + i * place;
    bulk_load(to, static_cast<const T*>(a.h) + row * a.ldh + from_col, bytes, &full[i]);
    bulk_load(to + bytes, static_cast<const T*>(a.dy) + row * a.lddy + from_col, bytes, &full[i]);
    if (skip) bulk_load(to + 2 * bytes, static_cast<const T*>(a.dh) + row * a.lddh + from_col, bytes, &full[i]);
  };
  long row = first;  // the grid has no more blocks (or clusters) than there are rows
  if (t == 0)
    for (int i = 0; i < kRing; ++i) request(row + i * step, i);

  float2 g[8], acc[8], accb[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    g[k] = on ? *reinterpret_cast<const float2*>(a.gamma + from_col + (k < 4 ? c : half + c - 8) + 2 * k) : splat(0.f);
    acc[k] = accb[k] = splat(0.f);
  }
  auto pair = [](uint32_t w) {
    const T* e = reinterpret_cast<const T*>(&w);
    return make_float2(to_f(e[0]), to_f(e[1]));
  };
  auto take = [&](uint32_t from, uint32_t (&w)[8]) {
    const uint32_t at = from + c * 2;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(at) : "memory");
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7]) : "r"(at + half * 2) : "memory");
  };
  float inv = a.inv[row], mean = a.mean[row];
  int par = 0, slot = 0;
  uint32_t phase = 0, meet = 0;
  bool ok = true;
  for (; row < a.rows; row += step, par ^= 1) {
    const float2 iv = splat(inv), mu = splat(-mean);
    if (row + step < a.rows) {
      inv = a.inv[row + step];
      mean = a.mean[row + step];
    } else {
      pdl_release();
    }
    uint32_t h[8], d[8], s[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) h[k] = d[k] = s[k] = 0u;
    ok = ok && wait(&full[slot], phase, a.err, kSiteLayerBwd);  // (one that ran out leaves garbage and its mark)
    if (on) {
      const uint32_t from = base + slot * place;
      take(from, h);
      take(from + bytes, d);
      if (skip) take(from + 2 * bytes, s);
    }
    float2 dot = splat(0.f), sum = splat(0.f);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float2 n = __fmul2_rn(__fadd2_rn(pair(h[k]), mu), iv), y = pair(d[k]), w = __fmul2_rn(y, g[k]);
      acc[k] = __ffma2_rn(y, n, acc[k]);
      accb[k] = __fadd2_rn(accb[k], y);
      dot = __ffma2_rn(w, n, dot);
      sum = __fadd2_rn(sum, w);
    }
    // past the row's end dy is zero, so it counts in no sum
    float2 both = make_float2(warp_sum(dot.x + dot.y), warp_sum(sum.x + sum.y));
    // Once a row all warps meet: the next row writes the other half of part, this row's place is free. In a cluster each
    // warp sends its sums to every CTA, whose barrier counts the bytes; what is sent orders nothing before it, so the warp
    // arrives there itself too, once it has read the row's place.
    if constexpr (CL > 1) {
      const int lane = t & 31;
      if (lane < CL)
        send_pair(mapa_shared(smem_u32(&part[par][rank * nw + (t >> 5)]), static_cast<uint32_t>(lane)), both,
                  mapa_shared(smem_u32(&met[par]), static_cast<uint32_t>(lane)));
      __syncwarp();
      if (lane == 0) mbar_arrive(&met[par]);
      ok = ok && wait_cluster(&met[par], meet, a.err, kSiteLayerBwd);
      if (t == 0) mbar_arrive_expect_tx(&met[par], sent);  // for the row after next: none sends its sums before this warp
      if (par) meet ^= 1;
    } else {
      if ((t & 31) == 0) part[par][t >> 5] = both;
      __syncthreads();
    }
    if (t == 0) request(row + kRing * step, slot);
    if (++slot == kRing) {
      slot = 0;
      phase ^= 1;
    }
    if (!a.dx) continue;
    both = splat(0.f);
#pragma unroll 8
    for (int w = 0; w < CL * nw; ++w) both = __fadd2_rn(both, part[par][w]);
    const float2 md = splat(-both.x * over), ms = splat(-both.y * over);
    if (on) {
      uint32_t o[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float2 n = __fmul2_rn(__fadd2_rn(pair(h[k]), mu), iv);
        float2 v = __ffma2_rn(n, md, __ffma2_rn(pair(d[k]), g[k], ms));
        v = a.dh ? __ffma2_rn(v, iv, pair(s[k])) : __fmul2_rn(v, iv);
        T* e = reinterpret_cast<T*>(&o[k]);
        e[0] = from_f<T>(v.x);
        e[1] = from_f<T>(v.y);
      }
      T* x = static_cast<T*>(a.dx) + row * a.lddx + from_col + c;
      *reinterpret_cast<uint4*>(x) = make_uint4(o[0], o[1], o[2], o[3]);
      *reinterpret_cast<uint4*>(x + half) = make_uint4(o[4], o[5], o[6], o[7]);
    }
  }
  if (!ok && t == 0) {  // gave up: the copies in flight land before the block goes; row n of this block in place n % kRing
    const long n = (a.rows - first + step - 1) / step;
    for (long i = n > kRing ? n - kRing : 0; i < n; ++i)
      (void)wait(&full[i % kRing], static_cast<uint32_t>(i / kRing) & 1u, a.err, kSiteLayerBwd);
  }
  if (CL > 1) cluster_sync();  // (after a wait that ran out: no CTA goes while another may still send to it)
  if (!on) return;
  auto partials = [&](float* sums, const float2 (&v)[8]) {
    if (!sums) return;
    float* p = sums + first * a.cols + from_col + c;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      float* q = k < 2 ? p + 4 * k : p + half + 4 * (k - 2);
      *reinterpret_cast<float4*>(q) = make_float4(v[2 * k].x, v[2 * k].y, v[2 * k + 1].x, v[2 * k + 1].y);
    }
  };
  partials(a.part, acc);
  partials(a.partb, accb);
}
// The same for rows of any length and type, whose starts may lie anywhere: a block's rows are a multiple of eight apart, so
// that they all start `m` features behind a 16-byte boundary, and a thread has the same features in each. A copy takes whole
// 16 bytes; what is of the rows beside is set to zero where it is taken, and the end of the last row, behind which nothing
// may be read, comes feature by feature, as do the ends of a row of dx go. Those ends hold the whole block up: 8192 x 4088
// bf16, which has none, 63 us, 8192 x 4095 100 (floor 40; 8192 x 4096 in layer_bwd_kernel 49).
template <typename T, int MT, int MB, int CL>
__global__ void __launch_bounds__(MT, MB) layer_bwd_shift_kernel(const NormBwdArgs a) {
  constexpr int V = 16 / static_cast<int>(sizeof(T));  // features of a vector; a thread has two vectors, V pairs
  extern __shared__ uint4 ring[];                      // [kRing][h, dy, dh][n]
  __shared__ uint64_t full[kRing], met[2];
  __shared__ float2 part[2][CL * MT / 32];
  const int t = static_cast<int>(threadIdx.x), nw = static_cast<int>(blockDim.x) >> 5;
  const int rank = CL > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const long step = gridDim.x / CL, first = blockIdx.x / CL;
  const int m = static_cast<int>(first * a.ldh % V);
  const int all = (m + a.cols + V - 1) / V, per = (all + CL - 1) / CL, v0 = rank * per, n = min(per, all - v0);
  const int half = (n + 1) / 2, c0 = (v0 + t) * V - m, c1 = c0 + half * V;  // the first columns of the thread's vectors
  const bool on0 = t < half, on1 = t < n - half, skip = a.dh && a.dx;
  const bool whole0 = c0 >= 0 && c0 + V <= a.cols, whole1 = c1 + V <= a.cols;  // (no second vector is the row's first)
  const bool edge = (on0 && !whole0) || (on1 && !whole1);
  const float over = 1.f / static_cast<float>(a.cols);
  const uint32_t bytes = static_cast<uint32_t>(n) * 16u, place = 3u * bytes, base = smem_u32(ring);
  // of the last row: without the vector that its end cuts
  const uint32_t bytes_end = bytes - (v0 + n == all && (m + a.cols) % V ? 16u : 0u);
  const uint32_t sent = static_cast<uint32_t>(CL * nw) * 8u;
  if (t == 0) {
    for (int i = 0; i < kRing; ++i) mbar_init(&full[i], 1);
    if (CL > 1)
      for (int i = 0; i < 2; ++i) mbar_init(&met[i], 1 + static_cast<uint32_t>(nw));  // the bytes' count, and this CTA's warps
    fence_mbar_init();
    if (CL > 1)
      for (int i = 0; i < 2; ++i) mbar_arrive_expect_tx(&met[i], sent);
  }
  pdl_entry();
  if (CL > 1)
    cluster_sync();
  else
    __syncthreads();
  auto request = [&](long row, int i) {  // one thread
    if (row >= a.rows) return;
    const uint32_t b = row == a.rows - 1 ? bytes_end : bytes;
    mbar_arrive_expect_tx(&full[i], (skip ? 3u : 2u) * b);
    if (b == 0) return;
    const uint32_t to = base + i * place;
    const long at = static_cast<long>(v0) * V - m;
    bulk_load(to, static_cast<const T*>(a.h) + row * a.ldh + at, b, &full[i]);
    bulk_load(to + bytes, static_cast<const T*>(a.dy) + row * a.lddy + at, b, &full[i]);
    if (skip) bulk_load(to + 2 * bytes, static_cast<const T*>(a.dh) + row * a.lddh + at, b, &full[i]);
  };
  long row = first;
  if (t == 0)
    for (int i = 0; i < kRing; ++i) request(row + i * step, i);

  auto column = [&](int e) { return e < V ? c0 + e : c1 + e - V; };  // of the thread's feature e
  auto there = [&](int e) { return (e < V ? on0 : on1) && column(e) >= 0 && column(e) < a.cols; };
  uint32_t valid = 0;  // the thread's features that are there
#pragma unroll
  for (int e = 0; e < 2 * V; ++e) valid |= there(e) ? 1u << e : 0u;
  float2 g[V], acc[V], accb[V];
#pragma unroll
  for (int k = 0; k < V; ++k) {
    g[k] = make_float2(there(2 * k) ? a.gamma[column(2 * k)] : 0.f, there(2 * k + 1) ? a.gamma[column(2 * k + 1)] : 0.f);
    acc[k] = accb[k] = splat(0.f);
  }
  auto pair = [](const uint32_t (&w)[8], int k) {
    if constexpr (sizeof(T) == 2) {
      const T* e = reinterpret_cast<const T*>(&w[k]);
      return make_float2(to_f(e[0]), to_f(e[1]));
    } else {
      return make_float2(__uint_as_float(w[2 * k]), __uint_as_float(w[2 * k + 1]));
    }
  };
  auto take = [&](uint32_t from, uint32_t (&w)[8]) {
    const uint32_t at = from + t * 16;
    if (on0) asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(at) : "memory");
    if (on1) asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7]) : "r"(at + half * 16) : "memory");
  };
  // Of a vector at an end of the row: only the features that are there.
  auto mask = [&](uint32_t* w, uint32_t there) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if constexpr (sizeof(T) == 2)
        w[k] &= (there >> 2 * k & 1u ? 0xffffu : 0u) | (there >> (2 * k + 1) & 1u ? 0xffff0000u : 0u);
      else
        w[k] = there >> k & 1u ? w[k] : 0u;
    }
  };
  // The end of the last row (at), which no copy brought: in place of what was taken.
  auto last = [&](const T* at, uint32_t (&w)[8]) {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      if ((k < 4 ? c0 : c1) + V <= a.cols) continue;
      if constexpr (sizeof(T) == 2) {
        const uint16_t* e = reinterpret_cast<const uint16_t*>(at) + column(2 * k);
        w[k] = (valid >> 2 * k & 1u ? e[0] : 0u) | (valid >> (2 * k + 1) & 1u ? static_cast<uint32_t>(e[1]) << 16 : 0u);
      } else {
        w[k] = valid >> k & 1u ? reinterpret_cast<const uint32_t*>(at)[column(k)] : 0u;
      }
    }
  };
  float inv = a.inv[row], mean = a.mean[row];
  int par = 0, slot = 0;
  uint32_t phase = 0, meet = 0;
  bool ok = true;
  for (; row < a.rows; row += step, par ^= 1) {
    const float2 iv = splat(inv), mu = splat(-mean);
    if (row + step < a.rows) {
      inv = a.inv[row + step];
      mean = a.mean[row + step];
    } else {
      pdl_release();
    }
    uint32_t h[8], d[8], s[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) h[k] = d[k] = s[k] = 0u;
    ok = ok && wait(&full[slot], phase, a.err, kSiteLayerBwd);
    const uint32_t from = base + slot * place;
    take(from, h);
    take(from + bytes, d);
    if (skip) take(from + 2 * bytes, s);
    if (edge) {
      if (row == a.rows - 1) {
        last(static_cast<const T*>(a.h) + row * a.ldh, h);
        last(static_cast<const T*>(a.dy) + row * a.lddy, d);
        if (skip) last(static_cast<const T*>(a.dh) + row * a.lddh, s);
      }
      if (on0 && !whole0) {
        mask(h, valid);
        mask(d, valid);
        mask(s, valid);
      }
      if (on1 && !whole1) {
        mask(h + 4, valid >> V);
        mask(d + 4, valid >> V);
        mask(s + 4, valid >> V);
      }
    }
    float2 dot = splat(0.f), sum = splat(0.f);
#pragma unroll
    for (int k = 0; k < V; ++k) {
      const float2 x = __fmul2_rn(__fadd2_rn(pair(h, k), mu), iv), y = pair(d, k), w = __fmul2_rn(y, g[k]);
      acc[k] = __ffma2_rn(y, x, acc[k]);
      accb[k] = __fadd2_rn(accb[k], y);
      dot = __ffma2_rn(w, x, dot);
      sum = __fadd2_rn(sum, w);
    }
    float2 both = make_float2(warp_sum(dot.x + dot.y), warp_sum(sum.x + sum.y));
    if constexpr (CL > 1) {
      const int lane = t & 31;
      if (lane < CL)
        send_pair(mapa_shared(smem_u32(&part[par][rank * nw + (t >> 5)]), static_cast<uint32_t>(lane)), both,
                  mapa_shared(smem_u32(&met[par]), static_cast<uint32_t>(lane)));
      __syncwarp();
      if (lane == 0) mbar_arrive(&met[par]);
      ok = ok && wait_cluster(&met[par], meet, a.err, kSiteLayerBwd);
      if (t == 0) mbar_arrive_expect_tx(&met[par], sent);
      if (par) meet ^= 1;
    } else {
      if ((t & 31) == 0) part[par][t >> 5] = both;
      __syncthreads();
    }
    if (t == 0) request(row + kRing * step, slot);
    if (++slot == kRing) {
      slot = 0;
      phase ^= 1;
    }
    if (!a.dx) continue;
    both = splat(0.f);
#pragma unroll 8
    for (int w = 0; w < CL * nw; ++w) both = __fadd2_rn(both, part[par][w]);
    const float2 md = splat(-both.x * over), ms = splat(-both.y * over);
    uint32_t o[8];
#pragma unroll
    for (int k = 0; k < V; ++k) {
      const float2 x = __fmul2_rn(__fadd2_rn(pair(h, k), mu), iv);
      float2 v = __ffma2_rn(x, md, __ffma2_rn(pair(d, k), g[k], ms));
      v = a.dh ? __ffma2_rn(v, iv, pair(s, k)) : __fmul2_rn(v, iv);
      T* e = reinterpret_cast<T*>(o) + 2 * k;
      e[0] = from_f<T>(v.x);
      e[1] = from_f<T>(v.y);
    }
    T* x = static_cast<T*>(a.dx) + row * a.lddx;
    auto put = [&](int col, bool whole, uint32_t there, const uint32_t* w) {
      if (whole) {
        *reinterpret_cast<uint4*>(x + col) = make_uint4(w[0], w[1], w[2], w[3]);
      } else {
#pragma unroll
        for (int e = 0; e < V; ++e)
          if (there >> e & 1u) x[col + e] = reinterpret_cast<const T*>(w)[e];
      }
    };
    if (on0) put(c0, whole0, valid, o);
    if (on1) put(c1, whole1, valid >> V, o + 4);
  }
  if (!ok && t == 0) {  // gave up: as above
    const long mine = (a.rows - first + step - 1) / step;
    for (long i = mine > kRing ? mine - kRing : 0; i < mine; ++i)
      (void)wait(&full[i % kRing], static_cast<uint32_t>(i / kRing) & 1u, a.err, kSiteLayerBwd);
  }
  if (CL > 1) cluster_sync();
  auto partials = [&](float* sums, const float2 (&v)[V]) {
    if (!sums) return;
    float* p = sums + first * a.cols;
#pragma unroll
    for (int e = 0; e < 2 * V; ++e)
      if (there(e)) p[column(e)] = e % 2 ? v[e / 2].y : v[e / 2].x;
  };
  partials(a.part, acc);
  partials(a.partb, accb);
}
// Blocks or clusters that are resident together: a later one would begin when the others end, with as many rows. CTAs of a
// cluster come from one GPC, so the device says how many clusters fit (36 of four here, not 38: 1024 x 32768 66 us, with 38
// 111).
template <typename T, int MT, int MB, int CL, bool SHIFT>
cudaError_t layer_bwd_launch(const NormBwdArgs& a, int threads, int vectors, long blocks, int* grid, cudaStream_t st) {
  const auto kernel = [] {
    if constexpr (SHIFT) return layer_bwd_shift_kernel<T, MT, MB, CL>;
    else return layer_bwd_kernel<T, MT, MB, CL>;
  }();
  static std::atomic<int> fit[64];  // by device; 0: not asked yet
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  int most = dev < 64 ? fit[dev].load(std::memory_order_relaxed) : 0;
  if (!most) {
    constexpr int bytes = kRing * 3 * 16 * 2 * MT;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    most = 1 << 30;
    if (CL > 1) {
      cudaLaunchAttribute at = {};
      at.id = cudaLaunchAttributeClusterDimension;
      at.val.clusterDim.x = CL;
      at.val.clusterDim.y = at.val.clusterDim.z = 1;
      cudaLaunchConfig_t cfg = {};
      cfg.gridDim = dim3(CL);
      cfg.blockDim = dim3(MT);
      cfg.dynamicSmemBytes = bytes;
      cfg.attrs = &at;
      cfg.numAttrs = 1;
      e = cudaOccupancyMaxActiveClusters(&most, kernel, &cfg);
      if (e != cudaSuccess) return e;
      if (most < 1) return cudaErrorInvalidConfiguration;
    }
    if (dev < 64) fit[dev].store(most, std::memory_order_relaxed);
  }
  blocks = std::min<long>(blocks, most);
  if (SHIFT) blocks = blocks_alike(blocks, a.rows);
  *grid = static_cast<int>(blocks);
  if (blocks == 0) return cudaSuccess;
  return launch_k(kernel, dim3(*grid * CL), dim3(threads), static_cast<size_t>(kRing) * 3 * 16 * vectors, st, CL, a);
}
// (grid 0: nothing was launched, because fewer than eight blocks fit the device, or the part of it that there is, and
// there are more rows)
template <typename T, bool SHIFT>
cudaError_t layer_bwd_ring(const NormBwdArgs& a, int cl, int threads, int vectors, int sms, int* grid, cudaStream_t st) {
  // no more blocks than the workspace has rows for
  const long blocks = std::min<long>(norm_bwd_blocks(a.rows, a.cols, sms),
                                     static_cast<long>(sms) * (cl > 1 ? 1 : 512 / threads));
  if (cl == 4) return layer_bwd_launch<T, 512, 1, 4, SHIFT>(a, threads, vectors, blocks, grid, st);
  if (cl == 2) return layer_bwd_launch<T, 512, 1, 2, SHIFT>(a, threads, vectors, blocks, grid, st);
  return threads <= 256 ? layer_bwd_launch<T, 256, 2, 1, SHIFT>(a, threads, vectors, blocks, grid, st)
                        : layer_bwd_launch<T, 512, 1, 1, SHIFT>(a, threads, vectors, blocks, grid, st);
}
// grid: rows of partial sums.
template <typename T>
cudaError_t layer_bwd(const NormBwdArgs& a, int sms, int* grid, cudaStream_t st) {
  constexpr int es = sizeof(T), V = 16 / es;
  auto whole = [&](const void* p, long ld) { return !p || vec_ok(p, ld, es, V); };
  auto alike = [&](const void* p, long ld) { return !p || ld % V == a.ldh % V; };
  const bool even = whole(a.h, a.ldh) && whole(a.dy, a.lddy) && whole(a.dx, a.lddx) && whole(a.dh, a.lddh);
  if constexpr (es == 2) {
    const int cl = a.cols <= 16 * 512 ? 1 : a.cols <= 2 * 16 * 512 ? 2 : 4;
    const int threads = (a.cols / (16 * cl) + 31) / 32 * 32;
    if (a.cols % (16 * cl) == 0 && threads >= 64 && threads <= 512 && even)
      return layer_bwd_ring<T, false>(a, cl, threads, a.cols / (8 * cl), sms, grid, st);
  }
  // vectors of a row that begins within one, of a CTA
  const long all = (static_cast<long>(a.cols) + 2 * V - 2) / V;
  const int cl = all <= 1024 ? 1 : all <= 2048 ? 2 : 4;
  const int vectors = static_cast<int>((all + cl - 1) / cl), threads = ((vectors + 1) / 2 + 31) / 32 * 32;
  // The alternative takes features one by one, or 16-byte vectors through the caches. us there and here: fp32 8192 x 1021 47
  // and 30, 8192 x 5119 255 and 139, 100 x 1021 level; bf16 8192 x 1021 36 and 27, 20000 x 601 80 and 39, but 2000 x 1021
  // 13.6 and 15.5; beyond 8,192 features bf16 2048 x 12001 162 and 70, fp32 16 x 13496 25 and 8, 2048 x 16384 level. Shorter
  // rows of whole vectors stay: bf16 8192 x 1000 22 and 25, fp32 8192 x 4096 87 and 114 to 127. (The 4,096 rows were fitted
  // at 601 to 1,021 features and are too many for long rows: 4095 x 8191, there, 154; 4096 x 8191, here, 105.)
  const bool better = a.cols > 8192 || ((!even || a.cols % V) && (es == 4 || a.rows >= 4096));
  if (better && threads >= 64 && threads <= 512 && alike(a.dy, a.lddy) && alike(a.dx, a.lddx) && alike(a.dh, a.lddh)) {
    const cudaError_t e = layer_bwd_ring<T, true>(a, cl, threads, vectors, sms, grid, st);
    if (e != cudaSuccess || *grid > 0) return e;
  }
  return norm_bwd_vec<T, true>(a, sms, grid, st);
}

}  // namespace
}  // namespace c2d

using namespace c2d;

extern "C" {

int conv2d_layer_norm_fwd(int64_t rows, int32_t cols, float eps, const conv2d_mat* x, const conv2d_mat* residual,
                          const float* gamma, const float* beta, const conv2d_mat* h, const conv2d_mat* y,
                          const conv2d_mat* q8, float* mean, float* inv_std, void* stream) {
  int rc = check_rows(rows, cols);
  if (rc) return rc;
  if (!(eps > 0.f) || !std::isfinite(eps) || !gamma) return CONV2D_ERR_INVALID_ARG;
  for (const float* p : {gamma, beta, static_cast<const float*>(mean), static_cast<const float*>(inv_std)})
    if (!aligned16(p)) return CONV2D_ERR_INVALID_ARG;
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
  a.beta = beta;
  if (y) {
    a.y = y->data;
    a.ldy = ld_of(y, cols);
  }
  if (q8) set_q8(a, q8, cols);
  a.mean = mean;
  a.inv = inv_std;
  a.rows = rows;
  a.cols = cols;
  a.wide = ((reinterpret_cast<uintptr_t>(gamma) | reinterpret_cast<uintptr_t>(beta)) & 31u) == 0;
  a.eps = eps;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  auto run = [&]() -> cudaError_t {
    if (x->type == CONV2D_BF16) return layer_any<__nv_bfloat16>(a, dev->sms, st);
    if (x->type == CONV2D_FP16) return layer_any<__half>(a, dev->sms, st);
    return layer_any<float>(a, dev->sms, st);
  };
  LAUNCH("layer_norm_fwd", st, run());
  return CONV2D_OK;
}

size_t conv2d_layer_norm_bwd_workspace_size(int64_t rows, int32_t cols) {
  if (check_rows(rows, cols)) return 0;
  return std::max<size_t>(256, 2 * static_cast<size_t>(norm_bwd_blocks(rows, cols, sms_for_sizing())) * cols * 4);
}

int conv2d_layer_norm_bwd(int64_t rows, int32_t cols, const conv2d_mat* h, const float* gamma, const float* mean,
                          const float* inv_std, const conv2d_mat* dy, const conv2d_mat* dh, const conv2d_mat* dx,
                          float* dgamma, float* dbeta, int accumulate, void* ws, size_t ws_bytes, void* stream) {
  int rc = check_rows(rows, cols);
  if (rc) return rc;
  const bool sums = dgamma || dbeta;
  if ((!dx && !sums) || !gamma || !aligned16(gamma) || !aligned16(dgamma) || !aligned16(dbeta))
    return CONV2D_ERR_INVALID_ARG;
  DevInfo* dev = nullptr;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (rows == 0) {
    if (!sums || accumulate) return CONV2D_OK;
    if ((rc = device_info(&dev))) return rc;
    for (float* out : {dgamma, dbeta})
      if (out) LAUNCH("zero", st, launch_zero_rows(1, cols, CONV2D_FP32, out, cols, 0, st));
    return CONV2D_OK;
  }
  if (!mean || !inv_std || !aligned16(mean) || !aligned16(inv_std)) return CONV2D_ERR_INVALID_ARG;
  if ((rc = check_mat(h, cols)) || (rc = check_mat(dy, cols))) return rc;
  if (!is_float(h->type) || dy->type != h->type) return CONV2D_ERR_INVALID_ARG;
  for (const conv2d_mat* m : {dh, dx})
    if (m && (check_mat(m, cols) || m->type != h->type)) return CONV2D_ERR_INVALID_ARG;
  if ((rc = device_info(&dev))) return rc;
  const size_t need = conv2d_layer_norm_bwd_workspace_size(rows, cols);
  if (sums && (!ws || ws_bytes < need || (reinterpret_cast<uintptr_t>(ws) & 255u))) return CONV2D_ERR_WORKSPACE;
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
  a.mean = mean;
  a.inv = inv_std;
  a.err = dev->err;
  a.part = dgamma ? static_cast<float*>(ws) : nullptr;
  a.partb = dbeta ? static_cast<float*>(ws) + need / 8 : nullptr;
  a.rows = rows;
  a.cols = cols;
  int grid = 0;
  auto run = [&]() -> cudaError_t {
    if (h->type == CONV2D_BF16) return layer_bwd<__nv_bfloat16>(a, dev->sms, &grid, st);
    if (h->type == CONV2D_FP16) return layer_bwd<__half>(a, dev->sms, &grid, st);
    return layer_bwd<float>(a, dev->sms, &grid, st);
  };
  LAUNCH("layer_norm_bwd", st, run());
  if (sums)
    LAUNCH("column_sum", st,
           launch_column_sum(dgamma ? a.part : a.partb, grid, cols, dgamma ? dgamma : dbeta, accumulate, 0, st, a.partb,
                             dgamma ? dbeta : nullptr));
  return CONV2D_OK;
}

}  // extern "C"
