// rows.cu - kernels over rows of features: 8-bit checkpoints (encode, decode),
// the backward through a dense layer's activation, and the column sums and
// joins behind it and the norms. All are bound by memory: each reads its inputs once and writes its
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
#include "rows_norm.cuh"

namespace c2d {
namespace {

// ------------------------------------------------------------------ 8 bits, 16-bit types in whole groups
// Encode (ENC) or decode of rows of whole groups (32 or 128 columns; TILE, decode only: tiles of 128 x 128): GL = 2 or 8
// threads a group, 16 values each, two groups of a thread in flight (200704 x 256 there and back in groups of 32: 46.5
// us, 0.99 of the copy rate; 59 us with 16-byte accesses).
// total = rows * cols / 16 < 2^31; x rows on 32-byte, q rows on 16-byte boundaries.
template <typename T, bool ENC, int GL, bool TILE, bool LATE>
__global__ void __launch_bounds__(256) q8_flat_kernel(T* x, long ldx, uint8_t* q, long ldq, uint8_t* scale,
                                                      uint32_t total, FastDiv div_nv) {
  if (!LATE) pdl_entry();
  pdl_release();
  constexpr int N = 2;
  const uint32_t step = gridDim.x * 256u;
  const int ng = static_cast<int>(div_nv.d / GL);
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
        sb[i] = scale[(TILE ? row[i] >> 7 : row[i]) * ng + v[i] / GL];
      }
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (j0 + i * step >= total) break;  // the threads of a group go on together (total is a multiple of them)
      float f[16];
      if constexpr (ENC) {
        const T* e = reinterpret_cast<const T*>(w[i]);
        float m = 0.f;
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          f[k] = to_f(e[k]);
          m = fmaxf(m, fabsf(f[k]));
        }
        const uint32_t group = ((1u << GL) - 1u) << (threadIdx.x & (32u - GL));
        auto join = [&](uint32_t x) {
#pragma unroll
          for (int o = 1; o < GL; o <<= 1) x = max(x, __shfl_xor_sync(group, x, o));
          return x;
        };
        uint32_t top = join(__float_as_uint(m));
        bool finite = true;
        if (top == 0x7f800000u) {
          finite = false;
          top = 0u;
#pragma unroll
          for (int k = 0; k < 16; ++k) top = max(top, finite_bits(f[k]));
          top = join(top);
        }
        const uint32_t byte = q8_scale_byte(top);
        const float inv = q8_inv_scale(byte);
        *reinterpret_cast<uint4*>(q + row[i] * ldq + v[i] * 16) =
            make_uint4(q8_pack4(f, inv, finite), q8_pack4(f + 4, inv, finite), q8_pack4(f + 8, inv, finite),
                       q8_pack4(f + 12, inv, finite));
        if (v[i] % GL == 0) scale[row[i] * ng + v[i] / GL] = static_cast<uint8_t>(byte);
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
  const int width = group == kQ8Tile ? 128 : group;
  if (width == 0 || (ENC && group == kQ8Tile) || cols % width != 0 || ldx % 16 != 0 || ldq % 16 != 0 ||
      reinterpret_cast<uintptr_t>(x) % 32 != 0 || rows * (cols / 16) > 0x7fffffffL)
    return false;
  const long total = rows * (cols / 16);
  auto go = [&](auto kernel) {
    return launch_k(kernel, dim3(stream_grid((total + 1) / 2)), dim3(256), 0, st, 1,
                    static_cast<T*>(const_cast<void*>(x)), ldx, static_cast<uint8_t*>(const_cast<void*>(q)), ldq, scale,
                    static_cast<uint32_t>(total), make_fastdiv(static_cast<uint32_t>(cols / 16)));
  };
  auto with = [&](auto gl, auto tile) {
    constexpr int GL = decltype(gl)::value;
    constexpr bool TILE = decltype(tile)::value;
    if constexpr (!ENC)
      if (late) return go(q8_flat_kernel<T, ENC, GL, TILE, true>);
    return go(q8_flat_kernel<T, ENC, GL, TILE, false>);
  };
  if (group == kQ8Group) *e = with(std::integral_constant<int, 2>{}, std::false_type{});
  else if (group == kQ8Wide) *e = with(std::integral_constant<int, 8>{}, std::false_type{});
  else if constexpr (!ENC) *e = with(std::integral_constant<int, 8>{}, std::true_type{});
  return true;
}

// ------------------------------------------------------------------ 8 bits, tiles of 128 x 128
// Encode with one scale for 128 rows by 128 columns: a block a tile, whose values stay in registers (64 a thread, all
// loads in flight at once) between their maximum and their output. V values a vector; zeros past the ends.
template <typename T, int V>
__global__ void __launch_bounds__(256, V == 1 || sizeof(T) == 4 ? 2 : 3) q8_tile_kernel(const T* x, long ldx, uint8_t* q, long ldq, uint8_t* scale,
                                                      long rows, int cols, int ng) {
  pdl_entry();
  constexpr int TPR = 128 / V, RP = 256 / TPR, N = 128 / RP;  // threads a row, rows a pass, passes
  __shared__ uint32_t red[8];
  const int tr = static_cast<int>(threadIdx.x) / TPR, tc = static_cast<int>(threadIdx.x) % TPR * V;
  const long tiles = (rows + 127) / 128 * ng;
  for (long tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    const long row0 = tile / ng * 128 + tr;
    const int c = static_cast<int>(tile % ng) * 128 + tc;
    // The values stay as they came: widened for the maximum and again for the output, not kept widened in between (83
    // registers and two blocks an SM then: 16384 x 4096 bf16 60 us).
    constexpr int W = V * sizeof(T) < 4 ? 1 : V * static_cast<int>(sizeof(T)) / 4;
    uint32_t e[N][W];
#pragma unroll
    for (int i = 0; i < N; ++i) {
#pragma unroll
      for (int k = 0; k < W; ++k) e[i][k] = 0u;
      if (c < cols && row0 + i * RP < rows) {
        const T* p = x + (row0 + i * RP) * ldx + c;
        if constexpr (W == 8) ld_32b(p, e[i]);
        else if constexpr (W == 4) *reinterpret_cast<uint4*>(e[i]) = *reinterpret_cast<const uint4*>(p);
        else if constexpr (sizeof(T) == 4) e[i][0] = *reinterpret_cast<const uint32_t*>(p);
        else e[i][0] = *reinterpret_cast<const uint16_t*>(p);
      }
    }
    pdl_release();
    auto widen = [&](int i, float (&f)[V]) {
#pragma unroll
      for (int k = 0; k < V; ++k) {
        if constexpr (sizeof(T) == 4) {
          f[k] = __uint_as_float(e[i][k]);
        } else {
          const uint16_t h = static_cast<uint16_t>(e[i][k / 2] >> (16 * (k & 1)));
          f[k] = to_f(*reinterpret_cast<const T*>(&h));
        }
      }
    };
    auto top = [&](auto&& of) {
      uint32_t m = 0u;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        float f[V];
        widen(i, f);
        m = max(m, of(f));
      }
      return row_max<256>(m, red);
    };
    uint32_t m = top([](const float (&f)[V]) { return absmax(f); });
    auto narrow = [&] {
#pragma unroll
      for (int i = 0; i < N; ++i)
#pragma unroll
        for (int k = 0; k < W; ++k) asm volatile("" : "+r"(e[i][k]));
    };
    narrow();
    const bool finite = m != kInf;
    if (!finite) {  // the same for the whole block
      m = top([](const float (&f)[V]) { return absmax_finite(f); });
      narrow();
    }
    const uint32_t byte = q8_scale_byte(m);
    const float inv = q8_inv_scale(byte);
    if (threadIdx.x == 0) scale[tile] = static_cast<uint8_t>(byte);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      float f[V];
      widen(i, f);
      if (c < cols && row0 + i * RP < rows) q8_store<V>(q + (row0 + i * RP) * ldq + c, f, inv, finite);
    }
  }
}
template <typename T, int V>
cudaError_t q8_tile_v(const NormArgs& a, cudaStream_t st) {
  const long tiles = (a.rows + 127) / 128 * a.ng;
  return launch_k(q8_tile_kernel<T, V>, dim3(static_cast<unsigned>(std::min(tiles, kMaxGridX))), dim3(256), 0, st, 1,
                  static_cast<const T*>(a.x), a.ldx, a.q, a.ldq, a.qs, a.rows, a.cols, a.ng);
}
template <typename T>
cudaError_t q8_tile(const NormArgs& a, cudaStream_t st) {
  constexpr int es = sizeof(T);
  if (rows_fwd_ok(a, es, 32 / es)) return q8_tile_v<T, 32 / es>(a, st);
  if (rows_fwd_ok(a, es, 16 / es)) return q8_tile_v<T, 16 / es>(a, st);
  return q8_tile_v<T, 1>(a, st);
}

// ------------------------------------------------------------------ decode / move
// V elements a thread and step of a [rows][cols] matrix, dense steps of the grid (E4M3 source: V bytes and
// their scale, two output vectors). rows * ceil(cols / V) below 2^31 (see to_rows).
template <typename T, int V, bool Q, bool LATE>
__global__ void __launch_bounds__(256) to_rows_kernel(const void* x, long ldx, const uint8_t* scale, Q8Layout ql,
                                                      long r0, uint32_t total, int cols, FastDiv div_nv, T* out, long ldo) {
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
        sc[i] = q8_scale(scale[((row[i] + r0) >> ql.row_shift) * ql.ng + (c[i] >> ql.col_shift)]);
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
__global__ void __launch_bounds__(256) to_rows_ragged_kernel(const void* x, long ldx, const uint8_t* scale, Q8Layout ql,
                                                             long r0, uint32_t total, FastDiv div_chunks, int cols, T* out,
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
        sb[k] = scale[((row + r0) >> ql.row_shift) * ql.ng + (c >> ql.col_shift)];  // W divides c and a group: one scale for the neighbours
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

template <typename T, bool Q, int W>
cudaError_t to_rows_ragged(const void* x, long ldx, const uint8_t* scale, Q8Layout ql, long rows, int cols,
                           void* out, long ldo, int late, cudaStream_t st) {
  const int chunks = (cols + ragged_chunk(W) - 1) / ragged_chunk(W);
  const long slab = std::max<long>(1, 0x7fffffffL / chunks);  // rows a launch indexes in 31 bits
  const FastDiv div = make_fastdiv(static_cast<uint32_t>(chunks));
  for (long r0 = 0; r0 < rows; r0 += slab) {
    const long n = std::min(slab, rows - r0);
    const uint32_t total = static_cast<uint32_t>(n * chunks);
    const dim3 grid(static_cast<unsigned>(std::min<long>((n * chunks + 7) / 8, 152L * 64)));
    const void* src = static_cast<const char*>(x) + r0 * ldx * (Q ? 1 : static_cast<long>(sizeof(T)));
    T* o = static_cast<T*>(out) + r0 * ldo;
    const cudaError_t e =
        late ? launch_k(to_rows_ragged_kernel<T, Q, W, true>, grid, dim3(256), 0, st, 1, src, ldx, scale, ql, r0, total,
                        div, cols, o, ldo)
             : launch_k(to_rows_ragged_kernel<T, Q, W, false>, grid, dim3(256), 0, st, 1, src, ldx, scale, ql, r0, total,
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
  const Q8Layout ql = q8_layout(q ? x.group : 0, cols);
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
        return q ? to_rows_ragged<T, true, 4>(x.data, ldx, x.scale, ql, rows, cols, out, ld, late, st)
                 : to_rows_ragged<T, false, 4>(x.data, ldx, nullptr, ql, rows, cols, out, ld, late, st);
      if (ld % 2 == 0)
        return q ? to_rows_ragged<T, true, 2>(x.data, ldx, x.scale, ql, rows, cols, out, ld, late, st)
                 : to_rows_ragged<T, false, 2>(x.data, ldx, nullptr, ql, rows, cols, out, ld, late, st);
    }
    return q ? to_rows_ragged<T, true, 1>(x.data, ldx, x.scale, ql, rows, cols, out, ld, late, st)
             : to_rows_ragged<T, false, 1>(x.data, ldx, nullptr, ql, rows, cols, out, ld, late, st);
  }
  const int nv = cols / V;
  const long slab = std::max<long>(1, 0x7fffffffL / nv);  // rows a launch indexes in 31 bits
  for (long r0 = 0; r0 < rows; r0 += slab) {
    const long n = std::min(slab, rows - r0);
    const uint32_t total = static_cast<uint32_t>(n * nv);
    const dim3 grid(stream_grid((n * nv + 1) / 2));
    const char* src = static_cast<const char*>(x.data) + r0 * ldx * (q ? 1 : static_cast<long>(sizeof(T)));
    T* o = static_cast<T*>(out) + r0 * ld;
    const uint8_t* sc = x.scale;
    const FastDiv div = make_fastdiv(static_cast<uint32_t>(nv));
#define TO_ROWS(V, Q)                                                                                                \
  (late ? launch_k(to_rows_kernel<T, V, Q, true>, grid, dim3(256), 0, st, 1, static_cast<const void*>(src), ldx, sc, \
                   ql, r0, total, cols, div, o, ld)                                                                  \
        : launch_k(to_rows_kernel<T, V, Q, false>, grid, dim3(256), 0, st, 1, static_cast<const void*>(src), ldx, sc, \
                   ql, r0, total, cols, div, o, ld))
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
                                                         const float* part2, float* out2, int accumulate, int late) {
  if (!late) pdl_entry();
  pdl_release();
  if (blockIdx.y) {
    part = part2;
    out = out2;
  }
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
  return to_rows_ragged<uint8_t, false, 1>(x, ldx, nullptr, Q8Layout{}, rows, cols, out, ldo, late, st);
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
                              cudaStream_t st, const float* part2, float* out2) {
  const dim3 grid((cols + 31) / 32, out2 ? 2 : 1);
  if (G > 320)
    return launch_k(column_sum_kernel<32>, grid, dim3(1024), 0, st, 1, part, G, cols, out, part2, out2, accumulate, late);
  return launch_k(column_sum_kernel<16>, grid, dim3(512), 0, st, 1, part, G, cols, out, part2, out2, accumulate, late);
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
  a.rows = rows;
  a.cols = cols;
  set_q8(a, q8, cols);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  auto run = [&]() -> cudaError_t {
    cudaError_t e = cudaSuccess;
    if (a.group == kQ8Tile)
      return x->type == CONV2D_BF16 ? q8_tile<__nv_bfloat16>(a, st) : x->type == CONV2D_FP16 ? q8_tile<__half>(a, st)
                                                                                           : q8_tile<float>(a, st);
    if (x->type == CONV2D_BF16 && q8_flat<__nv_bfloat16, true>(a.x, a.ldx, a.q, a.ldq, a.qs, a.group, rows, cols, 0, st, &e))
      return e;
    if (x->type == CONV2D_FP16 && q8_flat<__half, true>(a.x, a.ldx, a.q, a.ldq, a.qs, a.group, rows, cols, 0, st, &e))
      return e;
    return rows_fwd_any<kEncode>(a, x->type, st);
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

}  // extern "C"
