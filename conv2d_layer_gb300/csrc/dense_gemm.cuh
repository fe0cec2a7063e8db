// dense_gemm.cuh - the dense layer's matrix products on the 5th-generation
// tensor cores: out[m][n] = sum_k R[m][k] C[n][k] for the three products of a
// dense layer's step,
//   forward  y[M][N]  = x[M][K] w[N][K]^T           R = x,  C = w
//   dx       [M][K]   = dz[M][N] w[N][K]            R = dz, C = w (k along its rows)
//   dW       [N][K]   = dz[M][N]^T x[M][K]          R = dz, C = x (k along the rows of both)
// Both operands come by TMA into 128-byte swizzled tiles, K-major or MN-major
// as they lie in memory (no transposed copies); elements outside the matrices
// read as zero, so no size needs to be a multiple of a tile.
//
// Two kernels:
//   dense_pair_kernel     for outputs of many tiles: persistent CTA pairs (cta_group::2), 256 rows x BN columns a
//                         unit, two accumulators, so that the epilogue of a unit runs under the next one's
//                         MMAs. Rows of the output are accumulator lanes: a thread holds 32 neighbouring
//                         columns of its row (an 8-bit group) and packs them into a swizzled buffer of 32
//                         rows x 64 bytes, which a TMA store writes
//   dense_cluster_kernel  for few rows or few tiles: one unit for a cluster of `cluster` CTAs, which split the
//                         K loop and join their sums through distributed shared memory in rank order. Columns
//                         of the output are accumulator lanes (128), rows its columns (16 to 128), so that one
//                         token costs 16 MMA columns and not 128 lanes; a warp holds 32 neighbouring elements
//                         of a row and accesses memory directly
//
// Measured: pair kernel 9728 x 2048 x 8192 bf16 171 us, 1,906 TFLOP/s (the library's product of the same operands:
// 171 us), bound by the tensor cores with the operands' way from L2 (32 KB a CTA for 512 clocks of MMA) as close
// behind; 200704 x 1024 x 256 with relu and both z and y written 156 to 168 us, 0.81 to 0.87 of the copy rate; cluster
// kernel 1 x 16384 x 4096 23 us, 0.86 of the copy rate, 1 x 4096 x 4096 8 to 9 us.
#pragma once
#include "ptx.cuh"
#include "q8.cuh"

namespace c2d {

constexpr int kClusterThreads = 320;  // TMA warp, MMA warp, 8 epilogue warps
constexpr int kPairWarps = 16;        // epilogue warps of the pair kernel: four for each TMEM lane quarter
constexpr int kPairThreads = 64 + 32 * kPairWarps;
constexpr int kDenseMaxStages = 10;
constexpr int kPairBuffers = kPairWarps * 2048;  // the pair kernel's epilogue: 32 rows x 64 bytes a warp
enum : int { kSiteDenseFull = 11, kSiteDenseEmpty = 12, kSiteDenseTFull = 13, kSiteDenseTEmpty = 14, kSiteDenseJoin = 15 };
// The three products: how the operands lie (R is MN-major for dW, C for dx and dW) and the epilogue. kDenseDwAdd: dW
// added in T to what is there, by the pair kernel. A kernel of its own: as a branch of kDenseDw's epilogue it cost
// the overwriting one a tenth (8192 x 2048 x 8192 bf16: 155 us, 170 with the branch).
enum : int { kDenseForward = 0, kDenseDx = 1, kDenseDw = 2, kDenseDwAdd = 3 };
__host__ __device__ constexpr bool dense_r_mn(int mode) { return mode >= kDenseDw; }
__host__ __device__ constexpr bool dense_c_mn(int mode) { return mode != kDenseForward; }

struct DenseGemmParams {
  CUtensorMap tl, tc;   // the operands whose rows are the accumulator's lanes / columns
  // pair kernel: out and z (zq) as {columns, rows, splits} for stores of 32 rows x 64 bytes (zq: 32 bytes)
  CUtensorMap tout, tz;
  uint32_t fmt;         // instruction descriptor's operand format: fp16 0, bf16 1, e4m3 0
  int n;                // columns of the output
  long m;               // rows of the output
  int l_tiles, c_tiles, splits;
  int kb_total, kb_per_split;  // k-blocks of 128 bytes: 64 16-bit or 128 8-bit elements
  // pair kernel: the units from `full` on (fewer than half the pairs, the last wave) are cut into `parts` along k,
  // each run by a pair of its own; the one that ends up with the unit adds the others' sums from join_part
  // [unit][parts - 1][2][BN / 32][4][32 columns][32 rows] once their flags [unit][parts - 1][2][kPairWarps] are 1.
  // parts = 1: full is the number of units.
  int full, parts;
  float* join_part;
  uint32_t* join_flag;
  int BN, stages, cluster;
  // kDenseForward: v = acc * ns[n] * ms[m] + bias[n]; z = v; out = act(v) + res
  const uint8_t *ns, *ms;  // scale bytes of 8-bit operands (both or neither)
  const float* bias;
  int act;
  const void* res;
  void* z;
  uint8_t *zq, *zs;
  int zg;  // scale bytes a row of zq
  long ldr, ldz;
  // kDenseDx, kDenseDw: out = acc (+ out): type T, or fp32 when out_f32; split s at out + s * split_stride.
  // kDenseDwAdd reads out through res and ldr.
  int out_f32, accumulate;
  long split_stride;
  void* out;
  long ldo;
  int tma_out, vec_res, tma_z;  // rows of out / res / z (zq) start on 16-byte boundaries: tout, tz are set
  int late;   // runs beside the kernel before it (see pdl_entry)
  int early;  // leaves SMs idle: the kernel after this one may start at once
  int* err;
};

// One thread of a converged warp, in a way that tells the compiler so: the operands of the copies and MMAs it
// issues then stay in uniform registers.
__device__ __forceinline__ bool elect_one() {
  uint32_t ok;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(ok));
  return ok != 0;
}

// ---------------------------------------------------------------- tcgen05 forms the conv layers do not use
__device__ __forceinline__ void mma_f8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void mma_f8_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}

// 3-D tiled store of a box from shared memory; part of the thread's current bulk group.
__device__ __forceinline__ void tma_store_3d(const CUtensorMap* m, uint32_t src, int c0, int c1, int c2) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
                   reinterpret_cast<uint64_t>(m)),
               "r"(src), "r"(c0), "r"(c1), "r"(c2)
               : "memory");
}
// The same, added to what is there (fp32; sums below 2^-126 come out as zero).
__device__ __forceinline__ void tma_add_3d(const CUtensorMap* m, uint32_t src, int c0, int c1, int c2) {
  asm volatile("cp.reduce.async.bulk.tensor.3d.global.shared::cta.add.tile.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
                   reinterpret_cast<uint64_t>(m)),
               "r"(src), "r"(c0), "r"(c1), "r"(c2)
               : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
// Wait until this thread's bulk stores have read their shared memory / have completed.
__device__ __forceinline__ void bulk_wait_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void bulk_wait() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

// Arrive on an mbarrier of the cluster (shared::cluster address) without ordering this thread's memory accesses.
__device__ __forceinline__ void mbar_arrive_relaxed(uint32_t caddr) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(caddr) : "memory");
}

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ void st_shared_cluster_f32(uint32_t caddr, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(caddr), "f"(v) : "memory");
}
__device__ __forceinline__ float ld_shared_f32(uint32_t addr) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}

// ---------------------------------------------------------------- epilogue of the cluster kernel
// NC rows of the output (m0 ..) of one column (n; off: past the end) a thread. Warp-collective (the 8-bit form
// of z takes a maximum over the warp's 32 columns, which are one group).
template <typename T, int MODE, int NC>
__device__ __forceinline__ void dense_epilogue(const DenseGemmParams& p, float (&v)[NC], int n, long m0, int split,
                                               float2 nscale, float bias) {
  const int nc = static_cast<int>(p.m - m0 < NC ? p.m - m0 : NC);  // uniform
  const bool on = n < p.n;
  if constexpr (MODE == kDenseForward) {
    T res[NC];
    if (p.res) {
      const T* r = static_cast<const T*>(p.res) + m0 * p.ldr + n;
#pragma unroll
      for (int e = 0; e < NC; ++e)
        if (on && e < nc) res[e] = r[e * p.ldr];
    }
    if (p.ns) {
#pragma unroll
      for (int e = 0; e < NC; ++e) v[e] = e < nc ? v[e] * nscale.x * q8_scale(p.ms[m0 + e]) * nscale.y : 0.f;
    }
#pragma unroll
    for (int e = 0; e < NC; ++e) v[e] += bias;
    if (p.zq) {
#pragma unroll
      for (int e = 0; e < NC; ++e) {
        if (e >= nc) break;
        const uint32_t byte = q8_scale_byte(__reduce_max_sync(0xffffffffu, on ? finite_bits(v[e]) : 0u));
        if (on) p.zq[(m0 + e) * p.ldz + n] = static_cast<uint8_t>(q8_pack2(v[e] * q8_inv_scale(byte), 0.f));
        if (on && (n & (kQ8Group - 1)) == 0) p.zs[(m0 + e) * p.zg + n / kQ8Group] = static_cast<uint8_t>(byte);
      }
    } else if (p.z) {
      T* z = static_cast<T*>(p.z) + m0 * p.ldz + n;
#pragma unroll
      for (int e = 0; e < NC; ++e)
        if (on && e < nc) z[e * p.ldz] = from_f<T>(v[e]);
    }
    with_dense_act(p.act, [&](auto act) {
#pragma unroll
      for (int e = 0; e < NC; e += 2) {
        const float2 a = dense_act<decltype(act)::value>(make_float2(v[e], v[e + 1]));
        v[e] = a.x;
        v[e + 1] = a.y;
      }
    });
    T* y = static_cast<T*>(p.out) + m0 * p.ldo + n;
#pragma unroll
    for (int e = 0; e < NC; ++e)
      if (on && e < nc) y[e * p.ldo] = from_f<T>(p.res ? v[e] + to_f(res[e]) : v[e]);
  } else {
    if (!on) return;
    if (p.out_f32) {
      float* o = static_cast<float*>(p.out) + split * p.split_stride + m0 * p.ldo + n;
#pragma unroll
      for (int e = 0; e < NC; ++e)
        if (e < nc) o[e * p.ldo] = p.accumulate ? o[e * p.ldo] + v[e] : v[e];
    } else {
      T* o = static_cast<T*>(p.out) + m0 * p.ldo + n;
#pragma unroll
      for (int e = 0; e < NC; ++e)
        if (e < nc) o[e * p.ldo] = from_f<T>(p.accumulate ? to_f(o[e * p.ldo]) + v[e] : v[e]);
    }
  }
}

// ---------------------------------------------------------------- epilogue of the pair kernel
// A warp's buffer of 32 rows x RB bytes (64 or 32) in shared memory; 16-byte pieces are swizzled so that a
// thread's own row and the warp's whole rows are both accessed without bank conflicts.
template <int RB>
__device__ __forceinline__ uint32_t row_piece(int r, int j) {
  return RB == 64 ? static_cast<uint32_t>(r * 64 + ((j ^ ((r >> 1) & 3)) << 4))
                  : static_cast<uint32_t>(r * 32 + ((j ^ ((r >> 2) & 1)) << 4));
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ void sts128(uint32_t a, const uint4& v) { st_shared_v4(a, v.x, v.y, v.z, v.w); }

// The buffer's rows (nr of them) x nc elements of type E to memory at g (row length ld), for rows that start off
// 16-byte boundaries: in 4-byte words where they start on those, else element by element; accumulate (fp32): added
// to what is there.
template <typename E, int RB>
__device__ __forceinline__ void rows_out(uint32_t buf, E* g, long ld, int nr, int nc, bool accumulate, int lane) {
  constexpr int P = 4 / static_cast<int>(sizeof(E));  // elements a word
  if (P > 1 && !accumulate && ld % P == 0) {
    constexpr int WR = RB / 4;  // words a row
    const int word = lane % WR;
#pragma unroll 4
    for (int r = lane / WR; r < nr; r += 32 / WR) {
      uint32_t w;
      asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w) : "r"(buf + row_piece<RB>(r, word / 4) + (word % 4) * 4u) : "memory");
      E* o = g + r * ld + word * P;
      if ((word + 1) * P <= nc) {
        *reinterpret_cast<uint32_t*>(o) = w;
      } else {
#pragma unroll
        for (int k = 0; k < P; ++k)
          if (word * P + k < nc) o[k] = reinterpret_cast<const E*>(&w)[k];
      }
    }
    return;
  }
  constexpr int PE = 16 / static_cast<int>(sizeof(E));  // elements a piece
  constexpr int W = RB / static_cast<int>(sizeof(E));   // elements a row: 32 or 16
  const int col = lane % W;
  if (col >= nc) return;
#pragma unroll 4
  for (int r = lane / W; r < nr; r += 32 / W) {
    const uint32_t at = buf + row_piece<RB>(r, col / PE) + (col % PE) * static_cast<uint32_t>(sizeof(E));
    E e;
    if constexpr (sizeof(E) == 4) {
      asm volatile("ld.shared.f32 %0, [%1];" : "=f"(e) : "r"(at) : "memory");
    } else if constexpr (sizeof(E) == 2) {
      uint16_t b;
      asm volatile("ld.shared.u16 %0, [%1];" : "=h"(b) : "r"(at) : "memory");
      e = *reinterpret_cast<const E*>(&b);
    } else {
      uint32_t b;
      asm volatile("ld.shared.u8 %0, [%1];" : "=r"(b) : "r"(at) : "memory");
      e = static_cast<E>(b);
    }
    E* o = g + r * ld + col;
    if constexpr (sizeof(E) == 4) {
      if (accumulate) e += *o;
    }
    *o = e;
  }
}
// Takes the warp's buffer for writing: an earlier store has read it.
__device__ __forceinline__ void buffer_take(int lane) {
  if (lane == 0) bulk_wait_read();
  __syncwarp();
}
// Stores the written buffer: by TMA (whole rows, clipped at the matrix's ends; fp32 sums are added there), or word
// by word.
template <typename E, int RB>
__device__ __forceinline__ void buffer_store(uint32_t buf, bool tma, const CUtensorMap* map, int n, long m0, int split,
                                             E* g, long ld, int nr, int nc, bool accumulate, int lane) {
  if (tma) {
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) {
      if (sizeof(E) == 4 && accumulate) tma_add_3d(map, buf, n, static_cast<int>(m0), split);
      else tma_store_3d(map, buf, n, static_cast<int>(m0), split);
      bulk_commit();
    }
  } else {
    __syncwarp();
    rows_out<E, RB>(buf, g + m0 * ld + n, ld, nr, nc, accumulate, lane);
    __syncwarp();
  }
}
// Packs 8 values as T.
template <typename T>
__device__ __forceinline__ uint4 pack8(const float* v) {
  uint4 w;
  T* e = reinterpret_cast<T*>(&w);
#pragma unroll
  for (int k = 0; k < 8; ++k) e[k] = from_f<T>(v[k]);
  return w;
}

// The residual of 32 rows x 32 columns on its way to the buffer, in 16 registers: as 16-byte pieces where the rows
// allow it, as pairs where they start on those, else the elements of rows `from` .. from + 15, one column a lane.
template <typename T>
__device__ __forceinline__ void residual_load(const DenseGemmParams& p, uint32_t (&w)[16], long m0, int n, int nr, int nc,
                                              int from, int lane) {
  if (p.vec_res && nc == 32) {
    const T* r = static_cast<const T*>(p.res) + (m0 + (lane >> 2)) * p.ldr + n + (lane & 3) * 8;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i * 8 + (lane >> 2) < nr)
        *reinterpret_cast<uint4*>(w + 4 * i) = *reinterpret_cast<const uint4*>(r + i * 8 * p.ldr);
  } else if (p.ldr % 2 == 0) {
    const int c = (lane & 15) * 2;
    const uint16_t* r = static_cast<const uint16_t*>(p.res) + (m0 + (lane >> 4)) * p.ldr + n + c;
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (i * 2 + (lane >> 4) < nr && c < nc)
        w[i] = c + 1 < nc ? *reinterpret_cast<const uint32_t*>(r + i * 2 * p.ldr) : r[i * 2 * p.ldr];
  } else if (lane < nc) {
    const uint16_t* r = static_cast<const uint16_t*>(p.res) + (m0 + from) * p.ldr + n + lane;
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (from + i < nr) w[i] = r[i * p.ldr];
  }
}
template <typename T>
__device__ __forceinline__ void residual_store(const DenseGemmParams& p, uint32_t (&w)[16], uint32_t buf, long m0, int n,
                                               int nr, int nc, int lane) {
  if (p.vec_res && nc == 32) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      st_shared_v4(buf + row_piece<64>(i * 8 + (lane >> 2), lane & 3), w[4 * i], w[4 * i + 1], w[4 * i + 2],
                   w[4 * i + 3]);
    return;
  }
  if (p.ldr % 2 == 0) {
#pragma unroll
    for (int i = 0; i < 16; ++i)
      st_shared_b32(buf + row_piece<64>(i * 2 + (lane >> 4), (lane & 15) >> 2) + (lane & 3) * 4u, w[i]);
    return;
  }
#pragma unroll
  for (int from = 0; from < 32; from += 16) {
    if (from) residual_load<T>(p, w, m0, n, nr, nc, from, lane);
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (from + i < nr && lane < nc)
        asm volatile("st.shared.b16 [%0], %1;" ::"r"(buf + row_piece<64>(from + i, lane >> 3) + (lane & 7) * 2),
                     "h"(static_cast<uint16_t>(w[i]))
                     : "memory");
  }
}

// Adds this thread's row of the residual in the buffer to its 32 values.
template <typename T>
__device__ __forceinline__ void residual_add(uint32_t buf, float* v, int lane) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint4 w = lds128(buf + row_piece<64>(lane, j));
    const T* e = reinterpret_cast<const T*>(&w);
#pragma unroll
    for (int k = 0; k < 8; ++k) v[8 * j + k] += to_f(e[k]);
  }
}

// A warp's 32 rows (m0 ..) x up to 32 columns (n ..) of the accumulator at taddr; nr rows and nc columns count.
// res: the residual's registers, loaded for these columns and left loading for the columns from n + 128 (the
// warp's next), so that its way from memory is hidden by the main loop or by the columns before. taken(a) is
// called when the accumulator's columns are in a[] (it frees the accumulator, and adds other parts' sums).
template <typename T, int MODE, bool FP8, typename F>
__device__ __forceinline__ void pair_epilogue(const DenseGemmParams& p, uint32_t taddr, uint32_t buf, long m0, int n,
                                              int end, int nr, int split, uint32_t mscale, uint32_t (&res)[16], int lane,
                                              F&& taken) {
  const int nc = min(end - n, 32);
  if constexpr (MODE == kDenseForward) {
    float v[32];
    {
      uint32_t a[32];
      tmem_ld32(taddr, a);
      tmem_ld_wait32(a);
      taken(a);
#pragma unroll
      for (int e = 0; e < 32; ++e) v[e] = __uint_as_float(a[e]);
    }
    if constexpr (FP8) {
      const float2 f = q8_factors(mscale);
#pragma unroll
      for (int e = 0; e < 32; e += 2) {
        const float2 a = make_float2(e < nc ? q8_scale(p.ns[n + e]) : 1.f, e + 1 < nc ? q8_scale(p.ns[n + e + 1]) : 1.f);
        const float2 s = __fmul2_rn(__fmul2_rn(make_float2(v[e], v[e + 1]), splat(f.x)), a);
        v[e] = s.x;
        v[e + 1] = s.y;
      }
      if (__any_sync(0xffffffffu, f.y != 1.f)) {  // a scale of one of the rows is beyond 2^-100 or 2^80
#pragma unroll
        for (int e = 0; e < 32; ++e) v[e] *= f.y;
      }
    }
    if (p.bias) {
      if (nc == 32) {
#pragma unroll
        for (int e = 0; e < 32; e += 4) {
          const float4 b = *reinterpret_cast<const float4*>(p.bias + n + e);
          v[e] += b.x;
          v[e + 1] += b.y;
          v[e + 2] += b.z;
          v[e + 3] += b.w;
        }
      } else {
#pragma unroll
        for (int e = 0; e < 32; ++e)
          if (e < nc) v[e] += p.bias[n + e];
      }
    }
    if (p.zq) {
      // The largest magnitude: fmaxf passes NaN over; only where an infinity is among the values are they
      // looked at one by one.
      float top = 0.f;
      if (nc == 32) {
#pragma unroll
        for (int e = 0; e < 32; ++e) top = fmaxf(top, fabsf(v[e]));
      } else {
#pragma unroll
        for (int e = 0; e < 32; ++e) top = e < nc ? fmaxf(top, fabsf(v[e])) : top;
      }
      uint32_t bits = __float_as_uint(top);
      float inf0 = 0.f;  // times an infinity: NaN
      if (bits == 0x7f800000u) {
        bits = 0u;
        for (int e = 0; e < 32; ++e)
          if (e < nc) bits = max(bits, finite_bits(v[e]));
        inf0 = 1.f;
      }
      const uint32_t byte = q8_scale_byte(bits);
      const float inv = q8_inv_scale(byte);
      if (lane < nr) p.zs[(m0 + lane) * p.zg + n / kQ8Group] = static_cast<uint8_t>(byte);
      uint32_t w[8];
      if (inf0 == 0.f) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float* x = v + 4 * e;
          w[e] = q8_pack2_finite(x[0] * inv, x[1] * inv) | q8_pack2_finite(x[2] * inv, x[3] * inv) << 16;
        }
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float* x = v + 4 * e;
          w[e] = q8_pack2(x[0] * inv, x[1] * inv) | q8_pack2(x[2] * inv, x[3] * inv) << 16;
        }
      }
      buffer_take(lane);
      st_shared_v4(buf + row_piece<32>(lane, 0), w[0], w[1], w[2], w[3]);
      st_shared_v4(buf + row_piece<32>(lane, 1), w[4], w[5], w[6], w[7]);
      buffer_store<uint8_t, 32>(buf, p.tma_z, &p.tz, n, m0, 0, p.zq, p.ldz, nr, nc, false, lane);
    } else if (p.z) {
      buffer_take(lane);
#pragma unroll
      for (int j = 0; j < 4; ++j) sts128(buf + row_piece<64>(lane, j), pack8<T>(v + 8 * j));
      buffer_store<T, 64>(buf, p.tma_z, &p.tz, n, m0, 0, static_cast<T*>(p.z), p.ldz, nr, nc, false, lane);
    }
    with_dense_act(p.act, [&](auto act) {
#pragma unroll
      for (int e = 0; e < 32; e += 2) {
        const float2 a = dense_act<decltype(act)::value>(make_float2(v[e], v[e + 1]));
        v[e] = a.x;
        v[e + 1] = a.y;
      }
    });
    buffer_take(lane);
    if (p.res) {
      residual_store<T>(p, res, buf, m0, n, nr, nc, lane);
      if (n + 128 < end) residual_load<T>(p, res, m0, n + 128, nr, min(end - n - 128, 32), 0, lane);
      __syncwarp();
      residual_add<T>(buf, v, lane);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) sts128(buf + row_piece<64>(lane, j), pack8<T>(v + 8 * j));
    buffer_store<T, 64>(buf, p.tma_out, &p.tout, n, m0, 0, static_cast<T*>(p.out), p.ldo, nr, nc, false, lane);
  } else {
    uint32_t a[32];
    tmem_ld32(taddr, a);
    tmem_ld_wait32(a);
    taken(a);
    if constexpr (MODE == kDenseDwAdd) {
      // what is there (p.res = p.out) is added to the fp32 sums: the result is rounded to T once
      buffer_take(lane);
      residual_load<T>(p, res, m0, n, nr, nc, 0, lane);
      residual_store<T>(p, res, buf, m0, n, nr, nc, lane);
      __syncwarp();
      float v[32];
#pragma unroll
      for (int e = 0; e < 32; ++e) v[e] = __uint_as_float(a[e]);
      residual_add<T>(buf, v, lane);
#pragma unroll
      for (int j = 0; j < 4; ++j) sts128(buf + row_piece<64>(lane, j), pack8<T>(v + 8 * j));
      buffer_store<T, 64>(buf, p.tma_out, &p.tout, n, m0, 0, static_cast<T*>(p.out), p.ldo, nr, nc, false, lane);
    } else if (p.out_f32) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (16 * h >= nc) break;  // uniform
        buffer_take(lane);
#pragma unroll
        for (int j = 0; j < 4; ++j)
          st_shared_v4(buf + row_piece<64>(lane, j), a[16 * h + 4 * j], a[16 * h + 4 * j + 1], a[16 * h + 4 * j + 2],
                       a[16 * h + 4 * j + 3]);
        buffer_store<float, 64>(buf, p.tma_out, &p.tout, n + 16 * h, m0, split,
                                static_cast<float*>(p.out) + split * p.split_stride, p.ldo, nr, nc - 16 * h,
                                p.accumulate, lane);
      }
    } else {
      buffer_take(lane);
#pragma unroll
      for (int j = 0; j < 4; ++j) sts128(buf + row_piece<64>(lane, j), pack8<T>(reinterpret_cast<const float*>(a) + 8 * j));
      buffer_store<T, 64>(buf, p.tma_out, &p.tout, n, m0, 0, static_cast<T*>(p.out), p.ldo, nr, nc, false, lane);
    }
  }
}

// ---------------------------------------------------------------- operands
// One k-block of an operand's `rows` rows from row r0 into shared memory at dst. K-major: one box of 128
// bytes x rows. MN-major: panels of 64 rows (128 bytes) x 64 k, 8 KB each.
template <bool PAIR, bool MN>
__device__ __forceinline__ void dense_load(const CUtensorMap* m, uint32_t dst, uint64_t* bar, uint32_t pbar, int kelem,
                                           int r0, int rows) {
  if (MN) {
    for (int j = 0; j < rows; j += 64) {
      if (PAIR) tma_load_2d_pair(dst + j * 128, m, pbar, r0 + j, kelem);
      else tma_load_2d(dst + j * 128, m, bar, r0 + j, kelem);
    }
  } else {
    if (PAIR) tma_load_2d_pair(dst, m, pbar, kelem, r0);
    else tma_load_2d(dst, m, bar, kelem, r0);
  }
}
// Descriptor of the ring's first tile of an operand. A stage, a k-block and a 32-byte step of k are added to
// its address field (units of 16 bytes; the ring lies below 256 KB, so nothing carries into the next field):
// what the issuing thread does between two MMAs is time that the tensor core may stand still (making the
// descriptors anew for each MMA, with the layouts as variables, took 9728 x 2048 x 8192 from 179 to 210 us).
template <bool MN>
__device__ __forceinline__ uint64_t dense_desc(uint32_t addr) {
  return sdesc_sw128(addr, MN ? 8192u : 16u, 1024);
}
// The MMAs of the k-block `offset` bytes into the ring: four of 32 bytes of k (16 16-bit or 32 8-bit elements).
template <bool PAIR, bool FP8, bool LMN, bool CMN>
__device__ __forceinline__ void dense_mma(uint64_t l, uint64_t c, uint32_t d, uint32_t offset, uint32_t idesc,
                                          uint32_t acc) {
#pragma unroll
  for (int kk = 0; kk < 4; ++kk) {
    const uint64_t a = l + (offset >> 4) + kk * (LMN ? 128 : 2), b = c + (offset >> 4) + kk * (CMN ? 128 : 2);
    if (FP8) {
      if (PAIR) mma_f8_pair(d, a, b, idesc, kk ? 1u : acc);
      else mma_f8(d, a, b, idesc, kk ? 1u : acc);
    } else {
      if (PAIR) mma_bf16_pair(d, a, b, idesc, kk ? 1u : acc);
      else mma_bf16(d, a, b, idesc, kk ? 1u : acc);
    }
  }
}

// Columns of a unit that one CTA of its cluster joins: groups of four, owned in turn.
__host__ __device__ constexpr int dense_own_cols(int BN, int cluster) { return (BN / 4 + cluster - 1) / cluster * 4; }

// Unit u of the output: bands of 8 lane tiles are walked column tile by column tile, so that the units in
// flight at one time share their operands in L2.
__device__ __forceinline__ void dense_unit(const DenseGemmParams& p, int u, int& lt, int& ct, int& split) {
  const int per = p.l_tiles * p.c_tiles;
  split = u / per;
  u -= split * per;
  const int band = u / (8 * p.c_tiles);
  const int l0 = band * 8;
  const int h = min(8, p.l_tiles - l0);
  const int i = u - band * 8 * p.c_tiles;
  ct = i / h;
  lt = l0 + i - ct * h;
}

// The it-th piece of work of pair cid of ncl: a unit, or in the last wave a part of one.
struct DenseItem {
  int lt, ct, split, kb0, kb1;
  int tail, part;  // tail: index among the cut units, -1: a whole unit; part 0 ends up with the unit
};
__device__ __forceinline__ bool dense_item(const DenseGemmParams& p, int it, int cid, int ncl, DenseItem& o) {
  const int u = cid + it * ncl;
  if (u < p.full) {
    dense_unit(p, u, o.lt, o.ct, o.split);
    o.kb0 = o.split * p.kb_per_split;
    o.kb1 = min(p.kb_total, o.kb0 + p.kb_per_split);
    o.tail = -1;
    o.part = 0;
    return true;
  }
  if (p.parts <= 1) return false;
  const int rem = p.l_tiles * p.c_tiles - p.full;
  if (u >= p.full + ncl || cid >= rem * p.parts) return false;
  // The pairs that wait for others' sums are the last ones: blocks start in the order of their index, so those that
  // they wait for have started.
  const int q = cid / rem;
  o.tail = cid - q * rem;
  o.part = q == p.parts - 1 ? 0 : q + 1;
  dense_unit(p, p.full + o.tail, o.lt, o.ct, o.split);
  o.kb0 = static_cast<int>(static_cast<long>(p.kb_total) * o.part / p.parts);
  o.kb1 = static_cast<int>(static_cast<long>(p.kb_total) * (o.part + 1) / p.parts);
  return true;
}
// The slot of a warp's sums of columns c .. c + 31 of its unit's tile (column-major, so that a warp's accesses are
// whole lines).
__device__ __forceinline__ float* join_slot(const DenseGemmParams& p, int tail, int part, int rank, int q, int c) {
  const long tile = (static_cast<long>(tail) * (p.parts - 1) + part - 1) * 2 + rank;
  return p.join_part + ((tile * (p.BN / 32) + c / 32) * 4 + q) * 1024;
}
__device__ __forceinline__ uint32_t* join_flag(const DenseGemmParams& p, int tail, int part, int rank, int warp) {
  return p.join_flag + ((static_cast<long>(tail) * (p.parts - 1) + part - 1) * 2 + rank) * kPairWarps + warp;
}
__device__ __forceinline__ uint32_t ld_acquire(const uint32_t* p) {
  uint32_t v;
  asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ void st_release(uint32_t* p, uint32_t v) {
  asm volatile("st.release.gpu.global.u32 [%0], %1;" ::"l"(p), "r"(v) : "memory");
}
// Bounded wait for a flag (see wait()).
__device__ __forceinline__ bool wait_flag(const uint32_t* f, int* err) {
  const uint64_t t0 = globaltimer();
  for (uint32_t i = 1;; ++i) {
    if (ld_acquire(f) == 1u) return true;
    if ((i & 255u) == 0 && globaltimer() - t0 > kWaitLimitNs) {
      atomicCAS(err, 0, kSiteDenseJoin);
      return false;
    }
  }
}

template <typename T, int MODE, bool FP8>
__global__ void __launch_bounds__(kPairThreads, 1) dense_pair_kernel(const __grid_constant__ DenseGemmParams p) {
  constexpr bool RMN = dense_r_mn(MODE), CMN = dense_c_mn(MODE);
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int BN = p.BN, S = p.stages;
  // this CTA's halves: 128 rows and BN / 2 columns (whole panels of 64 when MN-major)
  const int c_rows = CMN ? (BN / 2 + 63) & ~63 : BN / 2;
  const uint32_t l_bytes = 128 * 128, c_bytes = static_cast<uint32_t>(c_rows) * 128;
  const uint32_t stage_bytes = l_bytes + c_bytes;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + S * stage_bytes + kPairBuffers);
  uint64_t* empty = full + kDenseMaxStages;
  uint64_t* tfull = empty + kDenseMaxStages;
  uint64_t* tempty = tfull + 2;
  uint32_t* slot = reinterpret_cast<uint32_t*>(tempty + 2);
  const uint32_t sbase = smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  const int cid = static_cast<int>(blockIdx.x >> 1), ncl = static_cast<int>(gridDim.x >> 1);
  const uint32_t tcols = tmem_cols_for(2 * BN);

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&tfull[b], 1);
      mbar_init(&tempty[b], 2 * kPairWarps);  // one arrival per epilogue warp of both CTAs
    }
    fence_mbar_init();
    tma_prefetch_desc(&p.tl);
    tma_prefetch_desc(&p.tc);
    if (p.tma_out) tma_prefetch_desc(&p.tout);
    if (p.tma_z) tma_prefetch_desc(&p.tz);
  }
  if (warp == 1) {
    tmem_alloc_pair(slot, tcols);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // the peer's barriers are initialised before any remote arrival
  tc_fence_after();
  const uint32_t tmem = *slot;
  if (!p.late) pdl_entry();  // the set-up above runs under the end of the kernel before
  if (p.early) pdl_release();

  if (warp == 0) {
    if (elect_one()) {
      int s = 0;
      uint32_t par = 0;
      bool alive = true;
      const int kelems = FP8 ? 128 : 64;
      DenseItem w;
      for (int it = 0; alive && dense_item(p, it, cid, ncl, w); ++it) {
        const int lr = w.lt * 256 + static_cast<int>(rank) * 128, cr = w.ct * BN + static_cast<int>(rank) * (BN / 2);
        for (int kb = w.kb0; kb < w.kb1; ++kb) {
          if (!wait(&empty[s], par ^ 1, p.err, kSiteDenseEmpty)) {
            alive = false;
            break;
          }
          // both members' loads complete on the even CTA's barrier, which expects them all
          const uint32_t bar = mapa_shared(smem_u32(&full[s]), 0);
          if (leader) mbar_arrive_expect_tx(&full[s], 2 * stage_bytes);
          const uint32_t l0 = sbase + s * stage_bytes;
          dense_load<true, RMN>(&p.tl, l0, nullptr, bar, kb * kelems, lr, 128);
          dense_load<true, CMN>(&p.tc, l0 + l_bytes, nullptr, bar, kb * kelems, cr, c_rows);
          if (++s == S) {
            s = 0;
            par ^= 1;
          }
        }
      }
      // the even CTA's commits land in this CTA's empty barriers: let every stage's last use (and so every
      // copy) finish before the CTA can exit
      for (int i = 0; i < S; ++i) {
        if (!wait(&empty[s], par ^ 1, p.err, kSiteDenseEmpty)) break;
        if (++s == S) {
          s = 0;
          par ^= 1;
        }
      }
    }
  } else if (warp == 1) {
    if (leader && elect_one()) {
      const uint32_t idesc = idesc_f32acc(256, BN, p.fmt, RMN, CMN);
      const uint64_t l = dense_desc<RMN>(sbase), c = dense_desc<CMN>(sbase + l_bytes);
      int s = 0, tc = 0;
      uint32_t par = 0;
      bool alive = true;
      DenseItem w;
      for (; alive && dense_item(p, tc, cid, ncl, w); ++tc) {
        const int buf = tc & 1;
        if (!wait(&tempty[buf], ((tc >> 1) & 1) ^ 1, p.err, kSiteDenseTEmpty)) break;
        tc_fence_after();
        for (int kb = w.kb0; kb < w.kb1; ++kb) {
          if (!wait(&full[s], par, p.err, kSiteDenseFull)) {
            alive = false;
            break;
          }
          tc_fence_after();
          dense_mma<true, FP8, RMN, CMN>(l, c, tmem + buf * BN, s * stage_bytes, idesc, kb > w.kb0);
          mma_commit_pair(&empty[s]);
          if (++s == S) {
            s = 0;
            par ^= 1;
          }
        }
        if (alive) mma_commit_pair(&tfull[buf]);
      }
    }
  } else {
    // four warps per TMEM lane quarter, which take the unit's columns 32 at a time in turn
    const int q = warp & 3, part = (warp - 2) >> 2;
    const uint32_t buf0 = sbase + S * stage_bytes + static_cast<uint32_t>(warp - 2) * 2048u;
    DenseItem w;
    for (int tc = 0; dense_item(p, tc, cid, ncl, w); ++tc) {
      const int ct = w.ct;
      const long m0 = static_cast<long>(w.lt) * 256 + rank * 128 + q * 32;
      const int nr = static_cast<int>(min(p.m - m0, 32L));
      const uint32_t mscale = FP8 && lane < nr ? p.ms[m0 + lane] : 127u;
      const int end = min(p.n, ct * BN + BN);
      const int n0 = ct * BN + part * 32;
      uint32_t res[16];
      if (MODE == kDenseForward && p.res && w.part == 0 && nr > 0 && n0 < end)
        residual_load<T>(p, res, m0, n0, nr, min(end - n0, 32), 0, lane);
      const int buf = tc & 1;
      int ok = 1;
      if (lane == 0) ok = wait(&tfull[buf], (tc >> 1) & 1, p.err, kSiteDenseTFull) ? 1 : 0;
      if (!__shfl_sync(0xffffffffu, ok, 0)) break;
      tc_fence_after();
      // Frees the accumulator for the unit after next, once its last columns are in registers: before they are
      // written, and without waiting for what was (the arrival orders nothing but the TMEM reads; with release
      // semantics it waited for the stores to reach L2, and held the next MMAs back by as much).
      auto arrive = [&] {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_relaxed(mapa_shared(smem_u32(&tempty[buf]), 0));
      };
      const uint32_t t0 = tmem + (static_cast<uint32_t>(q * 32) << 16) + buf * BN - ct * BN;
      if (nr <= 0 || n0 >= end) {  // uniform
        arrive();
      } else if (w.part > 0) {
        // a part of a cut unit: the sums go to the pair that ends up with it
#pragma unroll 1
        for (int n = n0; n < end; n += 128) {
          uint32_t a[32];
          tmem_ld32(t0 + n, a);
          tmem_ld_wait32(a);
          if (n + 128 >= end) arrive();
          float* slot = join_slot(p, w.tail, w.part, static_cast<int>(rank), q, n - ct * BN) + lane;
#pragma unroll
          for (int e = 0; e < 32; ++e) slot[e * 32] = __uint_as_float(a[e]);
        }
        __threadfence();
        __syncwarp();
        if (lane == 0) st_release(join_flag(p, w.tail, w.part, static_cast<int>(rank), warp - 2), 1u);
      } else {
        if (w.tail >= 0) {
          ok = 1;
          for (int j = 1; j < p.parts; ++j)
            if (lane == 0 && ok) ok = wait_flag(join_flag(p, w.tail, j, static_cast<int>(rank), warp - 2), p.err) ? 1 : 0;
          __syncwarp();
        }
#pragma unroll 1
        for (int n = n0; n < end; n += 128)
          pair_epilogue<T, MODE, FP8>(p, t0 + n, buf0, m0, n, end, nr, w.split, mscale, res, lane,
                                 [&](uint32_t (&a)[32]) {
                                   if (w.tail >= 0) {
                                     for (int j = 1; j < p.parts; ++j) {
                                       const float* slot =
                                           join_slot(p, w.tail, j, static_cast<int>(rank), q, n - ct * BN) + lane;
#pragma unroll
                                       for (int e = 0; e < 32; ++e) a[e] = __float_as_uint(__uint_as_float(a[e]) + __ldcg(slot + e * 32));
                                     }
                                   }
                                   if (n + 128 >= end) arrive();
                                 });
      }
    }
    if (lane == 0) bulk_wait();  // the stores have read the buffers and are done
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // no remote arrival or MMA write into this CTA is still in flight
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, tcols);
  }
  if (p.late) pdl_entry();
}

template <typename T, int MODE, bool FP8>
__global__ void __launch_bounds__(kClusterThreads, 1) dense_cluster_kernel(const __grid_constant__ DenseGemmParams p) {
  constexpr bool LMN = dense_c_mn(MODE), CMN = dense_r_mn(MODE);  // the lanes are the output's columns
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int BN = p.BN, S = p.stages, CL = p.cluster;
  const uint32_t l_bytes = 128 * 128, c_bytes = static_cast<uint32_t>(BN) * 128;
  const uint32_t stage_bytes = l_bytes + c_bytes;
  // CL > 1: the sums that the cluster's CTAs hand this one, [CL][own_cols][128], behind the ring
  const int own_cols = dense_own_cols(BN, CL);
  const uint32_t join_bytes = CL > 1 ? static_cast<uint32_t>(CL * own_cols) * 512u : 0u;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + S * stage_bytes + join_bytes);
  uint64_t* empty = full + kDenseMaxStages;
  uint64_t* tfull = empty + kDenseMaxStages;
  uint32_t* slot = reinterpret_cast<uint32_t*>(tfull + 1);
  const uint32_t sbase = smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = CL > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const uint32_t tcols = tmem_cols_for(BN);

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(tfull, 1);
    fence_mbar_init();
    tma_prefetch_desc(&p.tl);
    tma_prefetch_desc(&p.tc);
  }
  if (warp == 1) {
    tmem_alloc(slot, tcols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  if (CL > 1) cluster_arrive();  // waited for before the other CTAs' shared memory is written
  tc_fence_after();
  const uint32_t tmem = *slot;
  if (!p.late) pdl_entry();  // the set-up above runs under the end of the kernel before
  if (p.early) pdl_release();

  int lt, ct, split;
  dense_unit(p, static_cast<int>(blockIdx.x) / CL, lt, ct, split);
  // this CTA's share of the split's k-blocks (maybe none)
  const int s0 = split * p.kb_per_split, s1 = min(p.kb_total, s0 + p.kb_per_split);
  const int kb0 = s0 + static_cast<int>(static_cast<long>(s1 - s0) * rank / CL);
  const int kb1 = s0 + static_cast<int>(static_cast<long>(s1 - s0) * (rank + 1) / CL);

  if (warp == 0) {
    if (elect_one()) {
      int s = 0;
      uint32_t par = 0;
      const int kelems = FP8 ? 128 : 64;
      int kb = kb0;
      for (; kb < kb1; ++kb) {
        if (!wait(&empty[s], par ^ 1, p.err, kSiteDenseEmpty)) break;
        mbar_arrive_expect_tx(&full[s], stage_bytes);
        const uint32_t l0 = sbase + s * stage_bytes;
        dense_load<false, LMN>(&p.tl, l0, &full[s], 0u, kb * kelems, lt * 128, 128);
        dense_load<false, CMN>(&p.tc, l0 + l_bytes, &full[s], 0u, kb * kelems, ct * BN, BN);
        if (++s == S) {
          s = 0;
          par ^= 1;
        }
      }
      if (kb < kb1) {  // gave up: the copies of the stages before land before the CTA goes on
        const int n = kb - kb0;  // stages filled
        for (int i = min(S, n); i > 0; --i) {
          const int j = n - i;
          (void)wait(&full[j % S], static_cast<uint32_t>(j / S) & 1u, p.err, kSiteDenseFull);
        }
      }
    }
  } else if (warp == 1) {
    if (elect_one()) {
      const uint32_t idesc = idesc_f32acc(128, BN, p.fmt, LMN, CMN);
      const uint64_t l = dense_desc<LMN>(sbase), c = dense_desc<CMN>(sbase + l_bytes);
      int s = 0;
      uint32_t par = 0;
      for (int kb = kb0; kb < kb1; ++kb) {
        if (!wait(&full[s], par, p.err, kSiteDenseFull)) break;
        tc_fence_after();
        dense_mma<false, FP8, LMN, CMN>(l, c, tmem, s * stage_bytes, idesc, kb > kb0);
        mma_commit(&empty[s]);
        if (++s == S) {
          s = 0;
          par ^= 1;
        }
      }
      if (kb1 > kb0) mma_commit(tfull);  // every MMA issued above
      else mbar_arrive(tfull);
    }
  } else {
    const int q = warp & 3, half = (warp - 2) >> 2;
    const int n = lt * 128 + q * 32 + lane;
    float2 nscale = splat(1.f);
    float bias = 0.f;
    if (MODE == kDenseForward && CL == 1 && n < p.n) {
      if (p.ns) nscale = q8_factors(p.ns[n]);
      if (p.bias) bias = p.bias[n];
    }
    int ok = 1;
    if (lane == 0) ok = wait(tfull, 0, p.err, kSiteDenseTFull) ? 1 : 0;
    ok = __shfl_sync(0xffffffffu, ok, 0);
    pdl_release();
    if (CL > 1) cluster_wait();  // the others have started
    if (ok) {
      tc_fence_after();
      const uint32_t t0 = tmem + (static_cast<uint32_t>(q * 32) << 16);
      const uint32_t join = sbase + S * stage_bytes;
      for (int c = half * 16; c < BN; c += 32) {
        const long m0 = static_cast<long>(ct) * BN + c;
        if (m0 >= p.m) break;  // uniform
        uint32_t r[16];
        tmem_ld16(t0 + c, r);
        tmem_ld_wait(r);
        float v[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) v[e] = kb1 > kb0 ? __uint_as_float(r[e]) : 0.f;
        if (CL == 1) {
          dense_epilogue<T, MODE, 16>(p, v, n, m0, split, nscale, bias);
        } else {
          // columns are owned four at a time in turn; each goes to its owner's slot for this CTA
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            const int quad = c / 4 + g;
            const uint32_t at = join + static_cast<uint32_t>(((rank * own_cols + quad / CL * 4) * 128 + q * 32 + lane) * 4);
            const uint32_t to = mapa_shared(at, static_cast<uint32_t>(quad % CL));
#pragma unroll
            for (int e = 0; e < 4; ++e) st_shared_cluster_f32(to + e * 512, v[4 * g + e]);
          }
        }
      }
    }
  }
  if (CL > 1) {
    __syncwarp();
    if (warp < 2) cluster_wait();
    __syncthreads();
    cluster_sync();  // every CTA's sums have arrived; from here on a CTA reads its own shared memory only
    // jobs of 4 columns x 32 lanes; the sums are added in rank order
    const int nc = static_cast<int>(min(static_cast<long>(BN), p.m - static_cast<long>(ct) * BN));
    const int quads = (nc + 3) / 4;
    const int own = (quads - rank + CL - 1) / CL;  // quads rank, rank + CL, ...
    const uint32_t join = sbase + S * stage_bytes;
    for (int j = warp; j < own * 4; j += kClusterThreads / 32) {
      const int q = j & 3, i = j >> 2;
      const int n = lt * 128 + q * 32 + lane;
      float2 nscale = splat(1.f);
      float bias = 0.f;
      if (MODE == kDenseForward && n < p.n) {
        if (p.ns) nscale = q8_factors(p.ns[n]);
        if (p.bias) bias = p.bias[n];
      }
      float v[4] = {0.f, 0.f, 0.f, 0.f};
      const uint32_t at = join + static_cast<uint32_t>((i * 4 * 128 + q * 32 + lane) * 4);
#pragma unroll 4
      for (int k = 0; k < CL; ++k) {
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] += ld_shared_f32(at + static_cast<uint32_t>((k * own_cols + e) * 512));
      }
      dense_epilogue<T, MODE, 4>(p, v, n, static_cast<long>(ct) * BN + (i * CL + rank) * 4, split, nscale, bias);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, tcols);
  }
  if (p.late) pdl_entry();
}

}  // namespace c2d
