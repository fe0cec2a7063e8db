// dense_gemm.cuh - the dense layer's matrix products on the 5th-generation
// tensor cores: out[m][n] = sum_k C[m][k] L[n][k] for the three products of a
// dense layer's step,
//   forward  y[M][N]  = x[M][K] w[N][K]^T           L = w,  C = x
//   dx       [M][K]   = dz[M][N] w[N][K]            L = w (k along its rows), C = dz
//   dW       [N][K]   = dz[M][N]^T x[M][K]          L = x (k along its rows), C = dz (likewise)
// L, the operand that runs along the output's rows (its contiguous dimension),
// takes the accumulator's lanes, C its columns. So the 32 lanes of an epilogue
// warp hold 32 neighbouring elements of one output row: it writes (and reads
// the residual) in whole sectors straight from the tensor memory layout, a
// bias is one register, and a group of 32 columns that shares an 8-bit scale
// is one warp, its maximum one redux instruction.
//
// Both operands come by TMA into 128-byte swizzled tiles, K-major or MN-major
// as they lie in memory (no transposed copies); elements outside the matrices
// read as zero, so no size needs to be a multiple of a tile.
//
// Two kernels:
//   dense_pair_kernel     persistent CTA pairs (cta_group::2), 256 lanes x BN columns a unit, two
//                         accumulators, so that the epilogue of a unit runs under the next one's MMAs
//   dense_cluster_kernel  one unit of 128 lanes x BN columns for a cluster of `cluster` CTAs, which
//                         split the K loop and join their sums through distributed shared memory in
//                         rank order: for outputs too small to give every SM a unit of its own
#pragma once
#include "ptx.cuh"
#include "q8.cuh"

namespace c2d {

constexpr int kDenseThreads = 320;  // TMA warp, MMA warp, 8 epilogue warps
constexpr int kDenseMaxStages = 10;
enum : int { kSiteDenseFull = 11, kSiteDenseEmpty = 12, kSiteDenseTFull = 13, kSiteDenseTEmpty = 14 };
enum : int { kDenseForward = 0, kDenseStore = 1 };  // epilogues

struct DenseGemmParams {
  CUtensorMap tl, tc;
  int l_mn, c_mn;       // operand lies MN-major (its k index runs along memory rows)
  int fp8;              // e4m3 operands (K-major only)
  uint32_t fmt;         // instruction descriptor's operand format: fp16 0, bf16 1, e4m3 0
  int lanes;            // n: length of an output row
  long cols;            // m: output rows
  int l_tiles, c_tiles, splits;
  int kb_total, kb_per_split;  // k-blocks of 128 bytes: 64 16-bit or 128 8-bit elements
  int BN, stages, cluster;
  // kDenseForward: v = acc * ls[n] * cs[m] + bias[n]; z = v; out = act(v) + res
  const uint8_t *ls, *cs;
  const float* bias;
  int act;
  const void* res;
  void* z;
  uint8_t *zq, *zs;
  int zg;  // scale bytes a row of zq
  long ldr, ldz;
  // kDenseStore: out = acc (+ out): type T, or fp32 when out_f32; split s at out + s * split_stride
  int out_f32, accumulate;
  long split_stride;
  void* out;
  long ldo;
  int* err;
};

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

__device__ __forceinline__ float ld_shared_cluster_f32(uint32_t caddr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(caddr) : "memory");
  return v;
}

// ---------------------------------------------------------------- epilogue
// NC columns (output rows m0 ..) of one lane (output column n; off: n is past the row's end). Warp-collective
// (the 8-bit form of z takes a maximum over the warp's 32 lanes, which are one group).
template <typename T, int EPI, int NC>
__device__ __forceinline__ void dense_epilogue(const DenseGemmParams& p, float (&v)[NC], int n, long m0, int split,
                                               float lscale, float bias) {
  const int nc = static_cast<int>(p.cols - m0 < NC ? p.cols - m0 : NC);  // uniform
  const bool on = n < p.lanes;
  if constexpr (EPI == kDenseForward) {
    T res[NC];
    if (p.res) {
      const T* r = static_cast<const T*>(p.res) + m0 * p.ldr + n;
#pragma unroll
      for (int e = 0; e < NC; ++e)
        if (on && e < nc) res[e] = r[e * p.ldr];
    }
    if (p.ls) {
#pragma unroll
      for (int e = 0; e < NC; ++e) v[e] = e < nc ? v[e] * lscale * q8_scale(p.cs[m0 + e]) : 0.f;
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
      for (int e = 0; e < NC; ++e) v[e] = dense_act<decltype(act)::value>(v[e]);
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

// ---------------------------------------------------------------- operands
// One k-block of an operand's `rows` rows from row r0 into shared memory at dst. K-major: one box of 128
// bytes x rows. MN-major: panels of 64 rows (128 bytes) x 64 k, 8 KB each.
template <bool PAIR>
__device__ __forceinline__ void dense_load(const CUtensorMap* m, uint32_t dst, uint64_t* bar, uint32_t pbar, bool mn,
                                           int kelem, int r0, int rows) {
  if (mn) {
    for (int j = 0; j < rows; j += 64) {
      if (PAIR) tma_load_2d_pair(dst + j * 128, m, pbar, r0 + j, kelem);
      else tma_load_2d(dst + j * 128, m, bar, r0 + j, kelem);
    }
  } else {
    if (PAIR) tma_load_2d_pair(dst, m, pbar, kelem, r0);
    else tma_load_2d(dst, m, bar, kelem, r0);
  }
}
// The four MMAs of a k-block (32 bytes of k each: 16 16-bit or 32 8-bit elements).
template <bool PAIR>
__device__ __forceinline__ void dense_mma(const DenseGemmParams& p, uint32_t d, uint32_t l0, uint32_t c0,
                                          uint32_t idesc, bool first) {
  const uint32_t lstep = p.l_mn ? 2048u : 32u, cstep = p.c_mn ? 2048u : 32u;
  const uint32_t llbo = p.l_mn ? 8192u : 16u, clbo = p.c_mn ? 8192u : 16u;
#pragma unroll
  for (int kk = 0; kk < 4; ++kk) {
    const uint64_t a = sdesc_sw128(l0 + kk * lstep, llbo, 1024);
    const uint64_t b = sdesc_sw128(c0 + kk * cstep, clbo, 1024);
    const uint32_t acc = first && kk == 0 ? 0u : 1u;
    if (p.fp8) {
      if (PAIR) mma_f8_pair(d, a, b, idesc, acc);
      else mma_f8(d, a, b, idesc, acc);
    } else {
      if (PAIR) mma_bf16_pair(d, a, b, idesc, acc);
      else mma_bf16(d, a, b, idesc, acc);
    }
  }
}

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

template <typename T, int EPI>
__global__ void __launch_bounds__(kDenseThreads, 1) dense_pair_kernel(const __grid_constant__ DenseGemmParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int BN = p.BN, S = p.stages;
  const uint32_t l_bytes = 128 * 128, c_bytes = static_cast<uint32_t>(BN / 2) * 128;  // this CTA's halves
  const uint32_t stage_bytes = l_bytes + c_bytes;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + S * stage_bytes);
  uint64_t* empty = full + kDenseMaxStages;
  uint64_t* tfull = empty + kDenseMaxStages;
  uint64_t* tempty = tfull + 2;
  uint32_t* slot = reinterpret_cast<uint32_t*>(tempty + 2);
  const uint32_t sbase = smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  const int cid = static_cast<int>(blockIdx.x >> 1), ncl = static_cast<int>(gridDim.x >> 1);
  const int units = p.l_tiles * p.c_tiles * p.splits;
  const uint32_t tcols = tmem_cols_for(2 * BN);

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&tfull[b], 1);
      mbar_init(&tempty[b], 16);  // one arrival per epilogue warp of both CTAs
    }
    fence_mbar_init();
    tma_prefetch_desc(&p.tl);
    tma_prefetch_desc(&p.tc);
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
  pdl_entry();  // the set-up above runs under the end of the kernel before

  if (warp == 0) {
    if (lane == 0) {
      int s = 0;
      uint32_t par = 0;
      bool alive = true;
      const int kelems = p.fp8 ? 128 : 64;
      for (int u = cid; u < units && alive; u += ncl) {
        int lt, ct, split;
        dense_unit(p, u, lt, ct, split);
        const int kb0 = split * p.kb_per_split, kb1 = min(p.kb_total, kb0 + p.kb_per_split);
        const int lr = lt * 256 + static_cast<int>(rank) * 128, cr = ct * BN + static_cast<int>(rank) * (BN / 2);
        for (int kb = kb0; kb < kb1; ++kb) {
          if (!wait(&empty[s], par ^ 1, p.err, kSiteDenseEmpty)) {
            alive = false;
            break;
          }
          // both members' loads complete on the even CTA's barrier, which expects them all
          const uint32_t bar = mapa_shared(smem_u32(&full[s]), 0);
          if (leader) mbar_arrive_expect_tx(&full[s], 2 * stage_bytes);
          const uint32_t l0 = sbase + s * stage_bytes;
          dense_load<true>(&p.tl, l0, nullptr, bar, p.l_mn, kb * kelems, lr, 128);
          dense_load<true>(&p.tc, l0 + l_bytes, nullptr, bar, p.c_mn, kb * kelems, cr, BN / 2);
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
    if (lane == 0 && leader) {
      const uint32_t idesc = idesc_f32acc(256, BN, p.fmt, p.l_mn, p.c_mn);
      int s = 0, tc = 0;
      uint32_t par = 0;
      bool alive = true;
      for (int u = cid; u < units && alive; u += ncl, ++tc) {
        int lt, ct, split;
        dense_unit(p, u, lt, ct, split);
        const int kb0 = split * p.kb_per_split, kb1 = min(p.kb_total, kb0 + p.kb_per_split);
        const int buf = tc & 1;
        if (!wait(&tempty[buf], ((tc >> 1) & 1) ^ 1, p.err, kSiteDenseTEmpty)) break;
        tc_fence_after();
        for (int kb = kb0; kb < kb1; ++kb) {
          if (!wait(&full[s], par, p.err, kSiteDenseFull)) {
            alive = false;
            break;
          }
          tc_fence_after();
          const uint32_t l0 = sbase + s * stage_bytes;
          dense_mma<true>(p, tmem + buf * BN, l0, l0 + l_bytes, idesc, kb == kb0);
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
    // two warps per TMEM lane quarter, one per half of the columns
    const int q = warp & 3, half = (warp - 2) >> 2;
    int tc = 0;
    for (int u = cid; u < units; u += ncl, ++tc) {
      int lt, ct, split;
      dense_unit(p, u, lt, ct, split);
      const int n = lt * 256 + static_cast<int>(rank) * 128 + q * 32 + lane;
      float lscale = 1.f, bias = 0.f;
      if (EPI == kDenseForward && n < p.lanes) {
        if (p.ls) lscale = q8_scale(p.ls[n]);
        if (p.bias) bias = p.bias[n];
      }
      const int buf = tc & 1;
      int ok = 1;
      if (lane == 0) ok = wait(&tfull[buf], (tc >> 1) & 1, p.err, kSiteDenseTFull) ? 1 : 0;
      if (!__shfl_sync(0xffffffffu, ok, 0)) break;
      tc_fence_after();
      const uint32_t t0 = tmem + (static_cast<uint32_t>(q * 32) << 16) + buf * BN;
      for (int c = half * (BN / 2); c < (half + 1) * (BN / 2); c += 32) {
        const long m0 = static_cast<long>(ct) * BN + c;
        if (m0 >= p.cols) break;  // uniform
        uint32_t r[32];
        tmem_ld32(t0 + c, r);
        tmem_ld_wait32(r);
        float v[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) v[e] = __uint_as_float(r[e]);
        dense_epilogue<T, EPI, 32>(p, v, n, m0, split, lscale, bias);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (leader) mbar_arrive(&tempty[buf]);
        else mbar_arrive_cluster(mapa_shared(smem_u32(&tempty[buf]), 0));
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // no remote arrival or MMA write into this CTA is still in flight
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, tcols);
  }
}

template <typename T, int EPI>
__global__ void __launch_bounds__(kDenseThreads, 1) dense_cluster_kernel(const __grid_constant__ DenseGemmParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int BN = p.BN, S = p.stages, CL = p.cluster;
  const uint32_t l_bytes = 128 * 128, c_bytes = static_cast<uint32_t>(BN) * 128;
  const uint32_t stage_bytes = l_bytes + c_bytes;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + S * stage_bytes);
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
  tc_fence_after();
  const uint32_t tmem = *slot;
  pdl_entry();  // the set-up above runs under the end of the kernel before

  int lt, ct, split;
  dense_unit(p, static_cast<int>(blockIdx.x) / CL, lt, ct, split);
  // this CTA's share of the split's k-blocks (maybe none)
  const int s0 = split * p.kb_per_split, s1 = min(p.kb_total, s0 + p.kb_per_split);
  const int kb0 = s0 + static_cast<int>(static_cast<long>(s1 - s0) * rank / CL);
  const int kb1 = s0 + static_cast<int>(static_cast<long>(s1 - s0) * (rank + 1) / CL);

  if (warp == 0) {
    if (lane == 0) {
      int s = 0;
      uint32_t par = 0;
      const int kelems = p.fp8 ? 128 : 64;
      int kb = kb0;
      for (; kb < kb1; ++kb) {
        if (!wait(&empty[s], par ^ 1, p.err, kSiteDenseEmpty)) break;
        mbar_arrive_expect_tx(&full[s], stage_bytes);
        const uint32_t l0 = sbase + s * stage_bytes;
        dense_load<false>(&p.tl, l0, &full[s], 0u, p.l_mn, kb * kelems, lt * 128, 128);
        dense_load<false>(&p.tc, l0 + l_bytes, &full[s], 0u, p.c_mn, kb * kelems, ct * BN, BN);
        if (++s == S) {
          s = 0;
          par ^= 1;
        }
      }
      if (kb < kb1) {  // gave up: the copies of the stages before land before the CTA goes on
        for (int i = min(S, kb - kb0); i > 0; --i) {
          const int j = (kb - kb0) - i;
          (void)wait(&full[j % S], static_cast<uint32_t>(j / S) & 1u, p.err, kSiteDenseFull);
        }
      }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      const uint32_t idesc = idesc_f32acc(128, BN, p.fmt, p.l_mn, p.c_mn);
      int s = 0;
      uint32_t par = 0;
      for (int kb = kb0; kb < kb1; ++kb) {
        if (!wait(&full[s], par, p.err, kSiteDenseFull)) break;
        tc_fence_after();
        const uint32_t l0 = sbase + s * stage_bytes;
        dense_mma<false>(p, tmem, l0, l0 + l_bytes, idesc, kb == kb0);
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
    float lscale = 1.f, bias = 0.f;
    if (EPI == kDenseForward && CL == 1 && n < p.lanes) {
      if (p.ls) lscale = q8_scale(p.ls[n]);
      if (p.bias) bias = p.bias[n];
    }
    int ok = 1;
    if (lane == 0) ok = wait(tfull, 0, p.err, kSiteDenseTFull) ? 1 : 0;
    if (__shfl_sync(0xffffffffu, ok, 0)) {
      tc_fence_after();
      const uint32_t t0 = tmem + (static_cast<uint32_t>(q * 32) << 16);
      float* part = reinterpret_cast<float*>(smem);  // CL > 1: [BN][128] sums over the ring, which is drained
      for (int c = half * 16; c < BN; c += 32) {
        const long m0 = static_cast<long>(ct) * BN + c;
        if (m0 >= p.cols) break;  // uniform
        uint32_t r[16];
        tmem_ld16(t0 + c, r);
        tmem_ld_wait(r);
        float v[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) v[e] = kb1 > kb0 ? __uint_as_float(r[e]) : 0.f;
        if (CL == 1) {
          dense_epilogue<T, EPI, 16>(p, v, n, m0, split, lscale, bias);
        } else {
#pragma unroll
          for (int e = 0; e < 16; ++e) part[(c + e) * 128 + q * 32 + lane] = v[e];
        }
      }
    }
  }
  if (CL > 1) {
    __syncthreads();
    cluster_sync();  // every CTA's sums are written
    // jobs of 4 columns x 32 lanes, spread over the cluster's warps
    const int nc = static_cast<int>(min(static_cast<long>(BN), p.cols - static_cast<long>(ct) * BN));
    const int jobs = (nc + 3) / 4 * 4;
    for (int j = rank + CL * warp; j < jobs; j += CL * (kDenseThreads / 32)) {
      const int q = j & 3, c = (j >> 2) * 4;
      const int n = lt * 128 + q * 32 + lane;
      float lscale = 1.f, bias = 0.f;
      if (EPI == kDenseForward && n < p.lanes) {
        if (p.ls) lscale = q8_scale(p.ls[n]);
        if (p.bias) bias = p.bias[n];
      }
      float v[4] = {0.f, 0.f, 0.f, 0.f};
      const uint32_t off = sbase + static_cast<uint32_t>((c * 128 + q * 32 + lane) * 4);
#pragma unroll 4
      for (int k = 0; k < CL; ++k) {
        const uint32_t at = mapa_shared(off, static_cast<uint32_t>(k));
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] += ld_shared_cluster_f32(at + e * 512);
      }
      dense_epilogue<T, EPI, 4>(p, v, n, static_cast<long>(ct) * BN + c, split, lscale, bias);
    }
    __syncthreads();
    cluster_sync();  // nobody reads this CTA's sums any more
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, tcols);
  }
}

}  // namespace c2d
