// moe.cuh - a mixture-of-experts layer for a few tokens, as three kernels that run into one another (programmatic
// dependent launch):
//
//   route_kernel          logits x R^T, the k largest of each token's, their weights (softmax); with 8-bit experts
//                         also x in 8 bits, a scale for 128 columns
//   expert_kernel, up     h = act(x w1^T + b1) [* (x w3^T + b3)], one unit for each chosen expert and 128 of its
//                         inner features
//   expert_kernel, down   y = sum over the chosen experts of weight (h w2^T + b2), + residual, one unit for each
//                         128 output features
//
// What bounds it is reading each chosen expert's weights once. So the weights' rows are the tensor core's 128 lanes and
// the tokens its columns (16 to 64): every token is multiplied with every chosen expert, which costs nothing beside the
// weights' way from memory, and what a token did not choose is left out of its sums (the accumulator's columns do not
// touch each other, so an expert's infinities stay with the tokens that chose it). The loop over k is split over the
// CTAs of a cluster, which join their sums through distributed shared memory in rank order; a unit of the down product
// walks through the experts, a segment of k each, with two accumulators, so that one expert's sums are weighted and added
// in fp32 registers under the next one's MMAs. Sums have a fixed order: by rank, within a rank by expert.
//
// The down kernel's CTAs start beside the last of the up kernel's (two an SM: at most 113 KB of shared memory and 256
// columns of tensor memory each) and fill their rings with w2 while that ends. They take the routing from the kernel
// before the up kernel, which that one has waited for. An up CTA releases them only once it holds its own tensor memory:
// they keep theirs until the up kernel has ended.
//
// Clusters that each hold tensor memory on one SM and wait for it on another would wait for ever, so what runs on an SM at
// once must never want more than its 512 columns together. Registers see to that: these kernels take 72 to 96 a thread, so a
// third CTA does not fit, nor the dense layer's beside two; beside one there is room for one forward CTA of at most 128
// columns or two of the gradients' (the block-scaled ones and the pairs fill an SM by themselves), or of the conv layer's
// kernels for a weight gradient of 64 columns.
//
// Measured: 16 tokens, 8 experts of (4096, 8192), gated, bf16: 1.6 GB in 241 to 255 us, 0.92 to 0.98 of the copy rate. One
// token, 8 of 64 experts of (2048, 1024): 101 MB in 33 us, where memory takes 15: three starts of 3 to 4 us each (launch,
// routing, first copies) and as much for the joins. As one kernel, whose down CTAs waited for counters that the up CTAs
// raised, 35 us (255 and 241 in the first case): the fences and the waiting took longer than the end of a kernel.
#pragma once
#include "dense_gemm.cuh"

namespace c2d {

constexpr int kMoeTokens = 64, kMoeExperts = 256, kMoeChosen = 16;
constexpr int kMoeThreads = 320;  // TMA warp, MMA warp, 8 epilogue warps; one more for the scales of blocks
constexpr int kMoeMaxStages = 8;
constexpr int kRouteThreads = 512, kRouteWarps = kRouteThreads / 32, kRouteCluster = 8;
enum : int { kSiteMoeFull = 16, kSiteMoeEmpty = 17, kSiteMoeTFull = 18, kSiteMoeTEmpty = 19 };

struct RouteParams {
  const void *x, *router;
  long ldx, ldr;
  int T, D, E, k, normalize;
  int32_t* experts;
  float* weights;
  uint8_t *xq, *xs;  // 8-bit form of x (null: none), rows of ldq bytes
  long ldq;
};

struct ExpertParams {
  CUtensorMap tl, tc;  // weights (rows are lanes) and tokens (rows are columns)
  DenseScales sl, sc;
  uint32_t fmt;
  int T, BN, E, k;
  int rows;      // rows of an expert's weights: F or 2 F (up), D (down)
  int second;    // up, gated: rows from a gate's row to its factor's
  int width;     // output features: F (up), D (down)
  int tiles;     // of 128 of them
  int kb_total;  // k-blocks of an expert
  int stages, cluster, act;
  const int32_t* experts;  // [T][k]
  const float* weights;    // [T][k]
  const float* bias;       // [E][rows], may be null
  // up: h [slots][T][F] in T or as e4m3 with a scale for 128 columns
  void* h;
  uint8_t *hq, *hs;
  // down
  const void* res;
  void* y;
  long ldres, ldy;
  int* err;
};

// ---------------------------------------------------------------- routing
// A logit's bits, ordered as the numbers are: NaN above all, both zeros equal. Never 0.
__device__ __forceinline__ uint32_t logit_key(float v) {
  if (v != v) return 0xffffffffu;
  const uint32_t b = __float_as_uint(v + 0.f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

// A cluster of eight CTAs takes NT tokens: each CTA an eighth of the experts, a warp two of them at a time (or a slice of
// their columns), for all NT tokens; token i's logits are gathered by CTA i, whose first warp chooses while the others
// bring the token to 8 bits. Bound by latency (two passes through memory and a cluster's meeting), so the tokens are spread
// over as many clusters as run at once (8 tokens, 128 experts of 4096: 64 us with eight tokens a cluster).
template <typename T, typename R, int NT>
__global__ void __launch_bounds__(kRouteThreads) route_kernel(const RouteParams p) {
  __shared__ float logits[kMoeExperts];
  __shared__ float part[kRouteWarps][2][NT];
  pdl_entry();
  pdl_release();
  cluster_arrive();  // waited for before the other CTAs' shared memory is written
  const int rank = static_cast<int>(cluster_ctarank()), t0 = static_cast<int>(blockIdx.x) / kRouteCluster * NT;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int mine = rank < p.E ? (p.E - rank + kRouteCluster - 1) / kRouteCluster : 0;  // experts rank, rank + 8, ...
  const int pairs = (mine + 1) / 2;
  const int slices = pairs >= kRouteWarps || pairs == 0 ? 1 : kRouteWarps / pairs;
  const int nv = p.D / 8;
  auto send = [&](int t, int e, float v) {
    const uint32_t at = mapa_shared(smem_u32(&logits[e]), static_cast<uint32_t>(t));
    st_shared_cluster_f32(at, v);
  };
  bool started = false;  // the other CTAs
  for (int pair = slices > 1 ? warp % pairs : warp; pair < pairs; pair += slices > 1 ? pairs : kRouteWarps) {
    const int slice = slices > 1 ? warp / pairs : 0;
    if (slice >= slices) break;
    const int e0 = rank + 2 * pair * kRouteCluster, e1 = min(e0 + kRouteCluster, p.E - 1);
    const R* r0 = static_cast<const R*>(p.router) + e0 * p.ldr;
    const R* r1 = static_cast<const R*>(p.router) + e1 * p.ldr;
    const T* x = static_cast<const T*>(p.x) + t0 * p.ldx;
    float acc[2][NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) acc[0][t] = acc[1][t] = 0.f;
#pragma unroll(NT >= 4 ? 2 : 4)
    for (int v = slice * 32 + lane; v < nv; v += 32 * slices) {
      float w[2][8];
      if constexpr (sizeof(R) == 4) {
#pragma unroll
        for (int i = 0; i < 8; i += 4) {
          *reinterpret_cast<float4*>(w[0] + i) = *reinterpret_cast<const float4*>(r0 + v * 8 + i);
          *reinterpret_cast<float4*>(w[1] + i) = *reinterpret_cast<const float4*>(r1 + v * 8 + i);
        }
      } else {
        R a[8], b[8];
        *reinterpret_cast<uint4*>(a) = *reinterpret_cast<const uint4*>(r0 + v * 8);
        *reinterpret_cast<uint4*>(b) = *reinterpret_cast<const uint4*>(r1 + v * 8);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          w[0][i] = to_f(a[i]);
          w[1][i] = to_f(b[i]);
        }
      }
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        if (t0 + t >= p.T) break;  // uniform
        T e[8];
        *reinterpret_cast<uint4*>(e) = *reinterpret_cast<const uint4*>(x + t * p.ldx + v * 8);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          acc[0][t] = fmaf(to_f(e[i]), w[0][i], acc[0][t]);
          acc[1][t] = fmaf(to_f(e[i]), w[1][i], acc[1][t]);
        }
      }
    }
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int o = 16; o; o >>= 1) acc[i][t] += __shfl_xor_sync(0xffffffffu, acc[i][t], o);
    if (slices > 1) {
      if (lane == 0)
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          part[warp][0][t] = acc[0][t];
          part[warp][1][t] = acc[1][t];
        }
      break;
    }
    if (!started) cluster_wait();
    started = true;
    if (lane < NT) {
#pragma unroll
      for (int t = 0; t < NT; ++t)
        if (lane == t) {
          send(t, e0, acc[0][t]);
          if (e0 + kRouteCluster < p.E) send(t, e0 + kRouteCluster, acc[1][t]);
        }
    }
  }
  __syncwarp();
  if (!started) cluster_wait();
  if (slices > 1) {  // the same for the whole CTA
    __syncthreads();
    for (int i = threadIdx.x; i < pairs * 2 * NT; i += kRouteThreads) {
      const int t = i % NT, half = i / NT % 2, pair = i / NT / 2, e = rank + (2 * pair + half) * kRouteCluster;
      float v = 0.f;
      for (int s = 0; s < slices; ++s) v += part[s * pairs + pair][half][t];
      if (e < p.E) send(t, e, v);
    }
  }
  cluster_sync();  // all logits are where they belong; from here on a CTA reads its own shared memory only
  const int t = t0 + rank;
  if (rank >= NT || t >= p.T) return;
  if (warp == 0) {
    uint32_t key[kMoeExperts / 32];
#pragma unroll
    for (int i = 0; i < kMoeExperts / 32; ++i) key[i] = lane + 32 * i < p.E ? logit_key(logits[lane + 32 * i]) : 0u;
    float chosen = 0.f, top = 0.f;
    int index = 0;
    for (int j = 0; j < p.k; ++j) {
      uint32_t best = 0u;
#pragma unroll
      for (int i = 0; i < kMoeExperts / 32; ++i) {
        if (32 * i >= p.E) break;  // uniform
        best = max(best, key[i]);
      }
      best = __reduce_max_sync(0xffffffffu, best);
      int at = kMoeExperts;
#pragma unroll
      for (int i = kMoeExperts / 32 - 1; i >= 0; --i)
        if (key[i] == best) at = lane + 32 * i;
      at = __reduce_min_sync(0xffffffffu, at);  // of equal ones the lowest
#pragma unroll
      for (int i = 0; i < kMoeExperts / 32; ++i)
        if (lane + 32 * i == at) key[i] = 0u;
      const float v = logits[at];
      if (j == 0) top = v;
      if (lane == j) {
        chosen = v;
        index = at;
      }
    }
    const float e = lane < p.k ? expf(chosen - top) : 0.f;
    float sum = e;
    if (!p.normalize) {
      sum = 0.f;
      for (int i = lane; i < p.E; i += 32) sum += expf(logits[i] - top);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane < p.k) {
      p.experts[t * p.k + lane] = index;
      p.weights[t * p.k + lane] = e / sum;
    }
  }
  if (p.xq) {
    const T* x = static_cast<const T*>(p.x) + t * p.ldx;
    const int groups = (p.D + 127) / 128;
    for (int g = warp; g < groups; g += kRouteThreads / 32) {
      const int c = g * 128 + lane * 4;
      float v[4] = {0.f, 0.f, 0.f, 0.f};
      if (c < p.D) {  // columns come in eights
        T e[4];
        *reinterpret_cast<uint2*>(e) = *reinterpret_cast<const uint2*>(x + c);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = to_f(e[i]);
      }
      uint32_t m = 0u;
#pragma unroll
      for (int i = 0; i < 4; ++i) m = max(m, finite_bits(v[i]));
      const uint32_t byte = q8_scale_byte(__reduce_max_sync(0xffffffffu, m));
      if (c < p.D) q8_store<4>(p.xq + t * p.ldq + c, v, q8_inv_scale(byte), false);
      if (lane == 0) p.xs[static_cast<long>(t) * groups + g] = static_cast<uint8_t>(byte);
    }
  }
}

// ---------------------------------------------------------------- experts' products
// A segment of a CTA's work: k-blocks kb0 .. kb1 - 1 of features f0 .. of the slot'th chosen expert.
struct Segment {
  int slot, f0, kb0, kb1;
};

// Bytes of a stage, of the scales' two sets and of the joined sums (in the ring's place, once it is free).
__host__ __device__ constexpr int moe_stage_bytes(int L, int BN) { return L * 16384 + BN * 128; }
__host__ __device__ constexpr int moe_slot_bytes(int L) { return 512 * (L + 1); }
constexpr int kMoeGroups = 2, kMoeSet = 4 * kMoeGroups;  // k-blocks of a set of scales: three stages fit beside its slots
__host__ __device__ constexpr int moe_slots_bytes(int L) { return 2 * kMoeGroups * moe_slot_bytes(L); }
__host__ __device__ constexpr int moe_join_bytes(int L, int BN, int cluster) {
  return cluster > 1 ? L * cluster * dense_own_cols(BN, cluster) * 512 : 0;
}
// Accumulators: two where a CTA has several segments, as far as 256 columns of tensor memory allow (two CTAs an SM).
__host__ __device__ constexpr int moe_buffers(bool up, int L, int BN, int cluster, int q) {
  return (up && cluster > 1) || (q == kBlockScaled && L * BN > 64) ? 1 : 2;
}
// Barriers (512 bytes), routing tables (down: gates too) and what the epilogue's warps tell each other.
__host__ __device__ constexpr int moe_fixed_bytes(bool up) {
  return 512 + kMoeTokens * kMoeChosen * (up ? 2 : 6) + kMoeExperts * 2 + 256;
}

template <typename T, bool UP, int L, int Q>
__global__ void __launch_bounds__(kMoeThreads + dense_scale_threads(Q), 2) expert_kernel(const __grid_constant__ ExpertParams p) {
  static_assert(UP || L == 1, "the down product has one matrix");
  constexpr bool BYTES = Q != kHalves;
  constexpr int kElems = BYTES ? 128 : 64;  // of k a k-block
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int BN = p.BN, S = p.stages, CL = p.cluster;
  const uint32_t stage_bytes = moe_stage_bytes(L, BN);
  const uint32_t slots = S * stage_bytes;  // the scales' two sets
  uint8_t* fixed = smem + slots + (Q == kBlockScaled ? moe_slots_bytes(L) : 0);
  uint64_t* full = reinterpret_cast<uint64_t*>(fixed);
  uint64_t* empty = full + kMoeMaxStages;
  uint64_t* tfull = empty + kMoeMaxStages;
  uint64_t* tempty = tfull + 2;
  uint64_t* sfull = tempty + 2;
  uint64_t* sempty = sfull + 2;
  uint32_t* tslot = reinterpret_cast<uint32_t*>(sempty + 2);
  uint32_t* mask = tslot + 1;              // chosen experts, one bit each
  float* gate = reinterpret_cast<float*>(fixed + 512);                                               // down: [T][k]
  int16_t* slot_of_choice = reinterpret_cast<int16_t*>(gate + (UP ? 0 : kMoeTokens * kMoeChosen));  // [T][k]
  int16_t* list = slot_of_choice + kMoeTokens * kMoeChosen;                         // chosen experts in order
  uint32_t* group_max = reinterpret_cast<uint32_t*>(list + kMoeExperts);            // [2][2][4][4]
  const uint32_t sbase = smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = CL > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int buffers = moe_buffers(UP, L, BN, CL, Q);
  const uint32_t tcols = tmem_cols_for(buffers * L * BN + (Q == kBlockScaled ? S * 4 * (L + 1) : 0));

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&tfull[b], 1);
      mbar_init(&tempty[b], 8);  // one arrival per epilogue warp
      mbar_init(&sfull[b], 1);
      mbar_init(&sempty[b], 1);
    }
    fence_mbar_init();
    tma_prefetch_desc(&p.tl);
    tma_prefetch_desc(&p.tc);
  }
  if (threadIdx.x < 8) mask[threadIdx.x] = 0u;
  // The down kernel reads the routing without waiting for the up kernel, which has waited for the one that wrote it.
  if (UP) pdl_entry();
  const int choices = p.T * p.k;
  // the first choice of each thread stays in a register (there are more than threads only from 20 tokens on)
  const int tid = static_cast<int>(threadIdx.x);
  const int choice = tid < choices ? __ldcg(p.experts + tid) : -1;
  const float weight = !UP && tid < choices ? __ldcg(p.weights + tid) : 0.f;
  if (warp == 1) {
    tmem_alloc(tslot, tcols);
    tmem_relinquish();
  }
  __syncthreads();
  auto each_choice = [&](auto&& f) {
    if (tid < choices) f(tid, choice, weight);
    for (int i = tid + static_cast<int>(blockDim.x); i < choices; i += blockDim.x)
      f(i, __ldcg(p.experts + i), UP ? 0.f : __ldcg(p.weights + i));
  };
  each_choice([&](int, int e, float) { atomicOr(&mask[e >> 5], 1u << (e & 31)); });
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tslot;
  int n = 0;  // chosen experts
#pragma unroll
  for (int i = 0; i < 8; ++i) n += __popc(mask[i]);
  // Units: tiles of the chosen experts (up), of the output (down). A CTA of its own takes one after the other (up), a
  // cluster one.
  const int unit0 = static_cast<int>(blockIdx.x) / CL, units = UP ? n * p.tiles : p.tiles;
  if (UP && unit0 >= units) {  // the whole cluster
    if (warp == 1) tmem_dealloc(tmem, tcols);
    return;
  }
  each_choice([&](int i, int e, float w) {
    // its order among the chosen ones
    int r = __popc(mask[e >> 5] & ((1u << (e & 31)) - 1u));
    for (int m = 0; m < e >> 5; ++m) r += __popc(mask[m]);
    list[r] = static_cast<int16_t>(e);  // by each token that chose it, the same
    slot_of_choice[i] = static_cast<int16_t>(r);
    if (!UP) gate[i] = w;
  });
  __syncthreads();
  // Not before the tensor memory is taken: the down kernel's CTAs hold theirs until this kernel has ended.
  if (UP) pdl_release();

  // This CTA's segments: units' k-blocks (up), or its share of all chosen experts' (down). In 32 bits (at most 256 experts
  // of 2^24 / 64 k-blocks between eight CTAs, E F at most 2^29; a cluster has a power of two of CTAs), because the first copies wait for this.
  const bool many = UP && CL == 1;
  const uint32_t all = UP ? p.kb_total : static_cast<uint32_t>(n) * p.kb_total, share = 31 - __clz(CL);
  const int g0 = static_cast<int>(all * rank >> share), g1 = static_cast<int>(all * (rank + 1) >> share);
  const int slot0 = UP ? 0 : g0 / p.kb_total;
  int segments = g1 > g0 ? 1 : 0;
  if (many) segments = (units - unit0 + static_cast<int>(gridDim.x) - 1) / static_cast<int>(gridDim.x);
  if (!UP && g1 > g0) segments = (g1 - 1) / p.kb_total - slot0 + 1;
  const int blocks = many ? segments * p.kb_total : g1 - g0;  // k-blocks of this CTA
  auto segment = [&](int i) {
    Segment w;
    if constexpr (UP) {
      const int u = unit0 + i * static_cast<int>(gridDim.x);
      w.slot = u / p.tiles;
      w.f0 = (u - w.slot * p.tiles) * 128;
      w.kb0 = g0;
      w.kb1 = g1;
    } else {
      w.slot = slot0 + i;
      const int base = w.slot * p.kb_total;
      w.kb0 = max(g0 - base, 0);
      w.kb1 = min(g1 - base, p.kb_total);
      w.f0 = unit0 * 128;
    }
    return w;
  };
  auto lane_row = [&](const Segment& w) { return list[w.slot] * p.rows + w.f0; };  // of the first matrix
  auto column_row = [&](const Segment& w) { return UP ? 0 : w.slot * p.T; };

  if (Q == kBlockScaled && warp == kMoeThreads / 32) {
    // The scales' warp (see scales_store): sets of eight k-blocks, two ahead of the MMAs, the next one's words on their way.
    int b = 0, i = 0, j = 0;
    uint32_t par = 0, words[4 * L + 2][kMoeGroups];
    Segment w = segment(0);
    auto weights = [&] {
#pragma unroll
      for (int l = 0; l < L; ++l) lane_words<kMoeGroups>(p.sl, lane_row(w) + l * p.second, j, p.kb_total, words + 4 * l, lane);
    };
    auto tokens = [&] {
#pragma unroll
      for (int r = 0; r < 2; ++r)
        if (32 * r < BN) scale_words<kMoeGroups>(p.sc, column_row(w) + lane + 32 * r, j, p.kb_total, words[4 * L + r]);
    };
#pragma unroll
    for (int g = 0; g < kMoeGroups; ++g) words[4 * L + 1][g] = 0x7f7f7f7fu;
    j = w.kb0 / kMoeSet;
    if (segments > 0) weights();
    if (!UP) pdl_entry();  // h's scales
    if (segments > 0) tokens();
    while (i < segments) {
      int ok = 1;
      if (lane == 0) ok = wait(&sempty[b], par ^ 1, p.err, kSiteMoeEmpty) ? 1 : 0;
      if (!__shfl_sync(0xffffffffu, ok, 0)) break;
#pragma unroll
      for (int g = 0; g < kMoeGroups; ++g) {
        const uint32_t slot = sbase + slots + b * (moe_slots_bytes(L) / 2) + g * moe_slot_bytes(L) + lane * 16;
#pragma unroll
        for (int l = 0; l < L; ++l)
          st_shared_v4(slot + 512 * l, words[4 * l][g], words[4 * l + 1][g], words[4 * l + 2][g], words[4 * l + 3][g]);
        st_shared_v4(slot + 512 * L, words[4 * L][g], words[4 * L + 1][g], 0x7f7f7f7fu, 0x7f7f7f7fu);
      }
      fence_proxy_async_smem();  // they are read by tcgen05.cp
      __syncwarp();
      if (lane == 0) mbar_arrive(&sfull[b]);
      b ^= 1;
      if (b == 0) par ^= 1;
      if (++j * kMoeSet >= w.kb1) {
        if (++i >= segments) break;
        w = segment(i);
        j = w.kb0 / kMoeSet;
      }
      weights();
      tokens();
    }
    __syncwarp();
  } else if (warp == 0) {
    if (elect_one()) {
      int s = 0;
      uint32_t par = 0;
      auto lanes = [&](const Segment& w, int kb, int st) {
        mbar_arrive_expect_tx(&full[st], stage_bytes);
#pragma unroll
        for (int l = 0; l < L; ++l)
          tma_load_2d(sbase + st * stage_bytes + l * 16384, &p.tl, &full[st], kb * kElems, lane_row(w) + l * p.second);
      };
      auto columns = [&](const Segment& w, int kb, int st) {
        tma_load_2d(sbase + st * stage_bytes + L * 16384, &p.tc, &full[st], kb * kElems, column_row(w));
      };
      // The ring's first round: the weights, then (down: once the up kernel has ended) the tokens.
      int i = 0, kb = 0;
      const int first = min(S, blocks);
      for (int pass = 0; pass < 2; ++pass) {
        if (pass == 1 && !UP) pdl_entry();
        i = 0;
        Segment w = segment(0);
        kb = w.kb0;
        for (int st = 0; st < first; ++st) {
          if (pass == 0) lanes(w, kb, st);
          else columns(w, kb, st);
          if (++kb == w.kb1 && ++i < segments) {
            w = segment(i);
            kb = w.kb0;
          }
        }
      }
      if (first == S) par = 1;
      else s = first;
      bool alive = blocks > first;
      int done = first;
      while (alive) {
        const Segment w = segment(i);
        for (; kb < w.kb1; ++kb) {
          if (!wait(&empty[s], par ^ 1, p.err, kSiteMoeEmpty)) {
            alive = false;
            break;
          }
          lanes(w, kb, s);
          columns(w, kb, s);
          ++done;
          if (++s == S) {
            s = 0;
            par ^= 1;
          }
        }
        if (alive && ++i < segments) kb = segment(i).kb0;
        else if (alive) break;
      }
      if (!alive && blocks > first)  // gave up: the copies of the stages before land before the CTA goes on
        for (int j = max(0, done - S); j < done; ++j)
          (void)wait(&full[j % S], static_cast<uint32_t>(j / S) & 1u, p.err, kSiteMoeFull);
    }
  } else if (warp == 1) {
    if (elect_one()) {
      const uint32_t idesc = Q == kBlockScaled ? idesc_block(128, BN, false, false) : idesc_f32acc(128, BN, p.fmt, false, false);
      const uint64_t l = dense_desc<false, BYTES>(sbase), c = dense_desc<false, BYTES>(sbase + L * 16384);
      [[maybe_unused]] uint32_t sf = 0, sb = 0, spar = 0;
      [[maybe_unused]] ScalePlaces places = {static_cast<uint32_t>(S), 0};
      int s = 0;
      uint32_t par = 0;
      bool alive = true;
      for (int i = 0; alive && i < segments; ++i) {
        const Segment w = segment(i);
        const int buf = buffers == 2 ? i & 1 : 0, round = buffers == 2 ? i >> 1 : i;
        if (!wait(&tempty[buf], (round & 1) ^ 1, p.err, kSiteMoeTEmpty)) break;
        tc_fence_after();
        for (int kb = w.kb0; kb < w.kb1; ++kb) {
          if (!wait(&full[s], par, p.err, kSiteMoeFull) ||
              (Q == kBlockScaled && set_begins<kMoeSet>(kb, w.kb0) && !wait(&sfull[sb], spar, p.err, kSiteMoeFull))) {
            alive = false;
            break;
          }
          tc_fence_after();
          const uint32_t acc = kb > w.kb0, d = tmem + buf * L * BN;
          if constexpr (Q == kBlockScaled) {
            if (scales_begin(kb, w.kb0)) {
              sf = tmem + buffers * L * BN + places.next() * 4 * (L + 1);
              const uint32_t slot = sbase + slots + sb * (moe_slots_bytes(L) / 2) + (kb % kMoeSet / 4) * moe_slot_bytes(L);
#pragma unroll
              for (int m = 0; m <= L; ++m) tmem_copy_scales<false>(sf + 4 * m, scales_desc(slot + 512 * m));
            }
            const uint32_t byte = kb & 3, id = idesc | byte << 4 | byte << 29;
#pragma unroll
            for (int m = 0; m < L; ++m)
              dense_mma<false, Q, false, false>(l + m * 1024, c, d + m * BN, s * stage_bytes, id, acc, sf + 4 * m, sf + 4 * L);
            if (set_ends<kMoeSet>(kb, w.kb1)) {
              mma_commit(&sempty[sb]);
              sb ^= 1;
              if (sb == 0) spar ^= 1;
            }
          } else {
#pragma unroll
            for (int m = 0; m < L; ++m)
              dense_mma<false, Q, false, false>(l + m * 1024, c, d + m * BN, s * stage_bytes, idesc, acc);
          }
          mma_commit(&empty[s]);
          if (++s == S) {
            s = 0;
            par ^= 1;
          }
        }
        if (alive) mma_commit(&tfull[buf]);
      }
    }
  }

  // ---------------- epilogue: warps 2 .. 9, two groups of 128 lanes
  const int q = warp & 3, group = (warp - 2) >> 2;
  const bool epilogue = warp >= 2 && warp < kMoeThreads / 32;
  const int feature = unit0 * 128 + q * 32 + lane;  // down
  const bool on = feature < p.width;
  const uint32_t t0 = tmem + (static_cast<uint32_t>(q * 32) << 16);
  int ok = 1;
  float v[UP ? 1 : 2][16];

  // Up: four tokens' sums of one feature a thread (m0 ..): bias, activation, factor, 16 or 8 bits; for the tokens that
  // chose the expert. Collective over a group (the 8-bit form takes a maximum over its 128 features).
  [[maybe_unused]] int flip = 0;
  [[maybe_unused]] auto up_finish = [&](const Segment& w, float (&a)[4], float (&b)[4], int m0) {
    const int feature = w.f0 + q * 32 + lane;
    const bool on = feature < p.width;
    // lanes 0 .. 3 look whether their token is among those
    bool mine = false;
    if (lane < 4 && m0 + lane < p.T)
      for (int j = 0; j < p.k; ++j) mine |= slot_of_choice[(m0 + lane) * p.k + j] == w.slot;
    const uint32_t chose = __ballot_sync(0xffffffffu, mine);
    const float* bias = p.bias ? p.bias + static_cast<long>(list[w.slot]) * p.rows + feature : nullptr;
    if (bias && on) {
      const float b1 = bias[0], b3 = L == 2 ? bias[p.second] : 0.f;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        a[e] += b1;
        if (L == 2) b[e] += b3;
      }
    }
    with_dense_act(p.act, [&](auto act) {
#pragma unroll
      for (int e = 0; e < 4; e += 2) {
        const float2 o = dense_act<decltype(act)::value>(make_float2(a[e], a[e + 1]));
        a[e] = o.x;
        a[e + 1] = o.y;
      }
    });
    if (L == 2) {
#pragma unroll
      for (int e = 0; e < 4; ++e) a[e] *= b[e];
    }
    [[maybe_unused]] uint32_t top[4];
    if constexpr (Q == kBlockScaled) {
      uint32_t* box = group_max + (group * 2 + flip) * 16;  // two, in turn: one meeting a call
      flip ^= 1;
#pragma unroll
      for (int e = 0; e < 4; ++e) top[e] = __reduce_max_sync(0xffffffffu, on ? finite_bits(a[e]) : 0u);
      if (lane < 4) box[lane * 4 + q] = lane == 0 ? top[0] : lane == 1 ? top[1] : lane == 2 ? top[2] : top[3];
      named_bar_sync(1 + group, 128);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint4 m = *reinterpret_cast<const uint4*>(box + e * 4);
        top[e] = max(max(m.x, m.y), max(m.z, m.w));
      }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (!(chose >> e & 1u)) continue;
      const long row = static_cast<long>(w.slot) * p.T + m0 + e;
      if constexpr (Q == kBlockScaled) {
        const uint32_t byte = q8_scale_byte(top[e]);
        if (on) p.hq[row * p.width + feature] = static_cast<uint8_t>(q8_pack2(a[e] * q8_inv_scale(byte), 0.f));
        if (q == 0 && lane == 0) p.hs[row * p.tiles + w.f0 / 128] = static_cast<uint8_t>(byte);
      } else {
        if (on) static_cast<T*>(p.h)[row * p.width + feature] = from_f<T>(a[e]);
      }
    }
  };
  // Down: the chosen experts' biases, the residual.
  [[maybe_unused]] auto down_finish = [&](float a, int t) {
    if (!on || t >= p.T) return;
    if (p.bias)
      for (int j = 0; j < p.k; ++j)
        a = fmaf(gate[t * p.k + j], p.bias[static_cast<long>(list[slot_of_choice[t * p.k + j]]) * p.rows + feature], a);
    if (p.res) a += to_f(static_cast<const T*>(p.res)[t * p.ldres + feature]);
    static_cast<T*>(p.y)[t * p.ldy + feature] = from_f<T>(a);
  };

  if (epilogue) {
    if constexpr (UP) {
      // (A wait that ran out leaves garbage and its mark: a group's warps go on together.)
      if (CL > 1) {
        if (segments > 0 && lane == 0) (void)wait(&tfull[0], 0, p.err, kSiteMoeTFull);
        __syncwarp();
        tc_fence_after();
      }
      for (int i = 0; CL == 1 && i < segments; ++i) {
        const Segment w = segment(i);
        const int buf = buffers == 2 ? i & 1 : 0, round = buffers == 2 ? i >> 1 : i;
        if (lane == 0) (void)wait(&tfull[buf], round & 1, p.err, kSiteMoeTFull);
        __syncwarp();
        tc_fence_after();
#pragma unroll 1
        for (int c = group * 16; c < BN && c < p.T; c += 32) {
          uint32_t r[L][16];
#pragma unroll
          for (int m = 0; m < L; ++m) {
            tmem_ld16(t0 + (buf * L + m) * BN + c, r[m]);
            tmem_ld_wait(r[m]);
          }
#pragma unroll
          for (int e = 0; e < 16; e += 4) {
            if (c + e >= p.T) break;  // uniform
            float o[L][4];
#pragma unroll
            for (int m = 0; m < L; ++m)
#pragma unroll
              for (int j = 0; j < 4; ++j) o[m][j] = __uint_as_float(r[m][e + j]);
            up_finish(w, o[0], o[L - 1], c + e);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&tempty[buf]);
      }
    } else {
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int e = 0; e < 16; ++e) v[j][e] = 0.f;
      for (int i = 0; i < segments && ok; ++i) {
        const int buf = i & 1, slot = segment(i).slot;  // two accumulators
        if (lane == 0) ok = wait(&tfull[buf], (i >> 1) & 1, p.err, kSiteMoeTFull) ? 1 : 0;
        ok = __shfl_sync(0xffffffffu, ok, 0);
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int c = group * 16 + 32 * j;
          if (c >= BN || c >= p.T) break;  // uniform
          // lane e has the weight of token c + e for this expert; below zero: not chosen
          float g = -1.f;
          const int t = c + (lane & 15);
          if (t < p.T)
            for (int m = 0; m < p.k; ++m)
              if (slot_of_choice[t * p.k + m] == slot) g = gate[t * p.k + m];
          uint32_t r[16];
          tmem_ld16(t0 + buf * BN + c, r);
          tmem_ld_wait(r);
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const float w = __shfl_sync(0xffffffffu, g, e);
            if (!(w < 0.f)) v[j][e] = fmaf(w, __uint_as_float(r[e]), v[j][e]);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&tempty[buf]);
      }
      pdl_release();
    }
  }
  if (!UP) pdl_entry();  // y may lie where the up kernel reads

  // The sums of a group's columns c .. c + 15 of matrix m.
  auto sums = [&](int j, int c, int m, float (&o)[16]) {
    if constexpr (UP) {
      uint32_t r[16];
      tmem_ld16(t0 + m * BN + c, r);
      tmem_ld_wait(r);
#pragma unroll
      for (int e = 0; e < 16; ++e) o[e] = segments > 0 ? __uint_as_float(r[e]) : 0.f;
    } else {
#pragma unroll
      for (int e = 0; e < 16; ++e) o[e] = v[UP ? 0 : j][e];
    }
  };
  if (CL == 1) {
    if (!UP && epilogue) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int c = group * 16 + 32 * j;
        if (c >= BN || c >= p.T) break;  // uniform
        float o[16];
        sums(j, c, 0, o);
#pragma unroll
        for (int e = 0; e < 16; ++e) down_finish(o[e], c + e);
      }
    }
  } else {
    // The ring's place takes the sums that the cluster's CTAs hand this one, [matrix][CL][own_cols][128], once every CTA's
    // MMAs are done with theirs; columns are owned four at a time in turn.
    const int own_cols = dense_own_cols(BN, CL);
    __syncwarp();
    cluster_sync();
    if (epilogue) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int c = group * 16 + 32 * j;
        if (c >= BN || c >= p.T) break;  // uniform
#pragma unroll
        for (int m = 0; m < L; ++m) {
          float o[16];
          sums(j, c, m, o);
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            const int quad = c / 4 + g;
            if (quad * 4 >= p.T) break;  // uniform
            const uint32_t at = sbase + static_cast<uint32_t>((((m * CL + rank) * own_cols + quad / CL * 4) * 128 + q * 32 + lane) * 4);
            const uint32_t to = mapa_shared(at, static_cast<uint32_t>(quad % CL));
#pragma unroll
            for (int e = 0; e < 4; ++e) st_shared_cluster_f32(to + e * 512, o[4 * g + e]);
          }
        }
      }
    }
    __syncwarp();
    cluster_sync();  // every CTA's sums have arrived; from here on a CTA reads its own shared memory only
    if (epilogue) {
      const int quads = (p.T + 3) / 4, own = quads > rank ? (quads - rank + CL - 1) / CL : 0;
      for (int i = group; i < own; i += 2) {
        float o[L][4];
#pragma unroll
        for (int m = 0; m < L; ++m) {
#pragma unroll
          for (int e = 0; e < 4; ++e) o[m][e] = 0.f;
          const uint32_t at = sbase + static_cast<uint32_t>(((m * CL * own_cols + i * 4) * 128 + q * 32 + lane) * 4);
#pragma unroll 4
          for (int r = 0; r < CL; ++r)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[m][e] += ld_shared_f32(at + static_cast<uint32_t>((r * own_cols + e) * 512));
        }
        const int m0 = (i * CL + rank) * 4;
        if constexpr (UP) {
          up_finish(segment(0), o[0], o[L - 1], m0);
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) down_finish(o[0][e], m0 + e);
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, tcols);
  }
}

}  // namespace c2d
