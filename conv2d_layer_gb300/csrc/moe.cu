// moe.cu - the mixture-of-experts layer's C entry points: validation, plan,
// tensor maps and the three launches (moe.cuh).
#include <algorithm>
#include <atomic>
#include <climits>
#include <cmath>

#include "conv2d.h"
#include "dense.h"
#include "host.h"
#include "kernels.h"
#include "moe.cuh"

using namespace c2d;

namespace {

long ceil_div(long a, long b) { return (a + b - 1) / b; }
bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
long ld_of(const conv2d_mat* m, int cols) { return m->ld ? m->ld : cols; }

constexpr size_t kMoeSmem = 113 * 1024;  // two CTAs an SM

int check_desc(const conv2d_moe_desc* d) {
  if (!d || d->T < 0 || d->D < 1 || d->F < 1 || d->E < 1 || d->k < 1 || d->k > d->E || d->act < 0 ||
      d->act > CONV2D_ACT_SILU || (d->dtype != CONV2D_BF16 && d->dtype != CONV2D_FP16))
    return CONV2D_ERR_INVALID_ARG;
  if (d->T > kMoeTokens || d->E > kMoeExperts || d->k > kMoeChosen || d->D % 8 != 0 || d->F % 8 != 0)
    return CONV2D_ERR_UNSUPPORTED;
  // TMA coordinates and the kernels' counts of k-blocks are 32-bit
  if (d->D > (1 << 24) || d->F > (1 << 24) || 2L * d->E * d->F > INT_MAX / 2 || static_cast<long>(d->E) * d->D > INT_MAX / 2) return CONV2D_ERR_UNSUPPORTED;
  return CONV2D_OK;
}
int check_weights(const conv2d_moe_desc* d, const conv2d_mat* w1, const conv2d_mat* w2) {
  if (!w1 || !w2 || w1->type != w2->type || (w1->ld != 0 && w1->ld < d->D) || (w2->ld != 0 && w2->ld < d->F))
    return CONV2D_ERR_INVALID_ARG;
  if (w1->type == CONV2D_E4M3) {
    if (w1->group != kQ8Tile || w2->group != kQ8Tile) return CONV2D_ERR_INVALID_ARG;
    // an expert's rows (and its gate's) are whole tiles; rows start on 16-byte boundaries
    return d->D % 128 == 0 && d->F % 128 == 0 && w1->ld % 16 == 0 && w2->ld % 16 == 0 ? CONV2D_OK : CONV2D_ERR_UNSUPPORTED;
  }
  if (w1->type != d->dtype) return CONV2D_ERR_INVALID_ARG;
  return w1->ld % 8 == 0 && w2->ld % 8 == 0 ? CONV2D_OK : CONV2D_ERR_UNSUPPORTED;
}

struct MoePlan {
  bool q8;
  int slots;  // experts that may be chosen
  size_t xq, xs, h, hs, total;
};
MoePlan plan(const conv2d_moe_desc& d, bool q8) {
  MoePlan p = {};
  p.q8 = q8;
  p.slots = static_cast<int>(std::min<long>(d.E, static_cast<long>(d.T) * d.k));
  auto take = [&](size_t bytes) {
    const size_t at = p.total;
    p.total += (bytes + 255) / 256 * 256;
    return at;
  };
  const size_t rows = static_cast<size_t>(p.slots) * d.T;
  if (q8) {
    p.xq = take(static_cast<size_t>(d.T) * d.D);
    p.xs = take(static_cast<size_t>(d.T) * ceil_div(d.D, 128));
    p.hs = take(rows * ceil_div(d.F, 128));
  }
  p.h = take(rows * d.F * (q8 ? 1 : 2));
  p.total = std::max<size_t>(p.total, 256);
  return p;
}

// CTAs that split a unit's k-blocks (kb of them): as many as keep two on each SM, two k-blocks each at least (one
// token, 8 of 64 experts of (2048, 1024) bf16 25.7 us from L2, 27.6 with one on each). units: those expected to have work.
int cluster_for(double units, long kb, int sms) {
  int cl = 8;
  while (cl > 1 && (units * cl > 2.0 * sms || kb < 2L * cl)) cl /= 2;
  return cl;
}

template <typename T, bool UP, int L, int Q>
cudaError_t launch_experts(ExpertParams& p, int units, long kb, int sms, cudaStream_t st) {
  const auto kernel = expert_kernel<T, UP, L, Q>;
  static std::atomic<uint64_t> done{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (!(done.load(std::memory_order_relaxed) >> dev & 1)) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kMoeSmem));
    if (e != cudaSuccess) return e;
    done.fetch_or(uint64_t(1) << dev);
  }
  const size_t stage = moe_stage_bytes(L, p.BN);
  const size_t fixed = 1024 + moe_fixed_bytes(UP) + (Q == kBlockScaled ? moe_slots_bytes(L) : 0);
  // k-blocks of a CTA, but never less than two stages: the joined sums take the ring's place
  p.stages = static_cast<int>(std::min<size_t>({static_cast<size_t>(kMoeMaxStages), (kMoeSmem - fixed) / stage,
                                                static_cast<size_t>(std::max<long>(2, ceil_div(kb, p.cluster)))}));
  static_assert(2 * moe_stage_bytes(L, 16) >= moe_join_bytes(L, 16, 8) && 2 * moe_stage_bytes(L, 32) >= moe_join_bytes(L, 32, 8) &&
                    2 * moe_stage_bytes(L, 64) >= moe_join_bytes(L, 64, 8) && 2 * moe_stage_bytes(L, 64) >= moe_join_bytes(L, 64, 2),
                "the joined sums lie in the ring");
  // CTAs without a cluster walk through the up product's units; the down product has one for each
  const int grid = UP && p.cluster == 1 ? std::min(units, 2 * sms) : units * p.cluster;
  return launch_k(kernel, dim3(static_cast<unsigned>(grid)), dim3(kMoeThreads + dense_scale_threads(Q)),
                  p.stages * stage + fixed, st, p.cluster, p);
}
template <bool UP, int L>
cudaError_t launch_experts(ExpertParams& p, int dt, bool q8, int units, long kb, int sms, cudaStream_t st) {
  if (dt == CONV2D_BF16)
    return q8 ? launch_experts<__nv_bfloat16, UP, L, kBlockScaled>(p, units, kb, sms, st)
              : launch_experts<__nv_bfloat16, UP, L, kHalves>(p, units, kb, sms, st);
  return q8 ? launch_experts<__half, UP, L, kBlockScaled>(p, units, kb, sms, st)
            : launch_experts<__half, UP, L, kHalves>(p, units, kb, sms, st);
}

template <typename T, typename R>
cudaError_t route(const RouteParams& p, cudaStream_t st) {
  auto go = [&](auto kernel, int nt) {
    return launch_k(kernel, dim3(static_cast<unsigned>(ceil_div(p.T, nt) * kRouteCluster)), dim3(kRouteThreads), 0, st,
                    kRouteCluster, p);
  };
  if (p.T <= 16) return go(route_kernel<T, R, 1>, 1);
  if (p.T <= 32) return go(route_kernel<T, R, 2>, 2);
  return go(route_kernel<T, R, 4>, 4);
}

}  // namespace

extern "C" {

size_t conv2d_moe_fwd_workspace_size(const conv2d_moe_desc* d, const conv2d_mat* w1, const conv2d_mat* w2) {
  if (check_desc(d) || check_weights(d, w1, w2)) return 0;
  return plan(*d, w1->type == CONV2D_E4M3).total;
}

int conv2d_moe_fwd(const conv2d_moe_desc* d, const conv2d_mat* x, const conv2d_mat* router, const conv2d_mat* w1,
                   const float* b1, const conv2d_mat* w2, const float* b2, const conv2d_mat* residual, const conv2d_mat* y,
                   int32_t* experts, float* weights, void* ws, size_t ws_bytes, void* stream) {
  int rc = check_desc(d);
  if (rc || (rc = check_weights(d, w1, w2))) return rc;
  if (!x || !router || !y || x->type != d->dtype || y->type != d->dtype || (residual && residual->type != d->dtype) ||
      (router->type != d->dtype && router->type != CONV2D_FP32))
    return CONV2D_ERR_INVALID_ARG;
  for (const conv2d_mat* m : {x, router, y, residual})
    if (m && m->ld != 0 && m->ld < d->D) return CONV2D_ERR_INVALID_ARG;
  if (x->ld % 8 != 0 || router->ld % 8 != 0) return CONV2D_ERR_UNSUPPORTED;  // their rows are read in 16 bytes
  if (!aligned16(b1) || !aligned16(b2)) return CONV2D_ERR_INVALID_ARG;
  if (d->T == 0) return CONV2D_OK;
  for (const conv2d_mat* m : {x, router, w1, w2, y, residual})
    if (m && (!m->data || !aligned16(m->data) || (m->type == CONV2D_E4M3 && !m->scale))) return CONV2D_ERR_INVALID_ARG;
  if (!experts || !weights || !aligned16(experts) || !aligned16(weights)) return CONV2D_ERR_INVALID_ARG;
  DevInfo* dev = nullptr;
  if ((rc = device_info(&dev))) return rc;
  const bool q8 = w1->type == CONV2D_E4M3;
  const MoePlan pl = plan(*d, q8);
  if (!ws || ws_bytes < pl.total || (reinterpret_cast<uintptr_t>(ws) & 255u)) return CONV2D_ERR_WORKSPACE;
  char* base = static_cast<char*>(ws);
  uint8_t *xq = reinterpret_cast<uint8_t*>(base + pl.xq), *xs = reinterpret_cast<uint8_t*>(base + pl.xs);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool f32 = router->type == CONV2D_FP32;
  const int bn = d->T <= 16 ? 16 : d->T <= 32 ? 32 : 64, es8 = q8 ? static_cast<int>(CONV2D_E4M3) : d->dtype;
  const int up_rows = d->F * (d->gated ? 2 : 1), up_tiles = static_cast<int>(ceil_div(d->F, 128));
  const int down_tiles = static_cast<int>(ceil_div(d->D, 128));
  const long rows = static_cast<long>(pl.slots) * d->T;

  RouteParams r = {};
  r.x = x->data;
  r.ldx = ld_of(x, d->D);
  r.router = router->data;
  r.ldr = ld_of(router, d->D);
  r.T = d->T;
  r.D = d->D;
  r.E = d->E;
  r.k = d->k;
  r.normalize = d->normalize;
  r.experts = experts;
  r.weights = weights;
  if (q8) {
    r.xq = xq;
    r.xs = xs;
    r.ldq = d->D;
  }
  ExpertParams up = {}, down = {};
  for (ExpertParams* p : {&up, &down}) {
    p->fmt = d->dtype == CONV2D_BF16 ? 1u : 0u;
    p->T = d->T;
    p->BN = bn;
    p->E = d->E;
    p->k = d->k;
    p->act = d->act;
    p->experts = experts;
    p->weights = weights;
    p->err = dev->err;
  }
  const int kblock = q8 ? 128 : 64;
  // experts that T tokens choose where all are as likely
  const double likely = d->E * (1.0 - std::pow(1.0 - static_cast<double>(d->k) / d->E, d->T));
  up.rows = up_rows;
  up.second = d->gated ? d->F : 0;
  up.width = d->F;
  up.tiles = up_tiles;
  up.kb_total = static_cast<int>(ceil_div(d->D, kblock));
  up.cluster = cluster_for(likely * up_tiles, up.kb_total, dev->sms);
  up.bias = b1;
  up.h = base + pl.h;
  up.hq = reinterpret_cast<uint8_t*>(base + pl.h);
  up.hs = reinterpret_cast<uint8_t*>(base + pl.hs);
  down.rows = down.width = d->D;
  down.tiles = down_tiles;
  down.kb_total = static_cast<int>(ceil_div(d->F, kblock));
  const long down_kb = static_cast<long>(likely * down.kb_total) + 1;
  down.cluster = cluster_for(down_tiles, down_kb, dev->sms);
  down.bias = b2;
  down.y = y->data;
  down.ldy = ld_of(y, d->D);
  if (residual) {
    down.res = residual->data;
    down.ldres = ld_of(residual, d->D);
  }
  if (q8) {
    up.sl = block_scales(w1->scale, kQ8Tile, static_cast<long>(d->E) * up_rows, d->D, false);
    up.sc = block_scales(xs, kQ8Wide, d->T, d->D, false);
    down.sl = block_scales(w2->scale, kQ8Tile, static_cast<long>(d->E) * d->D, d->F, false);
    down.sc = block_scales(up.hs, kQ8Wide, rows, d->F, false);
  }
  if (!encode_operand(&up.tl, w1->data, es8, static_cast<long>(d->E) * up_rows, d->D, ld_of(w1, d->D), false, 128) ||
      !encode_operand(&up.tc, q8 ? static_cast<const void*>(xq) : x->data, es8, d->T, d->D, q8 ? d->D : ld_of(x, d->D), false, bn) ||
      !encode_operand(&down.tl, w2->data, es8, static_cast<long>(d->E) * d->D, d->F, ld_of(w2, d->F), false, 128) ||
      !encode_operand(&down.tc, base + pl.h, es8, rows, d->F, d->F, false, bn))
    return CONV2D_ERR_CUDA;

  auto run_route = [&]() -> cudaError_t {
    if (d->dtype == CONV2D_BF16) return f32 ? route<__nv_bfloat16, float>(r, st) : route<__nv_bfloat16, __nv_bfloat16>(r, st);
    return f32 ? route<__half, float>(r, st) : route<__half, __half>(r, st);
  };
  LAUNCH("moe_route", st, run_route());
  auto run_up = [&] {
    return d->gated ? launch_experts<true, 2>(up, d->dtype, q8, pl.slots * up_tiles, up.kb_total, dev->sms, st)
                    : launch_experts<true, 1>(up, d->dtype, q8, pl.slots * up_tiles, up.kb_total, dev->sms, st);
  };
  auto run_down = [&] {
    return launch_experts<false, 1>(down, d->dtype, q8, down_tiles, down_kb, dev->sms, st);
  };
  LAUNCH("moe_up", st, run_up());
  LAUNCH("moe_down", st, run_down());
  return CONV2D_OK;
}

}  // extern "C"
