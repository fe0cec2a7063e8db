// dense.cu - the dense layer's C entry points: validation, workspace plan,
// choice of kernel and tile, tensor maps, and the launch sequence.
//
//   conv2d_dense_fwd: [decode / repack x, w] -> GEMM (epilogue: scales, bias,
//                     z in 16 or 8 bits, activation, residual)
//   conv2d_dense_bwd: [decode / repack w, x] and [dz = dy act'(z), column
//                     partials] side by side -> dx GEMM, dW GEMM and column
//                     sums (dbias) side by side -> [join of dW's splits]
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <cmath>

#include "conv2d.h"
#include "dense.h"
#include "host.h"
#include "rows.h"

namespace c2d {

// Row-major matrix [rows][cols] of row length ld as a GEMM operand, 128-byte swizzle: K-major, boxes of 128
// bytes x box_rows; MN-major, boxes of 128 bytes x a k-block: 64 x 64 of 16 bits, 128 x 128 of 8.
bool encode_operand(CUtensorMap* m, const void* base, int type, long rows, long cols, long ld, bool mn, int box_rows) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  const int es = type == CONV2D_E4M3 ? 1 : 2;
  cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
  cuuint64_t strides[1] = {static_cast<cuuint64_t>(ld) * es};
  cuuint32_t box[2] = {static_cast<cuuint32_t>(128 / es), static_cast<cuuint32_t>(mn ? 128 / es : box_rows)};
  cuuint32_t estr[2] = {1, 1};
  const CUtensorMapDataType dt = type == CONV2D_E4M3   ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                                 : type == CONV2D_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                                       : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  return fn(m, dt, 2, const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Scales of an 8-bit matrix [rows][cols] with a scale for 128 columns or a tile, as an operand summed over its columns, or
// (down) over its rows, which are tiled.
DenseScales block_scales(const uint8_t* scale, int group, long rows, long cols, bool down) {
  const long ng = (cols + kQ8Wide - 1) / kQ8Wide;
  DenseScales s = {};
  s.p = scale;
  s.row_shift = down || group == kQ8Tile ? 7 : 0;
  s.row_step = down ? 1 : ng;
  s.block_step = down ? ng : 1;
  s.rows = down ? cols : rows;
  if (!down) {
    const uintptr_t at = reinterpret_cast<uintptr_t>(scale);
    s.words = ng % 16 == 0 && at % 16 == 0 ? 4 : ng % 4 == 0 && at % 4 == 0 ? 1 : 0;
  }
  return s;
}

}  // namespace c2d

using namespace c2d;

namespace {

long ceil_div(long a, long b) { return (a + b - 1) / b; }
long round_up(long a, long b) { return ceil_div(a, b) * b; }
bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
long ld_of(const conv2d_mat* m, int cols) { return m->ld ? m->ld : cols; }

// ------------------------------------------------------------------ tiles
// The longest K loop (k-blocks of 64 rows) one accumulator sums for a weight gradient, by its type. The tensor core's
// fp32 sums are truncated, so terms of one sign lose up to 2^-23.3 of the sum at every MMA of 16 rows (fp16 operands;
// 2^-24.4 with bf16 until the sums are long): 4,096 rows 2.3e-5, 16,384 rows 1e-4 (a fifth of fp16's half step),
// 131,072 rows 8e-4 (a fifth of bf16's). Terms of either sign lose far less: 4,096 rows 5e-6 in the 2-norm. Longer
// products are split and the splits joined with ordinary fp32 additions, rounded once.
constexpr int kFp32SplitKb = 64, kFp16SplitKb = 256, kBf16SplitKb = 2048;
// k-blocks whose sum is off by a quarter of that (1,024 rows: 5e-6, and 1.3e-6 in the 2-norm), taken for fp32 where it
// costs little: everywhere, 8192 x 2048 x 8192 would take 276 us instead of 176.
constexpr int kFp32ShortKb = 16;

struct GemmPlan {
  bool pair;
  int BN, cluster, splits, kb_total, kb_per_split, l_tiles, c_tiles, stages, grid;
  int full, parts;    // pair kernel: units run whole, and into how many parts the others are cut
  size_t smem;
  size_t join_bytes;  // workspace for the parts' sums, then their flags
  size_t join_flags;  // number of flags
};

// Kernel, tile, cluster size and splits by an estimate of each choice's clocks, fitted to timings of square and
// skewed products (16 to 8,192 in each direction; the choice was within 10 % of the fastest in all of them). A
// k-block takes a CTA what its MMAs or its operands' way from L2 take, whichever is longer, which comes to a line
// in BN; a unit has a fixed cost (launch, first operands, epilogue); clusters pay for joining their sums. Units
// run in waves over the SMs; the pair kernel hides its epilogue under the next unit's loop. can_split: the product
// may be split over k, with fp32 partials in the workspace; max_kb: bound on one accumulator's k-blocks, short_kb: those
// it had better not pass (0: none).
GemmPlan plan_gemm(int mode, long m, long n, int kb, int sms, int q = kHalves, bool can_split = false, int max_kb = 0,
                   int short_kb = 0) {
  const bool r_mn = dense_r_mn(mode), c_mn = dense_c_mn(mode), blocks = q == kBlockScaled;
  GemmPlan best = {};
  double best_t = 1e300;
  auto consider = [&](bool pair, int BN, int cl, int splits) {
    GemmPlan g = {};
    g.pair = pair;
    g.BN = BN;
    g.cluster = cl;
    g.kb_total = kb;
    g.kb_per_split = static_cast<int>(ceil_div(kb, splits));
    g.splits = static_cast<int>(ceil_div(kb, g.kb_per_split));
    if (max_kb > 0 && ceil_div(g.kb_per_split, cl) > max_kb) return;
    g.l_tiles = static_cast<int>(pair ? ceil_div(m, 256) : ceil_div(n, 128));
    g.c_tiles = static_cast<int>(ceil_div(pair ? n : m, BN));
    const double units = static_cast<double>(g.l_tiles) * g.c_tiles * g.splits;
    if (units * cl > INT_MAX / 4) return;
    const double loop = static_cast<double>(ceil_div(g.kb_per_split, cl));
    double t;
    if (pair) {
      const double epi = 1500 + 10.0 * BN, block = 188 + 1.35 * BN, unit = std::max(loop * block, epi);
      const long pairs = sms / 2, whole = static_cast<long>(units) / pairs, rem = static_cast<long>(units) % pairs;
      t = 8300 + 12.0 * BN + whole * unit;
      g.full = static_cast<int>(units);
      g.parts = 1;
      if (rem > 0) {
        // a last wave that leaves half of the pairs or more idle is cut along k: a part's sums go through memory
        // (about 3 us with the zeroing of the flags)
        const int parts = static_cast<int>(std::min<long>(std::min<long>(4, pairs / rem), g.kb_total / 8));
        const double cut = parts > 1 && g.splits == 1 && whole > 0 ? loop / parts * block + 9000 : 1e300;
        if (cut < unit) {
          g.full = static_cast<int>(whole * pairs);
          g.parts = parts;
        }
        t += std::min(unit, cut);
      }
    } else {
      // CTAs that are resident at once: clusters of 4 and 8 leave SMs of a GPC over
      const double fit = cl == 8 ? sms * 15 / 19 : cl == 4 ? sms * 18 / 19 : sms;
      t = std::ceil(units * cl / fit) * (6300 + 38.0 * BN + loop * ((r_mn ? 480 : 300) + 0.45 * BN) + (cl > 1 ? 3500 + 22.0 * BN : 0));
    }
    // the join is a launch of its own and waits for everything beside it (1777 x 1000 x 333 with dx: 19.7 us in 4
    // splits, 17.3 in one; 4096 x 512 x 512: 22.1 in 8, 18.7 as a cluster of 4); it reads a value's partials in turn
    if (g.splits > 1) t += 8000 + 100.0 * g.splits + static_cast<double>(m) * n * 4 * 2 * g.splits / 7000;
    // up to a tenth of the time goes into short fp32 sums
    if (short_kb > 0 && ceil_div(g.kb_per_split, cl) > short_kb) t *= 1.1;
    if (t < best_t) {
      best_t = t;
      best = g;
    }
  };
  // splits to look at: none, the fewest that keep an accumulator within max_kb, and those that fill one to three
  // waves of SMs (or pairs)
  auto splits_of = [&](bool pair, int BN, int cl) {
    consider(pair, BN, cl, 1);
    if (!can_split) return;
    if (max_kb > 0) consider(pair, BN, cl, static_cast<int>(ceil_div(kb, static_cast<long>(max_kb) * cl)));
    const long tiles = pair ? ceil_div(m, 256) * ceil_div(n, BN) : ceil_div(n, 128) * ceil_div(m, BN) * cl;
    for (int w = 1; w <= 3; ++w) {
      const long s = std::min<long>(w * (pair ? sms / 2 : sms) / tiles, kb);
      if (s > 1) consider(pair, BN, cl, static_cast<int>(s));
    }
  };
  for (int BN : {256, 224, 192, 160, 128})
    if (!blocks || BN < 256) splits_of(true, BN, 1);  // blocks' scales need columns of the tensor memory beside the sums
  for (int BN : {128, 64, 32, 16}) {
    if (r_mn && BN < 64) continue;  // MN-major tiles are panels of 64
    for (int cl : {1, 2, 4, 8})
      if (cl == 1 || kb >= 2 * cl) splits_of(false, BN, cl);
  }
  int c_rows = best.BN;  // columns of C a CTA brings: MN-major in whole panels of 64
  if (best.pair) c_rows = c_mn ? static_cast<int>(round_up(best.BN / 2, q == kHalves ? 64 : 128)) : best.BN / 2;
  const int need = static_cast<int>(ceil_div(best.kb_per_split, best.cluster));  // k-blocks of a CTA
  const int stage = (128 + c_rows) * 128;
  const int slots = blocks ? dense_slots_bytes(best.BN) : 0;
  const int room = static_cast<int>(kMaxDynSmem) - 1536 - (best.pair ? kPairBuffers : 0) - slots;
  const long units = static_cast<long>(best.l_tiles) * best.c_tiles * best.splits;
  const int join = best.cluster > 1 ? best.cluster * dense_own_cols(best.BN, best.cluster) * 512 : 0;
  if (best.pair) {
    best.grid = 2 * static_cast<int>(std::min<long>(units, sms / 2));
    best.stages = std::min(kDenseMaxStages, room / stage);
    if (blocks) best.stages = std::min(best.stages, (512 - 2 * best.BN) / dense_slot_cols(best.BN));
  } else {
    best.grid = static_cast<int>(units) * best.cluster;
    best.stages = std::max(2, std::min({kDenseMaxStages, (room - join) / stage, need}));
  }
  if (best.parts > 1) {
    const size_t rem = static_cast<size_t>(units - best.full) * (best.parts - 1) * 2;
    best.join_bytes = rem * 128 * best.BN * 4;
    best.join_flags = rem * kPairWarps;
  }
  // alignment slack, barriers
  best.smem = static_cast<size_t>(best.stages) * stage + 1024 + 512 + slots + (best.pair ? kPairBuffers : join);
  return best;
}

// ------------------------------------------------------------------ tensor maps
// Output [splits][rows][cols] of row length ld for the pair kernel's stores: boxes of 32 rows x RB bytes, swizzled
// over RB bytes (32 or 64).
bool encode_output(CUtensorMap* m, const void* base, int type, long rows, long cols, long ld, long splits) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  const int es = type == CONV2D_E4M3 ? 1 : type == CONV2D_FP32 ? 4 : 2;
  const int rb = type == CONV2D_E4M3 ? 32 : 64;
  cuuint64_t dims[3] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows), static_cast<cuuint64_t>(splits)};
  cuuint64_t strides[2] = {static_cast<cuuint64_t>(ld) * es, static_cast<cuuint64_t>(ld) * rows * es};
  cuuint32_t box[3] = {static_cast<cuuint32_t>(rb / es), 32, 1};
  cuuint32_t estr[3] = {1, 1, 1};
  const CUtensorMapDataType dt = type == CONV2D_E4M3   ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                                 : type == CONV2D_FP32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                 : type == CONV2D_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                                       : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  return fn(m, dt, 3, const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            rb == 32 ? CU_TENSOR_MAP_SWIZZLE_32B : CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// An operand ready for the tensor core: type BF16 / FP16 / E4M3, row length a multiple of 16 bytes.
struct Operand {
  const void* data;
  int type;
  long rows, cols, ld;
  DenseScales scales;  // of a block-scaled product
};

// out[m][n] = sum_k R[m][k] C[n][k]. The rows of the output are the accumulator's lanes in the pair kernel and its
// columns in the cluster kernel.
int run_gemm(DenseGemmParams& p, const GemmPlan& g, const Operand& r, const Operand& c, int dt, int mode, void* join,
             bool late, const char* name, const DevInfo* dev, cudaStream_t st) {
  const bool r_mn = dense_r_mn(mode), c_mn = dense_c_mn(mode);
  const Operand &lo = g.pair ? r : c, &co = g.pair ? c : r;
  if (!encode_operand(&p.tl, lo.data, lo.type, lo.rows, lo.cols, lo.ld, g.pair ? r_mn : c_mn, 128) ||
      !encode_operand(&p.tc, co.data, co.type, co.rows, co.cols, co.ld, g.pair ? c_mn : r_mn, g.pair ? g.BN / 2 : g.BN))
    return CONV2D_ERR_CUDA;
  const int q = r.type != CONV2D_E4M3 ? kHalves : r.scales.p ? kBlockScaled : kRowScaled;
  p.sl = lo.scales;
  p.sc = co.scales;
  p.fmt = r.type == CONV2D_BF16 ? 1u : 0u;
  p.m = r_mn ? r.cols : r.rows;
  p.n = static_cast<int>(c_mn ? c.cols : c.rows);
  if (g.pair && p.accumulate && !p.out_f32) {
    mode = kDenseDwAdd;
    p.res = p.out;
    p.ldr = p.ldo;
  }
  p.vec_res = p.ldr % 8 == 0;
  if (g.pair) {
    const int zt = p.zq ? static_cast<int>(CONV2D_E4M3) : dt, ot = p.out_f32 ? static_cast<int>(CONV2D_FP32) : dt;
    const void* z = p.zq ? p.zq : p.z;
    p.tma_out = p.ldo % (p.out_f32 ? 4 : 8) == 0;
    p.tma_z = z && p.ldz % (p.zq ? 16 : 8) == 0;
    if ((p.tma_out && !encode_output(&p.tout, p.out, ot, p.m, p.n, p.ldo, g.splits)) ||
        (p.tma_z && !encode_output(&p.tz, z, zt, p.m, p.n, p.ldz, 1)))
      return CONV2D_ERR_CUDA;
  }
  p.full = g.full;
  p.parts = g.parts;
  if (g.parts > 1) {
    p.join_part = static_cast<float*>(join);
    p.join_flag = reinterpret_cast<uint32_t*>(static_cast<char*>(join) + g.join_bytes);
    LAUNCH("zero", st, launch_zero_rows(1, static_cast<int>(g.join_flags), CONV2D_FP32, p.join_flag,
                                        static_cast<long>(g.join_flags), late, st));
    late = false;  // the flags are waited for
  }
  p.late = late;
  p.early = g.grid <= dev->sms * 3 / 4;
  p.l_tiles = g.l_tiles;
  p.c_tiles = g.c_tiles;
  p.splits = g.splits;
  p.kb_total = g.kb_total;
  p.kb_per_split = g.kb_per_split;
  p.BN = g.BN;
  p.stages = g.stages;
  p.cluster = g.cluster;
  p.err = dev->err;
  LAUNCH(name, st, g.pair ? launch_dense_pair(p, dt, mode, q, g.grid, g.smem, st)
                          : launch_dense_cluster(p, dt, mode, q, g.grid, g.smem, st));
  return CONV2D_OK;
}

// ------------------------------------------------------------------ arguments
int check_desc(const conv2d_dense_desc* d) {
  if (!d || d->M < 0 || d->K < 1 || d->N < 1 || d->act < 0 || d->act > CONV2D_ACT_SILU ||
      (d->dtype != CONV2D_BF16 && d->dtype != CONV2D_FP16))
    return CONV2D_ERR_INVALID_ARG;
  // TMA coordinates and tile counts are 32-bit
  if (d->M > INT_MAX / 2 || d->K > (1 << 28) || d->N > (1 << 28)) return CONV2D_ERR_UNSUPPORTED;
  return CONV2D_OK;
}
// The shape part of a matrix argument: type among the layer's, ld at least cols, known group (wide: those of 128 too).
int check_shape(const conv2d_mat* m, int cols, int dtype, bool q8, bool wide = false) {
  if (!m || (m->ld != 0 && m->ld < cols)) return CONV2D_ERR_INVALID_ARG;
  if (m->type == CONV2D_E4M3)
    return q8 && (wide ? q8_known(m->group) : m->group == 0 || m->group == kQ8Group) ? CONV2D_OK : CONV2D_ERR_INVALID_ARG;
  return m->type == dtype ? CONV2D_OK : CONV2D_ERR_INVALID_ARG;
}
int check_data(const conv2d_mat* m) {
  return m->data && aligned16(m->data) && (m->type != CONV2D_E4M3 || m->scale) ? CONV2D_OK : CONV2D_ERR_INVALID_ARG;
}

// How the forward product runs: on the 8-bit operands as they are, where their scales allow it.
int product_kind(const conv2d_mat* x, const conv2d_mat* w) {
  if (x->type != CONV2D_E4M3 || w->type != CONV2D_E4M3) return kHalves;
  if (x->group == 0 && w->group == 0) return kRowScaled;
  return x->group == kQ8Wide && (w->group == kQ8Wide || w->group == kQ8Tile) ? kBlockScaled : kHalves;
}

// ------------------------------------------------------------------ workspace
// What a size query answers where nothing is kept in the workspace; ws may then be null. Anything that is kept makes
// it larger, so a caller can tell the two apart.
constexpr size_t kNoWorkspace = 256;
struct Carver {
  size_t total = 0;
  size_t take(size_t bytes) {
    const size_t at = total;
    total += static_cast<size_t>(round_up(static_cast<long>(bytes), 256));
    return at;
  }
  size_t size() const { return total ? std::max(total, 2 * kNoWorkspace) : kNoWorkspace; }
};
constexpr size_t kNone = ~static_cast<size_t>(0);

// Where an operand has to be copied (decoded, or moved to rows of a multiple of 16 bytes): offset, else kNone.
size_t plan_copy(Carver& c, const conv2d_mat* m, long rows, int cols, bool as_8bit) {
  if (as_8bit) return ld_of(m, cols) % 16 == 0 ? kNone : c.take(static_cast<size_t>(rows) * round_up(cols, 16));
  if (m->type != CONV2D_E4M3 && ld_of(m, cols) % 8 == 0) return kNone;
  return c.take(static_cast<size_t>(rows) * round_up(cols, 8) * 2);
}
// The operand itself, or its copy in the workspace; *started: a kernel of this call has been launched.
int make_operand(Operand* o, const conv2d_mat* m, long rows, int cols, bool as_8bit, int dt, size_t off, void* ws,
                 const char* name, bool* started, cudaStream_t st) {
  *o = {m->data, as_8bit ? static_cast<int>(CONV2D_E4M3) : dt, rows, cols, ld_of(m, cols), {}};
  if (off == kNone) return CONV2D_OK;
  char* to = static_cast<char*>(ws) + off;
  o->data = to;
  o->ld = round_up(cols, as_8bit ? 16 : 8);
  const int late = *started;  // nothing before it in the call touches these operands
  *started = true;
  if (as_8bit) LAUNCH(name, st, launch_move_bytes(m->data, ld_of(m, cols), rows, cols, to, o->ld, late, st));
  else LAUNCH(name, st, launch_to_rows(*m, rows, cols, dt, to, o->ld, late, st));
  return CONV2D_OK;
}

// Room for the cut units' sums and flags.
size_t plan_join(Carver& c, const GemmPlan& g) { return g.parts > 1 ? c.take(g.join_bytes + g.join_flags * 4) : kNone; }
void* at(void* ws, size_t off) { return off == kNone ? nullptr : static_cast<char*>(ws) + off; }

struct FwdPlan {
  int kind;
  size_t x, w, join, total;
  GemmPlan g;
};
void plan_fwd(const conv2d_dense_desc& d, const conv2d_mat* x, const conv2d_mat* w, int sms, FwdPlan* pl) {
  Carver c;
  pl->kind = product_kind(x, w);
  const bool as8 = pl->kind != kHalves;
  pl->x = plan_copy(c, x, d.M, d.K, as8);
  pl->w = plan_copy(c, w, d.N, d.K, as8);
  pl->g = plan_gemm(kDenseForward, d.M, d.N, static_cast<int>(ceil_div(d.K, as8 ? 128 : 64)), sms, pl->kind);
  pl->join = plan_join(c, pl->g);
  pl->total = c.size();
}

struct BwdPlan {
  bool dz_own;  // dz is formed in the workspace (else it is dy)
  bool dx8;     // dx is a product of 8-bit operands: dz goes to 8 bits, a scale for 128 columns
  long lddz, lddz8;
  size_t dz8, dz8s;
  long pass_rows;  // rows of a pass of dW (M: one pass)
  int planes;      // fp32 partials of dW in the workspace, joined at the end (0: dW is written by the product)
  size_t dz, x, w, dpart, spart, joinx, joinw, total;
  DactPlan dact;
  GemmPlan gx, gw;
};
void plan_bwd(const conv2d_dense_desc& d, const conv2d_mat* x, const conv2d_mat* w, const conv2d_mat* dy, bool dx,
              const conv2d_mat* dw, bool dbias, int sms, BwdPlan* pl) {
  Carver c;
  pl->dx8 = dx && w->type == CONV2D_E4M3 && w->group == kQ8Tile;
  pl->lddz8 = round_up(d.N, 16);
  pl->lddz = round_up(d.N, 8);
  // dy itself where it is dz, in rows that a product takes; the encoder takes any
  pl->dz_own = (dx || dw) && (d.act != CONV2D_ACT_IDENTITY || (ld_of(dy, d.N) % 8 != 0 && (dw || !pl->dx8)));
  pl->dz = pl->dz_own ? c.take(static_cast<size_t>(d.M) * pl->lddz * 2) : kNone;
  pl->dact = plan_dact(d.M, d.N, sms);
  pl->dpart = dbias ? c.take(static_cast<size_t>(pl->dact.strips) * d.N * 4) : kNone;
  pl->w = pl->x = pl->spart = pl->joinx = pl->joinw = kNone;
  if (dx) {
    pl->w = plan_copy(c, w, d.N, d.K, pl->dx8);
    if (pl->dx8) {
      pl->dz8 = c.take(static_cast<size_t>(d.M) * pl->lddz8);
      pl->dz8s = c.take(static_cast<size_t>(d.M) * ceil_div(d.N, kQ8Wide));
    }
    pl->gx = plan_gemm(kDenseDx, d.M, d.K, static_cast<int>(ceil_div(d.N, pl->dx8 ? 128 : 64)), sms,
                       pl->dx8 ? kBlockScaled : kHalves);
    pl->joinx = plan_join(c, pl->gx);
  }
  if (dw) {
    pl->x = plan_copy(c, x, d.M, d.K, false);
    // A dW over many rows is summed in pieces: side by side, joined afterwards, or one after the other, added to dW (16
    // bits: to one fp32 plane in the workspace, rounded at the end). The second saves the partials' traffic but idles
    // at each piece's last wave. It is taken in fp32 for up to 4 pieces whose waves are four fifths full (8192 x 2048 x 8192: 176 us against 188; 16384 x
    // 4096 x 4096: 344 to 358 against 353 to 355; 8 pieces, 32768 x 2048 x 8192: 722 against 674; waves 59 % full,
    // 9000 x 2304 x 2560: 97 against 86), and where the partials would take more than 2 GB.
    const bool f32 = dw->type == CONV2D_FP32;
    const int kb = static_cast<int>(ceil_div(d.M, 64));
    const int bound = f32 ? kFp32SplitKb : d.dtype == CONV2D_FP16 ? kFp16SplitKb : kBf16SplitKb;
    const long pairs = sms / 2, tiles = ceil_div(d.N, 256) * ceil_div(d.K, 256), waves = ceil_div(tiles, pairs);
    const long pieces = ceil_div(kb, bound);
    const bool passes = pieces > 1 && ((f32 && pieces <= 4 && tiles * 5 >= waves * pairs * 4) ||
                                       pieces * d.N * d.K * 4 > (2L << 30));
    pl->pass_rows = passes ? bound * 64L : d.M;
    pl->gw = passes ? plan_gemm(kDenseDw, d.N, d.K, bound, sms)
                    : plan_gemm(kDenseDw, d.N, d.K, kb, sms, kHalves, true, bound, f32 ? kFp32ShortKb : 0);
    pl->joinw = plan_join(c, pl->gw);
    pl->planes = passes ? (f32 ? 0 : 1) : pl->gw.splits > 1 ? pl->gw.splits : 0;
    if (pl->planes) pl->spart = c.take(static_cast<size_t>(pl->planes) * d.N * d.K * 4);
  }
  pl->total = c.size();
}

int check_bwd_shapes(const conv2d_dense_desc* d, const conv2d_mat* x, const conv2d_mat* w, const conv2d_mat* z,
                     const conv2d_mat* dy, const conv2d_mat* dx, const conv2d_mat* dw, const float* dbias) {
  int rc = check_desc(d);
  if (rc) return rc;
  if (!dx && !dw && !dbias) return CONV2D_ERR_INVALID_ARG;
  if ((rc = check_shape(dy, d->N, d->dtype, false))) return rc;
  if (d->act != CONV2D_ACT_IDENTITY && (rc = check_shape(z, d->N, d->dtype, true))) return rc;
  if (dx && ((rc = check_shape(dx, d->K, d->dtype, false)) || (rc = check_shape(w, d->K, d->dtype, true, true)))) return rc;
  if (dw) {
    if ((rc = check_shape(dw, d->K, dw->type == CONV2D_FP32 ? CONV2D_FP32 : d->dtype, false))) return rc;
    if ((rc = check_shape(x, d->K, d->dtype, true, true))) return rc;
  }
  return CONV2D_OK;
}

}  // namespace

extern "C" {

size_t conv2d_dense_fwd_workspace_size(const conv2d_dense_desc* d, const conv2d_mat* x, const conv2d_mat* w) {
  if (check_desc(d) || check_shape(x, d->K, d->dtype, true, true) || check_shape(w, d->K, d->dtype, true, true)) return 0;
  FwdPlan pl;
  plan_fwd(*d, x, w, sms_for_sizing(), &pl);
  return pl.total;
}

size_t conv2d_dense_bwd_workspace_size(const conv2d_dense_desc* d, const conv2d_mat* x, const conv2d_mat* w,
                                       const conv2d_mat* pre_act, const conv2d_mat* dy, const conv2d_mat* dx,
                                       const conv2d_mat* dw, const float* dbias) {
  if (check_bwd_shapes(d, x, w, pre_act, dy, dx, dw, dbias)) return 0;
  BwdPlan pl;
  plan_bwd(*d, x, w, dy, dx != nullptr, dw, dbias != nullptr, sms_for_sizing(), &pl);
  return pl.total;
}

int conv2d_dense_fwd(const conv2d_dense_desc* d, const conv2d_mat* x, const conv2d_mat* w, const float* bias,
                     const conv2d_mat* residual, const conv2d_mat* pre_act, const conv2d_mat* y, void* ws,
                     size_t ws_bytes, void* stream) {
  int rc = check_desc(d);
  if (rc) return rc;
  if ((rc = check_shape(x, d->K, d->dtype, true, true)) || (rc = check_shape(w, d->K, d->dtype, true, true)) ||
      (rc = check_shape(y, d->N, d->dtype, false)))
    return rc;
  if (residual && (rc = check_shape(residual, d->N, d->dtype, false))) return rc;
  if (pre_act && ((rc = check_shape(pre_act, d->N, d->dtype, true)) ||
                  (pre_act->type == CONV2D_E4M3 && pre_act->group != kQ8Group)))
    return CONV2D_ERR_INVALID_ARG;
  if (!aligned16(bias)) return CONV2D_ERR_INVALID_ARG;
  if (d->M == 0) return CONV2D_OK;
  for (const conv2d_mat* m : {x, w, y, residual, pre_act})
    if (m && (rc = check_data(m))) return rc;
  DevInfo* dev = nullptr;
  if ((rc = device_info(&dev))) return rc;
  FwdPlan pl;
  plan_fwd(*d, x, w, dev->sms, &pl);
  const bool uses_ws = pl.x != kNone || pl.w != kNone || pl.join != kNone;
  if (uses_ws && (!ws || ws_bytes < pl.total || (reinterpret_cast<uintptr_t>(ws) & 255u))) return CONV2D_ERR_WORKSPACE;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  Operand ox, ow;
  bool started = false;
  const bool as8 = pl.kind != kHalves;
  if ((rc = make_operand(&ox, x, d->M, d->K, as8, d->dtype, pl.x, ws, "dense_x", &started, st))) return rc;
  if ((rc = make_operand(&ow, w, d->N, d->K, as8, d->dtype, pl.w, ws, "dense_w", &started, st))) return rc;
  DenseGemmParams p = {};
  if (pl.kind == kRowScaled) {
    p.ns = w->scale;
    p.ms = x->scale;
  } else if (pl.kind == kBlockScaled) {
    ox.scales = block_scales(x->scale, x->group, d->M, d->K, false);
    ow.scales = block_scales(w->scale, w->group, d->N, d->K, false);
  }
  p.bias = bias;
  p.act = d->act;
  if (residual) {
    p.res = residual->data;
    p.ldr = ld_of(residual, d->N);
  }
  if (pre_act) {
    p.ldz = ld_of(pre_act, d->N);
    if (pre_act->type == CONV2D_E4M3) {
      p.zq = static_cast<uint8_t*>(pre_act->data);
      p.zs = pre_act->scale;
      p.zg = static_cast<int>(ceil_div(d->N, kQ8Group));
    } else {
      p.z = pre_act->data;
    }
  }
  p.out = y->data;
  p.ldo = ld_of(y, d->N);
  return run_gemm(p, pl.g, ox, ow, d->dtype, kDenseForward, at(ws, pl.join), false, "dense_fwd", dev, st);
}

int conv2d_dense_bwd(const conv2d_dense_desc* d, const conv2d_mat* x, const conv2d_mat* w, const conv2d_mat* pre_act,
                     const conv2d_mat* dy, const conv2d_mat* dx, const conv2d_mat* dw, float* dbias, void* ws,
                     size_t ws_bytes, void* stream) {
  int rc = check_bwd_shapes(d, x, w, pre_act, dy, dx, dw, dbias);
  if (rc) return rc;
  if (!aligned16(dbias)) return CONV2D_ERR_INVALID_ARG;
  if (dw && (rc = check_data(dw))) return rc;
  DevInfo* dev = nullptr;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (d->M == 0) {  // sums over no rows
    if (d->accumulate || (!dw && !dbias)) return CONV2D_OK;
    if ((rc = device_info(&dev))) return rc;
    if (dw) LAUNCH("zero", st, launch_zero_rows(d->N, d->K, dw->type, dw->data, ld_of(dw, d->K), 0, st));
    if (dbias) LAUNCH("zero", st, launch_zero_rows(1, d->N, CONV2D_FP32, dbias, d->N, 0, st));
    return CONV2D_OK;
  }
  const bool act = d->act != CONV2D_ACT_IDENTITY;
  if ((rc = check_data(dy)) || (act && (rc = check_data(pre_act)))) return rc;
  if (dx && ((rc = check_data(dx)) || (rc = check_data(w)))) return rc;
  if (dw && (rc = check_data(x))) return rc;
  if ((rc = device_info(&dev))) return rc;
  BwdPlan pl;
  plan_bwd(*d, x, w, dy, dx != nullptr, dw, dbias != nullptr, dev->sms, &pl);
  if (!ws || ws_bytes < pl.total || (reinterpret_cast<uintptr_t>(ws) & 255u)) return CONV2D_ERR_WORKSPACE;
  char* base = static_cast<char*>(ws);

  // What only reads the call's arguments goes first and side by side: the operands' copies and dz. Then dx, dW
  // beside it (they share their inputs only), and the bias gradient beside both.
  bool started = false;
  Operand ow, ox;
  if (dx && (rc = make_operand(&ow, w, d->N, d->K, pl.dx8, d->dtype, pl.w, ws, "dense_w", &started, st))) return rc;
  if (dw && (rc = make_operand(&ox, x, d->M, d->K, false, d->dtype, pl.x, ws, "dense_x", &started, st))) return rc;
  Operand odz = {dy->data, d->dtype, d->M, d->N, ld_of(dy, d->N), {}};
  float* part = dbias ? reinterpret_cast<float*>(base + pl.dpart) : nullptr;
  if (pl.dz_own || dbias) {
    void* dz = pl.dz_own ? base + pl.dz : nullptr;
    // beside the copies only where it does not fill the GPU by itself: a block that has finished waits for them
    const bool beside = started && d->M * d->N < (int64_t(1) << 22);
    LAUNCH("dense_dact", st,
           launch_dact(act ? pre_act : nullptr, *dy, d->M, d->N, d->dtype, d->act, dz, pl.lddz, part, pl.dact, beside,
                       st));
    if (dz) {
      odz.data = dz;
      odz.ld = pl.lddz;
    }
  }
  if (dx) {
    DenseGemmParams p = {};
    p.out = dx->data;
    p.ldo = ld_of(dx, d->K);
    Operand o = odz;
    if (pl.dx8) {
      const conv2d_mat dz = {const_cast<void*>(odz.data), odz.ld, d->dtype, 0, nullptr};
      const conv2d_mat dz8 = {base + pl.dz8, pl.lddz8, CONV2D_E4M3, kQ8Wide, reinterpret_cast<uint8_t*>(base + pl.dz8s)};
      if ((rc = conv2d_q8_encode(d->M, d->N, &dz, &dz8, stream))) return rc;
      o = {dz8.data, CONV2D_E4M3, d->M, d->N, pl.lddz8, block_scales(dz8.scale, kQ8Wide, d->M, d->N, false)};
      ow.scales = block_scales(w->scale, kQ8Tile, d->N, d->K, true);
    }
    if ((rc = run_gemm(p, pl.gx, o, ow, d->dtype, kDenseDx, at(ws, pl.joinx), false, "dense_dx", dev, st))) return rc;
  }
  const bool joined = dw && pl.planes > 0;
  if (dw) {
    for (long r0 = 0; r0 < d->M; r0 += pl.pass_rows) {
      DenseGemmParams p = {};
      p.out = joined ? static_cast<void*>(base + pl.spart) : dw->data;
      p.ldo = joined ? d->K : ld_of(dw, d->K);
      p.out_f32 = joined || dw->type == CONV2D_FP32;
      p.accumulate = (d->accumulate && !joined) || r0 > 0;
      p.split_stride = static_cast<long>(d->N) * d->K;
      Operand oz = odz, oa = ox;
      oz.rows = oa.rows = std::min(pl.pass_rows, d->M - r0);
      oz.data = static_cast<const char*>(odz.data) + r0 * odz.ld * 2;  // row lengths are multiples of 16 bytes
      oa.data = static_cast<const char*>(ox.data) + r0 * ox.ld * 2;
      GemmPlan g = pl.gw;
      if (oz.rows < pl.pass_rows) {  // the last pass: fewer k-blocks, whole units
        g.kb_total = g.kb_per_split = static_cast<int>(ceil_div(oz.rows, 64));
        g.full = g.l_tiles * g.c_tiles;
        g.parts = 1;
      }
      if ((rc = run_gemm(p, g, oz, oa, d->dtype, kDenseDw, at(ws, pl.joinw), r0 == 0 && dx, "dense_dw", dev, st)))
        return rc;
    }
  }
  if (dbias)
    LAUNCH("column_sum", st,
           launch_column_sum(part, pl.dact.strips, d->N, dbias, d->accumulate != 0, dx || dw, st));
  if (joined)
    LAUNCH("dense_dw_join", st,
           launch_split_join(reinterpret_cast<float*>(base + pl.spart), pl.planes, d->N, d->K, dw->type, dw->data,
                             ld_of(dw, d->K), d->accumulate != 0, st));
  return CONV2D_OK;
}

}  // extern "C"
