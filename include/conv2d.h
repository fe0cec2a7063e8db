/*
 * conv2d.h - C ABI of the GB300 (sm_103a) conv2d training-step library
 * (libconv2d.so).
 *
 * One NHWC 2D convolution layer: conv + bias, optional training-mode batch
 * norm, layer norm or group norm, activation; and its backward pass. The operation is the one defined by
 * the rl-tools conv2d layer pages ("operations_generic.h": `forward`,
 * `evaluate`, `backward`, `backward_input`, `backward_full`; the CUDA page
 * "operations_cuda.h" splits the same work into cuDNN calls and per-channel
 * kernels). The layer spec (N,H,W,IC,OC,KH,KW,stride,pad, normalization,
 * activation, eps, momentum, type policy) follows the template parameters
 * those pages read from their LayerSpec.
 *
 * Conventions (all calls):
 *   - Tensors are dense, contiguous NHWC: x [N][H][W][IC], y / pre_act / dy
 *     [N][OH][OW][OC], weights w [OC][KH][KW][IC]; OH = (H+2*pad-KH)/stride+1
 *     (floor), OW likewise; symmetric zero padding; cross-correlation (no
 *     kernel flip); no dilation, no groups.
 *   - x, w, pre_act, y, dy, dx have the element type named by desc->dtype
 *     (CONV2D_FP32: float; CONV2D_BF16: bfloat16). bias, gamma, beta, running
 *     statistics, saved statistics and every parameter gradient are float32.
 *   - Every pointer is a DEVICE pointer on the current CUDA device, aligned to
 *     16 bytes. The caller owns every buffer; the library allocates no device
 *     memory on any path. Scratch space is the caller's workspace `ws` of at
 *     least conv2d_workspace_size(desc, op) bytes (alignment 256 bytes); its
 *     contents need not be initialised and are clobbered.
 *   - Calls are asynchronous on `stream` (a cudaStream_t; NULL = legacy
 *     default stream). Buffers must not be touched by other work until the
 *     stream reaches the call. Calls that share a workspace must be ordered.
 *   - Return value: CONV2D_OK, or an error code from host-side validation or
 *     launch (no kernel is launched when validation fails). Device-side
 *     failures (a bounded wait that ran out) are reported later by
 *     conv2d_device_status().
 *   - Accumulate / overwrite semantics follow `backward_full`: dw, dbias,
 *     dgamma, dbeta are ACCUMULATED into (the caller zeroes them, as the
 *     pages' `zero_gradient` does); dx is OVERWRITTEN.
 *   - The library is stateless apart from per-device constant data; it is
 *     safe to call from several host threads.
 *   - Per-device data is looked up once, on the first call made on a device,
 *     and cached for the life of the process: the SM count, the device
 *     address of the library's error word and of the static scratch array of
 *     conv2d_fwd_train_noalloc. cudaDeviceReset() on a device invalidates
 *     those addresses, so resetting a device while this library is loaded in
 *     the process is not supported.
 */
#ifndef CONV2D_GB300_H
#define CONV2D_GB300_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Status codes. */
enum {
    CONV2D_OK = 0,
    CONV2D_ERR_INVALID_ARG = 1, /* bad size, NULL or misaligned pointer, bad enum, eps<=0, momentum outside [0,1] */
    CONV2D_ERR_UNSUPPORTED = 2, /* valid but not implemented (stride > 8, sizes beyond 2^31 elements) */
    CONV2D_ERR_WORKSPACE = 3,   /* ws NULL or smaller than conv2d_workspace_size() */
    CONV2D_ERR_CUDA = 4,        /* a CUDA runtime / driver call failed (launch, tensor-map encode) */
    CONV2D_ERR_TIMEOUT = 5      /* a device-side bounded wait expired (reported by conv2d_device_status) */
};

/* Normalization (the pages' `Normalization` enum, plus the group norm of the
 * WebGPU page's GroupNorm backward). BATCH: per-channel statistics over
 * N*OH*OW with running statistics. LAYER: per-image statistics over OH*OW*OC
 * of the stored pre-activations (the pages' LAYER_NORM branches), per-channel
 * gamma / beta, no running statistics. GROUP: desc.groups groups of OC/groups
 * consecutive channels, statistics per (image, group) over OH*OW*OC/groups
 * stored pre-activations, per-channel gamma / beta, no running statistics
 * (GROUP with groups = 1 computes LAYER). */
enum { CONV2D_NORM_NONE = 0, CONV2D_NORM_BATCH = 1, CONV2D_NORM_LAYER = 2, CONV2D_NORM_GROUP = 3 };

/* Activation applied after (optional) normalization. Conv layers take the
 * first four. */
enum {
    CONV2D_ACT_IDENTITY = 0,
    CONV2D_ACT_RELU = 1,
    CONV2D_ACT_TANH = 2,
    CONV2D_ACT_SIGMOID = 3,
    CONV2D_ACT_GELU = 4, /* dense layers only: z/2 (1 + tanh(sqrt(2/pi) (z + 0.044715 z^3))) */
    CONV2D_ACT_SILU = 5  /* dense layers only: z / (1 + exp(-z)) */
};

/* Element types. Conv layers (x, w, pre_act, y, dy, dx): FP32 or BF16. FP32 runs the contractions as
 * 3xTF32 (split operands, fp32 accumulation) for fp32 accuracy; BF16 runs
 * bf16 x bf16 -> fp32 accumulation. */
enum {
    CONV2D_FP32 = 0,
    CONV2D_BF16 = 1,
    CONV2D_FP16 = 2, /* conv2d_mat only */
    CONV2D_E4M3 = 3  /* conv2d_mat only: 8-bit floats (4 exponent, 3 mantissa bits, no infinities) with scales */
};

/* Operation selector for conv2d_workspace_size(). */
enum { CONV2D_OP_FWD_TRAIN = 0, CONV2D_OP_FWD_INFER = 1, CONV2D_OP_BWD = 2 };

/* Layer spec. eps is read for BATCH and LAYER norm (1/sqrt(var+eps), biased
 * variance); momentum only for BATCH
 * (running = (1-momentum)*running + momentum*batch, biased batch variance).
 * bn_eval != 0 selects batch norm in evaluation mode inside training (the
 * pages' mode::Evaluation): conv2d_fwd_train normalises with the running
 * statistics, writes them as save_mean / save_inv_std (= 1/sqrt(var+eps)) and
 * updates nothing; conv2d_bwd then uses the frozen-statistics backward
 * (d_conv = act'(bn) * dy * gamma * inv_std). Zero keeps training mode.
 * Layer and group norm have no evaluation mode on the pages: bn_eval is
 * ignored there. groups is read only for GROUP norm (1 <= groups, OC % groups
 * == 0). */
typedef struct {
    int32_t N, H, W, IC, OC, KH, KW, stride, pad;
    int32_t norm, act, dtype;
    float eps, momentum;
    int32_t bn_eval;
    int32_t groups;
} conv2d_desc;

/* Output spatial size. Returns CONV2D_OK or CONV2D_ERR_INVALID_ARG. */
int conv2d_out_hw(const conv2d_desc* desc, int32_t* OH, int32_t* OW);

/* Host-side validation of a layer spec alone (no pointers). */
int conv2d_validate(const conv2d_desc* desc);

/* Bytes of workspace needed by `op` for this spec (0 if the spec is invalid). */
size_t conv2d_workspace_size(const conv2d_desc* desc, int op);

/* Training forward (`forward` on the generic page; cuDNN conv + bias, batch
 * statistics, affine and activation kernels on the CUDA page).
 *   pre_act  [N][OH][OW][OC] out: conv + bias (the pages' `pre_activations`)
 *   y        [N][OH][OW][OC] out: activation(normalised pre_act)
 *   BATCH norm (else may be NULL):
 *     gamma, beta [OC] in; running_mean, running_var [OC] in/out (EMA update);
 *     save_mean, save_inv_std [OC] out: batch mean and 1/sqrt(var+eps) that
 *     conv2d_bwd needs.
 *   LAYER norm: gamma, beta [OC] in; save_mean, save_inv_std [N] out: the
 *     per-image mean and 1/sqrt(var+eps) of the stored pre_act;
 *     running_mean / running_var are not read and may be NULL.
 *   GROUP norm: as LAYER with save_mean, save_inv_std [N*groups] (index
 *     n*groups + g).
 *   bias may be NULL (treated as zero). */
int conv2d_fwd_train(const conv2d_desc* desc, const void* x, const void* w, const float* bias,
                     const float* gamma, const float* beta, float* running_mean, float* running_var,
                     void* pre_act, float* save_mean, float* save_inv_std, void* y,
                     void* ws, size_t ws_bytes, void* stream);

/* Training forward without a caller workspace. The pages have no counterpart
 * of this call; it exists for callers that cannot allocate device memory: a
 * process whose device memory is fixed at start-up and that may not allocate
 * afterwards (cudaMalloc / cudaFree can synchronise the device and can fail
 * mid-run), or code that is handed only the tensors it passes here and has
 * no way to obtain a scratch buffer.
 * Same arguments and results as conv2d_fwd_train minus ws / ws_bytes. Its
 * scratch is one static 32 MiB device array inside the library (every GPU
 * that loads the library holds it until the process exits). A spec whose
 * conv2d_workspace_size(desc, CONV2D_OP_FWD_TRAIN) exceeds 32 MiB is refused
 * with CONV2D_ERR_WORKSPACE before anything is launched. The first call on a
 * device looks up the array's device address (with that device current);
 * make that first call before any stream capture. All calls share the array
 * and a call rewrites every scratch byte it reads, so nothing is cleared
 * between calls, but calls that overlap on the GPU (several streams, several
 * host threads) race on it: order them. */
int conv2d_fwd_train_noalloc(const conv2d_desc* desc, const void* x, const void* w, const float* bias,
                             const float* gamma, const float* beta, float* running_mean, float* running_var,
                             void* pre_act, float* save_mean, float* save_inv_std, void* y, void* stream);

/* Inference forward (`evaluate`): y = act(norm(conv + bias)), batch norm with
 * the running statistics (`bn_stats_eval` / `bn_forward_eval_running` on the
 * CUDA page), layer / group norm with per-image (per-group) statistics of the
 * stored conv output computed on the fly; no state is written. gamma, beta
 * are read for BATCH, LAYER and GROUP norm, running_mean, running_var only
 * for BATCH. */
int conv2d_fwd_infer(const conv2d_desc* desc, const void* x, const void* w, const float* bias,
                     const float* gamma, const float* beta, const float* running_mean,
                     const float* running_var, void* y, void* ws, size_t ws_bytes, void* stream);

/* Backward (`backward_full`; `backward_input` when dw..dbeta are all NULL;
 * `backward` when dx is NULL). Inputs: x, w, pre_act and (BATCH / LAYER /
 * GROUP) gamma, beta, save_mean, save_inv_std from conv2d_fwd_train,
 * dy = dLoss/dy.
 *   dx [N][H][W][IC]   out (overwritten), may be NULL
 *   dw [OC][KH][KW][IC], dbias [OC]        accumulated, may be NULL together
 *   dgamma, dbeta [OC] (with a norm)        accumulated, may be NULL together
 * The norm backward uses the saved statistics, not recomputed ones; under
 * layer / group norm its projection sums run over each image (group): the
 * GroupNorm backward of the WebGPU page ("groupnorm_backward.wgsl") with the
 * activation derivative in front and the dgamma / dbeta it leaves out.
 * At least one of dx / dw must be non-NULL. */
int conv2d_bwd(const conv2d_desc* desc, const void* x, const void* w, const float* gamma,
               const float* beta, const void* pre_act, const float* save_mean,
               const float* save_inv_std, const void* dy, void* dx, float* dw, float* dbias,
               float* dgamma, float* dbeta, void* ws, size_t ws_bytes, void* stream);

/* ------------------------------------------------------------------------
 * The residual block: RMS norm, layer norm, dense layer, 8-bit activation
 * checkpoints.
 *
 * These calls take matrices of rows (tokens, or the pixels of an NHWC tensor:
 * N*H*W rows of C columns) by columns (features), each described by a
 * conv2d_mat. The conventions above hold (device pointers aligned to 16
 * bytes, caller-owned memory, asynchronous on `stream`, status codes), with
 * these differences: rows may be strided (what lies between the rows of an
 * output stays as it was), a row count of zero is valid (the
 * call writes nothing, except that gradients to be overwritten become zero),
 * and gradients are accumulated only where `accumulate` is nonzero and
 * overwritten otherwise.
 *
 * Sums (dot products, mean squares, column sums) are held in fp32; an output
 * of fewer bits is rounded once, to nearest even. Results do not depend on
 * timing: every sum is formed in a fixed order.
 * ------------------------------------------------------------------------ */

/* A row-major matrix in device memory.
 *   type   FP32, BF16, FP16 or E4M3
 *   ld     elements from the start of one row to the next, at least the
 *          number of columns; 0 stands for the number of columns
 *   group, scale   E4M3 only: columns that share a scale (32, 128, or 0 for a
 *          whole row) and the scales, one byte for each group, dense, row by
 *          row ([rows][ceil(columns / group)]): byte s stands for 2^(s - 127).
 *          The element (r, c) has the value data[r][c] * scale(r, c).
 *          With group CONV2D_TILE 128 rows by 128 columns share one
 *          ([ceil(rows / 128)][ceil(columns / 128)]). `scale` has no alignment
 *          rule. */
#define CONV2D_TILE (-128)
typedef struct {
    void* data;
    int64_t ld;
    int32_t type;
    int32_t group;
    uint8_t* scale;
} conv2d_mat;

/* 8-bit checkpoints. conv2d_q8_encode writes x (FP32, BF16 or FP16) as E4M3:
 * the scale of a group is the smallest power of two (2^-126 .. 2^127) that
 * keeps every finite value within 448 times the scale (1 for a group without
 * a finite nonzero value); values are rounded to nearest even (relative error
 * at most 2^-4 down to 2^-6 of the scale, absolute error at most 2^-10 of the
 * scale below); infinities and NaN become NaN. conv2d_q8_decode writes the
 * values it stands for, clamped to the largest finite value of the type (the
 * rounding to 8 bits may carry a value past it): exact otherwise in FP32, and
 * in BF16 for scales of 2^-124 or more; FP16 rounds what lies below its
 * normal range. */
int conv2d_q8_encode(int64_t rows, int32_t cols, const conv2d_mat* x, const conv2d_mat* q8, void* stream);
int conv2d_q8_decode(int64_t rows, int32_t cols, const conv2d_mat* q8, const conv2d_mat* x, void* stream);

/* Root-mean-square norm of the rows of h = x + residual:
 *   s = 1 / sqrt(mean_j h_j^2 + eps),   y_j = gamma_j h_j s
 *   x, residual, h, y   one type T of FP32, BF16, FP16. residual and h are
 *                given together or both NULL (then h = x and is not written);
 *                h is rounded to T, and the norm is taken of the rounded h.
 *                h may be the same buffer as x or as residual.
 *   q8           E4M3 form of y, from the unrounded y (see conv2d_q8_encode)
 *   inv_rms [rows]  s, for conv2d_rms_norm_bwd
 * y, q8 and inv_rms may be NULL; one of y and q8 is not. The squares are
 * summed in fp32: where that sum passes 3.4e38 (a root mean square of
 * 1.8e19 / sqrt(cols) and more), s and the row's finite y become 0. */
int conv2d_rms_norm_fwd(int64_t rows, int32_t cols, float eps, const conv2d_mat* x, const conv2d_mat* residual,
                        const float* gamma, const conv2d_mat* h, const conv2d_mat* y, const conv2d_mat* q8,
                        float* inv_rms, void* stream);

/* Bytes of workspace of conv2d_rms_norm_bwd (0 if the sizes are invalid). */
size_t conv2d_rms_norm_bwd_workspace_size(int64_t rows, int32_t cols);

/* Backward of conv2d_rms_norm_fwd. h, dy, dh, dx have one type T.
 *   dx = s gamma dy - h s^3 mean_j(gamma_j dy_j h_j) + dh  (the gradient of x
 *   and of residual); dgamma = sum over rows of dy h s.
 * dh, the gradient that reaches h beside the norm, may be NULL, and may be
 * the same buffer as dx. dx or dgamma may be NULL, not both. */
int conv2d_rms_norm_bwd(int64_t rows, int32_t cols, const conv2d_mat* h, const float* gamma, const float* inv_rms,
                        const conv2d_mat* dy, const conv2d_mat* dh, const conv2d_mat* dx, float* dgamma,
                        int accumulate, void* ws, size_t ws_bytes, void* stream);

/* Layer norm of the rows of h = x + residual:
 *   m = mean_j h_j,   s = 1 / sqrt(mean_j (h_j - m)^2 + eps),
 *   y_j = gamma_j (h_j - m) s + beta_j
 * beta may be NULL (zero); mean [rows] and inv_std [rows] receive m and s for
 * conv2d_layer_norm_bwd and may be NULL. The rest is as in
 * conv2d_rms_norm_fwd; the squares are those of the distances from m, summed
 * after it. */
int conv2d_layer_norm_fwd(int64_t rows, int32_t cols, float eps, const conv2d_mat* x, const conv2d_mat* residual,
                          const float* gamma, const float* beta, const conv2d_mat* h, const conv2d_mat* y,
                          const conv2d_mat* q8, float* mean, float* inv_std, void* stream);

/* Bytes of workspace of conv2d_layer_norm_bwd (0 if the sizes are invalid). */
size_t conv2d_layer_norm_bwd_workspace_size(int64_t rows, int32_t cols);

/* Backward of conv2d_layer_norm_fwd. With n = (h - m) s and g = gamma dy:
 *   dx = s (g - mean_j g_j - n mean_j(g_j n_j)) + dh  (the gradient of x and of
 *   residual); dgamma = sum over rows of dy n; dbeta = sum over rows of dy.
 * dh may be NULL, and may be the same buffer as dx. Of dx, dgamma and dbeta
 * one or two may be NULL; without the two sums ws may be NULL. */
int conv2d_layer_norm_bwd(int64_t rows, int32_t cols, const conv2d_mat* h, const float* gamma, const float* mean,
                          const float* inv_std, const conv2d_mat* dy, const conv2d_mat* dh, const conv2d_mat* dx,
                          float* dgamma, float* dbeta, int accumulate, void* ws, size_t ws_bytes, void* stream);

/* Dense layer: y = act(z) + residual, z = x w^T + bias.
 * x [M][K], w [N][K], residual, y, z [M][N]; dtype (BF16 or FP16) is the type
 * of residual, y, dx, dy and of operands that are not E4M3. Products of BF16 /
 * FP16 operands accumulate in fp32; the tensor cores truncate those sums, so
 * terms of one sign lose up to 2^-23.3 of the sum for every 16 of them (4,096
 * terms 2.4e-5, 65,536 terms 3.9e-4; terms of either sign far less). That holds
 * for y over K and dx over N; dw is summed in pieces over M, so that no more is
 * lost than 2.4e-5 in FP32 and a fifth of the rounding of FP16 or BF16.
 * Where x and w are both E4M3 with one scale a row, the product runs on the
 * 8-bit operands and the scales are applied to its sums. Where x has a scale
 * for each row and 128 columns, and w that or one for 128 rows by 128 columns
 * (CONV2D_TILE), it runs on the 8-bit operands too: the tensor core multiplies
 * the partial sums of every 32 columns by both scales (bytes 1 to 254, as
 * conv2d_q8_encode writes them) before it adds them up. Any other E4M3 operand
 * is decoded to dtype first. */
typedef struct {
    int64_t M;          /* rows of x and y */
    int32_t K, N;       /* features in and out */
    int32_t act, dtype;
    int32_t accumulate; /* backward: add to dw and dbias (1) or overwrite them (0) */
} conv2d_dense_desc;

/* Bytes of workspace (0 if the arguments are invalid); of the matrices only
 * data's alignment, ld, type and group are looked at. 256 stands for a call
 * that keeps nothing in it: conv2d_dense_fwd then takes ws = NULL. A call
 * that does needs more. */
size_t conv2d_dense_fwd_workspace_size(const conv2d_dense_desc* desc, const conv2d_mat* x, const conv2d_mat* w);
size_t conv2d_dense_bwd_workspace_size(const conv2d_dense_desc* desc, const conv2d_mat* x, const conv2d_mat* w,
                                       const conv2d_mat* pre_act, const conv2d_mat* dy, const conv2d_mat* dx,
                                       const conv2d_mat* dw, const float* dbias);

/* Forward. bias [N], residual and pre_act may be NULL. pre_act receives z for
 * the backward pass, in dtype or as E4M3 with groups of 32; y is computed
 * from the unrounded z. residual may be the same buffer as y. */
int conv2d_dense_fwd(const conv2d_dense_desc* desc, const conv2d_mat* x, const conv2d_mat* w, const float* bias,
                     const conv2d_mat* residual, const conv2d_mat* pre_act, const conv2d_mat* y, void* ws,
                     size_t ws_bytes, void* stream);

/* Backward: dz = dy act'(z), dx = dz w, dw = dz^T x, dbias = sum over rows of
 * dz (the gradient of residual is dy itself). x, w and pre_act may be E4M3
 * (checkpoints); pre_act may be NULL when act is IDENTITY. dz is stored in
 * dtype for the two products (with IDENTITY dz is dy); dbias sums the
 * unrounded dz. dx, dw, dbias may be NULL, not all; dw is FP32 or dtype.
 * Where w is E4M3 with CONV2D_TILE, dx is a product of 8-bit operands: dz, as
 * it is stored in dtype, goes to E4M3 with a scale for each row and 128
 * columns. Other E4M3 operands of the two products are decoded. */
int conv2d_dense_bwd(const conv2d_dense_desc* desc, const conv2d_mat* x, const conv2d_mat* w,
                     const conv2d_mat* pre_act, const conv2d_mat* dy, const conv2d_mat* dx, const conv2d_mat* dw,
                     float* dbias, void* ws, size_t ws_bytes, void* stream);

/* ------------------------------------------------------------------------
 * Mixture of experts, for a few tokens (serving).
 *   l = x R^T; a token's experts are the k largest of its logits (of equal ones
 *   the lower index first; NaN counts as the largest), their weights
 *   p = exp(l - max) / sum of exp(l - max) over the chosen experts (normalize)
 *   or over all
 *   h_e = act(x w1_e^T + b1_e), or gated: act(x w1_e^T + b1_e) times
 *   (x w3_e^T + b3_e), where w3_e follows w1_e: rows F .. 2F - 1
 *   y = sum over the chosen experts of p_e (h_e w2_e^T + b2_e) + residual
 * The logits and p are formed in fp32; h is rounded to dtype once, and the
 * experts' outputs are weighted and added in fp32. Experts in 8 bits take x
 * and h in 8 bits too, one scale for 128 columns (h from its fp32 values),
 * and run on the 8-bit operands. What an expert's weights hold reaches only
 * the tokens that chose it.
 * ------------------------------------------------------------------------ */
typedef struct {
    int32_t T;         /* tokens, at most 64 */
    int32_t D, F;      /* features of a token, inner features of an expert: multiples of 8 (8 bits: of 128) */
    int32_t E, k;      /* experts, at most 256, and chosen ones for each token, at most 16 */
    int32_t act;
    int32_t gated, normalize;
    int32_t dtype;     /* BF16 or FP16: x, residual, y, and weights that are not E4M3 */
} conv2d_moe_desc;

/* Bytes of workspace (0 if the arguments are invalid); of the matrices only
 * type, ld and group are looked at. */
size_t conv2d_moe_fwd_workspace_size(const conv2d_moe_desc* desc, const conv2d_mat* w1, const conv2d_mat* w2);

/* x, residual, y [T][D]; router [E][D] in dtype or FP32; w1 [E F][D] (gated:
 * [E 2F][D]) and w2 [E D][F], the experts' matrices below each other, both in
 * dtype or both E4M3 with group CONV2D_TILE; b1 [E][F] (gated: [E][2F]) and
 * b2 [E][D] fp32, or NULL; residual may be NULL, and may be the same buffer
 * as y. Rows of x, router, w1 and w2 start on 16-byte boundaries
 * (CONV2D_ERR_UNSUPPORTED otherwise). experts [T][k] and weights [T][k]
 * receive the chosen experts and p, the largest first. */
int conv2d_moe_fwd(const conv2d_moe_desc* desc, const conv2d_mat* x, const conv2d_mat* router, const conv2d_mat* w1,
                   const float* b1, const conv2d_mat* w2, const float* b2, const conv2d_mat* residual, const conv2d_mat* y,
                   int32_t* experts, float* weights, void* ws, size_t ws_bytes, void* stream);

/* Synchronises `stream`, then reads and clears this device's error word,
 * which kernels set when a bounded wait expires. Returns CONV2D_OK,
 * CONV2D_ERR_TIMEOUT (with *site, if non-NULL, set to the wait site code) or
 * CONV2D_ERR_CUDA. */
int conv2d_device_status(void* stream, int32_t* site);

/* Diagnostic for the device-side failure path (no counterpart on the pages).
 * Launches one block whose thread waits, with the library's bounded wait, on a
 * barrier that nothing completes. After the wait limit (about 2 s) the wait
 * gives up, records site 6 in the device error word and the kernel ends; no
 * fault, trap or hang is involved and the context stays usable.
 * conv2d_device_status then returns CONV2D_ERR_TIMEOUT with site 6. */
int conv2d_selftest_wait_limit(void* stream);

/* Human-readable name of a status code (static string). */
const char* conv2d_status_str(int status);

/* Kernel timing for measurement. While enabled (on != 0), every kernel the
 * library launches is bracketed by CUDA events on its stream and recorded in
 * a fixed ring of 256 launches. conv2d_prof_read synchronises the device and
 * copies up to `cap` records (oldest first): a static kernel name and the
 * elapsed milliseconds; it returns the number copied and clears the ring.
 * Off by default; when off no events are recorded. */
int conv2d_prof_enable(int on);
int conv2d_prof_read(const char** names, float* ms, int cap);

#ifdef __cplusplus
}
#endif
#endif /* CONV2D_GB300_H */
