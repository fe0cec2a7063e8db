"""The residual block's operators on torch tensors: RMS norm, layer norm, dense layer, 8-bit checkpoints, and a mixture
of experts.

Matrices are 2-D CUDA tensors of rows by features; rows may be strided (the last dimension is contiguous, the
first element on a 16-byte boundary). Outputs that are not handed in are allocated with torch; workspaces
and new outputs come from torch's allocator, in the pool of the stream the call runs on. Every argument is checked
before a launch (ValueError); a status of the library raises abi.Conv2dError. The checks are in csrc/binding.cpp,
the arithmetic in the library's kernels.

`stream`: a torch.cuda.Stream of the tensors' device, a raw stream handle (an int) of that device, or None for its
current stream. With another stream than the current one, the caller orders the two (as for any torch operation on a
side stream).
"""
import functools
from typing import NamedTuple, Optional

import torch

from . import abi, build

GROUP = 32  # columns of an 8-bit tensor that share a scale, when not a whole row (0)
WIDE = 128  # the wider group: what the 8-bit matrix product takes
TILE = abi.TILE  # a group of 128 rows by 128 columns, for weights
# gelu is the tanh form, z/2 (1 + tanh(sqrt(2/pi) (z + 0.044715 z^3))): torch's gelu(approximate="tanh"), not its default
ACTS = {"identity": abi.ACT_IDENTITY, "relu": abi.ACT_RELU, "tanh": abi.ACT_TANH, "sigmoid": abi.ACT_SIGMOID,
        "gelu": abi.ACT_GELU, "silu": abi.ACT_SILU}
_SAVES = {"none": 0, "full": 1, "q8": 2}
_module = None


def _binding():
    """The native binding; loads it (building first if needed) at the first call, and raises if that is impossible."""
    global _module
    if _module is None:
        abi.lib()
        m = build.load_binding()
        m.init(abi.lib_path())
        _module = m
    return _module


class Q8(NamedTuple):
    """A matrix in 8 bits: value(r, c) = q[r, c] * 2 ** (scale[r, c // group] - 127), scale[r, 0] with group 0, or
    scale[r // 128, c // 128] with group TILE."""
    q: torch.Tensor      # [rows, cols] torch.float8_e4m3fn
    scale: torch.Tensor  # [rows, ceil(cols / group)] (TILE: [ceil(rows / 128), ceil(cols / 128)]) torch.uint8, contiguous
    group: int = GROUP   # 32, 128 (WIDE), 0: one scale a row, or TILE

    @property
    def shape(self):
        return self.q.shape

    @property
    def device(self):
        return self.q.device


class RmsNorm(NamedTuple):
    h: torch.Tensor            # x + residual (x itself without a residual)
    y: Optional[torch.Tensor]
    q8: Optional[Q8]
    inv_rms: torch.Tensor      # [rows] fp32


class LayerNorm(NamedTuple):
    h: torch.Tensor            # x + residual (x itself without a residual)
    y: Optional[torch.Tensor]
    q8: Optional[Q8]
    mean: torch.Tensor         # [rows] fp32
    inv_std: torch.Tensor      # [rows] fp32


def q8_scales(cols, group):
    """Scale bytes a row (TILE: a row of tiles)."""
    if group not in (0, GROUP, WIDE, TILE):
        raise ValueError(f"group: 0 (a whole row), {GROUP}, {WIDE} or TILE, got {group!r}")
    return -(-cols // (WIDE if group == TILE else group)) if group else 1


def q8_empty(rows, cols, group=GROUP, device="cuda"):
    tall = -(-rows // 128) if group == TILE else rows
    return Q8(torch.empty((rows, cols), dtype=torch.float8_e4m3fn, device=device),
              torch.empty((tall, q8_scales(cols, group)), dtype=torch.uint8, device=device), group)


def _device_of(args):
    """The device of the first tensor (or Q8) among a call's arguments."""
    return next((a.device for a in args if isinstance(getattr(a, "device", None), torch.device)), None)


def _streamed(f):
    """Runs a call on `stream`: made current, so that what the call allocates belongs to it."""
    @functools.wraps(f)
    def call(*args, stream=None, **kw):
        if stream is None:
            return f(*args, **kw)
        dev = _device_of((*args, *kw.values()))
        if dev is None or dev.type != "cuda":
            return f(*args, **kw)  # refused there
        if isinstance(stream, int):
            stream = torch.cuda.ExternalStream(stream, device=dev)
        elif stream.device != dev:
            raise ValueError(f"stream: of {stream.device}, but the tensors are on {dev}")
        with torch.cuda.stream(stream):
            return f(*args, **kw)
    return call


def _act(act):
    if act not in ACTS:
        raise ValueError(f"act: one of {sorted(ACTS)}, got {act!r}")
    return ACTS[act]


# ------------------------------------------------------------------ 8-bit checkpoints
@_streamed
def q8_encode(x, group=GROUP, out=None):
    """x [rows, cols] (fp32, bf16, fp16) in 8 bits, with one scale for `group` columns (32, 128, or 0: a row) or for 128
    rows by 128 columns (TILE). out: an output Q8, whose group then counts."""
    r = _binding().q8_encode(x, group, out)
    return Q8(r[0], r[1], group) if r is not None else out


@_streamed
def q8_decode(q8, dtype=torch.bfloat16, out=None):
    """The values an 8-bit matrix stands for, in fp32, bf16 or fp16."""
    return _binding().q8_decode(q8, dtype, out)


# ------------------------------------------------------------------ RMS norm
@_streamed
def rms_norm_fwd(x, gamma, eps=1e-6, residual=None, y=True, group=None, h=None, q8=None, inv_rms=None):
    """h = x + residual; y = gamma * h / sqrt(mean(h^2) + eps), row by row.

    y: True (allocate), False (none) or an output tensor. group: None, or the group of an 8-bit form of y
    (32, 128, or 0: a row); q8: an output Q8 for it, whose group then counts. h: output for x + residual (may be x or residual itself).
    Returns RmsNorm(h, y, q8, inv_rms); h and inv_rms are what rms_norm_bwd takes."""
    h, y, q, scale, inv_rms = _binding().rms_norm_fwd(x, gamma, eps, residual, y, group, h, q8, inv_rms)
    return RmsNorm(h, y, q8 if q is None else Q8(q, scale, group), inv_rms)


@_streamed
def rms_norm_bwd(h, gamma, inv_rms, dy, dh=None, dx=None, dgamma=None, need_dx=True, need_dgamma=True):
    """(dx, dgamma) of rms_norm_fwd: dx is the gradient of x and of residual, dh the gradient that reaches h
    beside the norm. dx may be dh itself. A dgamma that is handed in is accumulated into."""
    return _binding().rms_norm_bwd(h, gamma, inv_rms, dy, dh, dx, dgamma, need_dx, need_dgamma)


# ------------------------------------------------------------------ layer norm
@_streamed
def layer_norm_fwd(x, gamma, beta=None, eps=1e-5, residual=None, y=True, group=None, h=None, q8=None, mean=None,
                   inv_std=None):
    """h = x + residual; y = gamma * (h - m) / sqrt(mean((h - m)^2) + eps) + beta, m = mean(h), row by row. beta may be
    None (zero).

    y, group, q8 and h as in rms_norm_fwd. Returns LayerNorm(h, y, q8, mean, inv_std); h, mean and inv_std are what
    layer_norm_bwd takes."""
    h, y, q, scale, mean, inv_std = _binding().layer_norm_fwd(x, gamma, beta, eps, residual, y, group, h, q8, mean, inv_std)
    return LayerNorm(h, y, q8 if q is None else Q8(q, scale, group), mean, inv_std)


@_streamed
def layer_norm_bwd(h, gamma, mean, inv_std, dy, dh=None, dx=None, dgamma=None, dbeta=None, need_dx=True, need_dgamma=True,
                   need_dbeta=True):
    """(dx, dgamma, dbeta) of layer_norm_fwd: dx is the gradient of x and of residual, dh the gradient that reaches h
    beside the norm. dx may be dh itself. dgamma and dbeta that are handed in (both, or the one that is asked for) are
    accumulated into."""
    return _binding().layer_norm_bwd(h, gamma, mean, inv_std, dy, dh, dx, dgamma, dbeta, need_dx, need_dgamma, need_dbeta)


# ------------------------------------------------------------------ dense layer
@_streamed
def dense_fwd(x, w, bias=None, act="identity", residual=None, save="none", dtype=None, y=None, pre_act=None):
    """y = act(x w^T + bias) + residual; x [M, K], w [N, K], residual and y [M, N], bias [N] fp32. act: one of ACTS
    (gelu is the tanh form).

    dtype (bf16 or fp16) is the type of y, residual and the operands that are not Q8; it is x's (or w's) where
    those are not Q8. Two Q8 operands run on the 8-bit tensor cores where both have one scale a row, or where x has one
    for 128 columns (WIDE) and w that or TILE; other Q8 operands are decoded first. save: "none", "full" or "q8" (groups of 32) keeps the activation's input for dense_bwd;
    pre_act: an output for it. residual may be y itself. Returns (y, pre_act)."""
    if save not in _SAVES:
        raise ValueError(f"save: one of {sorted(_SAVES)}, got {save!r}")
    y, z, scale = _binding().dense_fwd(x, w, bias, _act(act), residual, _SAVES[save], dtype, y, pre_act)
    if z is not None:
        pre_act = z if scale is None else Q8(z, scale, GROUP)
    return y, pre_act


@_streamed
def dense_bwd(x, w, dy, pre_act=None, act="identity", need_dx=True, need_dw=True, need_dbias=True,
              grad_dtype=torch.float32, dx=None, dw=None, dbias=None):
    """(dx, dw, dbias) of dense_fwd. x, w and pre_act may be Q8; pre_act is what dense_fwd saved (not needed
    without an activation). dw is fp32 or dy's type (grad_dtype); dw and dbias that are handed in (both, or all
    that is asked for) are accumulated into. The gradient of the residual is dy. With w of TILE dx is a product of 8-bit
    operands (dz with a scale for 128 columns); other Q8 operands are decoded first."""
    return _binding().dense_bwd(x, w, dy, pre_act, _act(act), grad_dtype, dx, dw, dbias, need_dx, need_dw, need_dbias)


# ------------------------------------------------------------------ mixture of experts
class Moe(NamedTuple):
    y: torch.Tensor
    experts: torch.Tensor   # [rows, k] int32, by falling weight
    weights: torch.Tensor   # [rows, k] fp32


def moe_encode(w):
    """Experts' weights [E, rows, cols] (multiples of 128) as the Q8 that moe_fwd takes: one scale for 128 rows by 128
    columns, none across two experts."""
    if not isinstance(w, torch.Tensor) or w.dim() != 3 or w.shape[1] % 128 or w.shape[2] % 128:
        got = f"shape {tuple(w.shape)}" if isinstance(w, torch.Tensor) else type(w).__name__
        raise ValueError(f"w: experts by rows by columns (multiples of 128), got {got}")
    q = q8_encode(w.reshape(-1, w.shape[2]), TILE)
    return Q8(q.q.view(w.shape), q.scale.view(w.shape[0], w.shape[1] // 128, -1), TILE)


@_streamed
def moe_fwd(x, router, w1, w2, k, b1=None, b2=None, act="silu", gated=False, normalize=True, residual=None, y=None):
    """A mixture-of-experts layer for 0 to 64 rows (decoded tokens): each goes through the k experts with the largest
    logits x router^T (of equal ones the lower index first), y = sum of p_e (h_e w2_e^T + b2_e) + residual,
    h_e = act(x w1_e^T + b1_e), times (x w3_e^T + b3_e) where gated.

    x, residual, y [rows, D] bf16 or fp16; router [E, D] of that type or fp32, at most 256 experts; w1 [E, F, D] (gated:
    [E, 2 F, D], w3's rows behind w1's) and w2 [E, D, F], of x's type, or both Q8 (moe_encode), which takes x and h to 8
    bits too, one scale for 128 features; b1 [E, F] (gated: [E, 2 F]) and b2 [E, D] fp32. D and F are multiples of 8 (Q8:
    of 128). p is the softmax over the chosen logits (normalize) or over all. residual may be y itself.
    Returns Moe(y, experts, weights). Nothing is saved for a backward pass."""
    return Moe(*_binding().moe_fwd(x, router, w1, w2, k, b1, b2, _act(act), gated, normalize, residual, y))


__all__ = ["Q8", "RmsNorm", "LayerNorm", "q8_empty", "q8_scales", "q8_encode", "q8_decode", "rms_norm_fwd", "rms_norm_bwd",
           "layer_norm_fwd", "layer_norm_bwd", "dense_fwd", "dense_bwd",
           "Moe", "moe_encode", "moe_fwd", "ACTS", "GROUP", "WIDE", "TILE"]
