"""The residual block's operators on torch tensors: RMS norm, dense layer, 8-bit checkpoints.

Matrices are 2-D CUDA tensors of rows by features; rows may be strided (the last dimension is contiguous, the
first element on a 16-byte boundary). Outputs that are not handed in are allocated with torch; workspaces
and new outputs come from torch's allocator, in the pool of the stream the call runs on. Every argument is checked before a launch
(ValueError); the arithmetic is in the library's kernels (conv2d_layer_gb300.abi).

`stream`: a torch.cuda.Stream or None for the current stream of the tensors' device. With another stream than
the current one, the caller orders the two (as for any torch operation on a side stream).
"""
import functools
from typing import NamedTuple, Optional

import torch

from . import abi

GROUP = 32  # columns of an 8-bit tensor that share a scale, when not a whole row (0)
ACTS = {"identity": abi.ACT_IDENTITY, "relu": abi.ACT_RELU, "tanh": abi.ACT_TANH, "sigmoid": abi.ACT_SIGMOID,
        "gelu": abi.ACT_GELU, "silu": abi.ACT_SILU}
_TYPES = {torch.float32: abi.FP32, torch.bfloat16: abi.BF16, torch.float16: abi.FP16}
_HALF = (torch.bfloat16, torch.float16)


class Q8(NamedTuple):
    """A matrix in 8 bits: value(r, c) = q[r, c] * 2 ** (scale[r, c // group] - 127), or scale[r, 0] with group 0."""
    q: torch.Tensor      # [rows, cols] torch.float8_e4m3fn
    scale: torch.Tensor  # [rows, ceil(cols / group)] torch.uint8, contiguous
    group: int = GROUP   # 32, or 0: one scale a row

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


def q8_scales(cols, group):
    """Scale bytes a row."""
    if group not in (0, GROUP):
        raise ValueError(f"group: 0 (a whole row) or {GROUP}, got {group!r}")
    return -(-cols // GROUP) if group else 1


def q8_empty(rows, cols, group=GROUP, device="cuda"):
    return Q8(torch.empty((rows, cols), dtype=torch.float8_e4m3fn, device=device),
              torch.empty((rows, q8_scales(cols, group)), dtype=torch.uint8, device=device), group)


# ------------------------------------------------------------------ checks
# These run on every call, a small call's time is mostly theirs: the common path tests and returns, what is wrong
# is found out afterwards.
def _mat(t, name, rows, cols, dtypes, device):
    """A checked matrix argument as conv2d_mat."""
    if type(t) is Q8:
        return _mat_q8(t, name, rows, cols, dtypes, device)
    if isinstance(t, torch.Tensor) and t.shape == (rows, cols) and t.dtype in dtypes and t.device == device \
            and t.dtype in _TYPES:
        ld, step = t.stride()
        ptr = t.data_ptr()
        if rows <= 1:
            ld = cols
        if (step == 1 or cols == 1) and ld >= cols and not ptr & 15:
            return abi.Mat(ptr, ld, _TYPES[t.dtype], 0, None)
    _refuse(t, name, rows, cols, dtypes, device)


def _mat_q8(t, name, rows, cols, dtypes, device):
    if torch.float8_e4m3fn not in dtypes:
        raise ValueError(f"{name}: an 8-bit matrix is not taken here")
    q, scale, group = t
    shape = (rows, q8_scales(cols, group))
    if not isinstance(scale, torch.Tensor) or scale.dtype != torch.uint8 or scale.shape != shape:
        raise ValueError(f"{name}: scales are uint8 of shape {shape}")
    if not scale.is_contiguous() or scale.device != device:
        raise ValueError(f"{name}: scales must be contiguous and on {device}")
    if isinstance(q, torch.Tensor) and q.shape == (rows, cols) and q.dtype == torch.float8_e4m3fn and q.device == device:
        ld, step = q.stride()
        ptr = q.data_ptr()
        if rows <= 1:
            ld = cols
        if (step == 1 or cols == 1) and ld >= cols and not ptr & 15:
            return abi.Mat(ptr, ld, abi.E4M3, group, scale.data_ptr())
    _refuse(q, name, rows, cols, _E4M3, device)


def _refuse(t, name, rows, cols, dtypes, device):
    """Says what is wrong with a matrix argument."""
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name}: expected a torch.Tensor, got {type(t).__name__}")
    if tuple(t.shape) != (rows, cols):
        raise ValueError(f"{name}: shape {tuple(t.shape)} does not match {(rows, cols)}")
    if t.dtype == torch.float8_e4m3fn and dtypes is not _E4M3:
        raise ValueError(f"{name}: 8-bit values need their scales (Q8)")
    if t.dtype not in dtypes:
        raise ValueError(f"{name}: dtype {t.dtype} is not one of {[str(d) for d in dtypes]}")
    if t.device != device:
        raise ValueError(f"{name}: must be on {device} (got {t.device})")
    if t.data_ptr() & 15:
        raise ValueError(f"{name}: must start on a 16-byte boundary")
    raise ValueError(f"{name}: features must be contiguous and rows must not overlap (strides {t.stride()})")


def _new(rows, cols, dtype, device):
    """A new matrix and its conv2d_mat."""
    t = torch.empty((rows, cols), dtype=dtype, device=device)
    return t, abi.Mat(t.data_ptr(), cols, _TYPES[dtype], 0, None)


def _vec(t, name, n, device):
    """A checked contiguous fp32 vector."""
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name}: expected a torch.Tensor, got {type(t).__name__}")
    if t.dtype != torch.float32 or t.shape != (n,) or not t.is_contiguous() or t.device != device:
        raise ValueError(f"{name}: expected a contiguous float32 tensor of shape ({n},) on {device}, got "
                         f"{t.dtype} {tuple(t.shape)} on {t.device}")
    if t.data_ptr() & 15:
        raise ValueError(f"{name}: must start on a 16-byte boundary")
    return t


def _source(t, name, dtypes):
    """(rows, cols, device) of the argument the others are checked against."""
    m = t.q if type(t) is Q8 else t
    if not isinstance(m, torch.Tensor):
        raise ValueError(f"{name}: expected a torch.Tensor or Q8, got {type(m).__name__}")
    if m.dim() != 2 or m.shape[1] < 1:
        raise ValueError(f"{name}: expected rows by at least one feature, got shape {tuple(m.shape)}")
    if m.dtype not in dtypes:
        raise ValueError(f"{name}: dtype {m.dtype} is not one of {[str(d) for d in dtypes]}")
    rows, cols = m.shape
    return rows, cols, m.device


def _streamed(f):
    """Runs a call on `stream`: made current, so that what the call allocates belongs to it."""
    @functools.wraps(f)
    def call(*args, stream=None, **kw):
        if stream is None:
            return f(*args, **kw)
        with torch.cuda.stream(torch.cuda.ExternalStream(stream) if isinstance(stream, int) else stream):
            return f(*args, **kw)
    return call


def _run(device, call, *args):
    """One library call on the current stream of `device`, where every checked tensor lies."""
    if device.type != "cuda":
        raise ValueError(f"the tensors must be in CUDA device memory (got {device})")
    s = torch._C._cuda_getCurrentRawStream(device.index)
    if torch.cuda.current_device() == device.index:
        abi.check(call(*args, stream=s), call.__name__)
    else:
        with torch.cuda.device(device):
            abi.check(call(*args, stream=s), call.__name__)


def _scratch(nbytes, device):
    return torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device)


def _act(act):
    if act not in ACTS:
        raise ValueError(f"act: one of {sorted(ACTS)}, got {act!r}")
    return ACTS[act]


_FLOATS = (torch.float32, torch.bfloat16, torch.float16)
_E4M3 = (torch.float8_e4m3fn,)


# ------------------------------------------------------------------ 8-bit checkpoints
@_streamed
def q8_encode(x, group=GROUP, out=None):
    """x [rows, cols] (fp32, bf16, fp16) in 8 bits, with one scale for `group` columns (32, or 0: a row)."""
    rows, cols, dev = _source(x, "x", _FLOATS)
    if out is None:
        out = q8_empty(rows, cols, group, dev)
    elif not isinstance(out, Q8):
        raise ValueError("out: expected a Q8")
    mx, mo = _mat(x, "x", rows, cols, _FLOATS, dev), _mat(out, "out", rows, cols, _E4M3, dev)
    _run(dev, abi.conv2d_q8_encode, rows, cols, mx, mo)
    return out


@_streamed
def q8_decode(q8, dtype=torch.bfloat16, out=None):
    """The values an 8-bit matrix stands for, in fp32, bf16 or fp16."""
    if not isinstance(q8, Q8):
        raise ValueError("q8: expected a Q8")
    rows, cols, dev = _source(q8, "q8", _E4M3)
    if dtype not in _FLOATS:
        raise ValueError(f"dtype: one of {[str(d) for d in _FLOATS]}, got {dtype}")
    mq = _mat(q8, "q8", rows, cols, _E4M3, dev)
    if out is None:
        out, mo = _new(rows, cols, dtype, dev)
    else:
        mo = _mat(out, "out", rows, cols, (dtype,), dev)
    _run(dev, abi.conv2d_q8_decode, rows, cols, mq, mo)
    return out


# ------------------------------------------------------------------ RMS norm
@_streamed
def rms_norm_fwd(x, gamma, eps=1e-6, residual=None, y=True, group=None, h=None, q8=None, inv_rms=None):
    """h = x + residual; y = gamma * h / sqrt(mean(h^2) + eps), row by row.

    y: True (allocate), False (none) or an output tensor. group: None, or the group of an 8-bit form of y
    (32, or 0: a row); q8: an output Q8 for it. h: output for x + residual (may be x or residual itself).
    Returns RmsNorm(h, y, q8, inv_rms); h and inv_rms are what rms_norm_bwd takes."""
    rows, cols, dev = _source(x, "x", _FLOATS)
    dt = (x.dtype,)
    _vec(gamma, "gamma", cols, dev)
    if y is True:
        y, my = _new(rows, cols, x.dtype, dev)
    elif y is False:
        y = my = None
    else:
        my = _mat(y, "y", rows, cols, dt, dev)
    if q8 is None and group is not None:
        q8 = q8_empty(rows, cols, group, dev)
    elif q8 is not None and not isinstance(q8, Q8):
        raise ValueError("q8: expected a Q8")
    if y is None and q8 is None:
        raise ValueError("y or an 8-bit form of it (group, q8) must be asked for")
    if residual is None:
        if h is not None:
            raise ValueError("h: an output of x + residual, but there is no residual")
        mr = mh = None
    else:
        mr = _mat(residual, "residual", rows, cols, dt, dev)
        if h is None:
            h, mh = _new(rows, cols, x.dtype, dev)
        else:
            mh = _mat(h, "h", rows, cols, dt, dev)
    if inv_rms is None:
        inv_rms = torch.empty(rows, dtype=torch.float32, device=dev)
    else:
        _vec(inv_rms, "inv_rms", rows, dev)
    mx = _mat(x, "x", rows, cols, dt, dev)
    mq = None if q8 is None else _mat(q8, "q8", rows, cols, _E4M3, dev)
    _run(dev, abi.conv2d_rms_norm_fwd, rows, cols, eps, mx, mr, gamma, mh, my, mq, inv_rms)
    return RmsNorm(x if residual is None else h, y, q8, inv_rms)


@_streamed
def rms_norm_bwd(h, gamma, inv_rms, dy, dh=None, dx=None, dgamma=None, need_dx=True, need_dgamma=True):
    """(dx, dgamma) of rms_norm_fwd: dx is the gradient of x and of residual, dh the gradient that reaches h
    beside the norm. dx may be dh itself. A dgamma that is handed in is accumulated into."""
    rows, cols, dev = _source(h, "h", _FLOATS)
    dt = (h.dtype,)
    _vec(gamma, "gamma", cols, dev)
    _vec(inv_rms, "inv_rms", rows, dev)
    if not need_dx and not need_dgamma:
        raise ValueError("need_dx or need_dgamma")
    mh, md = _mat(h, "h", rows, cols, dt, dev), _mat(dy, "dy", rows, cols, dt, dev)
    ms = None if dh is None else _mat(dh, "dh", rows, cols, dt, dev)
    mx = None
    if need_dx and dx is None:
        dx, mx = _new(rows, cols, h.dtype, dev)
    elif need_dx:
        mx = _mat(dx, "dx", rows, cols, dt, dev)
    accumulate = dgamma is not None
    if need_dgamma and dgamma is None:
        dgamma = torch.empty(cols, dtype=torch.float32, device=dev)
    if need_dgamma:
        _vec(dgamma, "dgamma", cols, dev)
    ws = _scratch(abi.conv2d_rms_norm_bwd_workspace_size(rows, cols), dev) if need_dgamma else None
    _run(dev, abi.conv2d_rms_norm_bwd, rows, cols, mh, gamma, inv_rms, md, ms, mx, dgamma if need_dgamma else None,
         accumulate, ws)
    return dx if need_dx else None, dgamma if need_dgamma else None


# ------------------------------------------------------------------ dense layer
@_streamed
def dense_fwd(x, w, bias=None, act="identity", residual=None, save="none", dtype=None, y=None, pre_act=None):
    """y = act(x w^T + bias) + residual; x [M, K], w [N, K], residual and y [M, N], bias [N] fp32.

    dtype (bf16 or fp16) is the type of y, residual and the operands that are not Q8; it is x's (or w's) where
    those are not Q8. Two Q8 operands with one scale a row run on the 8-bit tensor cores, other Q8 operands are
    decoded first. save: "none", "full" or "q8" (groups of 32) keeps the activation's input for dense_bwd;
    pre_act: an output for it. Returns (y, pre_act)."""
    M, K, dev = _source(x, "x", _HALF + _E4M3)
    N = _source(w, "w", _HALF + _E4M3)[0]
    for t in (x, w):
        if not isinstance(t, Q8):
            if dtype is not None and t.dtype != dtype:
                raise ValueError(f"dtype {dtype}, but an operand is {t.dtype}")
            dtype = t.dtype
    if dtype not in _HALF:
        raise ValueError("dtype: bfloat16 or float16 (needed where both operands are Q8)")
    if N < 1:
        raise ValueError("w: expected at least one output feature")
    code = _act(act)
    dt, any8 = (dtype,), (dtype,) + _E4M3
    mx, mw = _mat(x, "x", M, K, any8, dev), _mat(w, "w", N, K, any8, dev)
    if bias is not None:
        _vec(bias, "bias", N, dev)
    mr = None if residual is None else _mat(residual, "residual", M, N, dt, dev)
    if y is None:
        y, my = _new(M, N, dtype, dev)
    else:
        my = _mat(y, "y", M, N, dt, dev)
    if save not in ("none", "full", "q8"):
        raise ValueError(f"save: none, full or q8, got {save!r}")
    if pre_act is None:
        if save == "full":
            pre_act = torch.empty((M, N), dtype=dtype, device=dev)
        elif save == "q8":
            pre_act = q8_empty(M, N, GROUP, dev)
    elif save == "none" or isinstance(pre_act, Q8) != (save == "q8"):
        raise ValueError(f"pre_act: not an output for save={save!r}")
    mz = None if pre_act is None else _mat(pre_act, "pre_act", M, N, any8, dev)
    if isinstance(pre_act, Q8) and pre_act.group != GROUP:
        raise ValueError(f"pre_act: groups of {GROUP}")
    d = abi.DenseDesc(M, K, N, code, _TYPES[dtype], 0)
    n = abi.conv2d_dense_fwd_workspace_size(d, mx, mw)
    ws = _scratch(n, dev) if n > 256 else None  # 256: nothing to decode or repack
    _run(dev, abi.conv2d_dense_fwd, d, mx, mw, bias, mr, mz, my, ws)
    return y, pre_act


@_streamed
def dense_bwd(x, w, dy, pre_act=None, act="identity", need_dx=True, need_dw=True, need_dbias=True,
              grad_dtype=torch.float32, dx=None, dw=None, dbias=None):
    """(dx, dw, dbias) of dense_fwd. x, w and pre_act may be Q8; pre_act is what dense_fwd saved (not needed
    without an activation). dw is fp32 or dy's type (grad_dtype); dw and dbias that are handed in (both, or all
    that is asked for) are accumulated into. The gradient of the residual is dy."""
    M, N, dev = _source(dy, "dy", _HALF)
    dt, any8 = (dy.dtype,), (dy.dtype,) + _E4M3
    code = _act(act)
    if not (need_dx or need_dw or need_dbias):
        raise ValueError("need_dx, need_dw or need_dbias")
    K = _source(x if need_dw else w, "x" if need_dw else "w", _HALF + _E4M3)[1] if need_dx or need_dw else 1
    md = _mat(dy, "dy", M, N, dt, dev)
    mx = _mat(x, "x", M, K, any8, dev) if need_dw else None
    mw = _mat(w, "w", N, K, any8, dev) if need_dx else None
    if code != abi.ACT_IDENTITY and pre_act is None:
        raise ValueError(f"pre_act: needed behind {act}")
    mz = _mat(pre_act, "pre_act", M, N, any8, dev) if code != abi.ACT_IDENTITY else None
    given = [t is not None for t, need in ((dw, need_dw), (dbias, need_dbias)) if need]
    if any(given) and not all(given):
        raise ValueError("dw and dbias: hand in both to accumulate, or neither")
    accumulate = any(given)
    mdx = mdw = db = None
    if need_dx and dx is None:
        dx, mdx = _new(M, K, dy.dtype, dev)
    elif need_dx:
        mdx = _mat(dx, "dx", M, K, dt, dev)
    if need_dw and dw is None:
        if grad_dtype not in (torch.float32, dy.dtype):
            raise ValueError(f"grad_dtype: float32 or {dy.dtype}, got {grad_dtype}")
        dw, mdw = _new(N, K, grad_dtype, dev)
    elif need_dw:
        mdw = _mat(dw, "dw", N, K, dt + (torch.float32,), dev)
    if need_dbias:
        db = torch.empty(N, dtype=torch.float32, device=dev) if dbias is None else _vec(dbias, "dbias", N, dev)
    d = abi.DenseDesc(M, K, N, code, _TYPES[dy.dtype], int(accumulate))
    ws = _scratch(abi.conv2d_dense_bwd_workspace_size(d, mx, mw, mz, md, mdx, mdw, db), dev)
    _run(dev, abi.conv2d_dense_bwd, d, mx, mw, mz, md, mdx, mdw, db, ws)
    return dx if need_dx else None, dw if need_dw else None, db


__all__ = ["Q8", "RmsNorm", "q8_empty", "q8_scales", "q8_encode", "q8_decode", "rms_norm_fwd", "rms_norm_bwd",
           "dense_fwd", "dense_bwd", "ACTS", "GROUP"]
