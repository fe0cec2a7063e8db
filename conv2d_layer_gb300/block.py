"""FeedForward: the pre-norm residual block on the rows of a conv layer's output (or on tokens).

    h = x + residual                      (x alone without a residual)
    n = gamma * h / rms(h)
    u = act(n w1^T + b1)
    y = u w2^T + b2 + h

act is one of ops.ACTS; gelu is the tanh form (torch's gelu(approximate="tanh"), not its default).
PyTorch supplies device memory and the stream; every step runs in the library's kernels (conv2d_layer_gb300.ops).
The class holds the parameters, the gradients (fp32, accumulated until zero_grad, as in Conv2dLayer) and what the
forward pass saves for the backward pass. With checkpoint="q8" that is kept in 8 bits, one scale for 32 features:
the norm's output n (the input of w1) and the activation's input and output; with "full" in the layer's type. h is
the residual stream and is kept as it is. fwd_infer saves nothing.

An NHWC conv output [N, H, W, C] is N*H*W rows of C features: `rows(y)` views it so without a copy.
"""
import torch

from . import ops


def rows(y):
    """An NHWC tensor as a matrix of pixels by channels (a view)."""
    return y.view(-1, y.shape[-1])


class FeedForward:
    def __init__(self, gamma, w1, b1, w2, b2, act="gelu", dtype=torch.bfloat16, eps=1e-6, checkpoint="q8", device="cuda"):
        if checkpoint not in ("q8", "full"):
            raise ValueError(f"checkpoint: q8 or full, got {checkpoint!r}")
        if act not in ops.ACTS:
            raise ValueError(f"act: one of {sorted(ops.ACTS)}, got {act!r}")
        if dtype not in (torch.bfloat16, torch.float16):
            raise ValueError(f"dtype: torch.bfloat16 or torch.float16, got {dtype!r}")
        inner, width = w1.shape
        for name, t, shape in (("gamma", gamma, (width,)), ("b1", b1, (inner,)), ("w2", w2, (width, inner)),
                               ("b2", b2, (width,))):
            if tuple(t.shape) != shape:
                raise ValueError(f"{name}: shape {tuple(t.shape)} does not match {shape}")
        dev = torch.device(device)
        self.width, self.inner, self.act, self.eps, self.dtype, self.q8 = width, inner, act, eps, dtype, checkpoint == "q8"
        self.gamma, self.b1, self.b2 = (t.to(dev, torch.float32).contiguous() for t in (gamma, b1, b2))
        self.w1, self.w2 = (t.to(dev, dtype).contiguous() for t in (w1, w2))
        self.dgamma, self.db1, self.db2 = (torch.zeros_like(t) for t in (self.gamma, self.b1, self.b2))
        self.dw1, self.dw2 = (torch.zeros(t.shape, device=dev, dtype=torch.float32) for t in (self.w1, self.w2))
        self.saved = None
        self.w8 = self.w8_of = None

    def zero_grad(self):
        for t in (self.dgamma, self.dw1, self.db1, self.dw2, self.db2):
            t.zero_()

    def fwd_train(self, x, residual=None):
        """y [rows, width]; keeps what bwd needs."""
        n = ops.rms_norm_fwd(x, self.gamma, self.eps, residual=residual, group=ops.GROUP if self.q8 else None)
        u, z = ops.dense_fwd(n.y, self.w1, self.b1, self.act, save="q8" if self.q8 else "full")
        y, _ = ops.dense_fwd(u, self.w2, self.b2, residual=n.h)
        kept_n, kept_u = (n.q8, ops.q8_encode(u)) if self.q8 else (n.y, u)
        self.saved = (n.h, n.inv_rms, kept_n, z, kept_u)
        return y

    def bwd(self, dy):
        """The gradient of x (and of residual); accumulates the parameters' gradients. Uses up what was saved."""
        if self.saved is None:
            raise RuntimeError("bwd follows a fwd_train")
        (h, inv, n, z, u), self.saved = self.saved, None
        du, _, _ = ops.dense_bwd(u, self.w2, dy, dw=self.dw2, dbias=self.db2)
        dn, _, _ = ops.dense_bwd(n, self.w1, du, z, self.act, dw=self.dw1, dbias=self.db1)
        dx, _ = ops.rms_norm_bwd(h, self.gamma, inv, dn, dh=dy, dgamma=self.dgamma)
        return dx

    def saved_bytes(self):
        """Bytes kept for the backward pass, without h."""
        def size(t):
            return sum(size(p) for p in t[:2]) if isinstance(t, ops.Q8) else t.numel() * t.element_size()
        return 0 if self.saved is None else sum(size(t) for t in self.saved[1:])

    def _weights(self):
        # tensors made in inference mode carry no version
        return [(t, None if t.is_inference() else t._version) for t in (self.w1, self.w2)]

    def quantize(self):
        """Keeps 8-bit weights, one scale an output feature, for fwd_infer(bits8=True); again after each change of w1
        or w2. fwd_infer refuses 8-bit weights older than a change that torch has seen (not one through .data, a raw
        pointer, or of tensors made in inference mode)."""
        self.w8 = ops.q8_encode(self.w1, 0), ops.q8_encode(self.w2, 0)
        self.w8_of = self._weights()

    def fwd_infer(self, x, residual=None, bits8=False):
        """(y, h) without saving anything, for any number of rows (one for a decoded token). bits8: 8-bit weights
        (quantize) and activations, one scale a token, on the 8-bit tensor cores."""
        if not bits8:
            n = ops.rms_norm_fwd(x, self.gamma, self.eps, residual=residual)
            u, _ = ops.dense_fwd(n.y, self.w1, self.b1, self.act)
            return ops.dense_fwd(u, self.w2, self.b2, residual=n.h)[0], n.h
        if self.w8 is None:
            raise RuntimeError("bits8 follows quantize()")
        if self.w8_of and any(a is not b or u != v for (a, u), (b, v) in zip(self.w8_of, self._weights())):
            raise RuntimeError("w1 or w2 has changed: bits8 needs another quantize()")
        n = ops.rms_norm_fwd(x, self.gamma, self.eps, residual=residual, y=False, group=0)
        u, _ = ops.dense_fwd(n.q8, self.w8[0], self.b1, self.act, dtype=self.dtype)
        return ops.dense_fwd(ops.q8_encode(u, 0), self.w8[1], self.b2, residual=n.h, dtype=self.dtype)[0], n.h
