"""FeedForward: the pre-norm residual block on the rows of a conv layer's output (or on tokens).

    h = x + residual                      (x alone without a residual)
    n = gamma * h / rms(h)                (norm="layer": gamma * (h - mean(h)) / std(h) + beta)
    u = act(n w1^T + b1)
    y = u w2^T + b2 + h

MixtureFeedForward is the same block with a mixture of experts in place of w1 and w2, for serving.

act is one of ops.ACTS; gelu is the tanh form (torch's gelu(approximate="tanh"), not its default).
PyTorch supplies device memory and the stream; every step runs in the library's kernels (conv2d_layer_gb300.ops).
The class holds the parameters, the gradients (fp32, accumulated until zero_grad, as in Conv2dLayer) and what the
forward pass saves for the backward pass. With checkpoint="q8" that is kept in 8 bits, one scale for 32 features:
the norm's output n (the input of w1) and the activation's input and output; with "full" in the layer's type. h is
the residual stream and is kept as it is. fwd_infer saves nothing.

8-bit weights (quantize) have one scale an output feature, for fwd_infer, or (block=True) one for 128 x 128 of them, for
fwd_infer and for training: the products of fwd_train(bits8=True) and the two dx of its bwd then run on 8-bit operands.

An NHWC conv output [N, H, W, C] is N*H*W rows of C features: `rows(y)` views it so without a copy.
"""
import torch

from . import ops


def rows(y):
    """An NHWC tensor as a matrix of pixels by channels (a view)."""
    return y.view(-1, y.shape[-1])


class _Norm:
    """The norm of a block: RMS, or layer norm with gamma and beta."""

    def _norm_init(self, norm, gamma, beta, eps, dev):
        if norm not in ("rms", "layer"):
            raise ValueError(f"norm: rms or layer, got {norm!r}")
        if norm == "rms" and beta is not None:
            raise ValueError("beta: layer norm only")
        if beta is not None and beta.shape != gamma.shape:
            raise ValueError(f"beta: shape {tuple(beta.shape)} does not match {tuple(gamma.shape)}")
        self.layer, self.eps = norm == "layer", eps
        self.gamma = gamma.to(dev, torch.float32).contiguous()
        self.beta = None if beta is None else beta.to(dev, torch.float32).contiguous()

    def _norm(self, x, residual, **kw):
        if self.layer:
            return ops.layer_norm_fwd(x, self.gamma, self.beta, self.eps, residual=residual, **kw)
        return ops.rms_norm_fwd(x, self.gamma, self.eps, residual=residual, **kw)


class FeedForward(_Norm):
    def __init__(self, gamma, w1, b1, w2, b2, act="gelu", dtype=torch.bfloat16, eps=1e-6, checkpoint="q8", device="cuda",
                 norm="rms", beta=None):
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
        self.width, self.inner, self.act, self.dtype, self.q8 = width, inner, act, dtype, checkpoint == "q8"
        self._norm_init(norm, gamma, beta, eps, dev)
        self.b1, self.b2 = (t.to(dev, torch.float32).contiguous() for t in (b1, b2))
        self.w1, self.w2 = (t.to(dev, dtype).contiguous() for t in (w1, w2))
        self.dgamma, self.db1, self.db2 = (torch.zeros_like(t) for t in (self.gamma, self.b1, self.b2))
        self.dw1, self.dw2 = (torch.zeros(t.shape, device=dev, dtype=torch.float32) for t in (self.w1, self.w2))
        self.dbeta = None if self.beta is None else torch.zeros_like(self.beta)
        self.saved = self.trained = None
        self.w8 = self.w8_of = None

    def zero_grad(self):
        for t in (self.dgamma, self.dbeta, self.dw1, self.db1, self.dw2, self.db2):
            if t is not None:
                t.zero_()

    def fwd_train(self, x, residual=None, bits8=False):
        """y [rows, width]; keeps what bwd needs. bits8: products of 8-bit operands, weights from quantize(block=True)
        and activations with a scale for 128 features, whose 8-bit forms are what is kept."""
        save = "q8" if self.q8 else "full"
        if bits8:
            self._check8(True)
            n = self._norm(x, residual, y=False, group=ops.WIDE)
            u, z = ops.dense_fwd(n.q8, self.w8[0], self.b1, self.act, save=save, dtype=self.dtype)
            kept_n, kept_u = n.q8, ops.q8_encode(u, ops.WIDE)
            y, _ = ops.dense_fwd(kept_u, self.w8[1], self.b2, residual=n.h, dtype=self.dtype)
        else:
            n = self._norm(x, residual, group=ops.GROUP if self.q8 else None)
            u, z = ops.dense_fwd(n.y, self.w1, self.b1, self.act, save=save)
            y, _ = ops.dense_fwd(u, self.w2, self.b2, residual=n.h)
            kept_n, kept_u = (n.q8, ops.q8_encode(u)) if self.q8 else (n.y, u)
        self.saved = (n.h, n.inv_std if self.layer else n.inv_rms, kept_n, z, kept_u) + ((n.mean,) if self.layer else ())
        self.trained = self.w8 if bits8 else None
        return y

    def bwd(self, dy):
        """The gradient of x (and of residual); accumulates the parameters' gradients. Uses up what was saved."""
        if self.saved is None:
            raise RuntimeError("bwd follows a fwd_train")
        (h, inv, n, z, u, *mean), self.saved = self.saved, None
        (w1, w2), self.trained = self.trained or (self.w1, self.w2), None
        du, _, _ = ops.dense_bwd(u, w2, dy, dw=self.dw2, dbias=self.db2)
        dn, _, _ = ops.dense_bwd(n, w1, du, z, self.act, dw=self.dw1, dbias=self.db1)
        if self.layer:
            return ops.layer_norm_bwd(h, self.gamma, mean[0], inv, dn, dh=dy, dgamma=self.dgamma, dbeta=self.dbeta,
                                      need_dbeta=self.beta is not None)[0]
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

    def quantize(self, block=False):
        """Keeps 8-bit weights for bits8=True, one scale an output feature or (block) one for 128 x 128 of them; again
        after each change of w1 or w2. Calls with bits8 refuse 8-bit weights older than a change that torch has seen (not
        one through .data, a raw pointer, or of tensors made in inference mode)."""
        group = ops.TILE if block else 0
        self.w8 = ops.q8_encode(self.w1, group), ops.q8_encode(self.w2, group)
        self.w8_of = self._weights()
        self.w8_block = block

    def _check8(self, block):
        if self.w8 is None:
            raise RuntimeError("bits8 follows quantize()")
        if self.w8_of and any(a is not b or u != v for (a, u), (b, v) in zip(self.w8_of, self._weights())):
            raise RuntimeError("w1 or w2 has changed: bits8 needs another quantize()")
        if block and not self.w8_block:
            raise RuntimeError("training with bits8 follows quantize(block=True)")

    def fwd_infer(self, x, residual=None, bits8=False):
        """(y, h) without saving anything, for any number of rows (one for a decoded token). bits8: 8-bit weights
        (quantize) and activations, one scale a token (block: for 128 features), on the 8-bit tensor cores."""
        if not bits8:
            n = self._norm(x, residual)
            u, _ = ops.dense_fwd(n.y, self.w1, self.b1, self.act)
            return ops.dense_fwd(u, self.w2, self.b2, residual=n.h)[0], n.h
        self._check8(False)
        group = ops.WIDE if self.w8_block else 0
        n = self._norm(x, residual, y=False, group=group)
        u, _ = ops.dense_fwd(n.q8, self.w8[0], self.b1, self.act, dtype=self.dtype)
        return ops.dense_fwd(ops.q8_encode(u, group), self.w8[1], self.b2, residual=n.h, dtype=self.dtype)[0], n.h


class MixtureFeedForward(_Norm):
    """The residual block with experts, for serving: h = x + residual, n = norm(h), y = h + the mixture of n (ops.moe_fwd).

    gamma (and beta) [D], router [E, D], w1 [E, F, D] (gated: [E, 2 F, D]), w2 [E, D, F], b1 and b2 of one row an expert,
    or None; k experts a row. The weights are kept in dtype, the router in fp32."""
    ROWS = 64  # of one call of ops.moe_fwd

    def __init__(self, gamma, router, w1, w2, k, b1=None, b2=None, act="silu", gated=True, normalize=True,
                 dtype=torch.bfloat16, eps=1e-6, device="cuda", norm="rms", beta=None):
        if act not in ops.ACTS:
            raise ValueError(f"act: one of {sorted(ops.ACTS)}, got {act!r}")
        if dtype not in (torch.bfloat16, torch.float16):
            raise ValueError(f"dtype: torch.bfloat16 or torch.float16, got {dtype!r}")
        if router.dim() != 2 or w2.dim() != 3:
            raise ValueError("router: experts by width; w2: experts by width by inner features")
        (experts, width), inner = router.shape, w2.shape[2]
        up = inner * (2 if gated else 1)
        for name, t, shape in (("gamma", gamma, (width,)), ("w1", w1, (experts, up, width)), ("w2", w2, (experts, width, inner)),
                               ("b1", b1, (experts, up)), ("b2", b2, (experts, width))):
            if t is not None and tuple(t.shape) != shape:
                raise ValueError(f"{name}: shape {tuple(t.shape)} does not match {shape}")
        if not 1 <= experts <= 256:
            raise ValueError(f"router: 1 to 256 experts, got {experts}")
        if not isinstance(k, int) or not 1 <= k <= min(experts, 16):
            raise ValueError(f"k: 1 to {min(experts, 16)} experts, got {k!r}")
        for name, n in (("width", width), ("inner features", inner)):
            if n < 8 or n % 8:
                raise ValueError(f"{name}: a multiple of 8, got {n}")
        dev = torch.device(device)
        self.k, self.act, self.gated, self.normalize, self.dtype = k, act, gated, normalize, dtype
        self._norm_init(norm, gamma, beta, eps, dev)
        self.router = router.to(dev, torch.float32).contiguous()
        self.w1, self.w2 = (t.to(dev, dtype).contiguous() for t in (w1, w2))
        self.b1, self.b2 = (None if t is None else t.to(dev, torch.float32).contiguous() for t in (b1, b2))

    def quantize(self):
        """Takes the experts to 8 bits, one scale for 128 x 128 weights, in place of what they were (once: later calls change
        nothing). Width and inner features must be multiples of 128."""
        if isinstance(self.w1, ops.Q8):
            return
        width, inner = self.w2.shape[1:]
        if width % 128 or inner % 128:
            raise ValueError(f"8-bit experts have whole tiles: width and inner features in multiples of 128, got {width} and {inner}")
        self.w1, self.w2 = ops.moe_encode(self.w1), ops.moe_encode(self.w2)

    def fwd_infer(self, x, residual=None):
        """(y, h) for any number of rows, 64 of them at a time."""
        n = self._norm(x, residual)
        y = torch.empty_like(n.y)
        for r in range(0, x.shape[0], self.ROWS):
            part = slice(r, r + self.ROWS)
            ops.moe_fwd(n.y[part], self.router, self.w1, self.w2, self.k, b1=self.b1, b2=self.b2, act=self.act,
                        gated=self.gated, normalize=self.normalize, residual=n.h[part], y=y[part])
        return y, n.h
