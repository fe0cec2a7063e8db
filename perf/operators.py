"""The residual block's operators as they are measured: RMS norm, dense layer, 8-bit activation checkpoints.

A case names one call of `conv2d_layer_gb300.ops` and its sizes. `run` makes that call where `own` is true and
computes the same from elementary torch operations in 32 bits where it is false; `exact` is the definition in
64 bits. An 8-bit tensor is e4m3 values with one power-of-two scale for each group of columns of a row (32 of
them, or the whole row): scale 2^e with the smallest e for which no finite value of the group exceeds 448 * 2^e.
It is returned as the values it stands for."""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
ES = {"bf16": 2, "fp16": 2, "fp32": 4}
ACTS = ("identity", "relu", "tanh", "sigmoid", "gelu", "silu")
EPS = 1e-6


def listed():
    return [
        # one new token in front of an 8-bit dense layer: h for the residual stream, y in 8 bits with a row scale
        dict(name="norm token to 8 bits", op="norm", rows=1, cols=4096, dtype="bf16", residual=True, y=False, group=0),
        # a training step's norm: y for the matrix product, its 8-bit form kept for the backward pass
        dict(name="norm train", op="norm", rows=8192, cols=4096, dtype="bf16", residual=True, y=True, group=32),
        # odd sizes in 32 bits, no residual
        dict(name="norm odd fp32", op="norm", rows=1003, cols=1021, dtype="fp32", residual=False, y=True, group=-1),
        # its gradient, with the gradient that arrives through the residual stream
        dict(name="norm gradient", op="norm_bwd", rows=8192, cols=4096, dtype="bf16", residual=True),
        # decoding one sequence: the weights are read once for one row
        dict(name="dense token", op="dense", rows=1, cols=4096, out=16384, dtype="bf16", bits8=False, bias=True,
             act="silu", residual=False, save="none"),
        # decoding a batch from 8-bit weights and activations
        dict(name="dense batch 8 bits", op="dense", rows=24, cols=16384, out=4096, dtype="bf16", bits8=True, bias=True,
             act="identity", residual=True, save="none"),
        # a training step's first matrix product: the activation's input is kept in 8 bits
        dict(name="dense train", op="dense", rows=8192, cols=2048, out=8192, dtype="bf16", bits8=False, bias=True,
             act="gelu", residual=False, save="q8"),
        # the pixels of 64 conv outputs (56 x 56 x 256) as rows of a pointwise layer, input of the activation kept whole
        dict(name="dense pixels", op="dense", rows=200704, cols=256, out=1024, dtype="bf16", bits8=False, bias=True,
             act="relu", residual=False, save="full"),
        # ragged in every direction, fp16, with the residual
        dict(name="dense ragged fp16", op="dense", rows=777, cols=1001, out=1333, dtype="fp16", bits8=False, bias=True,
             act="tanh", residual=True, save="none"),
        # gradients from 8-bit checkpoints of both the layer's input and the activation's
        dict(name="dense gradient 8-bit", op="dense_bwd", rows=8192, cols=2048, out=8192, dtype="bf16", act="gelu", q8=True,
             grad="same"),
        # gradients of an output projection: no activation, weight gradient in 32 bits
        dict(name="dense gradient ragged", op="dense_bwd", rows=1777, cols=1000, out=333, dtype="bf16", act="identity",
             q8=False, grad="fp32"),
        # a conv layer's saved activations to 8 bits and back
        dict(name="checkpoint", op="q8", rows=200704, cols=256, dtype="bf16", group=32),
    ]


def _log(rng, low, high):
    """A whole number of [low, high], spread over its logarithm; a multiple of 8 as often as not."""
    v = int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))
    return max(low, v - v % 8) if v >= 16 and rng.random() < 0.5 else v


def draw(rng):
    op = rng.choice(["norm", "norm", "norm_bwd", "dense", "dense", "dense", "dense_bwd", "dense_bwd", "q8"])
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    if op in ("norm", "norm_bwd", "q8"):
        rows, cols = _log(rng, 1, 65536), _log(rng, 32, 16384)
        rows = max(1, min(rows, (1 << 25) // cols))
        c = dict(op=op, rows=rows, cols=cols, dtype=dtype)
        if op != "q8":
            c["residual"] = rng.random() < 0.7
        if op == "norm":
            c["group"] = rng.choice([-1, 0, 32])
            c["y"] = c["group"] < 0 or rng.random() < 0.5
        if op == "q8":
            c["group"] = rng.choice([0, 32])
        return c
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    rows, cols, out = _log(rng, 1, 16384), _log(rng, 32, 16384), _log(rng, 32, 16384)
    while 2.0 * rows * cols * out > 1.3e11:
        rows, cols, out = max(1, rows // 2), max(32, cols * 3 // 4), max(32, out * 3 // 4)
    c = dict(op=op, rows=rows, cols=cols, out=out, dtype=dtype, act=rng.choice(ACTS))
    if op == "dense":
        c.update(bits8=rng.random() < 0.3, bias=rng.random() < 0.8, residual=rng.random() < 0.5,
                 save=rng.choice(["none", "full", "q8"]))
    else:
        # behind an activation dz is stored in the element type, and so is the weight gradient made of it
        c.update(q8=rng.random() < 0.5, grad="fp32" if c["act"] == "identity" else "same")
    return c


def _groups(cols, group):
    return -(-cols // group) if group > 0 else 1


def work(c):
    rows, cols, es = c["rows"], c["cols"], ES[c["dtype"]]
    n = rows * cols
    if c["op"] == "norm":
        per = es * (1 + 2 * c["residual"] + c["y"]) + (c["group"] >= 0)
        scales = rows * _groups(cols, c["group"]) if c["group"] >= 0 else 0
        return {"bytes": n * per + scales + 4 * cols + 4 * rows, "flops": 4 * n}
    if c["op"] == "norm_bwd":
        return {"bytes": n * es * (3 + c["residual"]) + 8 * cols + 4 * rows, "flops": 8 * n}
    if c["op"] == "q8":
        return {"bytes": 2 * (n * (es + 1) + rows * _groups(cols, c["group"])), "flops": 2 * n}
    out, k = c["out"], n * c["out"]
    if c["op"] == "dense":
        ops = 1 if c["bits8"] else es
        save = {"none": 0, "full": es, "q8": 1 + 1 / 32}[c["save"]]
        return {"bytes": ops * (n + out * cols) + rows * out * (es * (1 + c["residual"]) + save) + 4 * out * c["bias"],
                "flops": 2 * k}
    z = 0 if c["act"] == "identity" else (1 + 1 / 32 if c["q8"] else es)
    x = 1 + 1 / 32 if c["q8"] else es
    return {"bytes": rows * out * (es + z) + n * (x + es) + out * cols * (es + (4 if c["grad"] == "fp32" else es)) + 4 * out,
            "flops": 4 * k}


# ------------------------------------------------------------------ 8 bits, plain form
def _encode(v, group):
    """(e4m3 values, scale bytes) of 32-bit values [rows, cols]."""
    rows, cols = v.shape
    group = group if group > 0 else cols
    n = _groups(cols, group)
    w = torch.zeros(rows, n * group, device=v.device)
    w[:, :cols] = v
    w = w.view(rows, n, group)
    amax = torch.where(w.isfinite(), w.abs(), 0).amax(2)
    m, x = torch.frexp(amax)
    e = torch.where(m > 0.875, x - 8, x - 9).clamp(-126, 127)  # 448 = 0.875 * 2^9
    e = torch.where(amax > 0, e, 0).to(torch.int32)
    down = ((127 - e) << 23).view(torch.float32)
    q = (w * down[..., None]).view(rows, n * group)[:, :cols].contiguous().to(torch.float8_e4m3fn)
    return q, (e + 127).to(torch.uint8)


def _decode(q, scale, group):
    rows, cols = q.shape
    group = group if group > 0 else cols
    up = (scale.to(torch.int32) << 23).view(torch.float32)
    return q.float() * up.repeat_interleave(group, 1)[:, :cols]


def _act(act, z):
    if act == "relu":
        return torch.where(z > 0, z, 0)
    if act == "tanh":
        return 1 - 2 / (1 + torch.exp(2 * z))
    if act == "sigmoid":
        return 1 / (1 + torch.exp(-z))
    if act == "gelu":
        return z / (1 + torch.exp(-2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    if act == "silu":
        return z / (1 + torch.exp(-z))
    return z


def _dact(act, z):
    if act == "relu":
        return (z > 0).float()
    if act == "tanh":
        t = 1 - 2 / (1 + torch.exp(2 * z))
        return 1 - t * t
    if act == "gelu":
        a = math.sqrt(2 / math.pi)
        s = 1 / (1 + torch.exp(-2 * a * (z + 0.044715 * z * z * z)))
        return s + z * s * (1 - s) * 2 * a * (1 + 3 * 0.044715 * z * z)
    s = 1 / (1 + torch.exp(-z))
    if act == "sigmoid":
        return s * (1 - s)
    return s * (1 + z * (1 - s)) if act == "silu" else torch.ones_like(z)


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[c["dtype"]]
    rows, cols = c["rows"], c["cols"]

    def normal(*shape, std=1.0):
        return torch.randn(*shape, generator=g, device="cuda") * std

    def features(*shape):
        """Activations: every feature has a width of its own, a few are far wider."""
        wide = torch.exp(0.5 * normal(shape[-1]))
        return normal(*shape) * wide

    s = dict(case=dict(c))
    if c["op"] in ("norm", "norm_bwd"):
        s["gamma"] = 1 + normal(cols, std=0.2)
        if c["op"] == "norm":
            s["x"] = features(rows, cols).to(dt)
            s["residual"] = features(rows, cols).to(dt) if c["residual"] else None
        else:
            s["h"] = features(rows, cols).to(dt)
            s["inv"] = torch.rsqrt(s["h"].float().square().mean(1) + EPS)
            s["dy"] = normal(rows, cols, std=1e-2).to(dt)
            s["dh"] = normal(rows, cols, std=1e-2).to(dt) if c["residual"] else None
        return s
    if c["op"] == "q8":
        s["x"] = features(rows, cols).to(dt)
        return s
    out = c["out"]
    x, w = features(rows, cols), normal(out, cols, std=1 / math.sqrt(cols))
    if c["op"] == "dense":
        # 8-bit operands: one scale for each row of x (a token) and of w (an output feature)
        s["x"] = _encode(x, 0) if c["bits8"] else x.to(dt)
        s["w"] = _encode(w, 0) if c["bits8"] else w.to(dt)
        s["bias"] = normal(out, std=0.1) if c["bias"] else None
        s["residual"] = normal(rows, out).to(dt) if c["residual"] else None
        return s
    s["w"] = w.to(dt)
    s["dy"] = normal(rows, out, std=0.1).to(dt)
    s["x"] = _encode(x, 32) if c["q8"] else x.to(dt)
    z = None if c["act"] == "identity" else normal(rows, out, std=1.5)
    s["z"] = z if z is None else _encode(z, 32) if c["q8"] else z.to(dt)
    return s


# ------------------------------------------------------------------ one pass
def run(state):
    return _own(state) if own else _plain(state)


def _own(s):
    from conv2d_layer_gb300 import ops

    c = s["case"]
    dt = DTYPES[c["dtype"]]

    def q8(v, group):
        return ops.Q8(v[0], v[1], group)

    if c["op"] == "norm":
        r = ops.rms_norm_fwd(s["x"], s["gamma"], EPS, residual=s["residual"], y=c["y"],
                             group=c["group"] if c["group"] >= 0 else None)
        back = ops.q8_decode(r.q8, dt) if r.q8 is not None else None
        return {"h": r.h if c["residual"] else None, "y": r.y, "q8": back, "inv_rms": r.inv_rms}
    if c["op"] == "norm_bwd":
        dx, dgamma = ops.rms_norm_bwd(s["h"], s["gamma"], s["inv"], s["dy"], dh=s["dh"])
        return {"dx": dx, "dgamma": dgamma}
    if c["op"] == "q8":
        return {"x": ops.q8_decode(ops.q8_encode(s["x"], c["group"]), dt)}
    if c["op"] == "dense":
        x, w = (q8(s["x"], 0), q8(s["w"], 0)) if c["bits8"] else (s["x"], s["w"])
        y, z = ops.dense_fwd(x, w, s["bias"], c["act"], residual=s["residual"], save=c["save"], dtype=dt)
        return {"y": y, "z": ops.q8_decode(z, dt) if c["save"] == "q8" else z}
    x = q8(s["x"], 32) if c["q8"] else s["x"]
    z = q8(s["z"], 32) if c["q8"] and s["z"] is not None else s["z"]
    dx, dw, db = ops.dense_bwd(x, s["w"], s["dy"], z, c["act"], grad_dtype=torch.float32 if c["grad"] == "fp32" else dt)
    return {"dx": dx, "dw": dw, "db": db}


def _plain(s):
    c = s["case"]
    dt = DTYPES[c["dtype"]]
    if c["op"] == "norm":
        h = s["x"]
        if c["residual"]:
            h = (h.float() + s["residual"].float()).to(dt)
        v = h.float()
        inv = torch.rsqrt(v.square().mean(1) + EPS)
        y = v * inv[:, None] * s["gamma"]
        back = _decode(*_encode(y, c["group"]), c["group"]).to(dt) if c["group"] >= 0 else None
        return {"h": h if c["residual"] else None, "y": y.to(dt) if c["y"] else None, "q8": back, "inv_rms": inv}
    if c["op"] == "norm_bwd":
        h, dy, inv = s["h"].float(), s["dy"].float(), s["inv"][:, None]
        g = dy * s["gamma"]
        dx = inv * g - h * inv.pow(3) * (g * h).mean(1, keepdim=True)
        if c["residual"]:
            dx = dx + s["dh"].float()
        return {"dx": dx.to(dt), "dgamma": (dy * h * inv).sum(0)}
    if c["op"] == "q8":
        return {"x": _decode(*_encode(s["x"].float(), c["group"]), c["group"]).to(dt)}
    if c["op"] == "dense":
        x, w = (_decode(*s[k], 0) if c["bits8"] else s[k].float() for k in ("x", "w"))
        z = x @ w.t()
        if c["bias"]:
            z = z + s["bias"]
        y = _act(c["act"], z)
        if c["residual"]:
            y = y + s["residual"].float()
        save = {"none": lambda: None, "full": lambda: z, "q8": lambda: _decode(*_encode(z, 32), 32)}[c["save"]]()
        return {"y": y.to(dt), "z": save.to(dt) if save is not None else None}
    x = _decode(*s["x"], 32) if c["q8"] else s["x"].float()
    dz = s["dy"].float()
    if s["z"] is not None:
        dz = dz * _dact(c["act"], _decode(*s["z"], 32) if c["q8"] else s["z"].float())
    dw = dz.t() @ x
    return {"dx": (dz @ s["w"].float()).to(dt), "dw": dw if c["grad"] == "fp32" else dw.to(dt), "db": dz.sum(0)}


# ------------------------------------------------------------------ the definition, in 64 bits
def _held8(v, group):
    """What 64-bit values are once they have been held in 8 bits."""
    rows, cols = v.shape
    group = group if group > 0 else cols
    pad = torch.nn.functional.pad(v, (0, -cols % group)).reshape(rows, -1, group)
    top = pad.abs().amax(2, keepdim=True)
    unit = torch.exp2(torch.ceil(torch.log2(top / 448)).clamp(-126, 127))
    unit = torch.where(448 * unit < top, 2 * unit, torch.where(448 * (unit / 2) >= top, unit / 2, unit))
    unit = torch.where(top > 0, unit, torch.ones_like(unit))
    t = pad / unit
    step = torch.exp2(torch.floor(torch.log2(t.abs().clamp(min=2.0 ** -6))) - 3)
    return (torch.round(t / step) * step * unit).reshape(rows, -1)[:, :cols]


def _act64(act, z):
    """(act(z), its derivative)"""
    if act == "relu":
        return z.clamp(min=0), (z > 0).double()
    if act == "tanh":
        return torch.tanh(z), 1 / torch.cosh(z) ** 2
    if act == "sigmoid":
        return torch.sigmoid(z), torch.sigmoid(z) * torch.sigmoid(-z)
    if act == "silu":
        return z * torch.sigmoid(z), torch.sigmoid(z) + z * torch.sigmoid(z) * torch.sigmoid(-z)
    if act == "gelu":
        a, b = math.sqrt(2 / math.pi), 0.044715
        t = torch.tanh(a * (z + b * z ** 3))
        return 0.5 * z * (1 + t), 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * a * (1 + 3 * b * z * z)
    return z, torch.ones_like(z)


def exact(case, seed):
    c, s = case, prepare(case, seed)

    def wide(v, group):
        if isinstance(v, tuple):
            q, scale = v
            n = group if group > 0 else q.shape[1]
            col = torch.arange(q.shape[1], device=q.device) // n
            return q.double() * torch.exp2(scale.double() - 127)[:, col]
        return v.double()

    if c["op"] == "norm":
        h = s["x"].double()
        if c["residual"]:
            h = (h + s["residual"].double()).to(DTYPES[c["dtype"]]).double()  # h is what the norm is taken of
        inv = 1 / torch.sqrt((h * h).sum(1) / c["cols"] + EPS)
        y = s["gamma"].double() * (h * inv[:, None])
        return {"h": h if c["residual"] else None, "y": y if c["y"] else None,
                "q8": _held8(y, c["group"]) if c["group"] >= 0 else None, "inv_rms": inv}
    if c["op"] == "norm_bwd":
        h, g, inv = s["h"].double(), s["dy"].double(), s["inv"].double()[:, None]
        n = h * inv
        gy = g * s["gamma"].double()
        dx = inv * (gy - n * (gy * n).sum(1, keepdim=True) / c["cols"])
        if c["residual"]:
            dx = dx + s["dh"].double()
        return {"dx": dx, "dgamma": torch.einsum("rc,rc->c", g, n)}
    if c["op"] == "q8":
        return {"x": _held8(s["x"].double(), c["group"])}
    if c["op"] == "dense":
        z = wide(s["x"], 0) @ wide(s["w"], 0).t()
        if c["bias"]:
            z = z + s["bias"].double()
        y = _act64(c["act"], z)[0]
        if c["residual"]:
            y = y + s["residual"].double()
        return {"y": y, "z": {"none": None, "full": z, "q8": _held8(z, 32) if c["save"] == "q8" else None}[c["save"]]}
    dz = s["dy"].double()
    if s["z"] is not None:
        dz = dz * _act64(c["act"], wide(s["z"], 32))[1]
    return {"dx": dz @ s["w"].double(), "dw": dz.t() @ wide(s["x"], 32), "db": dz.sum(0)}
