"""More of the residual block's operators as they are measured: layer norm, the matrix product in 8 bits with a scale
for each block of 128, and a mixture-of-experts layer for a few tokens.

A case names one call of `conv2d_layer_gb300.ops` and its sizes. `run` makes that call where `own` is true and
computes the same from elementary torch operations in 32 bits where it is false; `exact` is the definition in
64 bits. An 8-bit tensor is e4m3 values with one power-of-two scale for each group of columns of a row (32 or 128 of
them, or the whole row) or for each tile of 128 rows by 128 columns: scale 2^e with the smallest e for which no finite
value of the group exceeds 448 * 2^e. It is returned as the values it stands for (bf16 holds them exactly)."""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
ES = {"bf16": 2, "fp16": 2, "fp32": 4}
ACTS = ("identity", "relu", "tanh", "sigmoid", "gelu", "silu")
EPS = 1e-5
TILE = "tile"  # a scale for 128 rows by 128 columns


def listed():
    return [
        # one new token in front of an 8-bit layer: h for the residual stream, y in 8 bits
        dict(name="layer norm token to 8 bits", op="norm", rows=1, cols=4096, dtype="bf16", residual=True, beta=True,
             y=False, group=128),
        # a training step's norm
        dict(name="layer norm train", op="norm", rows=8192, cols=4096, dtype="bf16", residual=True, beta=True, y=True,
             group=-1),
        # odd sizes in 32 bits, no residual
        dict(name="layer norm odd fp32", op="norm", rows=1003, cols=1021, dtype="fp32", residual=False, beta=True, y=True,
             group=-1),
        # its gradient, with the gradient that arrives through the residual stream
        dict(name="layer norm gradient", op="norm_bwd", rows=8192, cols=4096, dtype="bf16", residual=True, beta=True),
        # decoding one sequence from 8-bit weights
        dict(name="block product token", op="dense", rows=1, cols=4096, out=16384, dtype="bf16", wgroup=TILE, bias=True,
             act="silu", residual=False, save="none"),
        # ragged in every direction, fp16, with the residual, weights with a scale for each row and 128 columns
        dict(name="block product ragged", op="dense", rows=203, cols=1001, out=1333, dtype="fp16", wgroup=128, bias=True,
             act="tanh", residual=True, save="none"),
        # a training step's first matrix product: the activation's input is kept
        dict(name="block product train", op="dense", rows=8192, cols=2048, out=8192, dtype="bf16", wgroup=TILE, bias=True,
             act="gelu", residual=False, save="full"),
        # gradients of an output projection whose input was kept in 8 bits: dx in 8 bits too
        dict(name="block product gradient", op="dense_bwd", rows=8192, cols=8192, out=2048, dtype="bf16", act="identity"),
        # a layer's weights to 8 bits and back, after a step of the optimizer
        dict(name="weights to tiles", op="q8", rows=16384, cols=4096, dtype="bf16", group=TILE),
        # one token through small experts
        dict(name="experts token", op="moe", rows=1, cols=2048, inner=1024, experts=64, k=8, dtype="bf16", bits8=False,
             gated=True, act="silu", bias=False, normalize=True, residual=True),
        # a batch of decoded tokens through large experts: nearly all of them are chosen
        dict(name="experts batch", op="moe", rows=16, cols=4096, inner=8192, experts=8, k=2, dtype="bf16", bits8=False,
             gated=True, act="silu", bias=False, normalize=True, residual=True),
        # ragged: odd numbers of tokens and experts, 8-bit weights and activations, biases, no gate
        dict(name="experts ragged 8 bits", op="moe", rows=37, cols=1152, inner=640, experts=23, k=3, dtype="bf16",
             bits8=True, gated=False, act="gelu", bias=True, normalize=False, residual=False),
    ]


def _log(rng, low, high, of=8):
    """A whole number of [low, high], spread over its logarithm; a multiple of `of` as often as not."""
    v = int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))
    return max(low, v - v % of) if v >= 2 * of and rng.random() < 0.5 else v


def _up(v, of):
    return -(-v // of) * of


def draw(rng):
    op = rng.choice(["norm", "norm", "norm_bwd", "dense", "dense", "dense_bwd", "q8", "moe", "moe", "moe"])
    if op in ("norm", "norm_bwd", "q8"):
        rows, cols = _log(rng, 1, 65536), _log(rng, 32, 16384)
        rows = max(1, min(rows, (1 << 25) // cols))
        c = dict(op=op, rows=rows, cols=cols, dtype=rng.choice(["bf16", "bf16", "fp16", "fp32"]))
        if op == "q8":
            c["group"] = rng.choice([128, TILE])
            return c
        c.update(residual=rng.random() < 0.7, beta=rng.random() < 0.8)
        if op == "norm":
            c["group"] = rng.choice([-1, 0, 32, 128])
            c["y"] = c["group"] < 0 or rng.random() < 0.5
        return c
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    if op == "moe":
        bits8 = rng.random() < 0.4
        cols, inner = _up(_log(rng, 128, 4096), 128 if bits8 else 8), _up(_log(rng, 128, 8192), 128 if bits8 else 8)
        experts = _log(rng, 2, 128)
        while experts * cols * inner > 8 * 4096 * 8192:
            experts = max(2, experts // 2)
        return dict(op=op, rows=_log(rng, 1, 64), cols=cols, inner=inner, experts=experts, k=rng.randint(1, min(8, experts)),
                    dtype=dtype, bits8=bits8, gated=rng.random() < 0.6, act=rng.choice(["gelu", "silu", "relu"]),
                    bias=rng.random() < 0.5, normalize=rng.random() < 0.5, residual=rng.random() < 0.5)
    rows, cols, out = _log(rng, 1, 16384), _log(rng, 32, 16384), _log(rng, 32, 16384)
    while 2.0 * rows * cols * out > 1.3e11:
        rows, cols, out = max(1, rows // 2), max(32, cols * 3 // 4), max(32, out * 3 // 4)
    c = dict(op=op, rows=rows, cols=cols, out=out, dtype=dtype)
    if op == "dense":
        c.update(wgroup=rng.choice([128, TILE, TILE]), bias=rng.random() < 0.8, act=rng.choice(ACTS),
                 residual=rng.random() < 0.5, save=rng.choice(["none", "full"]))
    else:
        c.update(act=rng.choice(["identity", "identity", "gelu", "silu"]))
    return c


def _scales(rows, cols, group):
    if group == TILE:
        return -(-rows // 128) * -(-cols // 128)
    return rows * (-(-cols // group) if group > 0 else 1)


def work(c):
    rows, cols, es = c["rows"], c["cols"], ES[c["dtype"]]
    n = rows * cols
    if c["op"] == "norm":
        per = es * (1 + 2 * c["residual"] + c["y"]) + (c["group"] >= 0)
        scales = _scales(rows, cols, c["group"]) if c["group"] >= 0 else 0
        return {"bytes": n * per + scales + 4 * cols * (1 + c["beta"]) + 8 * rows, "flops": 7 * n}
    if c["op"] == "norm_bwd":
        return {"bytes": n * es * (3 + c["residual"]) + 4 * cols * (2 + c["beta"]) + 8 * rows, "flops": 11 * n}
    if c["op"] == "q8":
        return {"bytes": 2 * (n * (es + 1) + _scales(rows, cols, c["group"])), "flops": 2 * n}
    if c["op"] == "moe":
        f, e, k = c["inner"], c["experts"], c["k"]
        chosen = e * (1 - (1 - k / e) ** rows)  # experts that at least one token chooses, where all are as likely
        per = f * cols * (2 + c["gated"])
        return {"bytes": chosen * (per * (1 if c["bits8"] else es) + c["bias"] * 4 * (f * (1 + c["gated"]) + cols))
                + es * (e * cols + n * (2 + c["residual"])) + 8 * rows * k, "flops": 2 * rows * (k * per + e * cols)}
    out = c["out"]
    if c["op"] == "dense":
        return {"bytes": n + _scales(rows, cols, 128) + out * cols + _scales(out, cols, c["wgroup"])
                + rows * out * es * (1 + c["residual"] + (c["save"] == "full")) + 4 * out * c["bias"], "flops": 2 * n * out}
    z = 0 if c["act"] == "identity" else es
    return {"bytes": rows * out * (es + z) + n * (1 + es) + out * cols * (1 + es) + 4 * out, "flops": 4 * n * out}


# ------------------------------------------------------------------ 8 bits, plain form
def _encode(v, group):
    """(e4m3 values, scale bytes) of 32-bit values [rows, cols]."""
    rows, cols = v.shape
    height, group = (128, 128) if group == TILE else (1, group if group > 0 else cols)
    w = torch.nn.functional.pad(v, (0, -cols % group, 0, -rows % height))
    w = w.view(w.shape[0] // height, height, w.shape[1] // group, group)
    amax = torch.where(w.isfinite(), w.abs(), 0).amax((1, 3))
    m, x = torch.frexp(amax)
    e = torch.where(m > 0.875, x - 8, x - 9).clamp(-126, 127)  # 448 = 0.875 * 2^9
    e = torch.where(amax > 0, e, 0).to(torch.int32)
    down = ((127 - e) << 23).view(torch.float32)
    q = (w * down[:, None, :, None]).view(w.shape[0] * height, -1)[:rows, :cols].contiguous().to(torch.float8_e4m3fn)
    return q, (e + 127).to(torch.uint8)


def _decode(q, scale, group, real=torch.float32):
    """The values, of matrices or of a stack of them."""
    rows, cols = q.shape[-2:]
    up = torch.exp2(scale.to(real) - 127)
    if group == TILE:
        up = up.repeat_interleave(128, -2)[..., :rows, :]
    return q.to(real) * up.repeat_interleave(128 if group == TILE else group if group > 0 else cols, -1)[..., :cols]


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
    if act == "gelu":
        a = math.sqrt(2 / math.pi)
        s = 1 / (1 + torch.exp(-2 * a * (z + 0.044715 * z * z * z)))
        return s + z * s * (1 - s) * 2 * a * (1 + 3 * 0.044715 * z * z)
    s = 1 / (1 + torch.exp(-z))
    return s * (1 + z * (1 - s))


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[c["dtype"]]
    rows, cols = c["rows"], c["cols"]

    def normal(*shape, std=1.0):
        return torch.randn(*shape, generator=g, device="cuda") * std

    def features(*shape):
        """Activations: every feature has a width and an offset of its own, a few are far wider."""
        wide = torch.exp(0.5 * normal(shape[-1]))
        return (normal(*shape) + 0.3 * normal(shape[-1])) * wide

    s = dict(case=dict(c))
    if c["op"] in ("norm", "norm_bwd"):
        s["gamma"] = 1 + normal(cols, std=0.2)
        s["beta"] = normal(cols, std=0.1) if c["beta"] else None
        if c["op"] == "norm":
            s["x"] = features(rows, cols).to(dt)
            s["residual"] = features(rows, cols).to(dt) if c["residual"] else None
        else:
            s["h"] = features(rows, cols).to(dt)
            h = s["h"].double()
            s["mean"] = h.mean(1).float()
            s["inv"] = torch.rsqrt((h - h.mean(1, keepdim=True)).square().mean(1) + EPS).float()
            s["dy"] = normal(rows, cols, std=1e-2).to(dt)
            s["dh"] = normal(rows, cols, std=1e-2).to(dt) if c["residual"] else None
        return s
    if c["op"] == "q8":
        s["x"] = normal(rows, cols, std=1 / math.sqrt(cols)).to(dt)
        return s
    if c["op"] == "moe":
        e, f = c["experts"], c["inner"]
        up = f * (1 + c["gated"])
        s["x"] = features(rows, cols).to(dt)
        s["router"] = normal(e, cols, std=1 / math.sqrt(cols)).to(dt)
        s["residual"] = normal(rows, cols).to(dt) if c["residual"] else None
        s["b1"] = normal(e, up, std=0.1) if c["bias"] else None
        s["b2"] = normal(e, cols, std=0.1) if c["bias"] else None
        for name, out, width in (("w1", up, cols), ("w2", cols, f)):
            w = normal(e, out, width, std=1 / math.sqrt(width))
            if c["bits8"]:  # rows of an expert are whole tiles
                q, scale = _encode(w.view(e * out, width), TILE)
                s[name] = q.view(e, out, width), scale.view(e, out // 128, -1)
            else:
                s[name] = w.to(dt)
        return s
    out = c["out"]
    x, w = features(rows, cols), normal(out, cols, std=1 / math.sqrt(cols))
    s["x"] = _encode(x, 128)
    if c["op"] == "dense":
        s["w"] = _encode(w, c["wgroup"])
        s["bias"] = normal(out, std=0.1) if c["bias"] else None
        s["residual"] = normal(rows, out).to(dt) if c["residual"] else None
        return s
    s["w"] = _encode(w, TILE)
    s["dy"] = normal(rows, out, std=0.1).to(dt)
    s["z"] = None if c["act"] == "identity" else normal(rows, out, std=1.5).to(dt)
    return s


# ------------------------------------------------------------------ one pass
def run(state):
    return _own(state) if own else _plain(state)


def _own(s):
    from conv2d_layer_gb300 import ops

    c = s["case"]
    dt = DTYPES[c["dtype"]]

    def q8(v, group):
        return ops.Q8(v[0], v[1], ops.TILE if group == TILE else group)

    if c["op"] == "norm":
        r = ops.layer_norm_fwd(s["x"], s["gamma"], s["beta"], EPS, residual=s["residual"], y=c["y"],
                               group=c["group"] if c["group"] >= 0 else None)
        back = ops.q8_decode(r.q8, torch.bfloat16) if r.q8 is not None else None
        return {"h": r.h if c["residual"] else None, "y": r.y, "q8": back, "mean": r.mean, "inv_std": r.inv_std}
    if c["op"] == "norm_bwd":
        dx, dgamma, dbeta = ops.layer_norm_bwd(s["h"], s["gamma"], s["mean"], s["inv"], s["dy"], dh=s["dh"],
                                               need_dbeta=c["beta"])
        return {"dx": dx, "dgamma": dgamma, "dbeta": dbeta}
    if c["op"] == "q8":
        return {"x": ops.q8_decode(ops.q8_encode(s["x"], ops.TILE if c["group"] == TILE else c["group"]), dt)}
    if c["op"] == "moe":
        w1, w2 = (q8(s[n], TILE) if c["bits8"] else s[n] for n in ("w1", "w2"))
        r = ops.moe_fwd(s["x"], s["router"], w1, w2, c["k"], b1=s["b1"], b2=s["b2"], act=c["act"], gated=c["gated"],
                        normalize=c["normalize"], residual=s["residual"])
        return {"y": r.y, "experts": r.experts, "weights": r.weights}
    if c["op"] == "dense":
        y, z = ops.dense_fwd(q8(s["x"], 128), q8(s["w"], c["wgroup"]), s["bias"], c["act"], residual=s["residual"],
                             save=c["save"], dtype=dt)
        return {"y": y, "z": z}
    dx, dw, db = ops.dense_bwd(q8(s["x"], 128), q8(s["w"], TILE), s["dy"], s["z"], c["act"], grad_dtype=dt)
    return {"dx": dx, "dw": dw, "db": db}


def _plain(s):
    c = s["case"]
    dt = DTYPES[c["dtype"]]
    if c["op"] == "norm":
        h = s["x"]
        if c["residual"]:
            h = (h.float() + s["residual"].float()).to(dt)
        v = h.float()
        mean = v.mean(1)
        d = v - mean[:, None]
        inv = torch.rsqrt(d.square().mean(1) + EPS)
        y = d * inv[:, None] * s["gamma"]
        if c["beta"]:
            y = y + s["beta"]
        back = _decode(*_encode(y, c["group"]), c["group"]).to(torch.bfloat16) if c["group"] >= 0 else None
        return {"h": h if c["residual"] else None, "y": y.to(dt) if c["y"] else None, "q8": back, "mean": mean, "inv_std": inv}
    if c["op"] == "norm_bwd":
        dy, inv = s["dy"].float(), s["inv"][:, None]
        n = (s["h"].float() - s["mean"][:, None]) * inv
        g = dy * s["gamma"]
        dx = inv * (g - g.mean(1, keepdim=True) - n * (g * n).mean(1, keepdim=True))
        if c["residual"]:
            dx = dx + s["dh"].float()
        return {"dx": dx.to(dt), "dgamma": (dy * n).sum(0), "dbeta": dy.sum(0) if c["beta"] else None}
    if c["op"] == "q8":
        return {"x": _decode(*_encode(s["x"].float(), c["group"]), c["group"]).to(dt)}
    if c["op"] == "moe":
        rows, f = c["rows"], c["inner"]
        # 64 bits: which expert is chosen must not hang on the rounding of a sum
        logits = s["x"].double() @ s["router"].double().t()
        _, order = torch.sort(logits, dim=1, descending=True, stable=True)  # equal ones: the lower index first
        chosen = order[:, :c["k"]]
        top = torch.gather(logits, 1, chosen)
        p = torch.exp(top - logits.amax(1, keepdim=True))
        p = (p / (p if c["normalize"] else torch.exp(logits - logits.amax(1, keepdim=True))).sum(1, keepdim=True)).float()
        x, w1, w2 = s["x"].float(), s["w1"], s["w2"]
        if c["bits8"]:
            x, w1, w2 = _decode(*_encode(x, 128), 128), _decode(*w1, TILE), _decode(*w2, TILE)
        u = torch.matmul(x[None], w1.float().transpose(1, 2))  # every expert with every token
        if c["bias"]:
            u = u + s["b1"][:, None]
        h = _act(c["act"], u[..., :f])
        if c["gated"]:
            h = h * u[..., f:]
        if c["bits8"]:
            h = _decode(*_encode(h.reshape(-1, f), 128), 128).view_as(h)
        o = torch.matmul(h, w2.float().transpose(1, 2))
        if c["bias"]:
            o = o + s["b2"][:, None]
        each = o[chosen, torch.arange(rows, device=o.device)[:, None]]  # [rows, k, cols]
        y = (p[..., None] * each).sum(1)
        if c["residual"]:
            y = y + s["residual"].float()
        return {"y": y.to(dt), "experts": chosen.to(torch.int32), "weights": p}
    if c["op"] == "dense":
        z = _decode(*s["x"], 128) @ _decode(*s["w"], c["wgroup"]).t()
        if c["bias"]:
            z = z + s["bias"]
        y = _act(c["act"], z)
        if c["residual"]:
            y = y + s["residual"].float()
        return {"y": y.to(dt), "z": z.to(dt) if c["save"] == "full" else None}
    dz = s["dy"].float()
    if s["z"] is not None:
        dz = dz * _dact(c["act"], s["z"].float())
    # dz is held in the element type, and for dx in 8 bits of that
    held = dz.to(dt).float()
    dx = _decode(*_encode(held, 128), 128) @ _decode(*s["w"], TILE)
    return {"dx": dx.to(dt), "dw": (held.t() @ _decode(*s["x"], 128)).to(dt), "db": dz.sum(0)}


# ------------------------------------------------------------------ the definition, in 64 bits
def _held8(v, group):
    """What 64-bit values are once they have been held in 8 bits."""
    rows, cols = v.shape
    tall, wide = (128, 128) if group == TILE else (1, group if group > 0 else cols)
    pad = torch.nn.functional.pad(v, (0, -cols % wide, 0, -rows % tall))
    pad = pad.unflatten(1, (-1, wide)).unflatten(0, (-1, tall))
    top = pad.abs().amax((1, 3), keepdim=True)
    unit = torch.exp2(torch.ceil(torch.log2(top / 448)).clamp(-126, 127))
    unit = torch.where(448 * unit < top, 2 * unit, torch.where(448 * (unit / 2) >= top, unit / 2, unit))
    unit = torch.where(top > 0, unit, torch.ones_like(unit))
    t = pad / unit
    step = torch.exp2(torch.floor(torch.log2(t.abs().clamp(min=2.0 ** -6))) - 3)
    return (torch.round(t / step) * step * unit).flatten(2, 3).flatten(0, 1)[:rows, :cols]


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


def _wide(v, group):
    """The values of an 8-bit matrix, in 64 bits."""
    q, scale = v
    r = torch.arange(q.shape[-2], device=q.device) // (128 if group == TILE else 1)
    k = torch.arange(q.shape[-1], device=q.device) // 128
    return q.double() * torch.exp2(scale.double() - 127)[..., r[:, None], k]


def _experts64(c, s):
    x, f = s["x"].double(), c["inner"]
    logits = torch.einsum("td,ed->te", x, s["router"].double())
    index = torch.argsort(logits, dim=1, descending=True, stable=True)[:, :c["k"]]
    probability = torch.softmax(logits, 1).gather(1, index)
    if c["normalize"]:
        probability = probability / probability.sum(1, keepdim=True)
    if c["bits8"]:
        x = _held8(x, 128)
    y = s["residual"].double() if c["residual"] else torch.zeros_like(x)
    for e in torch.unique(index).tolist():  # one expert after the other, with the tokens that chose it
        t, j = torch.nonzero(index == e, as_tuple=True)
        w1, w2 = (_wide((s[n][0][e], s[n][1][e]), TILE) if c["bits8"] else s[n][e].double() for n in ("w1", "w2"))
        u = x[t] @ w1.t()
        if c["bias"]:
            u = u + s["b1"][e].double()
        h = _act64(c["act"], u[:, :f])[0]
        if c["gated"]:
            h = h * u[:, f:]
        if c["bits8"]:
            h = _held8(h, 128)
        o = h @ w2.t()
        if c["bias"]:
            o = o + s["b2"][e].double()
        y = y.index_add(0, t, probability[t, j, None] * o)
    return {"y": y, "experts": index.to(torch.int32), "weights": probability}


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "norm":
        h = s["x"].double()
        if c["residual"]:
            h = (h + s["residual"].double()).to(DTYPES[c["dtype"]]).double()  # h is what the norm is taken of
        mean = h.sum(1) / c["cols"]
        inv = 1 / torch.sqrt(((h - mean[:, None]) ** 2).sum(1) / c["cols"] + EPS)
        y = s["gamma"].double() * ((h - mean[:, None]) * inv[:, None])
        if c["beta"]:
            y = y + s["beta"].double()
        return {"h": h if c["residual"] else None, "y": y if c["y"] else None,
                "q8": _held8(y, c["group"]) if c["group"] >= 0 else None, "mean": mean, "inv_std": inv}
    if c["op"] == "norm_bwd":
        g, inv = s["dy"].double(), s["inv"].double()[:, None]
        n = (s["h"].double() - s["mean"].double()[:, None]) * inv
        gy = g * s["gamma"].double()
        dx = inv * (gy - gy.sum(1, keepdim=True) / c["cols"] - n * (gy * n).sum(1, keepdim=True) / c["cols"])
        if c["residual"]:
            dx = dx + s["dh"].double()
        return {"dx": dx, "dgamma": torch.einsum("rc,rc->c", g, n), "dbeta": g.sum(0) if c["beta"] else None}
    if c["op"] == "q8":
        return {"x": _held8(s["x"].double(), c["group"])}
    if c["op"] == "moe":
        return _experts64(c, s)
    if c["op"] == "dense":
        z = _wide(s["x"], 128) @ _wide(s["w"], c["wgroup"]).t()
        if c["bias"]:
            z = z + s["bias"].double()
        y = _act64(c["act"], z)[0]
        if c["residual"]:
            y = y + s["residual"].double()
        return {"y": y, "z": z if c["save"] == "full" else None}
    dz = s["dy"].double()
    if s["z"] is not None:
        dz = dz * _act64(c["act"], s["z"].double())[1]
    held = dz.to(DTYPES[c["dtype"]]).double()  # dz is held in the element type
    return {"dx": _held8(held, 128) @ _wide(s["w"], TILE), "dw": held.t() @ _wide(s["x"], 128), "db": dz.sum(0)}
