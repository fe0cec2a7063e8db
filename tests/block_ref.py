"""Plain 64-bit forms of the residual block's operators (RMS norm, dense layer, 8-bit checkpoints), and the
bounds their tests hold the kernels to. A rounding is off by half a step, U[dtype] relative; sums held in fp32
lose at most a step (2^-23) of the sum of magnitudes for each addition (the tensor core adds 16 products at a
time and truncates)."""
import math

import torch

U = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.float32: 2.0 ** -150, torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25}  # half the smallest step
STEP = 2.0 ** -23


def q8_ref(v, group):
    """(values in 64 bits, scale bytes) of v [rows, cols] (64 bits) in 8 bits, by counting: the scale from the
    largest finite magnitude, each value to the nearest multiple of its step, ties to even."""
    rows, cols = v.shape
    g = group if group else max(cols, 1)
    pad = torch.nn.functional.pad(v, (0, -cols % g)).reshape(rows, -1, g)
    top = torch.where(pad.isfinite(), pad.abs(), 0).amax(2)
    e = torch.full_like(top, -126)
    for k in range(-126, 128):  # the smallest e with top <= 448 * 2^e
        e = torch.where(top > 448 * 2.0 ** (k - 1), float(k), e) if k > -126 else e
    e = torch.where(top > 0, e, 0)
    t = pad / torch.exp2(e)[..., None]
    mag = t.abs().clamp(min=2.0 ** -6)
    step = torch.exp2(torch.floor(torch.log2(mag)) - 3)
    q = torch.where(t.isfinite(), torch.round(t / step) * step, math.nan)
    return (q * torch.exp2(e)[..., None]).reshape(rows, -1)[:, :cols], (e + 127).to(torch.uint8)


def q8_values(q8):
    """What an 8-bit matrix stands for, in 64 bits."""
    cols = q8.q.shape[1]
    g = q8.group if q8.group else max(cols, 1)
    col = torch.arange(cols, device=q8.q.device) // g
    return q8.q.double() * torch.exp2(q8.scale.double() - 127)[:, col]


def act_ref(act, z):
    if act == "relu":
        return torch.where(z > 0, z, torch.where(z <= 0, 0.0, z))
    if act == "tanh":
        return torch.tanh(z)
    if act == "sigmoid":
        return torch.sigmoid(z)
    if act == "silu":
        return z * torch.sigmoid(z)
    if act == "gelu":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    return z.clone()


def dact_ref(act, z):
    if act == "relu":
        return torch.where(z > 0, 1.0, torch.where(z <= 0, 0.0, z))
    if act == "tanh":
        return 1 / torch.cosh(z) ** 2
    if act == "sigmoid":
        return torch.sigmoid(z) * torch.sigmoid(-z)
    if act == "silu":
        return torch.sigmoid(z) * (1 + z * torch.sigmoid(-z))
    if act == "gelu":
        a, b = math.sqrt(2 / math.pi), 0.044715
        t = torch.tanh(a * (z + b * z ** 3))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * a * (1 + 3 * b * z * z)
    return torch.ones_like(z)


def rms_ref(h, gamma, eps):
    inv = 1 / torch.sqrt((h * h).mean(1) + eps)
    return gamma * h * inv[:, None], inv


def rms_bwd_ref(h, gamma, inv, dy, dh=None):
    n = h * inv[:, None]
    g = dy * gamma
    dx = inv[:, None] * (g - n * (g * n).mean(1, keepdim=True))
    return (dx if dh is None else dx + dh), (dy * n).sum(0)


def close(got, ref, tol, name=""):
    """Every element of got within tol of ref; infinities and NaN in the same places."""
    got = got.double()
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    fine = ref.isfinite()
    assert torch.equal(fine, got.isfinite()), f"{name}: infinities or NaN differ"
    off = torch.where(fine, (got - ref).abs() - tol, -1.0)
    if off.numel():
        i = int(off.argmax())
        assert float(off.flatten()[i]) <= 0, (name, i, float(got.flatten()[i]), float(ref.flatten()[i]),
                                              float(torch.as_tensor(tol).expand_as(ref).flatten()[i]))


def rounded(ref, dtype, extra=0.0):
    """Bound of a value that is `extra` off before it is rounded to dtype."""
    return U[dtype] * (ref.abs() + extra) + TINY[dtype] + extra
