"""Plain 64-bit forms of layer norm, of 8-bit matrices with wide groups and tiles, and of the mixture-of-experts layer."""
import torch

from block_ref import act_ref, q8_ref


def q8_wide_ref(v, group):
    """(values in 64 bits, scale bytes) of v [rows, cols] (64 bits) with one scale for 128 columns (128) or 128 rows by
    128 columns (-128): each group laid out as a row of its own, and counted as one there."""
    rows, cols = v.shape
    tall = 128 if group < 0 else 1
    p = torch.nn.functional.pad(v, (0, -cols % 128, 0, -rows % tall))
    a, b = p.shape[0] // tall, p.shape[1] // 128
    flat = p.view(a, tall, b, 128).transpose(1, 2).reshape(a * b, tall * 128)
    values, scale = q8_ref(flat, 0)
    values = values.view(a, b, tall, 128).transpose(1, 2).reshape(a * tall, b * 128)
    return values[:rows, :cols], scale.view(a, b)


def q8_wide_values(q8):
    """What an 8-bit matrix (or a stack of them) with wide groups or tiles stands for, in 64 bits."""
    q, s = q8.q.double(), torch.exp2(q8.scale.double() - 127)
    if q8.group < 0:
        s = s.repeat_interleave(128, -2)[..., :q.shape[-2], :]
    return q * s.repeat_interleave(128, -1)[..., :q.shape[-1]]


def layer_ref(h, gamma, beta, eps):
    """(y, mean, inv_std)"""
    mean = h.mean(1)
    inv = 1 / torch.sqrt((h - mean[:, None]).square().mean(1) + eps)
    y = gamma * (h - mean[:, None]) * inv[:, None]
    return (y if beta is None else y + beta), mean, inv


def layer_bwd_ref(h, gamma, mean, inv, dy, dh=None):
    """(dx, dgamma, dbeta)"""
    n = (h - mean[:, None]) * inv[:, None]
    g = dy * gamma
    dx = inv[:, None] * (g - g.mean(1, keepdim=True) - n * (g * n).mean(1, keepdim=True))
    return (dx if dh is None else dx + dh), (dy * n).sum(0), dy.sum(0)


def moe_ref(x, router, w1, w2, k, b1, b2, act, gated, normalize, residual, hold):
    """The layer in 64 bits, token by token: (y, experts, weights, magnitudes of y's terms). hold(v): what rows of 64-bit
    values are once they are stored for the second product."""
    T, D = x.shape
    F = w2.shape[2]
    logits = x @ router.t()
    ys, mags, experts, weights = [], [], [], []
    for t in range(T):
        order = sorted(range(router.shape[0]), key=lambda e: (-float(logits[t, e]), e))[:k]
        p = torch.softmax(logits[t, order] if normalize else logits[t], 0)
        p = p if normalize else p[order]
        y = torch.zeros(D, dtype=torch.float64, device=x.device) if residual is None else residual[t].clone()
        mag = y.abs()
        for j, e in enumerate(order):
            z = w1[e] @ x[t] + (0 if b1 is None else b1[e])
            h = act_ref(act, z[:F])
            if gated:
                h = h * z[F:]
            h = hold(h[None])[0]
            y = y + p[j] * (w2[e] @ h + (0 if b2 is None else b2[e]))
            mag = mag + p[j] * (w2[e].abs() @ h.abs() + (0 if b2 is None else b2[e].abs()))
        ys.append(y)
        mags.append(mag)
        experts.append(order)
        weights.append(p)
    return torch.stack(ys), torch.tensor(experts, dtype=torch.int32, device=x.device), torch.stack(weights), torch.stack(mags)
