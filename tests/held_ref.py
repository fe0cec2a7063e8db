"""What a value that is known within an error may be once it is held in 8 bits."""
import torch


def exponents(top):
    """The scales' exponents of groups whose largest magnitudes are `top` (finite): the smallest e with top <= 448 * 2^e."""
    e = torch.ceil(torch.log2(torch.clamp(top, min=2.0 ** -126) / 448))
    e = torch.where(top > 448 * torch.exp2(e), e + 1, e)
    e = torch.where(top <= 448 * torch.exp2(e - 1), e - 1, e)
    return torch.where(top > 0, e.clamp(min=-126), 0)


def at_scale(v, e):
    """v to the nearest e4m3 value times 2^e, ties to even."""
    t = v / torch.exp2(e)
    step = torch.exp2(torch.floor(torch.log2(t.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(t / step) * step * torch.exp2(e)


def held_between(v, err, dtype=None):
    """(least, greatest) of what v [rows, cols], off by up to err, is in 8 bits with a scale for 128 columns, rounded to
    dtype before: rounding keeps the order, so the ends of v's interval bound it, each with the least and the greatest
    scale that the group may have."""
    lo, hi = v - err, v + err
    if dtype is not None:
        lo, hi = lo.to(dtype).double(), hi.to(dtype).double()
    cols = v.shape[1]

    def groups(t):
        return torch.nn.functional.pad(t, (0, -cols % 128)).view(t.shape[0], -1, 128).amax(2)

    least = torch.where((lo < 0) & (hi > 0), 0.0, torch.minimum(lo.abs(), hi.abs()))
    ends = []
    for top in (groups(least), groups(torch.maximum(lo.abs(), hi.abs()))):
        e = exponents(top).repeat_interleave(128, 1)[:, :cols]
        ends += [at_scale(lo, e), at_scale(hi, e)]
    ends = torch.stack(ends)
    return ends.amin(0), ends.amax(0)
