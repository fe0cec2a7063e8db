"""Layer norm of rows, and 8-bit matrices with a scale for 128 columns or a tile of 128 x 128, against their 64-bit
forms, at the sizes, strides and values where they can go wrong."""
import os
import subprocess
import sys

import pytest
import torch

from block_ref import STEP, TINY, U, close, q8_ref, q8_values, rounded
from conv2d_layer_gb300 import abi, ops
from more_ref import layer_bwd_ref, layer_ref, q8_wide_ref, q8_wide_values

pytestmark = pytest.mark.gpu
BF, HF, FP = torch.bfloat16, torch.float16, torch.float32
EPS = 1e-5


def normal(seed, *shape, std=1.0, dtype=FP):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)


def strided(t, pad):
    """The same values with `pad` more elements from row to row, which hold NaN."""
    if not pad or t is None:
        return t
    wide = torch.full((t.shape[0], t.shape[1] + pad), float("nan"), device=t.device).to(t.dtype)
    wide[:, :t.shape[1]] = t
    return wide[:, :t.shape[1]]


@pytest.fixture(autouse=True)
def device_clean():
    yield
    assert abi.conv2d_device_status() == (abi.OK, 0)


# ------------------------------------------------------------------ 8 bits
@pytest.mark.parametrize("group", [128, ops.TILE])
@pytest.mark.parametrize("rows,cols,dtype,pad", [
    (1, 1, BF, 0), (3, 31, HF, 0), (5, 128, FP, 0), (2, 129, BF, 0), (130, 256, BF, 0), (4, 1000, HF, 8), (129, 2056, BF, 3),
    (2, 4096, FP, 4), (257, 384, HF, 16), (2, 16384, BF, 0), (2, 20000, HF, 0), (1, 5001, FP, 0), (3, 200, BF, 0),
    (2, 9001, BF, 0), (2, 17000, HF, 1), (70000, 40, BF, 0), (300, 1021, HF, 0)])
def test_q8_wide_encode_decode(rows, cols, dtype, group, pad):
    x = normal(rows + cols, rows, cols) * torch.exp2(torch.randint(-12, 12, (rows, 1), device="cuda").float())
    x = x.to(dtype)
    q = ops.q8_encode(strided(x, pad), group)
    ref, scale = q8_wide_ref(x.double(), group)
    assert torch.equal(q.scale, scale)
    assert torch.equal(q8_wide_values(q), ref)
    assert torch.equal(ops.q8_decode(q, FP).double(), ref)
    assert torch.equal(ops.q8_decode(q, BF).double(), ref)
    out = strided(torch.empty(rows, cols, dtype=dtype, device="cuda"), 3)
    ops.q8_decode(q, dtype, out=out)
    close(out, ref, U[HF] * ref.abs() + 2.0 ** -25 if dtype == HF else 0.0 * ref, "decode into rows of odd length")
    given = ops.Q8(strided(q.q.float(), 5).to(torch.float8_e4m3fn), torch.empty_like(q.scale), group)
    assert ops.q8_encode(x, out=given) is given
    assert torch.equal(given.q.float(), q.q.float()) and torch.equal(given.scale, q.scale)


@pytest.mark.parametrize("group", [128, ops.TILE])
@pytest.mark.parametrize("cols", [384, 387, 1029])
def test_q8_wide_special_values(group, cols):
    x = torch.zeros(6, cols, device="cuda")
    x[0, 3], x[0, 4], x[0, 5] = float("inf"), float("-inf"), float("nan")  # beside ordinary values
    x[0, 6] = 3.0
    x[1, :128] = float("nan")          # a group without a finite value
    x[2, 128:256] = 1e-42              # subnormal
    x[3, 256:384] = torch.finfo(FP).max
    x[4, 0], x[4, 1] = 448.0, 449.0   # just past the largest value at scale 1
    q = ops.q8_encode(x, group)
    ref, scale = q8_wide_ref(x.double(), group)
    assert torch.equal(q.scale, scale)
    ref = torch.where(ref.isfinite(), ref.clamp(-torch.finfo(FP).max, torch.finfo(FP).max), ref)
    close(ops.q8_decode(q, FP), ref, torch.zeros_like(ref), "special")


# ------------------------------------------------------------------ layer norm
NORMS = [(1, 1, FP, 0), (1, 4096, BF, 0), (3, 7, HF, 0), (9, 33, BF, 0), (5, 64, FP, 0), (300, 128, HF, 0), (17, 256, BF, 8),
         (33, 512, BF, 0), (4, 1000, HF, 3), (6, 1021, FP, 0), (5, 2048, FP, 0), (3, 5120, BF, 0), (2, 8192, HF, 0),
         (3, 12000, BF, 0), (2, 16384, BF, 0), (2, 20000, BF, 0), (2, 9001, FP, 0), (1000, 40, FP, 4), (2, 17001, HF, 0)]


def bounds(h, gamma, beta, mean, inv):
    """(mean, inv, y): how far the fp32 arithmetic is off. A thread adds up to cols / 32 terms, then the threads' sums
    are joined (ten steps): `adds` of the sum of magnitudes. An error e of the mean moves the sum of squares by
    cols e^2 only, and each distance by e."""
    cols = h.shape[1]
    adds = (cols / 32 + 10) * STEP
    e = (adds + U[FP]) * h.abs().mean(1) + U[FP] * mean.abs() + TINY[FP]
    half = 0.5 * (adds + 4 * U[FP] + e * e * inv * inv) + 3 * U[FP]
    n = (h - mean[:, None]) * inv[:, None]
    y = gamma.abs() * (e * inv)[:, None] * 1.01 + (half[:, None] + 4 * U[FP]) * (gamma * n).abs()
    if beta is not None:
        y = y + U[FP] * (gamma * n + beta).abs()
    return e, half * inv, y


@pytest.mark.parametrize("rows,cols,dtype,pad", NORMS)
@pytest.mark.parametrize("residual,offset,has_beta", [(False, 0.0, True), (True, 5.0, True), (True, 0.0, False)])
@pytest.mark.parametrize("group", [None, 32, 128, 0])
def test_layer_norm_fwd(rows, cols, dtype, pad, residual, offset, has_beta, group):
    x, gamma = normal(1, rows, cols, std=3.0) + offset, normal(2, cols)
    x = x.to(dtype)
    beta = normal(5, cols) if has_beta else None
    r = normal(3, rows, cols, dtype=dtype) if residual else None
    out = ops.layer_norm_fwd(strided(x, pad), gamma, beta, EPS, residual=strided(r, pad), group=group)
    h = x.double()
    if residual:
        h = (x.float() + r.float()).to(dtype)  # one fp32 addition, rounded: the definition of h
        assert torch.equal(out.h, h)
        h = h.double()
    b64 = None if beta is None else beta.double()
    y, mean, inv = layer_ref(h, gamma.double(), b64, EPS)
    bm, bi, by = bounds(h, gamma.double(), b64, mean, inv)
    close(out.mean, mean, bm, "mean")
    close(out.inv_std, inv, bi, "inv_std")
    close(out.y, y, rounded(y, dtype, by), "y")
    if group is not None:
        # half a step off: 2^-4 of the value or 2^-10 of the scale (of which the bound of the largest value is a part);
        # the scale may be the next one where y's own error carries it over 448
        s = torch.exp2(out.q8.scale.double() - 127).repeat_interleave(group or cols, 1)[:, :cols]
        got = q8_wide_values(out.q8) if group == 128 else q8_values(out.q8)
        close(got, y, torch.maximum(2.0 ** -4 * y.abs(), 2.0 ** -10 * s) + 2 * by, "q8")
        # the 8-bit form is that of the unrounded y: fp32's y is the same numbers
        if dtype == FP:
            ref, scale = (q8_wide_ref if group == 128 else q8_ref)(out.y.double(), group)
            assert torch.equal(out.q8.scale, scale) and torch.equal(got, ref)
        only = ops.layer_norm_fwd(x, gamma, beta, EPS, residual=r, y=False, group=group)
        assert only.y is None and torch.equal(only.q8.q.view(torch.uint8), out.q8.q.view(torch.uint8))
        assert torch.equal(only.q8.scale, out.q8.scale)


@pytest.mark.parametrize("rows,cols,dtype", [(3, 4096, BF), (5, 1021, HF), (2, 9001, FP), (9, 100, BF), (2, 20000, BF)])
def test_rms_norm_to_wide_groups(rows, cols, dtype):
    x, gamma = normal(1, rows, cols, dtype=dtype), normal(2, cols)
    out = ops.rms_norm_fwd(x, gamma, group=128)
    plain = ops.rms_norm_fwd(x.float(), gamma)  # the same fp32 numbers, kept
    ref, scale = q8_wide_ref(plain.y.double(), 128)
    # fp32 rows take other threads than 16-bit ones, so the sums may differ by their error, and a value on a border fall
    # to the other side
    s = torch.exp2(out.q8.scale.double() - 127).repeat_interleave(128, 1)[:, :cols]
    got = q8_wide_values(out.q8)
    close(got, plain.y.double(), torch.maximum(2.0 ** -4 * plain.y.double().abs(), 2.0 ** -10 * s) + 1e-4 * plain.y.double().abs(), "q8")
    assert float((got != ref).double().mean()) < 1e-3


def test_layer_norm_in_place_and_special_rows():
    x, r, gamma, beta = normal(1, 6, 512, dtype=BF), normal(2, 6, 512, dtype=BF), normal(3, 512), normal(4, 512)
    want = ops.layer_norm_fwd(x, gamma, beta, residual=r)
    r2 = r.clone()
    got = ops.layer_norm_fwd(x, gamma, beta, residual=r2, h=r2)
    assert torch.equal(got.h, want.h) and torch.equal(r2, want.h) and torch.equal(got.y, want.y)
    x = torch.zeros(5, 300, device="cuda")
    x[1, 5] = float("inf")
    x[2, 6] = float("nan")
    x[3] = 7.0
    x[4] = 1e4 + (torch.arange(300, device="cuda") % 2)  # far from zero: 10000 and 10001
    g, b = torch.ones(300, device="cuda"), torch.full((300,), 2.0, device="cuda")
    out = ops.layer_norm_fwd(x, g, b, 1e-5, group=32)
    assert torch.equal(out.y[0], b) and torch.equal(out.y[3], b)  # constant rows: the mean is exact there
    assert bool(out.y[1].isnan().all()) and bool(out.y[2].isnan().all())
    y, mean, inv = layer_ref(x[4:].double(), g.double(), b.double(), 1e-5)
    close(out.mean[4:], mean, torch.full_like(mean, 2.0 ** -9), "mean")  # half a step of 10000 at the last division, and the sums'
    # an error of 2^-9 of the mean moves each distance (1/2) and so y (1) by 2^-8, and the deviation by its square
    close(out.y[4:], y, torch.full_like(y, 2.0 ** -7), "far row")


@pytest.mark.parametrize("rows,cols,dtype,pad", NORMS + [(3000, 256, BF, 0), (700, 2048, BF, 0), (37, 528, BF, 0), (37, 768, HF, 0),
                                                         (900, 1024, BF, 0), (37, 1040, BF, 0), (37, 2576, BF, 0),
                                                         (400, 5120, BF, 0), (37, 6144, HF, 0), (37, 8208, BF, 0),
                                                         (37, 1032, HF, 8), (37, 2056, BF, 0), (37, 2568, BF, 8),
                                                         (37, 6152, BF, 0), (37, 516, FP, 0), (400, 1000, FP, 0),
                                                         (37, 1536, FP, 0), (37, 2052, FP, 0), (37, 4100, FP, 0),
                                                         (40, 12001, BF, 0), (5, 4097, FP, 0),
                                                         (700, 1021, BF, 0), (1, 513, HF, 0), (2, 514, BF, 0), (37, 777, HF, 3),
                                                         (400, 528, BF, 3), (333, 1000, BF, 0), (3, 8191, BF, 0), (2, 8192, HF, 1),
                                                         (1500, 2047, HF, 1), (310, 4095, BF, 0), (1, 8224, BF, 0),
                                                         (76, 8224, HF, 8), (153, 10240, BF, 0), (700, 16384, HF, 0),
                                                         (2, 16416, BF, 0), (39, 16448, BF, 0), (200, 32768, HF, 0),
                                                         (7, 32832, BF, 0),
                                                         (37, 1021, BF, 8), (300, 4099, FP, 4), (20, 9001, HF, 16),
                                                         (5, 30001, BF, 8), (16, 13496, FP, 0), (900, 4093, BF, 0),
                                                         (160, 8195, FP, 0), (90, 16391, BF, 0), (41, 15999, HF, 0)])
@pytest.mark.parametrize("skip", [False, True])
def test_layer_norm_bwd(rows, cols, dtype, pad, skip):
    h, gamma, dy = (normal(1, rows, cols) + 0.5).to(dtype), normal(2, cols), normal(3, rows, cols, dtype=dtype)
    dh = normal(4, rows, cols, dtype=dtype) if skip else None
    h64, dy64, g64 = h.double(), dy.double(), gamma.double()
    _, mean, inv = layer_ref(h64, g64, None, EPS)
    mean, inv = mean.float(), inv.float()
    dx, dg, db = ops.layer_norm_bwd(strided(h, pad), gamma, mean, inv, strided(dy, pad), dh=strided(dh, pad))
    m64, i64 = mean.double(), inv.double()
    rx, rg, rb = layer_bwd_ref(h64, g64, m64, i64, dy64, None if dh is None else dh.double())
    n = (h64 - m64[:, None]) * i64[:, None]
    g = dy64 * g64
    # both means: their terms' magnitudes, added as in the forward; then the difference, two products and the sum with
    # dh. n itself carries two roundings, g one.
    adds = (cols / 32 + 14) * STEP
    es, ed = adds * g.abs().mean(1, keepdim=True), adds * (g * n).abs().mean(1, keepdim=True)
    s, d = g.mean(1, keepdim=True), (g * n).mean(1, keepdim=True)
    extra = i64[:, None] * (es + n.abs() * ed + 6 * U[FP] * (g.abs() + s.abs() + (n * d).abs()))
    if skip:
        extra = extra + U[FP] * rx.abs()
    close(dx, rx, rounded(rx, dtype, extra), "dx")
    # at most rows additions in a thread, eight warps and up to 304 blocks after them, five roundings a term
    count = (min(rows, 304) / 8 + rows / 304 + 20) * STEP
    close(dg, rg, count * (dy64 * n).abs().sum(0) + 1e-300, "dgamma")
    close(db, rb, count * dy64.abs().sum(0) + 1e-300, "dbeta")
    if skip:  # in place of the incoming gradient, accumulating; then one result at a time
        ag, ab, buf = dg.clone(), db.clone(), dh.clone()
        x2, g2, b2 = ops.layer_norm_bwd(h, gamma, mean, inv, dy, dh=buf, dx=buf, dgamma=ag, dbeta=ab)
        assert x2 is buf and g2 is ag and b2 is ab
        if not pad:
            assert torch.equal(x2, dx) and torch.equal(g2, dg + dg) and torch.equal(b2, db + db)
        only = ops.layer_norm_bwd(h, gamma, mean, inv, dy, dh=dh, need_dgamma=False, need_dbeta=False)
        assert only[1:] == (None, None) and torch.equal(only[0], x2)
        only = ops.layer_norm_bwd(h, gamma, mean, inv, dy, need_dx=False, need_dbeta=False)
        assert only[0] is None and only[2] is None and (pad or torch.equal(only[1], dg))
        only = ops.layer_norm_bwd(h, gamma, mean, inv, dy, need_dx=False, need_dgamma=False)
        assert only[:2] == (None, None) and (pad or torch.equal(only[2], db))


FIRST_CALL_CAPTURED = """
import torch
from conv2d_layer_gb300 import ops
g = torch.Generator(device="cuda").manual_seed(0)
n = lambda *s: torch.randn(*s, generator=g, device="cuda")
h, dy, gamma, mean, inv = n(5, COLS).half(), n(5, COLS).half(), n(COLS), n(5), n(5).abs()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    out = ops.layer_norm_bwd(h, gamma, mean, inv, dy, dh=dy)
for t in out:
    t.zero_()
graph.replay()
want = ops.layer_norm_bwd(h, gamma, mean, inv, dy, dh=dy)
assert all(torch.equal(a, b) and bool(a.any()) for a, b in zip(out, want))
"""


@pytest.mark.parametrize("cols", [2048, 8224, 20480])
def test_layer_norm_bwd_first_called_under_capture(cols):
    """What a kernel's first launch asks the device for is asked during a capture as well."""
    subprocess.run([sys.executable, "-c", FIRST_CALL_CAPTURED.replace("COLS", str(cols))], check=True, timeout=300,
                   cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))


@pytest.mark.parametrize("rows,cols,dtype", [(40, 1021, BF), (37, 9001, HF), (37, 5119, FP), (4100, 777, BF), (500, 257, FP),
                                             (9, 20001, BF)])
def test_odd_rows_do_not_mix(rows, cols, dtype):
    """Rows of NaN and infinities between others: those come out bit by bit as beside rows of zeros, and the columns behind
    a strided output's rows stay as they were."""
    gamma, beta = normal(1, cols), normal(2, cols)
    x, r, dy = (normal(3 + i, rows, cols, dtype=dtype) for i in range(3))
    bad = torch.arange(rows, device="cuda") % 2 == 1

    def out():
        return torch.full((rows, cols + 8), 7.0, device="cuda", dtype=dtype)

    def run(v):
        a, b, d = (torch.where(bad[:, None], torch.full_like(t, v), t) for t in (x, r, dy))
        h, y, dx = out(), out(), out()
        n = ops.layer_norm_fwd(strided(a, 8), gamma, beta, EPS, residual=strided(b, 8), h=h[:, :cols], y=y[:, :cols])
        ops.layer_norm_bwd(h[:, :cols], gamma, n.mean, n.inv_std, strided(d, 8), dh=strided(d, 8), dx=dx[:, :cols],
                           need_dgamma=False, need_dbeta=False)
        return h, y, dx

    zero = run(0.0)
    for v in (float("nan"), float("inf")):
        for got, want in zip(run(v), zero):
            assert torch.equal(got[~bad], want[~bad]) and bool(got[~bad].isfinite().all())
            assert bool((got[:, cols:] == 7).all())


def test_layer_norm_without_rows():
    x, gamma = torch.empty(0, 64, device="cuda", dtype=BF), torch.ones(64, device="cuda")
    out = ops.layer_norm_fwd(x, gamma, gamma, residual=x, group=128)
    assert out.y.shape == (0, 64) and out.q8.scale.shape == (0, 1)
    dx, dg, db = ops.layer_norm_bwd(x, gamma, out.mean, out.inv_std, x)
    assert dx.shape == (0, 64) and not bool(dg.any()) and not bool(db.any())
    acc = torch.ones(64, device="cuda")
    _, dg, db = ops.layer_norm_bwd(x, gamma, out.mean, out.inv_std, x, dgamma=acc, dbeta=acc.clone())
    assert torch.equal(dg, torch.ones_like(dg)) and torch.equal(db, dg)


def test_layer_norm_captured_and_on_another_stream():
    x, gamma, beta = normal(1, 64, 1000, dtype=BF), normal(2, 1000), normal(3, 1000)
    dy = normal(4, 64, 1000, dtype=BF)

    def step(stream=None):
        o = ops.layer_norm_fwd(x, gamma, beta, group=128, stream=stream)
        return (o.y, o.q8.q.view(torch.uint8), o.q8.scale, *ops.layer_norm_bwd(o.h, gamma, o.mean, o.inv_std, dy, stream=stream))

    want = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = step(side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    x.add_(normal(9, 64, 1000, dtype=BF))
    for _ in range(2):
        graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(step(), held))
