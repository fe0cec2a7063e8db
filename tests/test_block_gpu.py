"""RMS norm, dense layer and 8-bit checkpoints against their 64-bit forms, at the sizes, strides and values
where they can go wrong."""
import pytest
import torch

from block_ref import (STEP, U, act_ref, close, dact_ref, q8_ref, q8_values, rms_bwd_ref, rms_ref, rounded)
from conv2d_layer_gb300 import abi, ops

pytestmark = pytest.mark.gpu
BF, HF, FP = torch.bfloat16, torch.float16, torch.float32


def normal(seed, *shape, std=1.0, dtype=FP):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)


def strided(t, pad):
    """The same values with `pad` more elements from row to row, which hold NaN."""
    if not pad:
        return t
    wide = torch.full((t.shape[0], t.shape[1] + pad), float("nan"), device=t.device).to(t.dtype)
    wide[:, :t.shape[1]] = t
    return wide[:, :t.shape[1]]


@pytest.fixture(autouse=True)
def device_clean():
    yield
    assert abi.conv2d_device_status() == (abi.OK, 0)


# ------------------------------------------------------------------ 8 bits
@pytest.mark.parametrize("group", [32, 0])
@pytest.mark.parametrize("rows,cols,dtype,pad", [
    (1, 1, BF, 0), (3, 31, HF, 0), (5, 32, FP, 0), (2, 33, BF, 0), (7, 256, BF, 0), (4, 1000, HF, 8), (3, 2056, BF, 3),
    (2, 4096, FP, 4), (2, 16384, BF, 0), (2, 20000, HF, 0), (1, 5001, FP, 0), (70000, 40, BF, 0)])
def test_q8_encode_decode(rows, cols, dtype, group, pad):
    x = normal(rows + cols, rows, cols) * torch.exp2(torch.randint(-12, 12, (rows, 1), device="cuda").float())
    x = x.to(dtype)
    q = ops.q8_encode(strided(x, pad), group)
    ref, scale = q8_ref(x.double(), group)
    assert torch.equal(q.scale, scale)
    assert torch.equal(q8_values(q), ref)
    # the stated error: 2^-4 of the value, or 2^-10 of the scale
    s = torch.exp2(scale.double() - 127).repeat_interleave(group or cols, 1)[:, :cols]
    close(ref, x.double(), torch.maximum(2.0 ** -4 * x.double().abs(), 2.0 ** -10 * s), "encode")
    assert torch.equal(ops.q8_decode(q, FP).double(), ref)
    assert torch.equal(ops.q8_decode(q, BF).double(), ref)
    out = strided(torch.empty(rows, cols, dtype=dtype, device="cuda"), 3)
    ops.q8_decode(q, dtype, out=out)
    close(out, ref, U[HF] * ref.abs() + 2.0 ** -25 if dtype == HF else 0.0 * ref, "decode into rows of odd length")


def test_q8_special_values():
    x = torch.zeros(6, 96, device="cuda")
    x[0, 3], x[0, 4], x[0, 5] = float("inf"), float("-inf"), float("nan")  # beside ordinary values
    x[0, 6] = 3.0
    x[1, :32] = float("nan")          # a group without a finite value
    x[2, :32] = 1e-42                 # subnormal
    x[3, :32] = torch.finfo(FP).max
    x[4, 0], x[4, 1] = 448.0, 449.0   # just past the largest value at scale 1
    x[5, 0], x[5, 1] = 448.0, -0.0
    for group in (32, 0):
        q = ops.q8_encode(x, group)
        ref, scale = q8_ref(x.double(), group)
        assert torch.equal(q.scale, scale)
        # the largest fp32 value rounds up to 2^128 in 8 bits, and decodes to the largest fp32 value
        ref = torch.where(ref.isfinite(), ref.clamp(-torch.finfo(FP).max, torch.finfo(FP).max), ref)
        close(ops.q8_decode(q, FP), ref, torch.zeros_like(ref), "special")
        assert int(q.scale[5, 0]) == 127 and int(q.scale[4, 0]) == 128
    assert int(ops.q8_encode(x, 32).scale[0, 1]) == 127  # an empty group
    # fp16: the largest values round up to 65536 in 8 bits, and decode to the largest fp16
    big = torch.full((1, 32), 65504.0, device="cuda", dtype=HF)
    assert torch.equal(ops.q8_decode(ops.q8_encode(big), HF), big)


# ------------------------------------------------------------------ RMS norm
NORMS = [(1, 1, FP, 0), (1, 4096, BF, 0), (3, 7, HF, 0), (9, 33, BF, 0), (5, 64, FP, 0), (300, 128, HF, 0), (17, 256, BF, 8),
         (33, 512, BF, 0), (4, 1000, HF, 3), (6, 1021, FP, 0), (5, 2048, FP, 0), (3, 5120, BF, 0), (2, 8192, HF, 0),
         (3, 12000, BF, 0), (2, 16384, BF, 0), (2, 20000, BF, 0), (2, 9001, FP, 0), (1000, 40, FP, 4)]


def norm_bound(cols):
    """Relative error of the normalised value: a thread adds up to cols / 32 squares, then the threads' sums
    are joined (ten steps); half of the sum's error reaches the root, and a few roundings follow."""
    return 0.5 * (cols / 32 + 10) * STEP + 4 * U[FP]


@pytest.mark.parametrize("rows,cols,dtype,pad", NORMS)
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("group", [None, 32, 0])
def test_rms_norm_fwd(rows, cols, dtype, pad, residual, group):
    x, gamma = normal(1, rows, cols, std=3.0, dtype=dtype), normal(2, cols)
    r = normal(3, rows, cols, dtype=dtype) if residual else None
    out = ops.rms_norm_fwd(strided(x, pad), gamma, 1e-6, residual=None if r is None else strided(r, pad), group=group)
    h = x.double()
    if residual:
        h = (x.float() + r.float()).to(dtype)  # one fp32 addition, rounded: the definition of h
        assert torch.equal(out.h, h)
        h = h.double()
    y, inv = rms_ref(h, gamma.double(), 1e-6)
    b = norm_bound(cols)
    close(out.inv_rms, inv, b * inv, "inv_rms")
    close(out.y, y, rounded(y, dtype, b * y.abs()), "y")
    if group is not None:
        # the 8-bit values are half a step off: 2^-4 of the value or 2^-10 of the scale (of which the bound of
        # the largest value is a part); the scale may be the next one where y's own error carries it over 448
        s = torch.exp2(out.q8.scale.double() - 127).repeat_interleave(group or cols, 1)[:, :cols]
        close(q8_values(out.q8), y, torch.maximum(2.0 ** -4 * y.abs(), 2.0 ** -10 * s) + 2 * b * y.abs(), "q8")
        only = ops.rms_norm_fwd(x, gamma, 1e-6, residual=r, y=False, group=group)
        assert only.y is None and torch.equal(only.q8.q.view(torch.uint8), out.q8.q.view(torch.uint8))
        assert torch.equal(only.q8.scale, out.q8.scale)


def test_rms_norm_in_place_and_special_rows():
    x, r, gamma = normal(1, 6, 512, dtype=BF), normal(2, 6, 512, dtype=BF), normal(3, 512)
    want = ops.rms_norm_fwd(x, gamma, residual=r)
    r2 = r.clone()
    got = ops.rms_norm_fwd(x, gamma, residual=r2, h=r2)
    assert torch.equal(got.h, want.h) and torch.equal(r2, want.h) and torch.equal(got.y, want.y)
    x = torch.zeros(4, 300, device="cuda")
    x[1, 5] = float("inf")
    x[2, 6] = float("nan")
    x[3] = 1e-30
    g = torch.ones(300, device="cuda")
    out = ops.rms_norm_fwd(x, g, 1e-5, group=32)
    assert torch.equal(out.y[0], torch.zeros(300, device="cuda"))  # a row of zeros stays zero
    assert bool(out.y[1, 5].isnan()) and bool((out.y[1, :5] == 0).all())
    assert bool(out.y[2].isnan().all())
    ref = 1e-30 / (1e-5 ** 0.5)
    close(out.y[3], torch.full((300,), ref, dtype=torch.float64, device="cuda"), 1e-6 * ref, "tiny row")


@pytest.mark.parametrize("rows,cols,dtype,pad", NORMS + [(3000, 256, BF, 0), (700, 2048, BF, 0)])
@pytest.mark.parametrize("skip", [False, True])
def test_rms_norm_bwd(rows, cols, dtype, pad, skip):
    h, gamma, dy = normal(1, rows, cols, dtype=dtype), normal(2, cols), normal(3, rows, cols, dtype=dtype)
    dh = normal(4, rows, cols, dtype=dtype) if skip else None
    inv = torch.rsqrt(h.double().square().mean(1) + 1e-6).float()
    dx, dg = ops.rms_norm_bwd(strided(h, pad), gamma, inv, strided(dy, pad), dh=None if dh is None else strided(dh, pad))
    h64, dy64, i64 = h.double(), dy.double(), inv.double()
    rx, rg = rms_bwd_ref(h64, gamma.double(), i64, dy64, None if dh is None else dh.double())
    n = h64 * i64[:, None]
    g = dy64 * gamma.double()
    # the mean of g n: its terms' magnitudes, added as in the forward; then three products and the sum with dh
    dot = (cols / 32 + 12) * STEP * (g * n).abs().mean(1, keepdim=True)
    extra = i64[:, None] * (n.abs() * dot + 4 * U[FP] * (g.abs() + n.abs() * (g * n).mean(1, keepdim=True).abs()))
    if skip:
        extra = extra + U[FP] * rx.abs()
    close(dx, rx, rounded(rx, dtype, extra), "dx")
    # dgamma: at most rows additions in a thread, eight warps and up to 304 blocks after them, four roundings a term
    mag = (dy64 * n).abs().sum(0)
    close(dg, rg, (min(rows, 304) / 8 + rows / 304 + 20) * STEP * mag + 1e-300, "dgamma")
    if skip:  # in place of the incoming gradient, accumulating
        acc = dg.clone()
        buf = dh.clone()
        dx2, dg2 = ops.rms_norm_bwd(h, gamma, inv, dy, dh=buf, dx=buf, dgamma=acc)
        assert dx2 is buf and dg2 is acc
        if not pad:
            assert torch.equal(dx2, dx) and torch.equal(dg2, dg + dg)
        only, none = ops.rms_norm_bwd(h, gamma, inv, dy, dh=dh, need_dgamma=False)
        assert none is None and torch.equal(only, dx2)
        none, only = ops.rms_norm_bwd(h, gamma, inv, dy, need_dx=False)
        assert none is None and (pad or torch.equal(only, dg))


# one for each number of threads that a row gets: by length, type and alignment
LENGTHS = [(37, 528, BF, 0), (37, 768, HF, 0), (900, 1024, BF, 0), (37, 1040, BF, 0), (1300, 2048, HF, 0), (37, 1536, BF, 0),
           (37, 2576, BF, 0), (400, 5120, BF, 0), (37, 6144, HF, 0), (37, 8208, BF, 0), (37, 1000, BF, 0), (37, 1032, HF, 8),
           (37, 2056, BF, 0), (37, 2568, BF, 8), (37, 6152, BF, 0), (37, 8200, HF, 0), (37, 516, FP, 0), (400, 1000, FP, 0),
           (37, 1300, FP, 0), (37, 1536, FP, 0), (37, 2052, FP, 0), (37, 4100, FP, 0)]


@pytest.mark.parametrize("rows,cols,dtype,pad", LENGTHS)
def test_rms_norm_lengths(rows, cols, dtype, pad):
    for group in (32, 0):
        test_rms_norm_fwd(rows, cols, dtype, pad, True, group)
    test_rms_norm_bwd(rows, cols, dtype, pad, True)


def test_rms_norm_gradient_matches_differences():
    h, gamma, w = normal(1, 3, 48, dtype=FP).double(), normal(2, 48).double(), normal(3, 3, 48).double()
    _, inv = rms_ref(h, gamma, 1e-6)
    dx, dg = ops.rms_norm_bwd(h.float(), gamma.float(), inv.float(), w.float())

    def loss(h, gamma):
        return float((rms_ref(h, gamma, 1e-6)[0] * w).sum())

    for i in range(0, 144, 7):
        d = torch.zeros(144, dtype=torch.float64, device="cuda")
        d[i] = 1e-5
        d = d.view(3, 48)
        num = (loss(h + d, gamma) - loss(h - d, gamma)) / 2e-5
        assert abs(num - float(dx.flatten()[i])) < 1e-5 * (1 + abs(num))
    d = torch.zeros(48, dtype=torch.float64, device="cuda")
    d[11] = 1e-5
    num = (loss(h, gamma + d) - loss(h, gamma - d)) / 2e-5
    assert abs(num - float(dg[11])) < 1e-5 * (1 + abs(num))


# ------------------------------------------------------------------ dense layer
def mm_bound(a, b):
    """fp32 accumulation of a b^T: one truncated addition for every 16 products, and up to 20 joins."""
    return (a.shape[1] / 16 + 20) * STEP * (a.abs() @ b.abs().t())


ACT_ERR = 2e-5  # relative: __expf of arguments in the tens


DENSE = [  # M, K, N, dtype, act, bias, residual, save, pad
    (1, 1, 1, BF, "identity", True, False, "full", 0),
    (1, 4096, 4096, BF, "silu", True, True, "none", 0),
    (1, 64, 40, HF, "relu", False, True, "q8", 0),
    (2, 1001, 77, BF, "gelu", True, True, "q8", 0),
    (17, 333, 129, HF, "tanh", True, False, "full", 5),
    (33, 4096, 256, BF, "sigmoid", True, True, "full", 8),
    (64, 8192, 1024, BF, "identity", False, False, "none", 0),
    (100, 72, 1000, BF, "gelu", True, True, "q8", 8),
    (129, 128, 257, HF, "silu", True, True, "q8", 0),
    (300, 520, 2048, BF, "relu", True, False, "full", 0),
    (777, 1000, 1333, HF, "tanh", True, True, "none", 0),
    (2048, 256, 4096, BF, "gelu", True, False, "q8", 0),
    (4100, 136, 5000, BF, "silu", True, True, "full", 0),
    (5000, 1024, 3000, HF, "gelu", True, True, "q8", 0),
    (70001, 32, 64, BF, "relu", True, True, "q8", 0),
]


@pytest.mark.parametrize("M,K,N,dtype,act,has_bias,has_res,save,pad", DENSE)
@pytest.mark.parametrize("bits8", [False, True])
def test_dense_fwd(M, K, N, dtype, act, has_bias, has_res, save, pad, bits8):
    x, w = normal(1, M, K), normal(2, N, K, std=K ** -0.5)
    if bits8:
        x, w = ops.q8_encode(x, 0), ops.q8_encode(w, 0)
        x64, w64 = q8_values(x), q8_values(w)
        if pad:
            x = ops.Q8(strided(x.q.view(torch.uint8).float(), pad).to(torch.uint8).view(torch.float8_e4m3fn), x.scale, 0)
    else:
        x, w = x.to(dtype), w.to(dtype)
        x64, w64 = x.double(), w.double()
        x, w = strided(x, pad), strided(w, pad)
    bias = normal(3, N) if has_bias else None
    res = normal(4, M, N, dtype=dtype) if has_res else None
    y, z = ops.dense_fwd(x, w, bias, act, residual=None if res is None else strided(res, pad), save=save, dtype=dtype)
    z64 = x64 @ w64.t()
    err = mm_bound(x64, w64) + (2 * U[FP] * z64.abs() if bits8 else 0)
    if has_bias:
        z64 = z64 + bias.double()
        err = err + U[FP] * z64.abs()
    if save == "full":
        close(z, z64, rounded(z64, dtype, err), "z")
    elif save == "q8":
        s = torch.exp2(z.scale.double() - 127).repeat_interleave(32, 1)[:, :N]
        close(q8_values(z), z64, torch.maximum(2.0 ** -4 * z64.abs(), 2.0 ** -10 * s) + 2 * err, "z in 8 bits")
    else:
        assert z is None
    a = act_ref(act, z64)
    y64 = a + res.double() if has_res else a
    extra = 1.2 * err + ACT_ERR * a.abs() * (act not in ("identity", "relu")) + U[FP] * y64.abs()
    close(y, y64, rounded(y64, dtype, extra), "y")
    # into strided outputs, over the residual itself, bit for bit
    if has_res:
        buf = strided(res, pad or 3)
        got, _ = ops.dense_fwd(x, w, bias, act, residual=buf, y=buf, dtype=dtype)
        assert got is buf and torch.equal(buf, y)
        assert bool(torch.as_strided(buf, (M, 3), (buf.stride(0), 1), buf.storage_offset() + N).isnan()[:M - 1].all())


@pytest.mark.parametrize("M,K,N,dtype,act,has_res,save,bits8", [
    (2600, 4096, 2048, BF, "gelu", True, "q8", False), (2601, 4100, 2050, HF, "silu", True, "full", False),
    (2600, 8192, 2048, BF, "identity", False, "none", True), (8192, 2304, 2304, BF, "relu", False, "none", False)])
def test_dense_fwd_cut_units(M, K, N, dtype, act, has_res, save, bits8):
    """Outputs whose last wave of units leaves most of the SMs idle: its units are cut along k and joined."""
    test_dense_fwd(M, K, N, dtype, act, True, has_res, save, 0, bits8)


def test_dense_weights_in_8_bits_only():
    x, w = normal(1, 70, 200, dtype=BF), ops.q8_encode(normal(2, 96, 200, std=0.1), 32)
    y, _ = ops.dense_fwd(x, w)
    same, _ = ops.dense_fwd(x, ops.q8_decode(w, BF))
    assert torch.equal(y, same)
    both, _ = ops.dense_fwd(ops.q8_encode(x, 32), w, dtype=BF)
    close(both, q8_values(ops.q8_encode(x, 32)) @ q8_values(w).t(),
          rounded(both.double(), BF, mm_bound(q8_values(ops.q8_encode(x, 32)), q8_values(w))) * 2, "groups of 32")


def test_dense_special_values():
    """Infinities and NaN stay in their rows and columns; activations at the ends of their range."""
    x, w = torch.zeros(200, 100, device="cuda", dtype=BF), torch.zeros(150, 100, device="cuda", dtype=BF)
    x[:, 0], w[:, 0] = 1, 1
    x[7, 99] = float("nan")
    w[149, 0] = float("inf")
    y, _ = ops.dense_fwd(x, w)
    bad = torch.zeros(200, 150, dtype=torch.bool, device="cuda")
    bad[7], bad[:, 149] = True, True
    assert torch.equal(~y.isfinite(), bad)
    z = torch.tensor([[-3e38, -1e30, -200., -100., -20., -5., -1e-3, -1e-20, 0., 1e-20, 1e-3, 5., 20., 100., 200., 1e30, 3e38]],
                     device="cuda", dtype=BF)
    eye = torch.eye(17, device="cuda", dtype=BF)
    for act in ops.ACTS:
        got, _ = ops.dense_fwd(z, eye, None, act)
        ref = act_ref(act, z.double())
        close(got, ref, rounded(ref, BF, ACT_ERR * ref.abs() + 1e-37), act)
        one = torch.ones_like(z)
        dx, _, db = ops.dense_bwd(z, eye, one, z, act, need_dw=False)
        ref = dact_ref(act, z.double())
        close(db, ref[0], 1e-4 * ref[0].abs() + 1e-7, act + " derivative")  # 1e-7: cancellation about gelu's and silu's zero
        close(dx, ref, rounded(ref, BF, 1e-4 * ref.abs() + 1e-7), act + " gradient")


BWD = [  # M, K, N, dtype, act, q8, grad, pad
    (1, 1, 1, BF, "identity", False, FP, 0),
    (1, 300, 4096, BF, "silu", False, FP, 0),
    (3, 1001, 77, HF, "gelu", True, HF, 0),
    (65, 64, 200, BF, "tanh", True, FP, 0),
    (130, 333, 129, BF, "identity", False, FP, 5),
    (500, 264, 136, HF, "sigmoid", False, HF, 8),
    (1777, 520, 333, BF, "identity", False, FP, 0),
    (1000, 1000, 1000, BF, "relu", True, BF, 0),
    (4097, 256, 512, BF, "gelu", True, FP, 0),
    (3000, 2048, 1536, HF, "silu", False, HF, 0),
    (9000, 40, 72, BF, "identity", True, FP, 0),
    (30000, 256, 300, BF, "gelu", False, FP, 0),
]


@pytest.mark.parametrize("M,K,N,dtype,act,q8,grad,pad", BWD)
def test_dense_bwd(M, K, N, dtype, act, q8, grad, pad):
    x, w, dy = normal(1, M, K, dtype=dtype), normal(2, N, K, std=N ** -0.5, dtype=dtype), normal(3, M, N, dtype=dtype)
    z = normal(4, M, N, std=1.5, dtype=dtype) if act != "identity" else None
    if q8:
        x = ops.q8_encode(x, 32)
        z = ops.q8_encode(z, 32) if z is not None else None
    x64 = q8_values(x) if q8 else x.double()
    if q8 and dtype == HF:
        x64 = x64.to(HF).double()  # decoded to fp16 (values below its normal range are rounded)
    if pad:
        x, w, dy = strided(x, pad), strided(w, pad), strided(dy, pad)
        z = strided(z, pad) if z is not None else None
    dx, dw, db = ops.dense_bwd(x, w, dy, z, act, grad_dtype=grad)
    dz = dy.double()
    if z is not None:
        z64 = q8_values(z) if q8 else z.double()
        dz = dz * dact_ref(act, z64)
    w64 = w.double()
    # dz is stored in dtype: half a step of every term, and what its derivative is off before
    off = rounded(dz, dtype, 2e-5 * dz.abs() + 2e-7 * dy.double().abs()) if act != "identity" else 0 * dz
    near = dz.abs() + off
    ref = dz @ w64
    close(dx, ref, rounded(ref, dtype, off @ w64.abs() + mm_bound(near, w64.t())), "dx")
    ref = dz.t() @ x64
    steps = (M / 16 + 600) * STEP * (near.t() @ x64.abs())  # the splits' joins among them
    extra = off.t() @ x64.abs() + steps
    close(dw, ref, rounded(ref, grad, extra), "dw")
    # strips of 64 rows or more: rows / 8 additions in a thread of a strip, 8 row lanes, strips / 8 + 8
    pre = 2e-5 * dz.abs() + 2e-7 * dy.double().abs()
    close(db, dz.sum(0), pre.sum(0) + (M / 64 + 160 + 8 + 8) * STEP * dz.abs().sum(0) + 1e-300, "db")
    # accumulating
    dw2, db2 = dw.clone(), db.clone()
    ops.dense_bwd(x, w, dy, z, act, need_dx=False, dw=dw2, dbias=db2)
    close(dw2, 2 * dw.double(), 2 * U[grad] * 2 * dw.double().abs() + 2 * steps * 2.0 ** -4 + TINY_OF[grad], "dw twice")
    close(db2, 2 * db.double(), 2 * U[FP] * 2 * db.double().abs(), "db twice")
    # each alone
    assert torch.equal(ops.dense_bwd(None, w, dy, z, act, need_dw=False, need_dbias=False)[0], dx)
    assert torch.equal(ops.dense_bwd(x, None, dy, z, act, need_dx=False, need_dbias=False, grad_dtype=grad)[1], dw)
    assert torch.equal(ops.dense_bwd(None, None, dy, z, act, need_dx=False, need_dw=False)[2], db)


@pytest.mark.parametrize("M,K,N,dtype,act,q8,grad,pad", [
    (2600, 2048, 4096, BF, "gelu", True, BF, 0),    # dx
    (4096, 2601, 2050, HF, "identity", False, HF, 0),  # dw
])
def test_dense_bwd_cut_units(M, K, N, dtype, act, q8, grad, pad):
    test_dense_bwd(M, K, N, dtype, act, q8, grad, pad)


@pytest.mark.parametrize("M,K,N", [(9000, 2560, 3840), (4160, 2048, 8192)])
def test_dense_bwd_fp32_passes(M, K, N):
    """An fp32 dW that fills the GPU by itself is summed in passes of 4,096 rows; the workspace holds no partials."""
    x, dy = normal(1, M, K, dtype=BF), normal(2, M, N, dtype=BF)
    _, dw, _ = ops.dense_bwd(x, None, dy, need_dx=False, need_dbias=False)
    ref = dy.double().t() @ x.double()
    # at most 256 truncated additions (16 products each) in a pass, and three passes
    steps = (256 + 20 + 3) * STEP * (dy.double().abs().t() @ x.double().abs())
    close(dw, ref, rounded(ref, FP, steps), "dw")
    d = abi.DenseDesc(M, K, N, 0, abi.BF16, 0)
    m = abi.Mat(1 << 20, 0, abi.BF16, 0, None)
    f = abi.Mat(1 << 20, 0, abi.FP32, 0, None)
    assert abi.conv2d_dense_bwd_workspace_size(d, m, m, None, m, None, f, None) < 2 * N * K * 4
    again, db = dw.clone(), torch.zeros(N, device="cuda")
    ops.dense_bwd(x, None, dy, need_dx=False, dw=again, dbias=db)
    close(again, 2 * dw.double(), 8 * U[FP] * ref.abs() + steps * 2.0 ** -3, "dw twice")


@pytest.mark.parametrize("M,K,N", [(50, 136, 72), (600, 520, 1000)])
def test_dense_strided_outputs(M, K, N):
    """Every output into rows of a longer matrix: the same bits, nothing beside them."""
    x, w, dy = normal(1, M, K, dtype=BF), normal(2, N, K, std=K ** -0.5, dtype=BF), normal(3, M, N, dtype=BF)

    def wide(rows, cols, dtype, pad):
        t = torch.full((rows, cols + pad), 7.0, device="cuda").to(dtype)
        return t, t[:, :cols]

    for pad in (8, 16, 3):
        y0, z0 = ops.dense_fwd(x, w, None, "gelu", save="q8")
        g0 = ops.dense_bwd(x, w, dy, z0, "gelu", grad_dtype=BF)
        Y, y = wide(M, N, BF, pad)
        Q = torch.full((M, N + pad), 1, device="cuda", dtype=torch.uint8)
        z = ops.Q8(Q.view(torch.float8_e4m3fn)[:, :N], torch.empty_like(z0.scale), 32)
        ops.dense_fwd(x, w, None, "gelu", save="q8", y=y, pre_act=z)
        assert torch.equal(y, y0) and torch.equal(z.scale, z0.scale)
        assert torch.equal(Q[:, :N], z0.q.view(torch.uint8)) and bool((Q[:, N:] == 1).all())
        X, dx = wide(M, K, BF, pad)
        W, dw = wide(N, K, BF, pad)
        dw.zero_()
        db = torch.zeros(N, device="cuda")
        ops.dense_bwd(x, w, dy, z, "gelu", dx=dx, dw=dw, dbias=db)
        assert torch.equal(dx, g0[0]) and torch.equal(dw, g0[1]) and torch.equal(db, g0[2])
        for t, cols in ((Y, N), (X, K), (W, K)):
            assert bool((t[:, cols:] == 7).all())


TINY_OF = {BF: 2.0 ** -133, HF: 2.0 ** -24, FP: 2.0 ** -149}


def test_dense_gradient_matches_differences():
    M, K, N = 5, 24, 18
    x, w, b, t = normal(1, M, K, dtype=BF), normal(2, N, K, std=0.2, dtype=BF), normal(3, N), normal(4, M, N, dtype=BF)
    for act in ops.ACTS:
        z64 = x.double() @ w.double().t() + b.double()
        z = z64.to(BF)
        dx, dw, db = ops.dense_bwd(x, w, t, z, act)

        def loss(x, w, b):
            return float((act_ref(act, x @ w.t() + b) * t.double()).sum())

        args = [x.double(), w.double(), b.double()]
        for k, (grad, at) in enumerate(((dx, 31), (dw, 77), (db, 7))):
            d = torch.zeros_like(args[k]).flatten()
            d[at] = 1e-6
            d = d.view_as(args[k])
            num = (loss(*[a + d if i == k else a for i, a in enumerate(args)])
                   - loss(*[a - d if i == k else a for i, a in enumerate(args)])) / 2e-6
            # z and dz are held in bf16: their half steps through at most 24 terms of order one
            assert abs(num - float(grad.flatten()[at])) < 24 * 3 * U[BF], (act, k)


def test_zero_rows():
    e = lambda *s, dtype=BF: torch.empty(*s, device="cuda", dtype=dtype)  # noqa: E731
    y, z = ops.dense_fwd(e(0, 64), normal(1, 32, 64, dtype=BF), normal(2, 32), "gelu", save="q8")
    assert y.shape == (0, 32) and z.q.shape == (0, 32)
    dx, dw, db = ops.dense_bwd(e(0, 64), normal(1, 32, 64, dtype=BF), e(0, 32), z, "gelu")
    assert dx.shape == (0, 64) and bool((dw == 0).all()) and bool((db == 0).all())
    acc, acb = normal(1, 32, 64), normal(2, 32)
    keep, keeb = acc.clone(), acb.clone()
    ops.dense_bwd(e(0, 64), normal(1, 32, 64, dtype=BF), e(0, 32), z, "gelu", dw=acc, dbias=acb)
    assert torch.equal(acc, keep) and torch.equal(acb, keeb)
    assert ops.rms_norm_fwd(e(0, 64), normal(1, 64)).y.shape == (0, 64)
    _, dg = ops.rms_norm_bwd(e(0, 64), normal(1, 64), e(0, dtype=FP), e(0, 64))
    assert bool((dg == 0).all())
    assert ops.q8_decode(ops.q8_encode(e(0, 40))).shape == (0, 40)


def test_repeatable_on_side_streams_and_in_graphs():
    """The same bits on a side stream and from a captured graph; no call synchronises or allocates outside torch."""
    x, w, b, r = normal(1, 500, 1000, dtype=BF), normal(2, 333, 1000, dtype=BF), normal(3, 333), normal(4, 500, 333, dtype=BF)
    gamma, dy = normal(5, 333), normal(6, 500, 333, dtype=BF)

    def step():
        y, z = ops.dense_fwd(x, w, b, "gelu", residual=r, save="q8")
        n = ops.rms_norm_fwd(y, gamma, residual=r, group=32)
        dh, dg = ops.rms_norm_bwd(n.h, gamma, n.inv_rms, dy, dh=dy)
        dx, dw, db = ops.dense_bwd(ops.q8_encode(x), w, dh, z, "gelu")
        return [y, z.q.view(torch.uint8), z.scale, n.y, n.q8.q.view(torch.uint8), dh, dg, dx, dw, db]

    want = step()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y, _ = ops.dense_fwd(x, w, b, "gelu", residual=r, stream=side)
    side.synchronize()
    assert torch.equal(y, want[0])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step()
    for _ in range(2):
        for t in got:
            t.fill_(1)
        g.replay()
        torch.cuda.synchronize()
        for a, t in zip(want, got):
            assert torch.equal(a, t)


def test_offsets_past_32_bits():
    """Rows that start more than 2^32 bytes into a tensor: 8-bit values past 2^32 elements' worth of bf16 rows."""
    rows, cols, ld = 70000, 64, 1 << 16  # 70000 rows of 128 KB: 9 GB between first and last
    x = torch.empty(rows, ld, device="cuda", dtype=BF)[:, :cols]
    x.copy_(normal(1, rows, cols, dtype=BF))
    q = ops.q8_encode(x)
    assert torch.equal(q8_values(q)[-64:], q8_ref(x[-64:].double(), 32)[0])
    gamma = normal(2, cols)
    n = ops.rms_norm_fwd(x, gamma)
    y, _ = rms_ref(x[-64:].double(), gamma.double(), 1e-6)
    close(n.y[-64:], y, rounded(y, BF, 1e-6 * y.abs()), "last rows")
    w = normal(3, 96, cols, dtype=BF)
    out = torch.empty(rows, ld, device="cuda", dtype=BF)[:, :96]
    ops.dense_fwd(x, w, y=out)
    ref = x[-64:].double() @ w.double().t()
    close(out[-64:], ref, rounded(ref, BF, mm_bound(x[-64:].double(), w.double())), "dense, last rows")
