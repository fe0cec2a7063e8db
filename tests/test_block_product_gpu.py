"""The dense layer on 8-bit operands with a scale for each block of 128, against 64-bit sums of the values they stand
for."""
import pytest
import torch

from block_ref import STEP, U, act_ref, close, dact_ref, q8_values, rounded
from conv2d_layer_gb300 import abi, ops
from more_ref import q8_wide_ref, q8_wide_values
from test_block_gpu import ACT_ERR, mm_bound, normal, strided

pytestmark = pytest.mark.gpu
BF, HF, FP = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(autouse=True)
def device_clean():
    yield
    assert abi.conv2d_device_status() == (abi.OK, 0)


def padded(q, pad):
    """The same 8-bit matrix with rows `pad` bytes further apart; the bytes between them are NaN."""
    if not pad:
        return q
    rows, cols = q.shape
    wide = torch.full((rows, cols + pad), 0x7f, dtype=torch.uint8, device="cuda")
    wide[:, :cols] = q.q.view(torch.uint8)
    return q._replace(q=wide.view(torch.float8_e4m3fn)[:, :cols])


def operands(M, K, N, wgroup, seed=0, spread=8):
    """Operands whose blocks have scales of their own, far apart."""
    g = torch.Generator(device="cuda").manual_seed(seed)

    def blocks(rows, cols, tall):
        e = torch.randint(-spread, spread + 1, (-(-rows // tall), -(-cols // 128)), generator=g, device="cuda").float()
        return torch.exp2(e).repeat_interleave(tall, 0).repeat_interleave(128, 1)[:rows, :cols]

    x = torch.randn(M, K, generator=g, device="cuda") * blocks(M, K, 1)
    w = torch.randn(N, K, generator=g, device="cuda") * K ** -0.5 * blocks(N, K, 128)
    return ops.q8_encode(x, 128), ops.q8_encode(w, wgroup)


# M, K, N, dtype, act, bias, residual, save, pad
FWD = [
    (1, 16, 8, BF, "identity", False, False, "none", 0),
    (1, 128, 128, BF, "identity", False, False, "none", 0),
    (3, 129, 1, HF, "relu", True, True, "full", 0),
    (16, 512, 128, BF, "identity", True, False, "none", 0),
    (17, 640, 130, BF, "gelu", True, True, "q8", 0),
    (1, 4096, 4096, BF, "silu", True, True, "none", 0),
    (24, 16384, 512, BF, "identity", True, True, "none", 0),
    (64, 1001, 333, HF, "tanh", True, True, "full", 0),
    (130, 777, 257, BF, "sigmoid", False, True, "q8", 7),
    (100, 2048, 1024, HF, "identity", True, False, "none", 16),
    (300, 520, 700, BF, "gelu", True, True, "q8", 0),
    (1000, 1000, 1000, BF, "relu", True, False, "full", 0),
    (2100, 1536, 2300, HF, "silu", True, True, "q8", 0),
    (4096, 896, 4096, BF, "gelu", True, False, "full", 0),
    (5000, 128, 1024, BF, "identity", False, True, "none", 0),
    (20000, 256, 256, BF, "identity", True, True, "full", 0),
]


@pytest.mark.parametrize("wgroup", [128, ops.TILE])
@pytest.mark.parametrize("M,K,N,dtype,act,has_bias,has_res,save,pad", FWD)
def test_block_product(M, K, N, dtype, act, has_bias, has_res, save, pad, wgroup):
    x, w = operands(M, K, N, wgroup, seed=M + K)
    x64, w64 = q8_wide_values(x), q8_wide_values(w)
    bias = normal(3, N) if has_bias else None
    res = normal(4, M, N, dtype=dtype) if has_res else None
    if dtype == HF:  # within fp16's range
        w = w._replace(scale=w.scale - 6)
        w64 = w64 / 64
    y, z = ops.dense_fwd(padded(x, pad), padded(w, pad), bias, act, residual=res, save=save, dtype=dtype)
    z64 = x64 @ w64.t()
    err = mm_bound(x64, w64)
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


@pytest.mark.parametrize("M,K,N,act,has_res", [(2600, 8192, 2048, "identity", True), (2601, 4100, 2050, "gelu", False)])
def test_block_product_cut_units(M, K, N, act, has_res):
    """Outputs whose last wave of units leaves most of the SMs idle: its units are cut along k and joined."""
    test_block_product(M, K, N, BF, act, True, has_res, "none", 0, ops.TILE)


def test_scales_far_from_one():
    """Scales of 2^-120 and 2^120 that cancel, and blocks of zeros between them."""
    M, K, N = 150, 700, 260
    x, w = operands(M, K, N, ops.TILE, seed=1, spread=0)
    want, _ = ops.dense_fwd(x, w, dtype=BF)
    for e in (-112, 112):
        got, _ = ops.dense_fwd(x._replace(scale=x.scale + e), w._replace(scale=w.scale - e), dtype=BF)
        assert torch.equal(got, want)
    x.q.view(torch.uint8)[:, 128:256] = 0
    x.scale[:, 1] = 254
    got, _ = ops.dense_fwd(x, w, dtype=BF)
    x64, w64 = q8_wide_values(x), q8_wide_values(w)
    ref = x64 @ w64.t()
    close(got, ref, rounded(ref, BF, mm_bound(x64, w64)), "zeros of a large scale")


def test_nan_and_strided_outputs():
    M, K, N = 200, 384, 150
    x, w = operands(M, K, N, ops.TILE, seed=2, spread=2)
    x.q.view(torch.uint8)[7, 383] = 0x7f
    w.q.view(torch.uint8)[149, 0] = 0x7f
    y, _ = ops.dense_fwd(x, w, dtype=BF)
    bad = torch.zeros(M, N, dtype=torch.bool, device="cuda")
    bad[7], bad[:, 149] = True, True
    assert torch.equal(~y.isfinite(), bad)
    out = strided(torch.zeros(M, N, device="cuda", dtype=BF), 5)
    got, _ = ops.dense_fwd(x, w, dtype=BF, y=out)
    assert torch.equal(got.nan_to_num(0.0), y.nan_to_num(0.0))
    assert bool(torch.as_strided(out, (M, 5), (out.stride(0), 1), N).isnan()[:M - 1].all())


def test_scales_off_word_boundaries():
    """Scale arrays need no alignment; rows of any number of blocks."""
    for K in (512, 600, 1024):
        x, w = operands(70, K, 300, 128, seed=K)
        want, _ = ops.dense_fwd(x, w, dtype=BF)
        n = x.scale.numel()
        buf = torch.empty(n + 1, dtype=torch.uint8, device="cuda")
        buf[1:] = x.scale.flatten()
        got, _ = ops.dense_fwd(x._replace(scale=buf[1:].view(x.scale.shape)), w, dtype=BF)
        assert torch.equal(got, want)


def test_other_pairs_are_decoded():
    x, w = operands(70, 300, 96, ops.TILE, seed=3, spread=1)
    same, _ = ops.dense_fwd(ops.q8_decode(x, BF), ops.q8_decode(w, BF))
    for a, b in ((ops.q8_decode(x, BF), w), (x, ops.q8_decode(w, BF))):
        assert torch.equal(ops.dense_fwd(a, b)[0], same)
    t = ops.q8_encode(ops.q8_decode(x, FP), ops.TILE)
    want, _ = ops.dense_fwd(ops.q8_decode(t, BF), ops.q8_decode(w, BF))
    assert torch.equal(ops.dense_fwd(t, w, dtype=BF)[0], want)


# M, K, N, dtype, act, pad
BWD = [
    (1, 16, 8, BF, "identity", 0), (1, 300, 4096, BF, "silu", 0), (3, 1001, 77, HF, "gelu", 0), (65, 64, 200, BF, "tanh", 0),
    (130, 333, 129, BF, "identity", 5), (500, 264, 136, HF, "sigmoid", 8), (1000, 1000, 1000, BF, "relu", 0),
    (4097, 256, 512, BF, "gelu", 0), (3000, 2048, 1536, HF, "silu", 0), (2600, 2048, 4096, BF, "identity", 0),
    (700, 640, 384, BF, "identity", 0),
]


@pytest.mark.parametrize("M,K,N,dtype,act,pad", BWD)
def test_block_product_bwd(M, K, N, dtype, act, pad):
    x, w = operands(M, K, N, ops.TILE, seed=M + K, spread=3)
    dy = normal(3, M, N, dtype=dtype)
    z = normal(4, M, N, std=1.5, dtype=dtype) if act != "identity" else None
    dx, dw, db = ops.dense_bwd(padded(x, pad), padded(w, pad), strided(dy, pad), z, act, grad_dtype=dtype)
    dz = dy.double()
    if z is not None:
        dz = dz * dact_ref(act, z.double())
    off = rounded(dz, dtype, 2e-5 * dz.abs() + 2e-7 * dy.double().abs()) if act != "identity" else 0 * dz
    w64, x64 = q8_wide_values(w), q8_wide_values(x)
    if dtype == HF:
        x64 = x64.to(HF).double()  # decoded to fp16
    # dz in 8 bits: exactly these values where dz is dy; else a value may lie a step of 8 bits off
    held, scale = q8_wide_ref(dz if act == "identity" else dz.to(dtype).double(), 128)
    eight = 0 * dz
    if act != "identity":
        s = torch.exp2(scale.double() - 127).repeat_interleave(128, 1)[:, :N]
        eight = off + 2 * torch.maximum(2.0 ** -4 * (dz.abs() + off), 2.0 ** -10 * s)
    ref = held @ w64
    close(dx, ref, rounded(ref, dtype, eight @ w64.abs() + mm_bound(held.abs() + eight, w64.t())), "dx")
    if act == "identity":  # the same bits from operands encoded beforehand
        alone = ops.dense_bwd(None, w, dy, z, act, need_dw=False, need_dbias=False)[0]
        assert torch.equal(alone, dx)
    ref = dz.t() @ x64
    steps = (M / 16 + 600) * STEP * ((dz.abs() + off).t() @ x64.abs())
    close(dw, ref, rounded(ref, dtype, off.t() @ x64.abs() + steps), "dw")
    pre = 2e-5 * dz.abs() + 2e-7 * dy.double().abs()
    close(db, dz.sum(0), pre.sum(0) + (M / 64 + 160 + 16) * STEP * dz.abs().sum(0) + 1e-300, "db")
    # 16-bit weights, or those with a scale for each row: a 16-bit product
    plain = ops.dense_bwd(None, ops.q8_decode(w, dtype), dy, z, act, need_dw=False, need_dbias=False)[0]
    rows = ops.dense_bwd(None, ops.q8_encode(ops.q8_decode(w, FP), 128), dy, z, act, need_dw=False, need_dbias=False)[0]
    w16 = ops.q8_decode(w, dtype).double()
    ref = dz @ w16
    for got in (plain, rows):
        close(got, ref, rounded(ref, dtype, off @ w16.abs() + mm_bound(dz.abs() + off, w16.t())), "dx in 16 bits")


def test_gradient_by_differences():
    """dx against differences of the forward product: linear, so only the rounding of dy to 8 bits and of sums is between."""
    M, K, N = 40, 256, 200
    _, w = operands(M, K, N, ops.TILE, seed=5, spread=2)
    dy = normal(6, M, N, dtype=BF)
    held = q8_wide_values(ops.q8_encode(dy, 128))
    dx = ops.dense_bwd(None, w, dy, need_dw=False, need_dbias=False)[0]
    w64 = q8_wide_values(w)
    for c in (0, 100, 255):
        e = torch.zeros(M, K, device="cuda")
        e[:, c] = 1.0
        y, _ = ops.dense_fwd(ops.q8_encode(e, 128), w, dtype=BF)  # column c of w
        assert torch.equal(y, w64[:, c].to(BF).expand(M, N))
        num = (held * y.double()).sum(1)
        tol = rounded(num, BF, 2 * U[BF] * (held.abs() @ w64[:, c].abs()))
        close(dx[:, c], num, tol, "dx")


def test_captured_and_on_another_stream():
    x, w = operands(300, 640, 500, ops.TILE, seed=7, spread=2)
    dy = normal(8, 300, 500, dtype=BF)

    def step(stream=None):
        y, z = ops.dense_fwd(x, w, None, "gelu", save="full", dtype=BF, stream=stream)
        return (y, *ops.dense_bwd(x, w, dy, z, "gelu", grad_dtype=BF, stream=stream))

    want = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = step(side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    x.scale.add_(1)
    for _ in range(2):
        graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(step(), held))
