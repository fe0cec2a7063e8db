"""Products whose left operand the library itself takes to 8 bits on the way: h of the experts, dz of the block-scaled
gradient. A value's 8-bit form is known but where its own error reaches over the middle between two of them, so the bounds
stay a few percent of the results; and whole numbers, whose 8-bit forms are exact, have to come out bit by bit."""
import pytest
import torch

from block_ref import STEP, U, act_ref, close, dact_ref, rounded
from conv2d_layer_gb300 import abi, ops
from held_ref import held_between
from more_ref import q8_wide_ref, q8_wide_values

pytestmark = pytest.mark.gpu
BF, HF, FP = torch.bfloat16, torch.float16, torch.float32
ACT_ERR = 2e-5  # relative: __expf of arguments in the tens


@pytest.fixture(autouse=True)
def device_clean():
    yield
    assert abi.conv2d_device_status() == (abi.OK, 0)


def normal(seed, *shape, std=1.0, dtype=FP):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)


def up_bound(w1, x, b1, act, gated, F):
    """(h, its error) of one token and expert: sums of 16 terms truncated at a time and joined, the activation, the factor."""
    z = w1 @ x + (0 if b1 is None else b1)
    ze = (x.shape[0] / 16 + 20) * STEP * (w1.abs() @ x.abs()) + U[FP] * z.abs()
    h = act_ref(act, z[:F])
    he = 1.2 * ze[:F] + ACT_ERR * h.abs()
    if gated:
        he = he * z[F:].abs() + h.abs() * ze[F:] + he * ze[F:]
        h = h * z[F:]
        he = he + U[FP] * h.abs()
    return h, he


def down_bound(w2, low, high, b2):
    """(the second product of an h between low and high, its error)"""
    h, r = (low + high) / 2, (high - low) / 2
    o = w2 @ h + (0 if b2 is None else b2)
    F = h.shape[0]
    return o, w2.abs() @ r + (F / 16 + 20) * STEP * (w2.abs() @ (h.abs() + r)) + U[FP] * o.abs()


# T, D, F, E, k, dtype, gated, act, bias, residual
@pytest.mark.parametrize("T,D,F,E,k,dtype,gated,act,bias,has_res", [
    (1, 128, 128, 1, 1, BF, False, "identity", False, False),
    (1, 2048, 1024, 16, 4, BF, True, "silu", False, True),
    (7, 384, 256, 6, 2, HF, True, "silu", True, True),
    (16, 2304, 128, 8, 2, BF, False, "gelu", True, False),
    (37, 1152, 640, 23, 3, BF, False, "gelu", True, False),
    (40, 512, 896, 5, 2, HF, True, "silu", False, False),
    (64, 640, 4352, 4, 2, BF, True, "silu", False, True),
])
def test_experts_in_8_bits(T, D, F, E, k, dtype, gated, act, bias, has_res):
    up = F * (1 + gated)
    x, router = normal(1, T, D, dtype=dtype), normal(2, E, D, std=D ** -0.5, dtype=dtype)
    q1 = ops.moe_encode(normal(3, E, up, D, std=D ** -0.5, dtype=dtype))
    q2 = ops.moe_encode(normal(4, E, D, F, std=F ** -0.5, dtype=dtype))
    b1, b2 = (normal(5, E, up, std=0.2), normal(6, E, D, std=0.2)) if bias else (None, None)
    res = normal(7, T, D, dtype=dtype) if has_res else None
    got = ops.moe_fwd(x, router, q1, q2, k, b1=b1, b2=b2, act=act, gated=gated, residual=res)
    w1, w2 = q8_wide_values(q1), q8_wide_values(q2)
    xs, _ = q8_wide_ref(x.double(), 128)
    y = torch.zeros(T, D, dtype=torch.float64, device="cuda")
    tol = torch.zeros_like(y)
    for t in range(T):
        for j in range(k):
            e, w = int(got.experts[t, j]), float(got.weights[t, j])
            h, he = up_bound(w1[e], xs[t], None if b1 is None else b1[e].double(), act, gated, F)
            low, high = held_between(h[None], he[None])
            o, oe = down_bound(w2[e], low[0], high[0], None if b2 is None else b2[e].double())
            y[t] += w * o
            tol[t] += w * oe + 2 * U[FP] * (w * o).abs()
    assert float(tol.norm()) < 0.08 * float(y.norm())
    if has_res:
        y += res.double()
    tol += 2 * U[FP] * y.abs()
    close(got.y, y, rounded(y, dtype, tol), "y")


# T, D, F, pairs of experts, k, gated, residual
@pytest.mark.parametrize("T,D,F,pairs,k,gated,has_res", [
    (1, 128, 128, 1, 1, False, False), (1, 2048, 1024, 8, 2, True, True), (16, 2304, 128, 4, 1, False, True),
    (33, 2048, 1024, 4, 2, True, False), (37, 1152, 640, 11, 2, False, True), (64, 1152, 640, 3, 2, True, True),
    (64, 640, 4352, 2, 2, True, True), (20, 256, 2176, 2, 1, True, False), (64, 4096, 384, 2, 2, True, False),
])
def test_experts_of_whole_numbers(T, D, F, pairs, k, gated, has_res):
    """h is a power of two or zero, so its 8-bit form is exact; a token's two experts weigh 1/2 each."""
    g = torch.Generator(device="cuda").manual_seed(T + D + F)

    def ints(low, high, *shape):
        return torch.randint(low, high, shape, generator=g, device="cuda")

    def tiles(rows, cols):  # scales that differ from tile to tile
        e = (ints(0, 3, 2 * pairs, rows // 128, 1) + torch.arange(cols // 128, device="cuda")) % 3
        return (e + 127).to(torch.uint8), torch.exp2(e.double()).repeat_interleave(128, 1).repeat_interleave(128, 2)

    E, up = 2 * pairs, F * (1 + gated)
    x = ints(-1, 2, T, D) * torch.exp2((torch.arange(D, device="cuda") // 128 % 2).float())
    pair = torch.arange(T, device="cuda") % pairs  # a token's experts, told by its first columns
    x[:, :pairs] = 4.0 * torch.nn.functional.one_hot(pair, pairs)
    router = torch.zeros(E, D, device="cuda", dtype=BF)
    router[torch.arange(E), torch.arange(E) // 2] = 8.0
    one = torch.zeros(E, up, D, device="cuda")  # one element of x for each feature, with a sign
    one.scatter_(2, ints(0, D, E, up, 1), (2.0 * ints(0, 2, E, up, 1) - 1))
    s1, f1 = tiles(up, D)
    v2 = ints(-1, 2, E, D, F)
    s2, f2 = tiles(D, F)
    q1, q2 = ops.Q8(one.to(torch.float8_e4m3fn), s1, ops.TILE), ops.Q8(v2.to(torch.float8_e4m3fn), s2, ops.TILE)
    w1, w2 = one.double() * f1, v2.double() * f2
    res = ints(-64, 65, T, D).to(BF) if has_res else None
    b2 = ints(-9, 10, E, D).float()
    got = ops.moe_fwd(x.to(BF), router, q1, q2, k, b2=b2, act="identity", gated=gated, residual=res)
    want = torch.zeros(T, D, dtype=torch.float64, device="cuda") if res is None else res.double()
    for t in range(T):
        mine = [2 * int(pair[t]) + j for j in range(k)]
        assert got.experts[t].tolist() == mine and got.weights[t].tolist() == [1.0 / k] * k
        for e in mine:
            z = w1[e] @ x[t].double()
            h = z[:F] * z[F:] if gated else z
            assert torch.equal(h, q8_wide_ref(h[None], 128)[0][0])
            want[t] += (w2[e] @ h + b2[e].double()) / k
    assert float(want.abs().max()) < 2 ** 20
    assert torch.equal(got.y, want.float().to(BF))


@pytest.mark.parametrize("M,K,N,dtype,act", [(65, 64, 200, BF, "tanh"), (500, 264, 136, HF, "sigmoid"), (4097, 256, 512, BF, "gelu"),
                                             (3, 1001, 77, HF, "gelu"), (1, 300, 4096, BF, "silu"), (1000, 1000, 1000, BF, "silu")])
def test_gradient_from_dz_in_8_bits(M, K, N, dtype, act):
    w = ops.q8_encode(normal(1, N, K, std=K ** -0.5), ops.TILE)
    dy, z = normal(2, M, N, dtype=dtype), normal(3, M, N, std=1.5, dtype=dtype)
    dx, _, _ = ops.dense_bwd(None, w, dy, z, act, need_dw=False, need_dbias=False)
    dz = dy.double() * dact_ref(act, z.double())
    low, high = held_between(dz, 2e-5 * dz.abs() + 2e-7 * dy.double().abs(), dtype)
    h, r = (low + high) / 2, (high - low) / 2
    w64 = q8_wide_values(w)
    ref = h @ w64
    tol = r @ w64.abs() + (N / 16 + 20) * STEP * ((h.abs() + r) @ w64.abs())
    assert float(tol.norm()) < 0.02 * float(ref.norm())
    close(dx, ref, rounded(ref, dtype, tol), "dx")


@pytest.mark.parametrize("M,K,N,dtype", [(1, 64, 300, BF), (333, 520, 700, HF), (3000, 1024, 2300, BF)])
def test_gradient_behind_relu(M, K, N, dtype):
    """dz is dy or zero, without an error: the bits of the product of dz taken to 8 bits beforehand."""
    w = ops.q8_encode(normal(1, N, K, std=K ** -0.5), ops.TILE)
    dy, z = normal(2, M, N, dtype=dtype), normal(3, M, N, dtype=dtype)
    dx, _, _ = ops.dense_bwd(None, w, dy, z, "relu", need_dw=False, need_dbias=False)
    dz = torch.where(z > 0, dy, torch.zeros_like(dy))
    want, _, _ = ops.dense_bwd(None, w, dz, need_dw=False, need_dbias=False)
    assert torch.equal(dx, want)
    held = q8_wide_values(ops.q8_encode(dz, 128))
    assert torch.equal(held, q8_wide_ref(dz.double(), 128)[0])
    w64 = q8_wide_values(w)
    ref = held @ w64
    close(dx, ref, rounded(ref, dtype, (N / 16 + 20) * STEP * (held.abs() @ w64.abs())), "dx")
