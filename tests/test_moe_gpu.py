"""The mixture-of-experts layer against its 64-bit form, token by token."""
import pytest
import torch

from block_ref import STEP, U, close, rounded
from conv2d_layer_gb300 import abi, ops
from more_ref import moe_ref, q8_wide_ref, q8_wide_values
from test_block_gpu import ACT_ERR, normal, strided

pytestmark = pytest.mark.gpu
BF, HF, FP = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(autouse=True)
def device_clean():
    yield
    assert abi.conv2d_device_status() == (abi.OK, 0)


def layer(T, D, F, E, dtype, gated, bias, bits8=False, seed=0):
    n = lambda i, *s, std=1.0: normal(100 * seed + i, *s, std=std)  # noqa: E731
    up = F * (1 + gated)
    p = dict(x=n(1, T, D).to(dtype), router=n(2, E, D, std=D ** -0.5).to(dtype), w1=n(3, E, up, D, std=D ** -0.5).to(dtype),
             w2=n(4, E, D, F, std=F ** -0.5).to(dtype), b1=n(5, E, up, std=0.2) if bias else None,
             b2=n(6, E, D, std=0.2) if bias else None)
    if bits8:
        p["w1"], p["w2"] = ops.moe_encode(p["w1"]), ops.moe_encode(p["w2"])
    return p


def check(p, k, act, gated, normalize, residual, got, dtype, y64=None):
    """Against the 64-bit form. The logits: at most 64 additions in a lane, a few joins. h: the first product's sums (16
    terms truncated at a time, joins of the cluster), the activation, its rounding; then the second product's."""
    bits8 = isinstance(p["w1"], ops.Q8)
    x, router = p["x"].double(), p["router"].double()
    w1, w2 = (q8_wide_values(p[n]) if bits8 else p[n].double() for n in ("w1", "w2"))
    D, F = x.shape[1], w2.shape[2]
    xs = q8_wide_ref(x, 128)[0] if bits8 else x
    r64 = None if residual is None else residual.double()
    b1, b2 = (None if p[n] is None else p[n].double() for n in ("b1", "b2"))

    def hold(h):
        return q8_wide_ref(h, 128)[0] if bits8 else h

    # the logits decide on x itself, the experts take what is held of it
    logits = x @ router.t()
    _, experts, weights, _ = moe_ref(x, router, w1, w2, k, b1, b2, act, gated, normalize, r64, hold)
    sums = (D / 256 + 20) * STEP * (x.abs() @ router.abs().t())
    mine = got.experts.long()
    # which experts: those of the 64-bit logits, or ones nearer than the sums' error
    worst = torch.gather(logits, 1, experts.long()[:, -1:])
    off = sums.amax(1, keepdim=True) * 2
    assert bool((torch.gather(logits, 1, mine) >= worst - off).all())
    same = (got.experts == experts).all(1)
    assert float(same.double().mean()) > 0.9 or x.shape[0] < 10
    e = torch.gather(sums, 1, mine).amax(1, keepdim=True) * 2 + 8 * U[FP]
    close(got.weights[same], weights[same], (weights * (2 * e + 4 * sums.amax(1, keepdim=True)))[same] + 1e-30, "weights")
    # y with the experts and weights that were taken
    T = x.shape[0]
    for t in range(T):
        y = torch.zeros(D, dtype=torch.float64, device="cuda") if r64 is None else r64[t].clone()
        tol = torch.zeros_like(y)
        for j in range(k):
            ex, w = int(got.experts[t, j]), float(got.weights[t, j])
            z = w1[ex] @ xs[t] + (0 if b1 is None else b1[ex])
            zmag = w1[ex].abs() @ xs[t].abs()
            ze = (D / 16 + 20) * STEP * zmag + U[FP] * z.abs()
            from block_ref import act_ref
            h = act_ref(act, z[:F])
            he = 1.2 * ze[:F] + ACT_ERR * h.abs()
            if gated:
                he = he * z[F:].abs() + h.abs() * ze[F:] + he * ze[F:]
                h = h * z[F:]
                he = he + U[FP] * h.abs()
            if bits8:
                held, scale = q8_wide_ref(h[None], 128)
                s = torch.exp2(scale.double() - 127).repeat_interleave(128, 1)[0, :F]
                # the nearest 8-bit value, or its neighbour where the sums' error carries h over the middle between them:
                # few, so half a step of each that is as near as that
                mid = torch.maximum(2.0 ** -4 * h.abs(), 2.0 ** -10 * s)
                near = (h - held[0]).abs() >= mid * 0.5 - he
                he = torch.where(near, 2 * mid, 0.0) + he * 0
                h = held[0]
            else:
                he = he + rounded(h, dtype, he)
            o = w2[ex] @ h + (0 if b2 is None else b2[ex])
            oe = w2[ex].abs() @ he + (F / 16 + 20) * STEP * (w2[ex].abs() @ (h.abs() + he)) + U[FP] * o.abs()
            y = y + w * o
            tol = tol + w * oe + 2 * U[FP] * (w * o).abs()
        tol = tol + U[FP] * y.abs() * 2
        close(got.y[t], y, rounded(y, dtype, tol), f"y of token {t}")


# T, D, F, E, k, dtype, gated, act, bias, normalize, residual, bits8
CASES = [
    (1, 8, 8, 1, 1, BF, False, "relu", False, True, False, False),
    (1, 256, 128, 4, 2, BF, True, "silu", False, True, False, False),
    (1, 2048, 1024, 64, 8, BF, True, "silu", True, False, True, False),
    (2, 264, 200, 3, 3, HF, False, "gelu", True, True, True, False),
    (3, 520, 72, 5, 1, BF, True, "identity", True, False, False, False),
    (5, 128, 1000, 9, 4, BF, True, "tanh", True, True, True, False),
    (8, 1024, 512, 256, 16, BF, False, "silu", False, True, False, False),
    (16, 768, 264, 7, 2, HF, True, "silu", False, False, True, False),
    (17, 640, 384, 20, 3, BF, True, "sigmoid", True, True, True, False),
    (33, 512, 136, 16, 4, BF, False, "gelu", True, True, True, False),
    (64, 1152, 640, 12, 2, BF, True, "silu", False, True, True, False),
    (64, 200, 96, 40, 8, HF, True, "relu", True, False, False, False),
    (64, 128, 64, 256, 16, BF, True, "silu", True, True, False, False),
    (1, 128, 128, 1, 1, BF, False, "identity", False, True, False, True),
    (1, 2048, 1024, 16, 4, BF, True, "silu", False, True, True, True),
    (7, 384, 256, 6, 2, HF, True, "silu", True, False, True, True),
    (16, 2304, 128, 8, 2, BF, False, "gelu", True, True, False, True),
    (37, 1152, 640, 23, 3, BF, False, "gelu", True, False, False, True),
    (64, 640, 4352, 4, 2, BF, True, "silu", False, True, True, True),
]


@pytest.mark.parametrize("T,D,F,E,k,dtype,gated,act,bias,normalize,has_res,bits8", CASES)
def test_moe(T, D, F, E, k, dtype, gated, act, bias, normalize, has_res, bits8):
    p = layer(T, D, F, E, dtype, gated, bias, bits8, seed=T)
    res = normal(7, T, D, dtype=dtype) if has_res else None
    args = dict(b1=p["b1"], b2=p["b2"], act=act, gated=gated, normalize=normalize)
    got = ops.moe_fwd(p["x"], p["router"], p["w1"], p["w2"], k, residual=res, **args)
    check(p, k, act, gated, normalize, res, got, dtype)
    # the same bits again, over the residual itself, from strided rows
    buf = strided(torch.zeros(T, D, dtype=dtype, device="cuda") if res is None else res, 3)
    x = strided(p["x"], 16)
    again = ops.moe_fwd(x, p["router"], p["w1"], p["w2"], k, residual=buf if has_res else None, y=buf, **args)
    assert again.y is buf and torch.equal(buf, got.y) and torch.equal(again.experts, got.experts)
    assert bool(torch.as_strided(buf, (T, 3), (buf.stride(0), 1), D).isnan()[:T - 1].all())


def test_fp32_router_and_strided_weights():
    p = layer(6, 256, 192, 10, BF, True, True, seed=3)
    p["router"] = normal(9, 10, 256, std=1 / 16)
    wide1, wide2 = normal(1, 10, 384, 264, dtype=BF), normal(2, 10, 256, 200, dtype=BF)
    wide1[:, :, :256], wide2[:, :, :192] = p["w1"], p["w2"]
    want = ops.moe_fwd(p["x"], p["router"], p["w1"], p["w2"], 3, b1=p["b1"], b2=p["b2"], gated=True)
    check(p, 3, "silu", True, True, None, want, BF)
    got = ops.moe_fwd(p["x"], p["router"], wide1[:, :, :256], wide2[:, :, :192], 3, b1=p["b1"], b2=p["b2"], gated=True)
    assert torch.equal(got.y, want.y)


def test_choice_among_equals_and_special_logits():
    E, D = 70, 64
    router = torch.zeros(E, D, device="cuda", dtype=BF)
    router[:, 0] = torch.tensor([float(e % 7) for e in range(E)], device="cuda")
    router[5, 1] = -0.0
    x = torch.zeros(4, D, device="cuda", dtype=BF)
    x[0, 0], x[1, 0] = 1.0, -1.0
    x[3, 0] = float("nan")
    w1, w2 = normal(1, E, 64, D, dtype=BF), normal(2, E, D, 64, dtype=BF)
    got = ops.moe_fwd(x, router, w1, w2, 12)
    assert got.experts[0].tolist() == [6, 13, 20, 27, 34, 41, 48, 55, 62, 69, 5, 12]
    assert got.experts[1].tolist() == [0, 7, 14, 21, 28, 35, 42, 49, 56, 63, 1, 8]
    assert got.experts[2].tolist() == list(range(12))  # all equal
    assert torch.equal(got.weights[2], torch.full((12,), 1 / 12, device="cuda"))
    assert got.experts[3].tolist() == list(range(12)) and bool(got.weights[3].isnan().all()) and bool(got.y[3].isnan().all())
    assert bool(got.y[:3].isfinite().all())
    inf = torch.full((E,), -float("inf"), device="cuda", dtype=BF)  # one expert is left, the others' weight is zero
    inf[33] = 0
    router[:, 0] = inf
    got = ops.moe_fwd(x[:1], router, w1, w2, 3)
    assert got.experts[0].tolist() == [33, 0, 1] and got.weights[0].tolist() == [1.0, 0.0, 0.0]


@pytest.mark.parametrize("bits8", [False, True])
def test_what_an_expert_holds_stays_with_its_tokens(bits8):
    T, D, F, E = 20, 256, 128, 6
    p = layer(T, D, F, E, BF, True, False, bits8, seed=4)
    clean = ops.moe_fwd(p["x"], p["router"], p["w1"], p["w2"], 1, gated=True)
    bad = 3
    hit = (clean.experts == bad).any(1)
    assert 0 < int(hit.sum()) < T
    for name in ("w1", "w2"):
        spoiled = dict(p)
        if bits8:
            q = p[name].q.clone()
            q.view(torch.uint8)[bad, 7] = 0x7f  # NaN
            spoiled[name] = p[name]._replace(q=q)
        else:
            spoiled[name] = p[name].clone()
            spoiled[name][bad, 7] = float("inf")
        got = ops.moe_fwd(p["x"], p["router"], spoiled["w1"], spoiled["w2"], 1, gated=True)
        assert torch.equal(got.y[~hit], clean.y[~hit])
        assert not bool(got.y[hit].isfinite().all())
    x = p["x"].clone()
    x[2, 5] = float("nan")
    got = ops.moe_fwd(x, p["router"], p["w1"], p["w2"], 1, gated=True)
    keep = torch.arange(T, device="cuda") != 2
    assert torch.equal(got.y[keep], clean.y[keep]) and bool(got.y[2].isnan().all())


def test_no_tokens():
    p = layer(1, 128, 64, 4, BF, False, False)
    got = ops.moe_fwd(p["x"][:0], p["router"], p["w1"], p["w2"], 2)
    assert got.y.shape == (0, 128) and got.experts.shape == (0, 2) and got.weights.shape == (0, 2)


@pytest.mark.parametrize("bits8", [False, True])
def test_captured_on_another_stream_and_back_to_back(bits8):
    """Calls one after the other share nothing but the allocator's workspaces; a replayed graph takes the inputs of its
    time."""
    p = layer(9, 512, 256, 12, BF, True, True, bits8, seed=5)
    q = layer(3, 256, 1024, 30, BF, False, False, bits8, seed=6)

    def step(stream=None):
        a = ops.moe_fwd(p["x"], p["router"], p["w1"], p["w2"], 3, b1=p["b1"], b2=p["b2"], gated=True, stream=stream)
        b = ops.moe_fwd(q["x"], q["router"], q["w1"], q["w2"], 8, act="gelu", stream=stream)
        c = ops.moe_fwd(a.y, p["router"], p["w1"], p["w2"], 3, gated=True, residual=a.y, stream=stream)
        return (*a, *b, *c)

    want = step()
    torch.cuda.synchronize()
    for _ in range(20):
        assert all(torch.equal(a, b) for a, b in zip(want, step()))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = step(side)
    here = step()  # both at once
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) and torch.equal(a, c) for a, b, c in zip(want, got, here))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    p["x"].copy_(normal(50, 9, 512, dtype=BF))
    for _ in range(3):
        graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(step(), held))


def test_behind_a_dense_layer():
    """The layer right behind kernels that write its inputs, and before one that reads its output."""
    p = layer(16, 1024, 512, 8, BF, True, False, seed=8)
    w = normal(60, 1024, 1024, std=1 / 32, dtype=BF)
    src = normal(61, 16, 1024, dtype=BF)
    x, _ = ops.dense_fwd(src, w)
    torch.cuda.synchronize()
    m = ops.moe_fwd(x, p["router"], p["w1"], p["w2"], 2, gated=True)
    torch.cuda.synchronize()
    want, _ = ops.dense_fwd(m.y, w)
    torch.cuda.synchronize()
    for _ in range(20):
        a, _ = ops.dense_fwd(src, w)
        b = ops.moe_fwd(a, p["router"], p["w1"], p["w2"], 2, gated=True)
        c, _ = ops.dense_fwd(b.y, w)
        assert torch.equal(c, want)
