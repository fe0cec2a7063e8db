"""The residual block behind a conv layer, trained and served: FeedForward against 64-bit arithmetic on the same
values, with the checkpoints kept whole and in 8 bits."""
import pytest
import torch

from block_ref import U, act_ref, dact_ref, q8_values, rms_bwd_ref, rms_ref
from conv2d_layer_gb300 import abi
from conv2d_layer_gb300.abi import ACT_RELU, BF16, NORM_BATCH
from conv2d_layer_gb300.block import FeedForward, rows
from conv2d_layer_gb300.layer import Conv2dLayer
from conv2d_layer_gb300.workloads import LayerSpec, random_layer_inputs

WIDTH, INNER = 64, 256


def params(seed=0, width=WIDTH, inner=INNER):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s, std=1.0: torch.randn(*s, generator=g) * std  # noqa: E731
    return [1 + n(width, std=0.2), n(inner, width, std=width ** -0.5), n(inner, std=0.1), n(width, inner, std=inner ** -0.5),
            n(width, std=0.1)]


def test_construction_and_order():
    p = params()
    with pytest.raises(ValueError, match="checkpoint"):
        FeedForward(*p, checkpoint="half", device="cpu")
    with pytest.raises(ValueError, match="act"):
        FeedForward(*p, act="swish", device="cpu")
    with pytest.raises(ValueError, match="b1: shape"):
        FeedForward(p[0], p[1], p[4], p[3], p[4], device="cpu")
    ff = FeedForward(*p, device="cpu")
    with pytest.raises(RuntimeError, match="fwd_train"):
        ff.bwd(torch.zeros(2, WIDTH))
    with pytest.raises(RuntimeError, match="quantize"):
        ff.fwd_infer(torch.zeros(2, WIDTH), bits8=True)


def rel(a, b):
    return float((a.double() - b).norm() / b.norm())


def step64(ff, x, r, dy, stored):
    """The block and its gradients in 64 bits; the activation's derivative is taken at the stored input, as the
    layer defines it (relu's steps at zero, so another z of the same rounding may have another derivative)."""
    g, b1, b2 = (t.double() for t in (ff.gamma, ff.b1, ff.b2))
    w1, w2 = ff.w1.double(), ff.w2.double()
    h = x.double() + r.double()
    n, inv = rms_ref(h, g, ff.eps)
    z = n @ w1.t() + b1
    u = act_ref(ff.act, z)
    y = u @ w2.t() + b2 + h
    d = dy.double()
    du = d @ w2
    dz = du * dact_ref(ff.act, stored)
    dn = dz @ w1
    dx, dg = rms_bwd_ref(h, g, inv, dn, d)
    return dict(y=y, dx=dx, dgamma=dg, dw1=dz.t() @ n, db1=dz.sum(0), dw2=d.t() @ u, db2=d.sum(0))


# Relative errors in the 2-norm: a chain of at most eight bf16 roundings of half a step each (2^-8 at most, and
# independent of each other), or checkpoints that are off by up to 2^-4 in each of two factors of a product.
BOUND = {"full": 8 * U[torch.bfloat16], "q8": 2 * 2.0 ** -4}


@pytest.mark.gpu
@pytest.mark.parametrize("checkpoint", ["full", "q8"])
@pytest.mark.parametrize("act", ["gelu", "silu", "relu"])
def test_training_step_behind_a_conv_layer(checkpoint, act):
    spec = LayerSpec(N=4, H=14, W=14, IC=32, OC=WIDTH, KH=3, KW=3, stride=1, pad=1, norm=NORM_BATCH, act=ACT_RELU, dtype=BF16)
    inp = random_layer_inputs(spec, 5)
    li = inp["layers"][0]
    conv = Conv2dLayer(spec, li.w, li.b, li.gamma, li.beta)
    x = inp["x"].cuda()
    conv.zero_grad()
    c = rows(conv.fwd_train(x))
    ff = FeedForward(*params(), act=act, checkpoint=checkpoint)
    g = torch.Generator(device="cuda").manual_seed(3)
    r = torch.randn(c.shape, generator=g, device="cuda").bfloat16()
    dy = torch.randn(c.shape, generator=g, device="cuda").bfloat16()
    y = ff.fwd_train(c, r)
    whole = 2 * c.shape[0] * (WIDTH + 2 * INNER) + 4 * c.shape[0]
    assert ff.saved_bytes() == whole if checkpoint == "full" else ff.saved_bytes() < 0.53 * whole
    z = ff.saved[3]
    stored = q8_values(z) if checkpoint == "q8" else z.double()
    dc = ff.bwd(dy)
    ref = step64(ff, c, r, dy, stored)
    got = dict(y=y, dx=dc, dgamma=ff.dgamma, dw1=ff.dw1, db1=ff.db1, dw2=ff.dw2, db2=ff.db2)
    for k, v in got.items():
        assert rel(v, ref[k]) < (BOUND["full"] if k == "y" else BOUND[checkpoint]), k
    # the gradient goes on into the conv layer
    dx = conv.bwd(x, dc.view(spec.N, spec.OH, spec.OW, spec.OC))
    assert bool(dx.isfinite().all()) and float(dx.float().norm()) > 0
    # gradients accumulate until they are zeroed
    once = ff.dw1.clone()
    ff.fwd_train(c, r)
    ff.bwd(dy)
    assert rel(ff.dw1, 2 * once.double()) < 1e-6
    ff.zero_grad()
    assert not bool(ff.dw1.any())
    assert abi.conv2d_device_status() == (abi.OK, 0)


@pytest.mark.gpu
@pytest.mark.parametrize("n", [1, 7, 64, 333])
def test_serving_agrees_with_training(n):
    ff = FeedForward(*params(1, 256, 1024), act="silu", checkpoint="full")
    g = torch.Generator(device="cuda").manual_seed(n)
    x, r = (torch.randn(n, 256, generator=g, device="cuda").bfloat16() for _ in range(2))
    want = ff.fwd_train(x, r)
    y, h = ff.fwd_infer(x, r)
    assert torch.equal(h, ff.saved[0])
    # another number of rows, another kernel: the same products in another order, rounded to bf16 twice on the way
    assert rel(y, want.double()) < 4 * U[torch.bfloat16]
    ff.quantize()
    y8, _ = ff.fwd_infer(x, r, bits8=True)
    # four operands in 8 bits, each off by at most 2^-4 and independently of each other
    assert rel(y8, want.double()) < 2 * 2.0 ** -4


@pytest.mark.gpu
def test_step_replays_from_a_graph():
    """Forward and backward captured with no eager step alive beside them; two replays give the eager bits."""
    ff = FeedForward(*params(2), checkpoint="q8")
    g = torch.Generator(device="cuda").manual_seed(4)
    x, r, dy = (torch.randn(500, WIDTH, generator=g, device="cuda").bfloat16() for _ in range(3))

    def step():
        ff.zero_grad()
        y = ff.fwd_train(x, r)
        return y, ff.bwd(dy)

    want = [t.clone() for t in step()] + [ff.dw1.clone(), ff.dgamma.clone()]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, dx = step()
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(want, (y, dx, ff.dw1, ff.dgamma)):
            assert torch.equal(a, b)
