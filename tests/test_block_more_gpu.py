"""Layer norm, 8-bit blocks and experts together, as a model has them: FeedForward trained and served behind a conv
layer, MixtureFeedForward behind it."""
import pytest
import torch

from block_ref import U, act_ref, dact_ref, q8_values
from conv2d_layer_gb300 import abi, ops
from conv2d_layer_gb300.abi import ACT_RELU, BF16, NORM_BATCH
from conv2d_layer_gb300.block import FeedForward, MixtureFeedForward, rows
from conv2d_layer_gb300.layer import Conv2dLayer
from conv2d_layer_gb300.workloads import LayerSpec, random_layer_inputs
from more_ref import layer_bwd_ref, layer_ref, q8_wide_values
from test_block_gpu import normal
from test_feedforward_gpu import params, rel

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(autouse=True)
def device_clean():
    yield
    assert abi.conv2d_device_status() == (abi.OK, 0)


def step64(ff, h, dy, stored, n=None, u=None, w=None):
    """The block behind its h and its gradients in 64 bits; n, u, w: the operands that 8-bit products take."""
    g, b1, b2 = (t.double() for t in (ff.gamma, ff.b1, ff.b2))
    w1, w2 = w or (ff.w1.double(), ff.w2.double())
    beta = None if ff.beta is None else ff.beta.double()
    n_, mean, inv = layer_ref(h, g, beta, ff.eps)
    n = n_ if n is None else n
    z = n @ w1.t() + b1
    u = act_ref(ff.act, z) if u is None else u
    y = u @ w2.t() + b2 + h
    d = dy.double()
    dz = (d @ w2) * dact_ref(ff.act, stored)
    dx, dg, db = layer_bwd_ref(h, g, mean, inv, dz @ w1, d)
    return dict(y=y, dx=dx, dgamma=dg, dbeta=db, dw1=dz.t() @ n, db1=dz.sum(0), dw2=d.t() @ u, db2=d.sum(0))


# Relative errors in the 2-norm: a chain of at most eight bf16 roundings of half a step each (2^-8 at most, independent of
# each other); checkpoints off by up to 2^-4 in each of two factors; with 8-bit products dz and dy too, in the first dx.
BOUND = {"full": 8 * U[BF], "q8": 2 * 2.0 ** -4, "bits8": 4 * 2.0 ** -4}


@pytest.mark.parametrize("checkpoint,bits8", [("full", False), ("q8", False), ("full", True), ("q8", True)])
@pytest.mark.parametrize("act", ["gelu", "relu"])
def test_training_step_behind_a_conv_layer(checkpoint, bits8, act):
    width, inner = 160, 384
    spec = LayerSpec(N=4, H=14, W=14, IC=32, OC=width, KH=3, KW=3, stride=1, pad=1, norm=NORM_BATCH, act=ACT_RELU, dtype=BF16)
    inp = random_layer_inputs(spec, 5)
    li = inp["layers"][0]
    conv = Conv2dLayer(spec, li.w, li.b, li.gamma, li.beta)
    x = inp["x"].cuda()
    conv.zero_grad()
    c = rows(conv.fwd_train(x))
    p = params(0, width, inner)
    ff = FeedForward(*p, act=act, checkpoint=checkpoint, norm="layer", beta=0.1 * p[4], eps=1e-5)
    if bits8:
        ff.quantize(block=True)
    r, dy = normal(3, *c.shape, dtype=BF), normal(4, *c.shape, dtype=BF)
    y = ff.fwd_train(c, r, bits8=bits8)
    h, _, n, z, u, mean = ff.saved
    stored = q8_values(z) if checkpoint == "q8" else z.double()
    held = dict(n=q8_wide_values(n), u=q8_wide_values(u), w=tuple(q8_wide_values(w) for w in ff.w8)) if bits8 else {}
    dc = ff.bwd(dy)
    assert torch.equal(h, (c.float() + r.float()).to(BF))
    ref = step64(ff, h.double(), dy, stored, **held)
    got = dict(y=y, dx=dc, dgamma=ff.dgamma, dbeta=ff.dbeta, dw1=ff.dw1, db1=ff.db1, dw2=ff.dw2, db2=ff.db2)
    bound = BOUND["bits8" if bits8 else checkpoint]
    for k, v in got.items():
        assert rel(v, ref[k]) < (BOUND["full"] if k == "y" else bound), k
    # the gradient goes on into the conv layer
    dx = conv.bwd(x, dc.view(spec.N, spec.OH, spec.OW, spec.OC))
    assert bool(dx.isfinite().all()) and float(dx.float().norm()) > 0
    once = ff.dbeta.clone()
    ff.fwd_train(c, r, bits8=bits8)
    ff.bwd(dy)
    assert rel(ff.dbeta, 2 * once.double()) < 1e-6


@pytest.mark.parametrize("n", [1, 7, 64, 333])
@pytest.mark.parametrize("norm", ["rms", "layer"])
def test_serving_from_blocks(n, norm):
    ff = FeedForward(*params(1, 256, 1024), act="silu", checkpoint="full", norm=norm)
    x, r = normal(n, n, 256, dtype=BF), normal(n + 1, n, 256, dtype=BF)
    want, h = ff.fwd_infer(x, r)
    ff.quantize(block=True)
    y, h8 = ff.fwd_infer(x, r, bits8=True)
    assert torch.equal(h, h8)
    # four operands in 8 bits, each off by at most 2^-4 and independently of each other
    assert rel(y, want.double()) < 2 * 2.0 ** -4
    # the same operators by hand
    a = ff._norm(x, r, y=False, group=128)
    u, _ = ops.dense_fwd(a.q8, ops.q8_encode(ff.w1, ops.TILE), ff.b1, "silu", dtype=BF)
    by_hand, _ = ops.dense_fwd(ops.q8_encode(u, 128), ops.q8_encode(ff.w2, ops.TILE), ff.b2, residual=a.h, dtype=BF)
    assert torch.equal(y, by_hand)


@pytest.mark.parametrize("n", [0, 1, 64, 65, 200])
@pytest.mark.parametrize("norm", ["rms", "layer"])
def test_mixture(n, norm):
    D, F, E, k = 256, 128, 9, 3
    g = 1 + normal(1, D, std=0.2)
    m = MixtureFeedForward(g, normal(2, E, D, std=1 / 16), normal(3, E, 2 * F, D, std=1 / 16), normal(4, E, D, F, std=F ** -0.5),
                           k, b1=normal(5, E, 2 * F, std=0.1), b2=normal(6, E, D, std=0.1), norm=norm)
    x, r = normal(7, n, D, dtype=BF), normal(8, n, D, dtype=BF)
    y, h = m.fwd_infer(x, r)
    a = m._norm(x, r)
    assert torch.equal(h, a.h) and y.shape == (n, D)
    if n == 0:
        return
    # every row as if it came alone: the experts of a row do not hang on the others
    for i in {0, n // 2, n - 1}:
        one, _ = m.fwd_infer(x[i:i + 1], r[i:i + 1])
        # other splits of the sums over k: fp32 sums in another order, rounded to bf16 twice on the way
        assert rel(one, y[i:i + 1].double()) < 4 * U[BF]
    m.quantize()
    y8, _ = m.fwd_infer(x, r)
    # weights, n and h in 8 bits: four operands, each off by at most 2^-4 and independently of each other
    assert rel(y8 - h, (y - h).double()) < 3 * 2.0 ** -4


def test_a_block_and_experts_replay_from_a_graph():
    ff = FeedForward(*params(2, 256, 512), checkpoint="q8", norm="layer", beta=torch.zeros(256))
    ff.quantize(block=True)
    m = MixtureFeedForward(ff.gamma, normal(2, 8, 256, std=1 / 16), normal(3, 8, 256, 256, std=1 / 16),
                           normal(4, 8, 256, 128, std=0.1), 2, norm="layer")
    x, dy = normal(5, 48, 256, dtype=BF), normal(6, 48, 256, dtype=BF)

    def step():
        ff.zero_grad()
        y = ff.fwd_train(x, bits8=True)
        dx = ff.bwd(dy)
        return (y, dx, *m.fwd_infer(y)[:1], ff.dw1, ff.dgamma, ff.dbeta)

    want = [t.clone() for t in step()]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, got))
