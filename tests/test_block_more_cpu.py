"""FeedForward with layer norm and 8-bit blocks, and MixtureFeedForward, without a GPU: construction and order of calls."""
import pytest
import torch

from conv2d_layer_gb300 import ops
from conv2d_layer_gb300.block import FeedForward, MixtureFeedForward


def n(*s):
    return torch.randn(*s, generator=torch.Generator().manual_seed(0))


def feed_forward(**kw):
    return FeedForward(n(16), n(32, 16), n(32), n(16, 32), n(16), device="cpu", **kw)


def mixture(gated=True, **kw):
    a = dict(gamma=n(128), router=n(6, 128), w1=n(6, 512 if gated else 256, 128), w2=n(6, 128, 256), k=2)
    a.update(kw)
    return MixtureFeedForward(**a, gated=gated, device="cpu")


def test_norms():
    with pytest.raises(ValueError, match="norm: rms or layer"):
        feed_forward(norm="batch")
    with pytest.raises(ValueError, match="beta: layer norm only"):
        feed_forward(beta=n(16))
    with pytest.raises(ValueError, match="beta: shape"):
        feed_forward(norm="layer", beta=n(17))
    ff = feed_forward(norm="layer", beta=n(16))
    assert ff.dbeta.shape == (16,)
    ff.dbeta += 1
    ff.zero_grad()
    assert not bool(ff.dbeta.any())
    ff = feed_forward(norm="layer")
    assert ff.beta is None and ff.dbeta is None
    ff.zero_grad()


def test_training_in_8_bits_needs_tiles(monkeypatch):
    monkeypatch.setattr(ops, "q8_encode", lambda t, group: ("8-bit", t, group))
    ff, x = feed_forward(), torch.zeros(2, 16).bfloat16()
    with pytest.raises(RuntimeError, match="quantize"):
        ff.fwd_train(x, bits8=True)
    ff.quantize()
    with pytest.raises(RuntimeError, match="block=True"):
        ff.fwd_train(x, bits8=True)
    ff.quantize(block=True)
    assert ff.w8[0][2] == ops.TILE
    for call in (ff.fwd_train, ff.fwd_infer):  # the kernels are reached
        with pytest.raises(ValueError, match="CUDA device memory"):
            call(x, bits8=True)
    ff.w1.mul_(2)
    for call in (ff.fwd_train, ff.fwd_infer):
        with pytest.raises(RuntimeError, match="changed"):
            call(x, bits8=True)


@pytest.mark.parametrize("change,why", [
    (dict(act="swish"), "act"), (dict(dtype=torch.float32), "dtype"), (dict(router=n(128)), "router"), (dict(w2=n(128, 256)), "router"),
    (dict(w1=n(6, 256, 128)), "w1: shape"), (dict(w2=n(6, 120, 256)), "w2: shape"), (dict(b1=n(6, 256)), "b1: shape"),
    (dict(b2=n(5, 128)), "b2: shape"), (dict(gamma=n(64)), "gamma: shape"), (dict(k=0), "k: 1 to 6"), (dict(k=7), "k: 1 to 6"),
    (dict(beta=n(128)), "beta"), (dict(norm="none"), "norm")])
def test_mixture_refusals(change, why):
    with pytest.raises(ValueError, match=why):
        mixture(**change)


def test_mixture_reaches_the_kernels():
    m = mixture(gated=False, b1=n(6, 256), b2=n(6, 128), norm="layer", beta=n(128))
    with pytest.raises(ValueError, match="CUDA device memory"):
        m.fwd_infer(torch.zeros(3, 128).bfloat16())
