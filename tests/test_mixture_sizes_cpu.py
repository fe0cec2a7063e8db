"""MixtureFeedForward and moe_encode refuse what no step could run, when the layer is made or taken to 8 bits."""
import pytest
import torch

from conv2d_layer_gb300 import ops
from conv2d_layer_gb300.block import MixtureFeedForward


def mixture(D=128, F=256, E=6, k=2, gated=True, **kw):
    z = torch.zeros
    return MixtureFeedForward(z(D), z(E, D), z(E, 2 * F if gated else F, D), z(E, D, F), k, gated=gated, device="cpu", **kw)


@pytest.mark.parametrize("sizes,why", [
    (dict(E=257, D=8, F=8), "router: 1 to 256 experts"), (dict(E=0, k=1), "router: 1 to 256 experts"), (dict(E=20, k=17), "k: 1 to 16"),
    (dict(k=2.0), "k: 1 to 6"), (dict(D=132), "width: a multiple of 8"), (dict(D=0), "width: a multiple of 8"),
    (dict(F=100), "inner features: a multiple of 8"), (dict(F=0), "inner features: a multiple of 8")])
def test_sizes_are_refused_when_the_layer_is_made(sizes, why):
    with pytest.raises(ValueError, match=why):
        mixture(**sizes)


def test_largest_counts_are_taken():
    assert mixture(E=256, D=8, F=8, k=16).k == 16


@pytest.mark.parametrize("sizes", [dict(D=256, F=192), dict(D=256, F=64), dict(D=136, F=256), dict(D=136, F=256, gated=False)])
def test_quantize_refuses_parts_of_tiles_and_keeps_the_weights(sizes, monkeypatch):
    monkeypatch.setattr(ops, "q8_encode", lambda t, group: pytest.fail("encoded"))
    m = mixture(**sizes)
    w1, w2 = m.w1, m.w2
    with pytest.raises(ValueError, match="multiples of 128"):
        m.quantize()
    assert m.w1 is w1 and m.w2 is w2


def test_a_second_quantize_changes_nothing(monkeypatch):
    def encode(t, group):
        assert group == ops.TILE
        return ops.Q8(t.to(torch.float8_e4m3fn), torch.zeros(t.shape[0] // 128, t.shape[1] // 128, dtype=torch.uint8), group)

    monkeypatch.setattr(ops, "q8_encode", encode)
    m = mixture()
    m.quantize()
    held = m.w1, m.w2
    m.quantize()
    assert (m.w1, m.w2) == held and m.w1.q.shape == (6, 512, 128) and m.w1.scale.shape == (6, 4, 1)


@pytest.mark.parametrize("w", [torch.zeros(4, 128, 136), torch.zeros(4, 136, 128), torch.zeros(128, 128), None,
                               ops.Q8(torch.zeros(4, 128, 128), torch.zeros(4, 1, 1), ops.TILE)])
def test_moe_encode_takes_whole_tiles(w):
    with pytest.raises(ValueError, match="w: experts by rows by columns"):
        ops.moe_encode(w)
