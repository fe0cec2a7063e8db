"""The bounds of tests/test_held_in_8_bits_gpu.py: that they contain what they should, and that a product with a mistake in
it does not pass them."""
import pytest
import torch

from block_ref import U, act_ref, dact_ref
from held_ref import exponents, held_between
from more_ref import q8_wide_ref
from test_held_in_8_bits_gpu import down_bound, up_bound

BF = torch.bfloat16


def normal(seed, *shape, std=1.0):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed), dtype=torch.float64) * std


def test_exponents():
    top = torch.tensor([0.0, 1e-42, 448.0, 448.0001, 1.75, 1.7500001, 3.5, 896.0, 3e38], dtype=torch.float64)
    _, scale = q8_wide_ref(top[:, None], 128)
    assert torch.equal(exponents(top), scale[:, 0].double() - 127)


@pytest.mark.parametrize("dtype", [None, BF])
def test_interval_contains_what_is_held(dtype):
    v = normal(1, 200, 300, std=3.0) * torch.exp2(torch.arange(200.0, dtype=torch.float64) % 9)[:, None]
    err = 1e-3 * v.abs()
    low, high = held_between(v, err, dtype)
    for seed in range(20):
        w = v + err * (2 * torch.rand(v.shape, generator=torch.Generator().manual_seed(seed), dtype=torch.float64) - 1)
        held, _ = q8_wide_ref(w if dtype is None else w.float().to(dtype).double(), 128)
        assert bool((low <= held).all() and (held <= high).all())
    # exact values: one value each, and that one
    low, high = held_between(v.to(BF).double(), 0 * v, dtype)
    held, _ = q8_wide_ref(v.to(BF).double(), 128)
    assert torch.equal(low, held) and torch.equal(high, held)


@pytest.mark.parametrize("D,F,act,gated", [(128, 128, "identity", False), (2048, 1024, "silu", True), (384, 256, "silu", True),
                                           (2304, 128, "gelu", False), (1152, 640, "gelu", False), (640, 4352, "silu", True)])
def test_mistakes_in_the_experts_second_product_show(D, F, act, gated):
    x, _ = q8_wide_ref(normal(1, 1, D), 128)
    up = F * (1 + gated)
    w1, _ = q8_wide_ref(normal(2, up, D, std=D ** -0.5), -128)
    w2, _ = q8_wide_ref(normal(3, D, F, std=F ** -0.5), -128)
    h, he = up_bound(w1, x[0], None, act, gated, F)
    low, high = held_between(h[None], he[None])
    y, tol = down_bound(w2, low[0], high[0], None)
    tol = tol + U[BF] * (y.abs() + tol)
    assert float(tol.norm()) < 0.08 * float(y.norm())
    held, _ = q8_wide_ref(h[None], 128)
    assert bool(((w2 @ held[0] - y).abs() <= tol).all())

    def shows(wrong):
        return float(((wrong - y).abs() > tol).double().mean())

    assert shows(0 * y) > 0.8
    if F > 128:
        assert shows(w2[:, :-128] @ held[0, :-128]) > 0.5  # without the last k-block
    w = w2.clone()
    w[:, -128:] *= 2  # a tile's scale for another
    assert shows(w @ held[0]) > 0.5
    wrong = held[0].clone()
    wrong[:128] *= 2  # a scale of h for another
    assert shows(w2 @ wrong) > 0.5


def test_mistakes_in_the_gradients_8_bit_form_show():
    M, K, N = 40, 200, 640
    dy, z = normal(1, M, N).to(BF).double(), normal(2, M, N, std=1.5).to(BF).double()
    w, _ = q8_wide_ref(normal(3, N, K, std=N ** -0.5), -128)
    dz = dy * dact_ref("gelu", z)
    low, high = held_between(dz, 2e-5 * dz.abs() + 2e-7 * dy.abs(), BF)
    ref, tol = (low + high) / 2 @ w, (high - low) / 2 @ w.abs()
    tol = tol + U[BF] * (ref.abs() + tol)
    assert float(tol.norm()) < 0.02 * float(ref.norm())
    right, _ = q8_wide_ref(dz.float().to(BF).double(), 128)
    assert bool(((right @ w - ref).abs() <= tol).all())
    before, _ = q8_wide_ref(dz, 128)  # encoded before it is rounded to the element type
    wrong, _ = q8_wide_ref((dy * act_ref("sigmoid", z)).to(BF).double(), 128)
    for other in (before, wrong, dz):
        assert float(((other @ w - ref).abs() > tol).double().mean()) > 0.01
