"""Layer norm of rows and the 8-bit forms with wide groups and tiles without a GPU: refusals of the C entry points
and of the torch binding, workspace sizes, and the 64-bit forms pinned by differences."""
import math

import pytest
import torch

from block_ref import q8_ref
from conv2d_layer_gb300 import abi, ops
from more_ref import layer_bwd_ref, layer_ref, q8_wide_ref

BF, HF, FP = torch.bfloat16, torch.float16, torch.float32
P = 1 << 20  # stands for an aligned device pointer: never read, every call below is refused or sized
BAD, BIG, WS = abi.ERR_INVALID_ARG, abi.ERR_UNSUPPORTED, abi.ERR_WORKSPACE


def mat(type=abi.BF16, ld=0, data=P):
    return abi.Mat(data, ld, type, 0, None)


def q8(group=128, ld=0, scale=P):
    return abi.Mat(P, ld, abi.E4M3, group, scale)


@pytest.mark.parametrize("change", [
    dict(eps=0.0), dict(eps=float("nan")), dict(gamma=None), dict(gamma=P + 4), dict(beta=P + 4), dict(mean=P + 4),
    dict(inv=P + 8), dict(y=None), dict(residual=mat()), dict(h=mat()), dict(residual=mat(abi.FP16), h=mat()),
    dict(y=mat(abi.FP32)), dict(y=q8()), dict(q=mat()), dict(x=q8()), dict(x=mat(data=P + 2)), dict(y=mat(ld=32)),
    dict(q=q8(abi.TILE)), dict(q=q8(64)), dict(q=q8(scale=None)), dict(x=None),
])
def test_layer_norm_fwd_refusals(change):
    a = dict(eps=1e-6, x=mat(), residual=None, gamma=P, beta=P, h=None, y=mat(), q=None, mean=P, inv=P)
    a.update(change)
    assert abi.conv2d_layer_norm_fwd(4, 64, a["eps"], a["x"], a["residual"], a["gamma"], a["beta"], a["h"], a["y"], a["q"],
                                     a["mean"], a["inv"], stream=0) == BAD


@pytest.mark.parametrize("change", [
    dict(h=q8()), dict(dy=mat(abi.FP16)), dict(dh=mat(abi.FP32)), dict(dx=mat(ld=8)), dict(gamma=None), dict(inv=None),
    dict(mean=None), dict(inv=P + 8), dict(dx=None, dgamma=None, dbeta=None), dict(dgamma=P + 4), dict(dbeta=P + 4),
])
def test_layer_norm_bwd_refusals(change):
    a = dict(h=mat(), gamma=P, mean=P, inv=P, dy=mat(), dh=None, dx=mat(), dgamma=None, dbeta=None)
    a.update(change)
    assert abi.conv2d_layer_norm_bwd(4, 64, a["h"], a["gamma"], a["mean"], a["inv"], a["dy"], a["dh"], a["dx"], a["dgamma"],
                                     a["dbeta"], 0, P, 1 << 30, stream=0) == BAD


def test_rms_norm_takes_wide_groups_but_no_tiles():
    for group, code in ((abi.TILE, BAD), (64, BAD), (-1, BAD)):
        assert abi.conv2d_rms_norm_fwd(4, 64, 1e-6, mat(), None, P, None, mat(), q8(group), P, stream=0) == code


def test_no_rows_and_sizes():
    assert abi.conv2d_layer_norm_fwd(0, 64, 1e-6, mat(), None, P, None, None, mat(), None, None, None, stream=0) == abi.OK
    assert abi.conv2d_layer_norm_bwd(0, 64, mat(), P, P, P, mat(), None, mat(), None, None, 0, None, stream=0) == abi.OK
    assert abi.conv2d_layer_norm_bwd(0, 64, mat(), P, P, P, mat(), None, mat(), P, P, 1, None, stream=0) == abi.OK
    assert abi.conv2d_layer_norm_fwd(1 << 31, 64, 1e-6, mat(), None, P, None, None, mat(), None, None, None, stream=0) == BIG
    assert abi.conv2d_layer_norm_bwd_workspace_size(1 << 31, 64) == 0
    one, two = abi.conv2d_rms_norm_bwd_workspace_size(500, 64), abi.conv2d_layer_norm_bwd_workspace_size(500, 64)
    assert two == 2 * one  # the partial sums of dgamma and of dbeta


def z(*shape, dtype=BF):
    return torch.zeros(*shape, dtype=dtype)


def q(rows, cols, group):
    return ops.q8_empty(rows, cols, group, device="cpu")


G8, G4 = z(8, dtype=FP), z(4, dtype=FP)
REFUSED = [
    (lambda: ops.layer_norm_fwd(z(4, 8), z(8)), "gamma: expected a contiguous float32"),
    (lambda: ops.layer_norm_fwd(z(4, 8), G8, z(7, dtype=FP)), "beta: expected"),
    (lambda: ops.layer_norm_fwd(z(4, 8), G8, G8, y=False), "must be asked for"),
    (lambda: ops.layer_norm_fwd(z(4, 8), G8, G8, h=z(4, 8)), "h: "),
    (lambda: ops.layer_norm_fwd(z(4, 8), G8, G8, residual=z(4, 8, dtype=HF)), "residual: dtype"),
    (lambda: ops.layer_norm_fwd(z(4, 8), G8, G8, group=ops.TILE), "group: a norm's rows share no scale"),
    (lambda: ops.layer_norm_fwd(z(4, 8), G8, G8, q8=q(4, 8, ops.TILE)), "q8: a norm's rows share no scale"),
    (lambda: ops.rms_norm_fwd(z(4, 8), G8, group=ops.TILE), "group: a norm's rows share no scale"),
    (lambda: ops.layer_norm_fwd(z(4, 8), G8, G8, mean=z(3, dtype=FP)), "mean: expected"),
    (lambda: ops.layer_norm_fwd(z(4, 8), G8, G8, inv_std=z(4)), "inv_std: expected"),
    (lambda: ops.layer_norm_fwd(z(4, 8), G8, G8), "CUDA device memory"),
    (lambda: ops.layer_norm_bwd(z(4, 8), G8, G4, G4, z(4, 8, dtype=HF)), "dy: dtype"),
    (lambda: ops.layer_norm_bwd(z(4, 8), G8, z(5, dtype=FP), G4, z(4, 8)), "mean: expected"),
    (lambda: ops.layer_norm_bwd(z(4, 8), G8, G4, G4, z(4, 8), need_dx=False, need_dgamma=False, need_dbeta=False), "need_"),
    (lambda: ops.layer_norm_bwd(z(4, 8), G8, G4, G4, z(4, 8), dgamma=G8), "hand in both"),
    (lambda: ops.layer_norm_bwd(z(4, 8), G8, G4, G4, z(4, 8), dbeta=G4, need_dgamma=False), "dbeta: expected"),
    (lambda: ops.layer_norm_bwd(z(4, 8), G8, G4, G4, z(4, 8)), "CUDA device memory"),
    (lambda: ops.q8_encode(z(4, 8), group=64), "group: 0"),
    (lambda: ops.q8_encode(z(4, 8), group=1 << 70), "group: 0"),
    (lambda: ops.q8_encode(z(130, 8), out=q(130, 8, ops.TILE)._replace(scale=z(1, 1, dtype=torch.uint8))), "out: scales are uint8 of shape (2, 1)"),
    (lambda: ops.q8_encode(z(130, 8), ops.TILE), "CUDA device memory"),
    (lambda: ops.q8_decode(q(4, 200, 128)._replace(group=32)), "q8: scales are uint8 of shape (4, 7)"),
    (lambda: ops.q8_decode(q(4, 200, ops.TILE)), "CUDA device memory"),
]


@pytest.mark.parametrize("i", range(len(REFUSED)))
def test_binding_refuses_before_a_launch(i):
    call, why = REFUSED[i]
    with pytest.raises(ValueError, match=why.replace("(", r"\(").replace(")", r"\)")):
        call()


def test_shapes_of_wide_groups_and_tiles():
    assert q(4, 200, 128).scale.shape == (4, 2) and q(4, 200, 128).shape == (4, 200)
    assert q(300, 200, ops.TILE).scale.shape == (3, 2)
    with pytest.raises(ValueError, match="group"):
        ops.q8_scales(8, 64)


# ------------------------------------------------------------------ the 64-bit forms
def test_wide_references_by_groups():
    g = torch.Generator().manual_seed(0)
    v = torch.randn(200, 300, generator=g).double() * torch.exp2(torch.randint(-9, 9, (200, 300), generator=g).double())
    values, scale = q8_wide_ref(v, 128)
    tiles, tscale = q8_wide_ref(v, -128)
    for c in range(3):
        part, s = q8_ref(v[:, 128 * c:128 * c + 128], 0)
        assert torch.equal(values[:, 128 * c:128 * c + 128], part) and torch.equal(scale[:, c:c + 1], s)
        for r in range(2):
            box = v[128 * r:128 * r + 128, 128 * c:128 * c + 128]
            part, s = q8_ref(box.reshape(1, -1), 0)
            assert torch.equal(tiles[128 * r:128 * r + 128, 128 * c:128 * c + 128], part.view(box.shape))
            assert int(tscale[r, c]) == int(s)


def test_layer_references_by_differences():
    g = torch.Generator().manual_seed(1)
    h, gamma, beta, dy, dh = (torch.randn(*s, generator=g).double() for s in ((3, 10), (10,), (10,), (3, 10), (3, 10)))
    _, mean, inv = layer_ref(h, gamma, beta, 1e-3)
    dx, dg, db = layer_bwd_ref(h, gamma, mean, inv, dy, dh)

    def loss(h, gamma, beta):
        return float((layer_ref(h, gamma, beta, 1e-3)[0] * dy + h * dh).sum())

    for i in range(30):
        d = torch.zeros(30, dtype=torch.float64)
        d[i] = 1e-6
        num = (loss(h + d.view(3, 10), gamma, beta) - loss(h - d.view(3, 10), gamma, beta)) / 2e-6
        assert math.isclose(num, float(dx.flatten()[i]), abs_tol=1e-7)
    for i in range(10):
        d = torch.zeros(10, dtype=torch.float64)
        d[i] = 1e-6
        assert math.isclose((loss(h, gamma + d, beta) - loss(h, gamma - d, beta)) / 2e-6, float(dg[i]), abs_tol=1e-7)
        assert math.isclose((loss(h, gamma, beta + d) - loss(h, gamma, beta - d)) / 2e-6, float(db[i]), abs_tol=1e-7)
