"""RMS norm, dense layer and 8-bit checkpoints without a GPU: refusals of the C entry points and of the torch
binding (nothing is launched when an argument is refused), workspace sizes, and the 64-bit forms that the GPU
tests compare against, pinned by counting and by differences."""
import math

import pytest
import torch

from block_ref import act_ref, dact_ref, q8_ref, rms_bwd_ref, rms_ref
from conv2d_layer_gb300 import abi, ops

BF, HF, FP = torch.bfloat16, torch.float16, torch.float32
P = 1 << 20  # stands for an aligned device pointer: never read, every call below is refused or sized


def mat(cols=64, type=abi.BF16, ld=0, group=0, data=P, scale=None):
    return abi.Mat(data, ld, type, group, scale)


def q8(cols=64, group=32, ld=0, data=P, scale=P):
    return abi.Mat(data, ld, abi.E4M3, group, scale)


def dense(M=8, K=64, N=32, act=abi.ACT_GELU, dtype=abi.BF16, accumulate=0):
    return abi.DenseDesc(M, K, N, act, dtype, accumulate)


BAD, BIG, WS = abi.ERR_INVALID_ARG, abi.ERR_UNSUPPORTED, abi.ERR_WORKSPACE


@pytest.mark.parametrize("rows,cols,x,q,code", [
    (-1, 64, mat(), q8(), BAD), (4, 0, mat(), q8(), BAD), (1 << 31, 64, mat(), q8(), BIG),
    (4, (1 << 28) + 1, mat(), q8(), BIG), (4, 64, None, q8(), BAD), (4, 64, mat(), None, BAD),
    (4, 64, mat(data=None), q8(), BAD), (4, 64, mat(data=P + 8), q8(), BAD), (4, 64, mat(ld=63), q8(), BAD),
    (4, 64, mat(type=4), q8(), BAD), (4, 64, mat(), q8(group=16), BAD), (4, 64, mat(), q8(scale=None), BAD),
    (4, 64, mat(), mat(), BAD), (4, 64, q8(), q8(), BAD),
])
def test_q8_refusals(rows, cols, x, q, code):
    assert abi.conv2d_q8_encode(rows, cols, x, q, stream=0) == code
    assert abi.conv2d_q8_decode(rows, cols, q, x, stream=0) == code


def test_no_rows_is_no_work():
    assert abi.conv2d_q8_encode(0, 64, mat(), q8(), stream=0) == abi.OK
    assert abi.conv2d_rms_norm_fwd(0, 64, 1e-6, mat(), None, P, None, mat(), None, None, stream=0) == abi.OK
    assert abi.conv2d_rms_norm_bwd(0, 64, mat(), P, P, mat(), None, mat(), None, 0, None, stream=0) == abi.OK
    assert abi.conv2d_rms_norm_bwd(0, 64, mat(), P, P, mat(), None, mat(), P, 1, None, stream=0) == abi.OK
    d = dense(M=0)
    assert abi.conv2d_dense_fwd(d, mat(), mat(), None, None, None, mat(), None, stream=0) == abi.OK
    assert abi.conv2d_dense_bwd(d, mat(), mat(), mat(), mat(), mat(), None, None, None, stream=0) == abi.OK
    d.accumulate = 1
    assert abi.conv2d_dense_bwd(d, mat(), mat(), mat(), mat(), mat(), mat(type=abi.FP32), P, None, stream=0) == abi.OK


@pytest.mark.parametrize("change", [
    dict(eps=0.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(gamma=None), dict(gamma=P + 4),
    dict(inv=P + 4), dict(y=None), dict(residual=mat()), dict(h=mat()), dict(residual=mat(type=abi.FP16), h=mat()),
    dict(y=mat(type=abi.FP32)), dict(y=q8()), dict(q=mat()), dict(x=q8()), dict(x=mat(data=P + 2)), dict(y=mat(ld=32)),
])
def test_rms_norm_fwd_refusals(change):
    a = dict(eps=1e-6, x=mat(), residual=None, gamma=P, h=None, y=mat(), q=None, inv=P)
    a.update(change)
    assert abi.conv2d_rms_norm_fwd(4, 64, a["eps"], a["x"], a["residual"], a["gamma"], a["h"], a["y"], a["q"], a["inv"],
                                   stream=0) == BAD


@pytest.mark.parametrize("change", [
    dict(h=q8()), dict(dy=mat(type=abi.FP16)), dict(dh=mat(type=abi.FP32)), dict(dx=mat(ld=8)), dict(gamma=None),
    dict(inv=None), dict(inv=P + 8), dict(dx=None, dgamma=None), dict(dgamma=P + 4),
])
def test_rms_norm_bwd_refusals(change):
    a = dict(h=mat(), gamma=P, inv=P, dy=mat(), dh=None, dx=mat(), dgamma=None)
    a.update(change)
    assert abi.conv2d_rms_norm_bwd(4, 64, a["h"], a["gamma"], a["inv"], a["dy"], a["dh"], a["dx"], a["dgamma"], 0, P,
                                   1 << 30, stream=0) == BAD


@pytest.mark.parametrize("change", [
    dict(d=dense(M=-1)), dict(d=dense(K=0)), dict(d=dense(N=0)), dict(d=dense(act=6)), dict(d=dense(act=-1)),
    dict(d=dense(dtype=abi.FP32)), dict(d=dense(dtype=abi.E4M3)), dict(x=None), dict(w=None), dict(y=None),
    dict(x=mat(type=abi.FP16)), dict(x=mat(ld=63)), dict(w=mat(ld=63)), dict(y=mat(ld=31)), dict(y=q8()),
    dict(x=q8(group=8)), dict(x=q8(scale=None)), dict(x=mat(data=P + 8)), dict(residual=q8()), dict(residual=mat(ld=1)),
    dict(z=q8(group=0)), dict(z=mat(type=abi.FP32)), dict(bias=P + 4), dict(y=mat(data=None)),
])
def test_dense_fwd_refusals(change):
    a = dict(d=dense(), x=mat(), w=mat(), bias=P, residual=None, z=None, y=mat())
    a.update(change)
    assert abi.conv2d_dense_fwd(a["d"], a["x"], a["w"], a["bias"], a["residual"], a["z"], a["y"], P, 1 << 40, stream=0) == BAD


@pytest.mark.parametrize("change", [
    dict(d=dense(N=-3)), dict(dx=None, dw=None, db=None), dict(dy=None), dict(dy=q8()), dict(dy=mat(type=abi.FP16)),
    dict(z=None), dict(z=mat(ld=16)), dict(z=q8(group=64)), dict(x=mat(type=abi.FP32)), dict(w=mat(ld=60)),
    dict(dx=q8()), dict(dx=mat(ld=63)), dict(dw=mat(type=abi.FP16)), dict(dw=q8()), dict(dw=mat(data=P + 4)),
    dict(db=P + 4), dict(w=mat(data=None)), dict(x=q8(scale=None)),
])
def test_dense_bwd_refusals(change):
    a = dict(d=dense(), x=mat(), w=mat(), z=mat(), dy=mat(), dx=mat(), dw=mat(type=abi.FP32), db=P)
    a.update(change)
    assert abi.conv2d_dense_bwd(a["d"], a["x"], a["w"], a["z"], a["dy"], a["dx"], a["dw"], a["db"], P, 1 << 40, stream=0) == BAD


def test_sizes_beyond_the_kernels():
    assert abi.conv2d_dense_fwd_workspace_size(dense(M=1 << 31), mat(), mat()) == 0
    assert abi.conv2d_dense_fwd(dense(M=1 << 31), mat(), mat(), None, None, None, mat(), None, stream=0) == BIG
    assert abi.conv2d_rms_norm_bwd_workspace_size(1 << 31, 64) == 0


def test_workspace_sizes():
    # aligned operands need none of their own (256 stands for that); odd rows are moved, 8-bit ones decoded
    assert abi.conv2d_dense_fwd_workspace_size(dense(), mat(), mat()) == 256
    assert abi.conv2d_dense_fwd_workspace_size(dense(K=65), mat(), mat(ld=72)) >= 8 * 72 * 2
    assert abi.conv2d_dense_fwd_workspace_size(dense(), q8(group=0), q8(group=0)) == 256
    assert abi.conv2d_dense_fwd_workspace_size(dense(), q8(), q8(group=0)) >= 8 * 64 * 2 + 32 * 64 * 2
    a = [dense(), mat(), mat(), mat(), mat()]
    assert abi.conv2d_dense_bwd_workspace_size(*a, None, None, None) == 0
    assert abi.conv2d_dense_bwd_workspace_size(*a, mat(), None, None) >= 8 * 32 * 2  # dz
    a[0] = dense(act=abi.ACT_IDENTITY)
    assert abi.conv2d_dense_bwd_workspace_size(*a, mat(), None, None) == 256  # dz is dy
    # an fp32 weight gradient over many rows is split, with one fp32 partial for each split
    many = dense(M=100000, act=abi.ACT_IDENTITY)
    assert abi.conv2d_dense_bwd_workspace_size(many, mat(), mat(), None, mat(), None, mat(type=abi.FP32), None) >= 3 * 64 * 32 * 4


def test_conv_layers_keep_their_types_and_activations():
    for dtype in (abi.FP16, abi.E4M3):
        assert abi.conv2d_validate(abi.desc(2, 8, 8, 3, 4, 3, 3, pad=1, dtype=dtype)) == BAD
    for act in (abi.ACT_GELU, abi.ACT_SILU):
        assert abi.conv2d_validate(abi.desc(2, 8, 8, 3, 4, 3, 3, pad=1, act=act)) == BAD


# ------------------------------------------------------------------ binding
def z(*shape, dtype=BF):
    return torch.zeros(*shape, dtype=dtype)


def q(rows, cols, group=32):
    return ops.q8_empty(rows, cols, group, device="cpu")


REFUSED = [
    (lambda: ops.q8_encode(3), "x: expected a torch.Tensor"),
    (lambda: ops.q8_encode(z(4)), "x: expected rows by"),
    (lambda: ops.q8_encode(z(4, 0)), "x: expected rows by"),
    (lambda: ops.q8_encode(z(4, 8, dtype=torch.int32)), "x: dtype"),
    (lambda: ops.q8_encode(z(4, 8), group=16), "group"),
    (lambda: ops.q8_encode(z(8, 4).t()), "x: features must be contiguous"),
    (lambda: ops.q8_encode(z(1, 8).expand(4, 8)), "x: features must be contiguous"),
    (lambda: ops.q8_encode(z(4, 9)[:, 1:]), "x: must start on a 16-byte boundary"),
    (lambda: ops.q8_encode(z(4, 8), out=z(4, 8)), "out: expected a Q8"),
    (lambda: ops.q8_encode(z(4, 8), out=q(4, 9)), "out: "),
    (lambda: ops.q8_encode(z(4, 8)), "CUDA device memory"),
    (lambda: ops.q8_decode(z(4, 8)), "q8: expected a Q8"),
    (lambda: ops.q8_decode(q(4, 8), torch.int8), "dtype"),
    (lambda: ops.q8_decode(q(4, 8)._replace(scale=z(4, 2, dtype=torch.uint8))), "q8: scales are uint8 of shape"),
    (lambda: ops.q8_decode(q(4, 64)._replace(scale=z(2, 4, dtype=torch.uint8).t())), "q8: scales must be contiguous"),
    (lambda: ops.q8_decode(q(4, 8)._replace(scale=None)), "q8: expected a torch.Tensor"),
    (lambda: ops.q8_decode(q(4, 8)._replace(q=z(4, 8))), "q8: dtype"),
    (lambda: ops.q8_decode(q(4, 8), out=z(4, 7)), "out: shape"),
    (lambda: ops.rms_norm_fwd(z(4, 8), z(8)), "gamma: expected a contiguous float32"),
    (lambda: ops.rms_norm_fwd(z(4, 8), z(7, dtype=FP)), "gamma: expected"),
    (lambda: ops.rms_norm_fwd(z(4, 8), z(8, dtype=FP), y=False), "must be asked for"),
    (lambda: ops.rms_norm_fwd(z(4, 8), z(8, dtype=FP), h=z(4, 8)), "h: "),
    (lambda: ops.rms_norm_fwd(z(4, 8), z(8, dtype=FP), residual=z(4, 8, dtype=HF)), "residual: dtype"),
    (lambda: ops.rms_norm_fwd(z(4, 8), z(8, dtype=FP), residual=z(3, 8)), "residual: shape"),
    (lambda: ops.rms_norm_fwd(z(4, 8), z(8, dtype=FP), group=7), "group"),
    (lambda: ops.rms_norm_fwd(z(4, 8), z(8, dtype=FP), y=z(4, 9)), "y: shape"),
    (lambda: ops.rms_norm_fwd(z(4, 8), z(8, dtype=FP), inv_rms=z(3, dtype=FP)), "inv_rms: expected"),
    (lambda: ops.rms_norm_fwd(z(4, 8), z(8, dtype=FP)), "CUDA device memory"),
    (lambda: ops.rms_norm_bwd(z(4, 8), z(8, dtype=FP), z(4, dtype=FP), z(4, 8, dtype=HF)), "dy: dtype"),
    (lambda: ops.rms_norm_bwd(z(4, 8), z(8, dtype=FP), z(4, dtype=FP), z(4, 8), need_dx=False, need_dgamma=False), "need_"),
    (lambda: ops.rms_norm_bwd(z(4, 8), z(8, dtype=FP), z(4, dtype=FP), z(4, 8), dgamma=z(9, dtype=FP)), "dgamma: expected"),
    (lambda: ops.dense_fwd(z(4, 8), z(3, 9)), "w: shape"),
    (lambda: ops.dense_fwd(z(4, 8, dtype=FP), z(3, 8, dtype=FP)), "x: dtype"),
    (lambda: ops.dense_fwd(z(4, 8), z(3, 8, dtype=HF)), "dtype torch.bfloat16, but an operand is torch.float16"),
    (lambda: ops.dense_fwd(z(4, 8), z(0, 8)), "w: expected at least one"),
    (lambda: ops.dense_fwd(q(4, 8, 0), q(3, 8, 0)), "dtype: bfloat16 or float16"),
    (lambda: ops.dense_fwd(q(4, 8).q, z(3, 8)), "x: 8-bit values need their scales"),
    (lambda: ops.dense_fwd(z(4, 8), z(3, 8), act="swish"), "act: one of"),
    (lambda: ops.dense_fwd(z(4, 8), z(3, 8), save="half"), "save: one of"),
    (lambda: ops.dense_fwd(z(4, 8), z(3, 8), bias=z(3)), "bias: expected"),
    (lambda: ops.dense_fwd(z(4, 8), z(3, 8), residual=z(4, 4)), "residual: shape"),
    (lambda: ops.dense_fwd(z(4, 8), z(3, 8), y=q(4, 3)), "y: an 8-bit matrix is not taken"),
    (lambda: ops.dense_fwd(z(4, 8), z(3, 8), pre_act=z(4, 3)), "pre_act: not an output"),
    (lambda: ops.dense_fwd(z(4, 8), z(3, 8), save="q8", pre_act=q(4, 3, 0)), "pre_act: groups of 32"),
    (lambda: ops.dense_fwd(z(4, 8), z(3, 8)), "CUDA device memory"),
    (lambda: ops.dense_bwd(z(4, 8), z(3, 8), q(4, 3)), "dy: dtype"),
    (lambda: ops.dense_bwd(z(4, 8), z(3, 8), z(4, 3), act="relu"), "pre_act: needed"),
    (lambda: ops.dense_bwd(z(4, 8), z(3, 7), z(4, 3)), "w: shape"),
    (lambda: ops.dense_bwd(z(5, 8), z(3, 8), z(4, 3)), "x: shape"),
    (lambda: ops.dense_bwd(z(4, 8), z(3, 8), z(4, 3), need_dx=False, need_dw=False, need_dbias=False), "need_dx"),
    (lambda: ops.dense_bwd(z(4, 8), z(3, 8), z(4, 3), dw=z(3, 8, dtype=FP)), "hand in both"),
    (lambda: ops.dense_bwd(z(4, 8), z(3, 8), z(4, 3), grad_dtype=HF), "grad_dtype"),
    (lambda: ops.dense_bwd(z(4, 8), z(3, 8), z(4, 3), dx=z(4, 9)), "dx: shape"),
    (lambda: ops.dense_bwd(z(4, 8), z(3, 8), z(4, 3)), "CUDA device memory"),
]


@pytest.mark.parametrize("i", range(len(REFUSED)))
def test_binding_refuses_before_a_launch(i):
    call, why = REFUSED[i]
    with pytest.raises(ValueError, match=why.replace("(", r"\(")):
        call()


# ------------------------------------------------------------------ the 64-bit forms
def test_q8_ref_counts():
    """Against the format written out: every e4m3 value by hand, the nearest one with ties to the even code."""
    codes = [(m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)) for e in range(16) for m in range(8)][:127]
    assert codes[-1] == 448.0
    g = torch.Generator().manual_seed(0)
    v = torch.cat([torch.randn(400, generator=g).double() * 30, torch.tensor(codes).double(),
                   (torch.tensor(codes[:-1]) + torch.tensor(codes[1:])).double() / 2, torch.tensor([448.0, 0.0]).double()])
    v = v.clamp(-448, 448)[None]
    values, scale = q8_ref(v, 0)
    assert int(scale) == 127
    for x, y in zip(v[0].tolist(), values[0].tolist()):
        off = [abs(abs(x) - c) for c in codes]
        best = min(off)
        nearest = [i for i, o in enumerate(off) if o == best]
        want = codes[nearest[0] if len(nearest) == 1 else next(i for i in nearest if i % 2 == 0)]
        assert abs(y) == want and (y == 0 or (y > 0) == (x > 0))
    # torch's own conversion agrees where nothing is scaled
    assert torch.equal(values, v.float().to(torch.float8_e4m3fn).double())


@pytest.mark.parametrize("top,e", [(448.0, 0), (448.0001, 1), (1.0, -8), (1.75, -8), (1.7501, -7), (2.0 ** -200, -126), (3e38, 120)])
def test_q8_ref_scales(top, e):
    v = torch.tensor([[top, -top / 3, 0.0]], dtype=torch.float64)
    values, scale = q8_ref(v, 32)
    assert int(scale) == e + 127
    assert bool((values.abs() <= 448 * 2.0 ** e).all())


def test_references_by_differences():
    for act in ops.ACTS:
        x = torch.tensor([-20.0, -3.1, -0.7, -1e-3, 2e-3, 0.4, 1.9, 15.0], dtype=torch.float64)
        num = (act_ref(act, x + 1e-6) - act_ref(act, x - 1e-6)) / 2e-6
        assert torch.allclose(num, dact_ref(act, x), atol=1e-8)
    g = torch.Generator().manual_seed(1)
    h, gamma, dy, dh = (torch.randn(*s, generator=g).double() for s in ((3, 10), (10,), (3, 10), (3, 10)))
    _, inv = rms_ref(h, gamma, 1e-3)
    dx, dg = rms_bwd_ref(h, gamma, inv, dy, dh)

    def loss(h, gamma):
        return float((rms_ref(h, gamma, 1e-3)[0] * dy + h * dh).sum())

    for i in range(30):
        d = torch.zeros(30, dtype=torch.float64)
        d[i] = 1e-6
        num = (loss(h + d.view(3, 10), gamma) - loss(h - d.view(3, 10), gamma)) / 2e-6
        assert math.isclose(num, float(dx.flatten()[i]), abs_tol=1e-7)
    d = torch.zeros(10, dtype=torch.float64)
    d[4] = 1e-6
    num = (loss(h, gamma + d) - loss(h, gamma - d)) / 2e-6
    assert math.isclose(num, float(dg[4]), abs_tol=1e-7)
