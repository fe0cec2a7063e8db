"""The mixture-of-experts layer without a GPU: refusals of the C entry point and of the torch binding, workspace sizes."""
import pytest
import torch

from conv2d_layer_gb300 import abi, ops

P = 1 << 20  # stands for an aligned device pointer: never read, every call below is refused or sized
BAD, BIG, WS = abi.ERR_INVALID_ARG, abi.ERR_UNSUPPORTED, abi.ERR_WORKSPACE
BF, HF, FP = torch.bfloat16, torch.float16, torch.float32


def mat(type=abi.BF16, ld=0, data=P):
    return abi.Mat(data, ld, type, 0, None)


def q8(group=abi.TILE, ld=0, scale=P):
    return abi.Mat(P, ld, abi.E4M3, group, scale)


def desc(T=4, D=128, F=256, E=8, k=2, act=abi.ACT_SILU, gated=1, normalize=1, dtype=abi.BF16):
    return abi.MoeDesc(T, D, F, E, k, act, gated, normalize, dtype)


def call(d=None, ws=P, ws_bytes=1 << 40, **change):
    a = dict(x=mat(), router=mat(), w1=mat(), b1=None, w2=mat(), b2=None, residual=None, y=mat(), experts=P, weights=P)
    a.update(change)
    return abi.conv2d_moe_fwd(d or desc(), a["x"], a["router"], a["w1"], a["b1"], a["w2"], a["b2"], a["residual"], a["y"],
                              a["experts"], a["weights"], ws, ws_bytes, stream=0)


@pytest.mark.parametrize("d,code", [
    (dict(T=-1), BAD), (dict(D=0), BAD), (dict(F=0), BAD), (dict(E=0), BAD), (dict(k=0), BAD), (dict(k=9), BAD), (dict(act=6), BAD),
    (dict(act=-1), BAD), (dict(dtype=abi.FP32), BAD), (dict(dtype=abi.E4M3), BAD), (dict(T=65), BIG), (dict(E=257), BIG),
    (dict(k=17, E=20), BIG), (dict(D=132), BIG), (dict(F=260), BIG), (dict(E=256, F=1 << 23), BIG), (dict(E=256, D=1 << 23), BIG)])
def test_descriptor_refusals(d, code):
    assert call(desc(**d)) == code
    assert abi.conv2d_moe_fwd_workspace_size(desc(**d), mat(), mat()) == 0


@pytest.mark.parametrize("change,code", [
    (dict(x=None), BAD), (dict(x=mat(abi.FP16)), BAD), (dict(x=mat(ld=64)), BAD), (dict(x=mat(ld=132)), BIG), (dict(x=mat(data=P + 8)), BAD),
    (dict(router=None), BAD), (dict(router=mat(abi.FP16)), BAD), (dict(router=mat(ld=130)), BIG), (dict(router=q8()), BAD),
    (dict(w1=None), BAD), (dict(w1=mat(abi.FP16)), BAD), (dict(w1=mat(ld=100)), BAD), (dict(w1=mat(ld=132)), BIG),
    (dict(w1=q8()), BAD), (dict(w2=q8()), BAD), (dict(w2=mat(ld=128)), BAD), (dict(w2=mat(ld=260)), BIG), (dict(w2=mat(abi.FP32)), BAD),
    (dict(w1=q8(128), w2=q8()), BAD), (dict(w1=q8(), w2=q8(0)), BAD), (dict(w1=q8(), w2=q8(scale=None)), BAD),
    (dict(w1=q8(ld=136), w2=q8()), BIG), (dict(w1=mat(data=None)), BAD), (dict(y=None), BAD), (dict(y=mat(abi.FP16)), BAD),
    (dict(y=mat(ld=127)), BAD), (dict(residual=mat(abi.FP16)), BAD), (dict(residual=mat(ld=1)), BAD), (dict(residual=mat(data=P + 2)), BAD),
    (dict(b1=P + 4), BAD), (dict(b2=P + 8), BAD), (dict(experts=None), BAD), (dict(weights=None), BAD), (dict(experts=P + 4), BAD)])
def test_argument_refusals(change, code):
    assert call(**change) == code


def test_8_bit_experts_are_whole_tiles():
    for d in (dict(D=136), dict(F=264), dict(D=64), dict(F=64)):
        assert call(desc(**d), w1=q8(), w2=q8()) == BIG
    assert abi.conv2d_moe_fwd_workspace_size(desc(), q8(), q8()) > 0


def test_no_tokens_and_workspace():
    assert call(desc(T=0), ws=None, ws_bytes=0) == abi.OK
    # h of at most E experts or T k choices, for T tokens
    assert abi.conv2d_moe_fwd_workspace_size(desc(), mat(), mat()) == 8 * 4 * 256 * 2
    assert abi.conv2d_moe_fwd_workspace_size(desc(T=1), mat(), mat()) == 2 * 256 * 2
    n = abi.conv2d_moe_fwd_workspace_size(desc(), q8(), q8())
    assert 8 * 4 * 256 + 4 * 128 < n < 8 * 4 * 256 * 2


def z(*shape, dtype=BF):
    return torch.zeros(*shape, dtype=dtype)


def experts(E, rows, cols):
    return ops.Q8(z(E, rows, cols, dtype=torch.float8_e4m3fn), z(E, rows // 128, cols // 128, dtype=torch.uint8), ops.TILE)


X, R, W1, W2 = z(3, 128), z(4, 128), z(4, 256, 128), z(4, 128, 256)
Q1, Q2 = experts(4, 256, 128), experts(4, 128, 256)
REFUSED = [
    (lambda: ops.moe_fwd(z(65, 128), R, W1, W2, 2), "x: at most 64 tokens"),
    (lambda: ops.moe_fwd(z(3, 128, dtype=FP), R, W1, W2, 2), "x: dtype"),
    (lambda: ops.moe_fwd(z(3, 126), z(4, 126), W1, W2, 2), "x: features in multiples of 8"),
    (lambda: ops.moe_fwd(z(3, 140)[:, :128], R, W1, W2, 2), "x: rows must start"),
    (lambda: ops.moe_fwd(X, z(4, 128, dtype=HF), W1, W2, 2), "router: dtype"),
    (lambda: ops.moe_fwd(X, z(4, 120), W1, W2, 2), "router: shape"),
    (lambda: ops.moe_fwd(X, z(257, 128), W1, W2, 2), "router: 1 to 256 experts"),
    (lambda: ops.moe_fwd(X, R, W1, W2, 0), "k: 1 to 16"),
    (lambda: ops.moe_fwd(X, R, W1, W2, 5), "k: 1 to 16"),
    (lambda: ops.moe_fwd(X, R, W1, W2, 2.0), "k: 1 to 16"),
    (lambda: ops.moe_fwd(X, R, W1, W2, 1 << 70), "k: 1 to 16"),
    (lambda: ops.moe_fwd(X, R, W1, z(512, 256), 2), "w2: expected experts"),
    (lambda: ops.moe_fwd(X, R, W1, z(4, 128, 252), 2), "w2: inner features in multiples of 8"),
    (lambda: ops.moe_fwd(X, R, z(4, 248, 128), W2, 2), "w1: shape"),
    (lambda: ops.moe_fwd(X, R, W1, W2, 2, gated=True), "w1: shape"),
    (lambda: ops.moe_fwd(X, R, z(4, 256, 128, dtype=HF), W2, 2), "w1: dtype"),
    (lambda: ops.moe_fwd(X, R, z(4, 128, 256).transpose(1, 2), W2, 2), "w1: features must be contiguous"),
    (lambda: ops.moe_fwd(X, R, z(8, 256, 128)[::2], W2, 2), "w1: features must be contiguous and the experts' rows"),
    (lambda: ops.moe_fwd(X, R, z(4, 256, 132)[:, :, :128], W2, 2), "w1: rows must start"),
    (lambda: ops.moe_fwd(X, R, Q1, W2, 2), "w1 and w2: both Q8"),
    (lambda: ops.moe_fwd(X, R, Q1._replace(group=128), Q2, 2), "w1: 8-bit experts have tiles"),
    (lambda: ops.moe_fwd(X, R, Q1._replace(scale=z(4, 1, 1, dtype=torch.uint8)), Q2, 2), "w1: scales are uint8 of shape"),
    (lambda: ops.moe_fwd(z(3, 144), z(4, 144), experts(4, 256, 144), experts(4, 144, 256), 2), "w1: 8-bit experts have whole tiles"),
    (lambda: ops.moe_fwd(X, R, W1, W2, 2, b1=z(4, 256)), "b1: expected a contiguous float32"),
    (lambda: ops.moe_fwd(X, R, W1, W2, 2, b2=z(4, 256, dtype=FP)), "b2: expected"),
    (lambda: ops.moe_fwd(X, R, W1, W2, 2, act="swish"), "act: one of"),
    (lambda: ops.moe_fwd(X, R, W1, W2, 2, residual=z(4, 128)), "residual: shape"),
    (lambda: ops.moe_fwd(X, R, W1, W2, 2, y=z(3, 128, dtype=HF)), "y: dtype"),
    (lambda: ops.moe_fwd(X, R, W1, W2, 2), "CUDA device memory"),
    (lambda: ops.moe_fwd(X, z(4, 128, dtype=FP), z(4, 512, 128), W2, 2, gated=True), "CUDA device memory"),
    (lambda: ops.moe_fwd(X, R, Q1, Q2, 2), "CUDA device memory"),
    (lambda: ops.moe_encode(z(4, 100, 128)), "w: experts by rows"),
    (lambda: ops.moe_encode(z(128, 128)), "w: experts by rows"),
]


@pytest.mark.parametrize("i", range(len(REFUSED)))
def test_binding_refuses_before_a_launch(i):
    run, why = REFUSED[i]
    with pytest.raises(ValueError, match=why.replace("(", r"\(")):
        run()
