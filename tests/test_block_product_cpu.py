"""The dense layer on 8-bit operands with a scale for each block of 128, without a GPU: which operands are taken as they
are, workspace sizes, refusals."""
import pytest
import torch

from conv2d_layer_gb300 import abi, ops

P = 1 << 20  # stands for an aligned device pointer: never read, every call below is refused or sized
BAD = abi.ERR_INVALID_ARG
BF, HF, FP = torch.bfloat16, torch.float16, torch.float32


def mat(type=abi.BF16, ld=0):
    return abi.Mat(P, ld, type, 0, None)


def q8(group, ld=0, scale=P):
    return abi.Mat(P, ld, abi.E4M3, group, scale)


def dense(M=8, K=64, N=32, act=abi.ACT_IDENTITY, dtype=abi.BF16):
    return abi.DenseDesc(M, K, N, act, dtype, 0)


def size(x, w, **kw):
    return abi.conv2d_dense_fwd_workspace_size(dense(**kw), x, w)


def test_operands_taken_as_they_are():
    """256: nothing is copied or decoded."""
    for w in (128, abi.TILE):
        assert size(q8(128), q8(w)) == 256
        assert size(q8(128, ld=64), q8(w), K=60) > 256  # w's rows of 60 bytes are moved to 16-byte boundaries
        assert size(q8(128, ld=64), q8(w, ld=80), K=60) == 256
    # other pairs are decoded: two copies of 16 bits
    for x, w in ((abi.TILE, abi.TILE), (128, 0), (0, 128), (128, 32), (32, abi.TILE), (0, abi.TILE)):
        assert size(q8(x), q8(w), M=256, N=256) >= 2 * 256 * 64 * 2
    assert 128 * 64 * 2 <= size(mat(), q8(abi.TILE), M=256, N=128) < 256 * 64 * 2


def test_gradients_of_tiled_weights():
    x, w, dy = q8(128), q8(abi.TILE), mat()
    d = dense(M=256, K=64, N=128)
    # dx: dy in 8 bits with its scales, the weights as they are; nothing in 16 bits
    n = abi.conv2d_dense_bwd_workspace_size(d, None, w, None, dy, mat(), None, None)
    assert 256 * 128 + 256 <= n < 256 * 128 * 2
    # weights with a scale for each row are decoded, dy is taken as it is
    n = abi.conv2d_dense_bwd_workspace_size(d, None, q8(128), None, dy, mat(), None, None)
    assert n == 128 * 64 * 2
    # dW: x is decoded
    assert abi.conv2d_dense_bwd_workspace_size(d, x, None, None, dy, None, mat(), None) == 256 * 64 * 2
    assert abi.conv2d_dense_bwd_workspace_size(d, q8(abi.TILE), None, None, dy, None, mat(), None) == 256 * 64 * 2


@pytest.mark.parametrize("change", [dict(x=q8(64)), dict(w=q8(-1)), dict(w=q8(abi.TILE, scale=None)), dict(z=q8(128)),
                                    dict(z=q8(abi.TILE)), dict(y=q8(128)), dict(residual=q8(128)), dict(x=q8(128, ld=60))])
def test_forward_refusals(change):
    a = dict(x=q8(128), w=q8(abi.TILE), z=None, y=mat(), residual=None)
    a.update(change)
    assert abi.conv2d_dense_fwd(dense(), a["x"], a["w"], None, a["residual"], a["z"], a["y"], P, 1 << 40, stream=0) == BAD


@pytest.mark.parametrize("change", [dict(dy=q8(128)), dict(z=q8(128)), dict(z=q8(abi.TILE)), dict(w=q8(96)), dict(x=q8(256)),
                                    dict(dx=q8(128)), dict(dw=q8(128))])
def test_backward_refusals(change):
    a = dict(x=q8(128), w=q8(abi.TILE), z=mat(), dy=mat(), dx=mat(), dw=mat())
    a.update(change)
    d = dense(act=abi.ACT_GELU)
    assert abi.conv2d_dense_bwd(d, a["x"], a["w"], a["z"], a["dy"], a["dx"], a["dw"], None, P, 1 << 40, stream=0) == BAD


def test_binding_refusals():
    def q(rows, cols, group):
        return ops.q8_empty(rows, cols, group, device="cpu")

    z = lambda *s: torch.zeros(*s, dtype=BF)  # noqa: E731
    for call, why in (
            (lambda: ops.dense_fwd(q(4, 200, 128), q(3, 200, ops.TILE)), "dtype: bfloat16 or float16"),
            (lambda: ops.dense_fwd(q(4, 200, 128), q(3, 201, ops.TILE), dtype=BF), "w: shape"),
            (lambda: ops.dense_fwd(q(4, 200, 128), q(300, 200, ops.TILE)._replace(scale=q(4, 200, 128).scale), dtype=BF),
             r"w: scales are uint8 of shape \(3, 2\)"),
            (lambda: ops.dense_fwd(q(4, 200, 128), q(3, 200, ops.TILE), dtype=BF, save="q8", pre_act=q(4, 3, 128)), "pre_act: groups of 32"),
            (lambda: ops.dense_bwd(q(4, 200, 128), q(3, 200, ops.TILE), z(4, 3), q(4, 3, 128), "relu"), "pre_act: groups of 32"),
            (lambda: ops.dense_fwd(q(4, 200, 128), q(3, 200, ops.TILE), dtype=BF), "CUDA device memory"),
            (lambda: ops.dense_bwd(q(4, 200, 128), q(3, 200, ops.TILE), z(4, 3)), "CUDA device memory")):
        with pytest.raises(ValueError, match=why):
            call()
