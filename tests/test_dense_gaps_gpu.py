"""The dense layer's outputs as columns of wider buffers: what lies beside them stays as it was, wherever their rows end."""
import pytest
import torch

from conv2d_layer_gb300 import abi, ops

pytestmark = pytest.mark.gpu
BF, HF, FP = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(autouse=True)
def device_clean():
    yield
    assert abi.conv2d_device_status() == (abi.OK, 0)


def normal(seed, *shape, std=1.0, dtype=FP):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)


class Beside:
    """rows x cols of a buffer of row length ld, filled with 7 (and three rows of it behind)."""

    def __init__(self, rows, cols, ld, dtype):
        self.all = torch.full((rows + 3, ld), 7.0, device="cuda").to(dtype)
        self.rows, self.cols, self.t = rows, cols, self.all[:rows, :cols]

    def kept(self):
        v = self.all.float()
        return bool((v[self.rows:] == 7).all()) and bool((v[:, self.cols:] == 7).all())


def up(n, to):
    return -(-n // to) * to


SIZES = [(2560, 11, 2485, HF), (485, 15, 15, BF), (896, 7, 448, HF), (485, 15, 24, BF), (3000, 7, 3001, BF), (2048, 520, 1030, BF),
         (1500, 2049, 700, HF), (600, 1001, 2003, BF), (5000, 100, 260, BF), (4, 100, 77, BF), (300, 65, 33, HF)]


@pytest.mark.parametrize("M,K,N,dtype", SIZES)
@pytest.mark.parametrize("act,save", [("identity", "none"), ("sigmoid", "full"), ("gelu", "q8")])
@pytest.mark.parametrize("operands", ["halves", "rows", "blocks"])
def test_forward(M, K, N, dtype, act, save, operands):
    x, w = normal(1, M, K, dtype=dtype), normal(2, N, K, std=K ** -0.5, dtype=dtype)
    if operands != "halves":
        x, w = (ops.q8_encode(x, 0), ops.q8_encode(w, 0)) if operands == "rows" else (ops.q8_encode(x, 128), ops.q8_encode(w, ops.TILE))
    bias, res = normal(3, N), normal(4, M, N, dtype=dtype)
    want, wz = ops.dense_fwd(x, w, bias, act, residual=res, save=save, dtype=dtype)
    for more in (0, 8):
        y, z = Beside(M, N, up(N, 8) + more, dtype), None
        if save == "full":
            z = Beside(M, N, up(N, 8) + more, dtype)
        elif save == "q8":
            z = Beside(M, N, up(N, 16) + 2 * more, torch.float8_e4m3fn)
        pre = None if z is None else ops.Q8(z.t, torch.empty_like(wz.scale), 32) if save == "q8" else z.t
        ops.dense_fwd(x, w, bias, act, residual=res, save=save, dtype=dtype, y=y.t, pre_act=pre)
        assert y.kept() and torch.equal(y.t, want)
        if save == "full":
            assert z.kept() and torch.equal(z.t, wz)
        elif save == "q8":
            assert z.kept() and torch.equal(z.t.float(), wz.q.float()) and torch.equal(pre.scale, wz.scale)


@pytest.mark.parametrize("M,K,N,dtype", SIZES + [(9000, 30, 1001, BF), (20000, 1003, 130, BF)])
@pytest.mark.parametrize("tiles", [False, True])
def test_backward(M, K, N, dtype, tiles):
    x, w, dy = normal(1, M, K, dtype=dtype), normal(2, N, K, std=K ** -0.5, dtype=dtype), normal(3, M, N, dtype=dtype)
    w = ops.q8_encode(w, ops.TILE) if tiles else w
    for grad in (FP, dtype):
        wx, ww, wb = ops.dense_bwd(x, w, dy, grad_dtype=grad)
        for more in (0, 8):
            dx, dw = Beside(M, K, up(K, 8) + more, dtype), Beside(N, K, up(K, 4 if grad == FP else 8) + more, grad)
            db = torch.zeros(N, device="cuda")
            dw.t.zero_()
            ops.dense_bwd(x, w, dy, dx=dx.t, dw=dw.t, dbias=db)
            assert dx.kept() and dw.kept()
            assert torch.equal(dx.t, wx) and torch.equal(dw.t, ww) and torch.equal(db, wb)


@pytest.mark.parametrize("N", [33, 260, 1001])
def test_two_layers_side_by_side(N):
    """Two products into neighbouring columns of one buffer, the left one last."""
    M, K = 3000, 256
    x, w = normal(1, M, K, dtype=BF), normal(2, 2 * N, K, std=1 / 16, dtype=BF)
    left, right = up(N, 8), N  # rows of the right one start on a boundary
    both = torch.empty(M, left + up(right, 8), device="cuda", dtype=BF)
    a, b = both[:, :N], both[:, left:left + right]
    ops.dense_fwd(x, w[N:].clone(), act="sigmoid", y=b)
    ops.dense_fwd(x, w[:N].clone(), act="sigmoid", y=a)
    assert torch.equal(a, ops.dense_fwd(x, w[:N].clone(), act="sigmoid")[0])
    assert torch.equal(b, ops.dense_fwd(x, w[N:].clone(), act="sigmoid")[0])
