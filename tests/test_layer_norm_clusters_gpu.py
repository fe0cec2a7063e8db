"""Layer norm's backward where a cluster of CTAs shares a row and brings its rows through a ring in shared memory, many
times round it: each row's dh is its own."""
import pytest
import torch

from block_ref import U
from conv2d_layer_gb300 import abi, ops

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def device_clean():
    yield
    assert abi.conv2d_device_status() == (abi.OK, 0)


@pytest.mark.parametrize("rows,cols,dtype", [(2500, 8224, torch.bfloat16), (2500, 16384, torch.float16), (1300, 32768, torch.bfloat16),
                                             (2500, 8211, torch.bfloat16), (1300, 20003, torch.float16), (1500, 9216, torch.float32)])
def test_rows_keep_their_own_gradient(rows, cols, dtype):
    g = torch.Generator(device="cuda").manual_seed(cols)
    h, dy = (torch.randn(rows, cols, generator=g, device="cuda").to(dtype) for _ in range(2))
    gamma = torch.randn(cols, generator=g, device="cuda")
    mean, inv = torch.zeros(rows, device="cuda"), torch.ones(rows, device="cuda")
    plain, dg, db = ops.layer_norm_bwd(h, gamma, mean, inv, dy)
    # 1 to 8, by the row and the column's 128: a value of another row or place is off by 1 at least
    dh = (1 + (torch.arange(rows, device="cuda")[:, None] * 3 + torch.arange(cols, device="cuda") // 128) % 8).to(dtype)
    first = None
    for _ in range(5):
        dx, g2, b2 = ops.layer_norm_bwd(h, gamma, mean, inv, dy, dh=dh)
        # dx and plain are rounded once each, of values up to |plain| + 8
        off = (dx.double() - plain.double() - dh.double()).abs()
        assert bool((off <= 2.01 * U[dtype] * (plain.double().abs() + 8) + 1e-6).all())
        assert torch.equal(g2, dg) and torch.equal(b2, db)
        first = dx if first is None else first
        assert torch.equal(dx, first)
