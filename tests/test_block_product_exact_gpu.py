"""Products of 8-bit operands with a scale for each block of 128, on whole numbers whose sums are exact: a scale that a
product took for another would show in the bits."""
import pytest
import torch

from conv2d_layer_gb300 import abi, ops

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(autouse=True)
def device_clean():
    yield
    assert abi.conv2d_device_status() == (abi.OK, 0)


def whole(rows, cols, group, seed):
    """(Q8, its values): -1, 0 and 1 with scales of 1, 2 and 4 that differ from block to block."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    v = torch.randint(-1, 2, (rows, cols), generator=g, device="cuda")
    tall = 128 if group == ops.TILE else 1
    down, across = -(-rows // tall), -(-cols // 128)
    e = (torch.randint(0, 3, (down, 1), generator=g, device="cuda") + torch.arange(across, device="cuda")) % 3
    q = ops.Q8(v.to(torch.float8_e4m3fn), (e + 127).to(torch.uint8), group)
    return q, v.double() * torch.exp2(e.double()).repeat_interleave(tall, 0).repeat_interleave(128, 1)[:rows, :cols]


# Several units a CTA pair with numbers of k-blocks on either side of the ring's; long sums of a few rows in clusters.
@pytest.mark.parametrize("wgroup", [128, ops.TILE])
@pytest.mark.parametrize("M,K,N", [(4096, 640, 4480), (4096, 1152, 4480), (4000, 1100, 4500), (4096, 1664, 4480), (4096, 2176, 2304),
                                   (3000, 768, 5000), (2600, 8192, 2048), (64, 16384, 512), (64, 16000, 128), (20, 9088, 640),
                                   (128, 6272, 256), (1, 16384, 256)])
def test_sums_of_whole_numbers(M, K, N, wgroup):
    x, x64 = whole(M, K, 128, 1)
    w, w64 = whole(N, K, wgroup, 2)
    # |sum| <= 16 K < 2^19: exact in fp32, whatever the order
    want = (x64 @ w64.t()).to(torch.float32).to(BF)
    for _ in range(3):
        y, _ = ops.dense_fwd(x, w, dtype=BF)
        assert torch.equal(y, want)


@pytest.mark.parametrize("M,K,N", [(4096, 4480, 1152), (4000, 4500, 1100), (4096, 2304, 1664), (3000, 5000, 640), (64, 512, 16384)])
def test_gradients_of_whole_numbers(M, K, N):
    w, w64 = whole(N, K, ops.TILE, 3)
    # dy is taken to 8 bits: whole numbers up to 15 times the power of two of their block, 0 and 1 times it among them
    g = torch.Generator(device="cuda").manual_seed(4)
    e = torch.arange(-(-N // 128), device="cuda") % 3
    dy = torch.randint(-1, 2, (M, N), generator=g, device="cuda") * torch.exp2(e.float()).repeat_interleave(128)[:N]
    dx, _, _ = ops.dense_bwd(None, w, dy.to(BF), need_dw=False, need_dbias=False)
    assert torch.equal(dx, (dy.double() @ w64).to(torch.float32).to(BF))
