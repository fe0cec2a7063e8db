"""The residual block's operators where a plan changes: one small copy in the workspace, accumulation into 16-bit
gradients by each kernel, sums over very many rows."""
import pytest
import torch

from block_ref import STEP, close, q8_values, rounded
from conv2d_layer_gb300 import abi, ops

pytestmark = pytest.mark.gpu
BF, HF, FP = torch.bfloat16, torch.float16, torch.float32


def normal(seed, *shape, std=1.0, dtype=FP):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)


@pytest.fixture(autouse=True)
def device_clean():
    yield
    assert abi.conv2d_device_status() == (abi.OK, 0)


def padded(t, ld):
    """The same values in rows of ld elements."""
    wide = torch.zeros(t.shape[0], ld, device="cuda", dtype=torch.uint8 if t.dtype == torch.float8_e4m3fn else t.dtype)
    wide = wide.view(t.dtype)
    wide.view(torch.uint8)[:, :t.shape[1] * t.element_size()] = t.contiguous().view(torch.uint8).view(t.shape[0], -1)
    return wide[:, :t.shape[1]]


def one_copy(kind):
    """(x, w) of which exactly one has to be copied, into 256 bytes or fewer."""
    if kind == "token in groups of 32":
        return ops.q8_encode(normal(1, 1, 128), 32), normal(2, 8, 128, dtype=BF)
    if kind == "one output in 8 bits":
        return normal(1, 4, 128, dtype=BF), ops.q8_encode(normal(2, 1, 128), 32)
    if kind == "two strided rows":
        return padded(normal(1, 2, 64, dtype=BF), 65), normal(2, 8, 64, dtype=BF)
    x, w = ops.q8_encode(normal(1, 1, 100), 0), ops.q8_encode(normal(2, 8, 100), 0)
    return x, ops.Q8(padded(w.q, 112), w.scale, 0)  # 8-bit operands, one of them in rows of 100 bytes


@pytest.mark.parametrize("kind", ["token in groups of 32", "one output in 8 bits", "two strided rows", "ragged 8 bits"])
def test_dense_fwd_with_one_small_copy(kind):
    x, w = one_copy(kind)
    y, _ = ops.dense_fwd(x, w, dtype=BF)
    x64, w64 = (q8_values(t) if isinstance(t, ops.Q8) else t.double() for t in (x, w))
    ref = x64 @ w64.t()
    # one truncated addition for 16 products and up to 20 joins
    err = (x64.shape[1] / 16 + 20) * STEP * (x64.abs() @ w64.abs().t())
    close(y, ref, rounded(ref, BF, err), kind)
