"""The residual block's operators where a plan changes: one small copy in the workspace, accumulation into 16-bit
gradients by each kernel, sums over very many rows."""
import pytest
import torch

from block_ref import STEP, close, q8_values, rounded
from conv2d_layer_gb300 import abi, ops
from conv2d_layer_gb300.block import FeedForward

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


@pytest.mark.parametrize("M,K,N,dtype", [
    (512, 2048, 2048, BF),    # whole units of the pair kernel, rows on 16-byte boundaries
    (512, 2048, 2048, HF),
    (500, 2050, 2000, HF),    # rows on 4-byte boundaries, ragged units
    (512, 2049, 2048, BF),    # rows on 2-byte boundaries
    (4096, 2600, 2048, BF),   # a last wave cut along k
    (100, 136, 72, BF),       # the cluster kernel
    (100, 137, 72, HF),
    (20000, 256, 256, HF),    # splits and their join
])
def test_accumulating_into_a_16_bit_dw_rounds_once(M, K, N, dtype):
    x, dy = normal(1, M, K, dtype=dtype), normal(2, M, N, dtype=dtype)
    old = normal(3, N, K, std=M ** 0.5, dtype=dtype)
    dw = old.clone()
    ops.dense_bwd(x, None, dy, need_dx=False, need_dbias=False, dw=dw)
    x64, dy64 = x.double(), dy.double()
    ref = old.double() + dy64.t() @ x64
    # what the fp32 sums lose (one truncated addition for 16 rows, up to 20 joins) and the fp32 addition of the old
    # value; then one rounding of the result
    extra = (M / 16 + 20) * STEP * (dy64.abs().t() @ x64.abs()) + STEP * old.double().abs()
    close(dw, ref, rounded(ref, dtype, extra), "dw")


@pytest.mark.parametrize("K,N", [(2048, 2048), (64, 40)])
def test_accumulated_fp16_sums_may_pass_the_type_on_the_way(K, N):
    """A product beyond 65504 onto an old value that brings it back."""
    x, dy = torch.full((64, K), 40.0, device="cuda", dtype=HF), torch.full((64, N), 32.0, device="cuda", dtype=HF)
    dw = torch.full((N, K), -60000.0, device="cuda", dtype=HF)
    ops.dense_bwd(x, None, dy, need_dx=False, need_dbias=False, dw=dw)
    assert torch.equal(dw, torch.full_like(dw, 64 * 40 * 32 - 60000))  # 21920: every sum on the way is exact


def test_fp16_dw_over_very_many_rows():
    """400,000 rows of positive terms: what the accumulators truncate must stay below the type's rounding.

    The mean relative error of n elements is what truncation leaves (it always points down) and the mean of n
    roundings of half a step at most each. Held to half of fp16's half step, 2^-12, and three standard deviations of
    that mean (half a step 2^-11, spread evenly: / sqrt(3 n))."""
    M, K, N = 400000, 2048, 2048
    g = torch.Generator(device="cuda").manual_seed(7)
    x = torch.rand(M, K, generator=g, device="cuda", dtype=HF)
    dy = torch.rand(M, N, generator=g, device="cuda", dtype=HF) * 0.25
    _, dw, _ = ops.dense_bwd(x, None, dy, need_dx=False, need_dbias=False, grad_dtype=HF)
    n = 64
    ref = dy[:, :n].double().t() @ x[:, :n].double()
    rel = (dw[:n, :n].double() - ref) / ref
    assert float(rel.mean().abs()) < 2.0 ** -12 + 3 * 2.0 ** -11 / (3 * n * n) ** 0.5
    assert float(rel.abs().max()) < 2.0 ** -11 + 2.0 ** -12


@pytest.mark.parametrize("accumulate", [False, True])
def test_fp16_dw_in_passes(accumulate):
    """Pieces whose partials would take more than 2 GB: one after the other onto one fp32 plane, rounded once."""
    M, K, N = 33000, 16384, 16128
    g = torch.Generator(device="cuda").manual_seed(8)
    x = torch.rand(M, K, generator=g, device="cuda", dtype=HF) - 0.5
    dy = torch.rand(M, N, generator=g, device="cuda", dtype=HF) - 0.5
    old = torch.rand(N, K, generator=g, device="cuda", dtype=HF) * 40 if accumulate else None
    dw = old.clone() if accumulate else None
    out = ops.dense_bwd(x, None, dy, need_dx=False, need_dbias=False, grad_dtype=HF, dw=dw)[1]
    assert out is dw or not accumulate
    n = 192
    for r, c in ((slice(0, n), slice(0, n)), (slice(N - n, N), slice(K - n, K))):
        ref = dy[:, r].double().t() @ x[:, c].double()
        mag = dy[:, r].double().abs().t() @ x[:, c].double().abs()
        # a pass adds 1,024 MMAs, each truncated; three passes are joined, then the old value
        extra = (1024 + 20 + 3) * STEP * mag
        if accumulate:
            ref = ref + old[r, c].double()
            extra = extra + STEP * old[r, c].double()
        close(out[r, c], ref, rounded(ref, HF, extra), "dw")


@pytest.mark.parametrize("M,N", [(3, 200), (2048, 4096)])
@pytest.mark.parametrize("up,down", [(118, -118), (-118, 118)])
def test_8_bit_scales_far_from_one(M, N, up, down):
    """Scales of either operand near the ends of their range: only their product is applied to the sums."""
    x, w = normal(1, M, 64).abs(), normal(2, N, 64).abs()
    near, _ = ops.dense_fwd(ops.q8_encode(x, 0), ops.q8_encode(w, 0), dtype=BF)
    far, _ = ops.dense_fwd(ops.q8_encode(x * 2.0 ** up, 0), ops.q8_encode(w * 2.0 ** down, 0), dtype=BF)
    assert torch.equal(near, far)


def test_on_a_raw_stream():
    x = normal(1, 300, 256, dtype=BF)
    want = ops.q8_encode(x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = ops.q8_encode(x, stream=side.cuda_stream)
    side.synchronize()
    assert torch.equal(got.scale, want.scale) and torch.equal(got.q.view(torch.uint8), want.q.view(torch.uint8))


def test_8_bit_weights_follow_the_weights():
    w1, w2 = normal(1, 64, 32, std=0.2), normal(2, 32, 64, std=0.2)
    make = lambda w: FeedForward(torch.ones(32), w, torch.zeros(64), w2, torch.zeros(32))  # noqa: E731
    ff, x = make(w1), normal(3, 5, 32, dtype=BF)
    ff.quantize()
    before = ff.fwd_infer(x, bits8=True)[0]
    ff.w1.mul_(-1)
    with pytest.raises(RuntimeError, match="quantize"):
        ff.fwd_infer(x, bits8=True)
    ff.quantize()
    other = make(-w1)
    other.quantize()
    after = ff.fwd_infer(x, bits8=True)[0]
    assert torch.equal(after, other.fwd_infer(x, bits8=True)[0]) and not torch.equal(after, before)
