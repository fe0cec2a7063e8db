"""The residual block's calls without a GPU, where a plan or a rule changes: workspace sizes, streams, stale 8-bit
weights."""
import contextlib
import ctypes
import subprocess

import pytest
import torch

from conv2d_layer_gb300 import abi, ops
from conv2d_layer_gb300.block import FeedForward

P = 1 << 20  # stands for an aligned device pointer: never read, every call below is sized or refused


def mat(type=abi.BF16, ld=0):
    return abi.Mat(P, ld, type, 0, None)


def q8(group=32, ld=0):
    return abi.Mat(P, ld, abi.E4M3, group, P)


def dense(M, K, N, act=abi.ACT_IDENTITY, dtype=abi.BF16):
    return abi.DenseDesc(M, K, N, act, dtype, 0)


@pytest.mark.parametrize("d,x,w", [
    (dense(1, 128, 8), q8(), mat()),                     # one token in groups of 32, decoded
    (dense(4, 128, 1), mat(), q8()),                     # one output feature, decoded
    (dense(2, 64, 8), mat(ld=65), mat()),                # two rows, moved to 16-byte boundaries
    (dense(1, 100, 2), q8(0, ld=112), q8(0)),            # 8-bit operands, one of them moved
    (dense(1, 1, 1), mat(), mat(ld=8)),
])
def test_a_copy_of_any_size_shows_in_the_workspace(d, x, w):
    """256 says that nothing is kept (no workspace need be handed in), so the smallest copy makes it more."""
    assert abi.conv2d_dense_fwd_workspace_size(d, x, w) > 256
    n = abi.conv2d_dense_fwd_workspace_size(d, x, w)
    assert abi.conv2d_dense_fwd_workspace_size(dense(d.M, 128, d.N), mat(), mat()) == 256 < n


@pytest.mark.parametrize("dtype,M,planes", [(abi.FP16, 16384, 0), (abi.FP16, 16448, 2), (abi.FP16, 200704, 13),
                                            (abi.BF16, 131072, 0), (abi.BF16, 200704, 2), (abi.BF16, 1000000, 8)])
def test_a_16_bit_dw_over_very_many_rows_is_summed_in_pieces(dtype, M, planes):
    """One accumulator sums at most 16,384 rows (fp16) or 131,072 (bf16): what it truncates stays below the rounding.
    Longer sums have an fp32 plane in the workspace for each piece (here the product fills the GPU by itself)."""
    d, m = dense(M, 2048, 2048, dtype=dtype), mat(dtype)
    n = abi.conv2d_dense_bwd_workspace_size(d, m, m, None, m, None, m, None)
    assert n // (2048 * 2048 * 4) == planes
    # partials of more than 2 GB: one plane, added to pass by pass
    d = dense(M, 16384, 16384, dtype=dtype)
    n = abi.conv2d_dense_bwd_workspace_size(d, m, m, None, m, None, m, None)
    one = 16384 * 16384 * 4
    assert n < one // 2 if planes == 0 else planes * one <= n < (planes + 1) * one if planes == 2 else one <= n < 2 * one


class OnDevice:
    """Stands for a tensor or a stream of a device that this machine lacks."""

    def __init__(self, device):
        self.device = torch.device(device)


@pytest.fixture
def streams(monkeypatch):
    """The streams made current around a call, as (pointer or object, device)."""
    seen = []

    class Binding:
        def q8_encode(self, x, group, out):
            return None

        def dense_bwd(self, *a):
            return None, None, None

    @contextlib.contextmanager
    def current(s):
        seen.append(s)
        yield

    monkeypatch.setattr(ops, "_binding", lambda: Binding())
    monkeypatch.setattr(torch.cuda, "stream", current)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda p, device=None: (p, device))
    return seen


def test_a_raw_stream_belongs_to_the_tensors_device(streams):
    ops.q8_encode(OnDevice("cuda:1"), stream=1234)
    ops.q8_encode(ops.Q8(OnDevice("cuda:2"), None), stream=5)
    # the first argument may be left out; the device is that of the first tensor there is
    ops.dense_bwd(None, None, dy=OnDevice("cuda:3"), need_dx=False, need_dw=False, stream=6)
    assert streams == [(1234, torch.device("cuda:1")), (5, torch.device("cuda:2")), (6, torch.device("cuda:3"))]


def test_a_stream_of_another_device_is_refused(streams):
    s = OnDevice("cuda:1")
    ops.q8_encode(OnDevice("cuda:1"), stream=s)
    assert streams == [s]
    with pytest.raises(ValueError, match="stream: of cuda:1, but the tensors are on cuda:0"):
        ops.q8_encode(OnDevice("cuda:0"), stream=s)
    assert streams == [s]


FAKE = """
#include <stddef.h>
int asked = 0;
size_t conv2d_rms_norm_bwd_workspace_size(long long rows, int cols) { ++asked; return 256; }
size_t conv2d_dense_fwd_workspace_size() { ++asked; return 256; }
size_t conv2d_dense_bwd_workspace_size() { ++asked; return 256; }
int conv2d_q8_encode() { return 1; }
int conv2d_q8_decode() { return 1; }
int conv2d_rms_norm_fwd() { return 1; }
int conv2d_rms_norm_bwd() { return 1; }
int conv2d_dense_fwd() { return 1; }
int conv2d_dense_bwd() { return 1; }
"""


def test_sizes_are_asked_for_on_the_tensors_device(tmp_path):
    """A workspace is sized for the current device (its SMs), so the library is asked only once the tensors' device
    has been made current: not at all for tensors that are refused before that. The library is a stand-in that counts."""
    src, path = tmp_path / "fake.c", str(tmp_path / "fake.so")
    src.write_text(FAKE)
    subprocess.run(["gcc", "-shared", "-fPIC", "-o", path, str(src)], check=True)
    h, gamma, inv = torch.zeros(4, 8), torch.ones(8), torch.ones(4)
    binding = ops._binding()
    binding.init(path)
    try:
        for call in (lambda: ops.rms_norm_bwd(h, gamma, inv, h), lambda: ops.dense_bwd(h.bfloat16(), h.bfloat16(), torch.zeros(4, 4).bfloat16()),
                     lambda: ops.dense_fwd(h.bfloat16(), h.bfloat16())):
            with pytest.raises(ValueError, match="CUDA device memory"):
                call()
    finally:
        binding.init(abi.lib_path())
    assert ctypes.c_int.in_dll(ctypes.CDLL(path), "asked").value == 0


def feed_forward(**kw):
    n = lambda *s: torch.randn(*s, generator=torch.Generator().manual_seed(0))  # noqa: E731
    return FeedForward(n(16), n(32, 16), n(32), n(16, 32), n(16), device="cpu", **kw)


def change_in_place(ff):
    ff.w1.mul_(2)


def change_by_assignment(ff):
    ff.w2 = ff.w2.clone()


@pytest.mark.parametrize("change", [change_in_place, change_by_assignment])
def test_8_bit_weights_are_not_served_once_the_weights_have_changed(monkeypatch, change):
    monkeypatch.setattr(ops, "q8_encode", lambda t, group: ("8-bit", t, group))
    ff, x = feed_forward(), torch.zeros(2, 16).bfloat16()
    ff.quantize()
    with pytest.raises(ValueError, match="CUDA device memory"):  # taken: the kernels are reached
        ff.fwd_infer(x, bits8=True)
    change(ff)
    with pytest.raises(RuntimeError, match="quantize"):
        ff.fwd_infer(x, bits8=True)
    ff.quantize()
    with pytest.raises(ValueError, match="CUDA device memory"):
        ff.fwd_infer(x, bits8=True)


def test_weights_made_in_inference_mode_can_be_quantized(monkeypatch):
    """Such tensors have no version; another tensor in their place is still seen."""
    monkeypatch.setattr(ops, "q8_encode", lambda t, group: ("8-bit", t, group))
    with torch.inference_mode():
        ff = feed_forward()
        ff.quantize()
        with pytest.raises(ValueError, match="CUDA device memory"):
            ff.fwd_infer(torch.zeros(2, 16).bfloat16(), bits8=True)
        change_by_assignment(ff)
        with pytest.raises(RuntimeError, match="quantize"):
            ff.fwd_infer(torch.zeros(2, 16).bfloat16(), bits8=True)


@pytest.mark.parametrize("dtype", [torch.float32, torch.float64, torch.int8])
def test_feed_forward_refuses_types_its_dense_layers_lack(dtype):
    with pytest.raises(ValueError, match="dtype: torch.bfloat16 or torch.float16"):
        feed_forward(dtype=dtype)
    assert feed_forward(dtype=torch.float16).w1.dtype == torch.float16
