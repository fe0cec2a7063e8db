"""The residual block's operators on several streams at once, of several sizes: the bits that they give alone."""
import threading

import pytest
import torch

from conv2d_layer_gb300 import abi, ops

pytestmark = pytest.mark.gpu
BF, HF, FP = torch.bfloat16, torch.float16, torch.float32


def normal(seed, *shape, std=1.0, dtype=FP):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)


def flat(o):
    if isinstance(o, torch.Tensor):
        return [o.view(torch.uint8) if o.dtype == torch.float8_e4m3fn else o]
    return [t for p in o for t in flat(p)] if isinstance(o, (tuple, list)) else []


def calls():
    """Functions of a stream; each makes its own outputs."""
    made = []
    for i, (M, K, N) in enumerate([(1, 4096, 512), (24, 8192, 256), (70, 640, 384), (2000, 512, 1024)]):
        x, w, dy = normal(10 * i, M, K, dtype=BF), normal(10 * i + 1, N, K, std=K ** -0.5, dtype=BF), normal(10 * i + 2, M, N, dtype=BF)
        for g, h in ((128, ops.TILE), (0, 0)):
            a, b = ops.q8_encode(x, g), ops.q8_encode(w, h)
            made.append(lambda s, a=a, b=b: ops.dense_fwd(a, b, act="gelu", save="full", dtype=BF, stream=s))
            made.append(lambda s, a=a, b=b, dy=dy: ops.dense_bwd(a, b, dy, stream=s))
        made.append(lambda s, x=x, w=w: ops.dense_fwd(x, w, act="silu", save="q8", stream=s))
    for i, (T, D, F, E, k) in enumerate([(1, 1024, 512, 16, 4), (16, 2048, 256, 8, 2), (64, 256, 1024, 6, 2), (40, 512, 128, 64, 8)]):
        x, r = normal(50 + i, T, D, dtype=BF), normal(60 + i, E, D, std=D ** -0.5)
        w1, w2 = normal(70 + i, E, 2 * F, D, std=D ** -0.5, dtype=BF), normal(80 + i, E, D, F, std=F ** -0.5, dtype=BF)
        for a, b in ((w1, w2), (ops.moe_encode(w1), ops.moe_encode(w2))):
            made.append(lambda s, x=x, r=r, a=a, b=b, k=k: ops.moe_fwd(x, r, a, b, k, gated=True, residual=x, stream=s))
    for i, (r, c) in enumerate([(3, 4096), (500, 1021), (300, 8224), (2000, 768)]):
        x, dy, g = normal(90 + i, r, c, dtype=BF), normal(95 + i, r, c, dtype=BF), normal(99, c)

        def norm(s, x=x, dy=dy, g=g):
            o = ops.layer_norm_fwd(x, g, group=128, residual=dy, stream=s)
            return o, ops.layer_norm_bwd(o.h, g, o.mean, o.inv_std, dy, dh=dy, stream=s)

        made.append(norm)
    return made


def test_all_at_once():
    made = calls()
    want = [[t.clone() for t in flat(f(None))] for f in made]
    torch.cuda.synchronize()
    wrong = []

    def work(n):
        try:
            stream = torch.cuda.Stream()
            for rnd in range(6):
                order = [(n * 7 + rnd * 5 + j * 11) % len(made) for j in range(len(made))]  # all of them, from elsewhere each time
                got = [(i, flat(made[i](stream))) for i in order]
                stream.synchronize()
                with torch.cuda.stream(stream):
                    wrong.extend(i for i, o in got if not all(torch.equal(a, b) for a, b in zip(want[i], o)))
        except Exception as e:  # noqa: BLE001 (a thread's failure is the test's)
            wrong.append(repr(e))

    threads = [threading.Thread(target=work, args=(n,)) for n in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong
    assert abi.conv2d_device_status() == (abi.OK, 0)
