"""Calls with adapters, back to back on one stream, without a wait of the host
between them: kernels that start beside the adapters' products read what the
kernels before those products wrote (prescaled activations, act, d gate and d
up). Each call's input is written on the stream just before it, so a kernel that
reads too early sees another call's values. The results have to be the bytes of
the same calls with the device idle in between."""
import numpy as np
import pytest

import weight_quantized_swiglu_gb300 as q
from helpers import bits_from_dev, to_dev
from test_gpu_lora import adapter, on_device, scaled_case, x_of

pytestmark = pytest.mark.gpu

CALLS = 12


@pytest.fixture(scope="module")
def torch(cuda_available):
    import torch
    from weight_quantized_swiglu_gb300 import build
    build.build()
    return torch


@pytest.mark.parametrize("fmt,K,I,M", [("nvfp4", 256, 512, 9), ("nvfp4", 256, 512, 17), ("fp8", 256, 512, 40),
                                       ("nvfp4", 1280, 2560, 61), ("fp8", 1280, 2560, 64), ("nvfp4", 1280, 2560, 130),
                                       ("nvfp4", 256, 512, 1), ("nvfp4", 1280, 2560, 5)])
def test_serving_calls_in_a_row(torch, fmt, K, I, M):
    rng = np.random.default_rng(M)
    mlp = q.QuantMLP.from_case(scaled_case(fmt, K, I, 61), max_M=max(M, 17))
    lora = q.LoraMLP(mlp, 3, 16)
    for s in range(3):
        lora.set(s, on_device(torch, adapter(rng, K, I, 16), 1.0))
    xs = [to_dev(x_of(rng, M, K)[0] ^ np.uint16(k & 1) * np.uint16(0x8000)) for k in range(CALLS)]
    ids = [torch.from_numpy(rng.integers(-1, 3, M).astype(np.int32)).cuda() for _ in range(CALLS)]
    x, at = torch.empty_like(xs[0]), torch.empty_like(ids[0])
    want = []
    for k in range(CALLS):
        out = torch.empty_like(x)
        torch.cuda.synchronize()
        lora.forward(xs[k], ids[k], out)
        torch.cuda.synchronize()
        want.append(bits_from_dev(out))
    outs = [torch.empty_like(x) for _ in range(CALLS)]
    torch.cuda.synchronize()
    for k in range(CALLS):
        x.copy_(xs[k])
        at.copy_(ids[k])
        lora.forward(x, at, outs[k])
    torch.cuda.synchronize()
    mlp.check()
    for k in range(CALLS):
        assert np.array_equal(bits_from_dev(outs[k]), want[k]), k
    lora.close()
    mlp.close()


@pytest.mark.parametrize("fmt,K,I,M", [("nvfp4", 256, 512, 20), ("fp8", 512, 1280, 100), ("nvfp4", 2048, 5632, 100),
                                       ("fp8", 512, 1280, 300)])
def test_training_steps_in_a_row(torch, fmt, K, I, M):
    rng = np.random.default_rng(M)
    mlp = q.QuantMLP.from_case(scaled_case(fmt, K, I, 62), max_M=768)
    t = q.TrainMLP(mlp, 16)
    ad = on_device(torch, adapter(rng, K, I, 16), 1.0)
    xs, dys = ([to_dev(x_of(rng, M, K)[0]) for _ in range(CALLS)] for _ in range(2))
    x, dy = torch.empty_like(xs[0]), torch.empty_like(dys[0])
    saved = torch.empty(t.saved_bytes(M), dtype=torch.uint8, device="cuda")

    def buffers():
        return (torch.empty_like(x), torch.empty_like(x),
                q.Adapter(1.0, **{n: torch.empty_like(p) for n, p in ad.parts.items()}))

    def step(a, b, bufs):
        t.forward(a, bufs[0], saved, adapter=ad)
        t.backward(a, saved, b, bufs[1], adapter=ad, grads=bufs[2])

    def bits(bufs):
        return [bits_from_dev(b.view(torch.int16)) for b in (*bufs[:2], *bufs[2].parts.values())]
    want = []
    for k in range(CALLS):
        b = buffers()
        torch.cuda.synchronize()
        step(xs[k], dys[k], b)
        torch.cuda.synchronize()
        want.append(bits(b))
    got = [buffers() for _ in range(CALLS)]
    torch.cuda.synchronize()
    for k in range(CALLS):
        x.copy_(xs[k])
        dy.copy_(dys[k])
        step(x, dy, got[k])
    torch.cuda.synchronize()
    mlp.check()
    for k in range(CALLS):
        assert all(np.array_equal(a, b) for a, b in zip(bits(got[k]), want[k])), k
    t.close()
    mlp.close()
