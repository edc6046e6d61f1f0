"""One buffer for what a forward keeps, for batches of different lengths."""
import numpy as np
import pytest

import weight_quantized_swiglu_gb300 as q
from helpers import bits_from_dev, to_dev
from test_gpu_lora import adapter, on_device, scaled_case, x_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch(cuda_available):
    import torch
    from weight_quantized_swiglu_gb300 import build
    build.build()
    return torch


def test_bytes_grow_with_the_tokens(torch):
    mlp = q.QuantMLP.from_case(scaled_case("nvfp4", 256, 512, 63), max_M=768)
    for r in (1, 64):
        t = q.TrainMLP(mlp, r)
        n = [t.saved_bytes(m) for m in range(1, 769)]
        assert all(b >= a for a, b in zip(n, n[1:]))
        t.close()
    mlp.close()


@pytest.mark.parametrize("fmt", ["nvfp4", "fp8"])
def test_a_buffer_for_long_batches_serves_short_ones(torch, fmt):
    """256 tokens, then fewer, in the buffer of 256: the steps of a buffer of
    their own, and nothing written behind its end. (Room behind it for twice as
    much keeps every write of this test inside one allocation.)"""
    K, I = 256, 512
    rng = np.random.default_rng(64)
    mlp = q.QuantMLP.from_case(scaled_case(fmt, K, I, 64), max_M=768)
    t = q.TrainMLP(mlp, 16)
    ad = on_device(torch, adapter(rng, K, I, 16), 1.0)
    size = t.saved_bytes(256)
    room = torch.empty(3 * size, dtype=torch.uint8, device="cuda")
    shared = room[:size]
    for M in (256, 255, 250, 225, 31, 1, 256):
        x, dy = to_dev(x_of(rng, M, K)[0]), to_dev(x_of(rng, M, K)[0])
        results = []
        for buf in (shared, torch.empty(t.saved_bytes(M), dtype=torch.uint8, device="cuda")):
            room[size:] = 0xA5
            out, dx = torch.empty_like(x), torch.empty_like(x)
            g = q.Adapter(1.0, **{n: torch.empty_like(p) for n, p in ad.parts.items()})
            t.forward(x, out, buf, adapter=ad)
            t.backward(x, buf, dy, dx, adapter=ad, grads=g)
            torch.cuda.synchronize()
            assert bool((room[size:] == 0xA5).all()), M
            results.append([bits_from_dev(b.view(torch.int16)) for b in (out, dx, *g.parts.values())])
        assert all(np.array_equal(a, b) for a, b in zip(*results)), M
    mlp.check()
    t.close()
    mlp.close()
