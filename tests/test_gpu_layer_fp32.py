"""Outputs in fp32, which keep fp32's precision: the mixture-of-experts layer's
intermediate in two fp16 words in every form of the kernel, INT4 projections in two
products; and outputs whose offsets pass 32 bits."""
import numpy as np
import pytest

import test_gpu_linear as linear
import test_gpu_moe_layer as moe_layer
import weight_quantized_swiglu_gb300 as q
from test_gpu_norm import torch  # noqa: F401 (the fixture)

pytestmark = pytest.mark.gpu

CASES = [  # E, S, K, I, topk, meta, score, bias, renorm, scale, gated, router, x, out, tokens
    (30, 0, 4096, 1024, 2, 4, "sigmoid", False, True, 1.0, False, "bf16", "bf16", "fp32", (16, 5, 1)),
    (20, 1, 1024, 896, 6, 3, "softmax", False, True, 1.0, True, "bf16", "fp16", "fp32", (16, 4, 3)),
    (40, 2, 1024, 352, 6, 3, "sigmoid", True, True, 2.5, False, "bf16", "fp16", "fp32", (16, 11, 2)),
    (12, 1, 8192, 64, 3, 4, "softmax", False, True, 1.0, True, "bf16", "bf16", "fp32", (1, 8)),
    (9, 0, 2048, 160, 8, 4, "softmax", False, False, 1.0, False, "bf16", "bf16", "fp32", (9, 1)),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_moe_layer(torch, case):  # noqa: F811
    moe_layer.test_layer(torch, case)


@pytest.mark.parametrize("G,N,K,tokens", [(32, 257, 2048, (65, 66, 128, 129, 255, 513)), (128, 5120, 640, (70, 300)),
                                          (64, 31, 192, (65, 400))])
def test_int4_projection(torch, G, N, K, tokens):  # noqa: F811
    linear.test_many_tokens(torch, ("int4", G, N, K, tokens, "fp16", "fp32", True))
    linear.test_many_tokens(torch, ("int4", G, N, K, tokens, "bf16", "fp32", False))


def test_weights_that_are_not_finite(torch):  # noqa: F811
    """A group's infinite scale reaches its row alone, as inf or NaN, in both forms."""
    N, K = 96, 256
    a, _ = linear.weights("int4", N, K, 64, 3)
    ok = {n: t.copy() if isinstance(t, np.ndarray) else t for n, t in a.items()}
    a["scale"][17, 2] = np.inf
    x = torch.randn((70, K), device="cuda").bfloat16()
    for M in (8, 40, 70):
        outs = []
        for w in (ok, a):
            lin = q.QuantLinear("int4", N, K, M, **w)
            out = torch.empty((M, N), device="cuda")
            lin.forward(x[:M], out)
            lin.check()
            lin.close()
            outs.append(out)
        rest = [n for n in range(N) if n != 17]
        assert torch.equal(outs[0][:, rest], outs[1][:, rest]) and not outs[1][:, 17].isfinite().any()


@pytest.mark.parametrize("fmt,G", [("int4", 128), ("nvfp4", 16)])
def test_more_than_2_31_outputs(torch, fmt, G):  # noqa: F811
    M, N, K = 33000, 70001, 128
    a, v = linear.weights(fmt, N, K, G, 5)
    lin = q.QuantLinear(fmt, N, K, M, **a)
    g = torch.Generator(device="cuda").manual_seed(6)
    x = torch.randn((M, K), generator=g, device="cuda").bfloat16()
    out = torch.empty((M, N), device="cuda", dtype=torch.bfloat16)
    lin.forward(x, out)
    lin.check()
    for m in (0, 30678, 32998):  # 30678 N is the first past 2^31
        linear.check(torch, x[m:m + 2].contiguous(), v, out[m:m + 2].contiguous(), more=2.0 ** -11 if fmt == "int4" else 0.0)
    lin.close()
