"""A token with an infinite value: the definition's infinities, of the definition's signs,
whatever the number of tokens, the output's type and the form of the kernel. No weight
that meets the infinity is zero, so that no output is a NaN."""
import numpy as np
import pytest

import weight_quantized_swiglu_gb300 as q
from test_gpu_linear import torch  # noqa: F401 (the fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", ["int4", "nvfp4"])
@pytest.mark.parametrize("N,K", [(96, 512), (301, 2176)])
def test_infinite_x(torch, fmt, N, K):  # noqa: F811
    r = np.random.default_rng(N)
    w = r.integers(0, 256, (N, K // 2), dtype=np.uint8)
    at = 6  # the k that is infinite: a low nibble
    code = r.integers(1, 8, N)  # int4: less a zero of 8 or 0; nvfp4: 0.5 to 6
    neg = r.integers(0, 2, N).astype(bool)
    if fmt == "int4":
        z = np.repeat(np.where(neg, 8, 0).astype(np.uint8)[:, None], K // 64, 1)
        a = dict(scale=(r.uniform(0.1, 0.4, (N, K // 64)) * K ** -0.5).astype(np.float16), zero=z, group=64)
    else:
        code = code | np.where(neg, 8, 0)
        a = dict(scale=r.integers(40, 80, (N, K // 16), dtype=np.uint8))
    w[:, at // 2] = (w[:, at // 2] & 0xF0) | code.astype(np.uint8)
    sign = torch.tensor(np.where(neg, -1.0, 1.0), device="cuda")
    lin = q.QuantLinear(fmt, N, K, 300, w, **a)
    for M in (1, 8, 40, 64, 65, 300):
        for dt in (torch.bfloat16, torch.float16):
            for ot in (torch.float32, torch.bfloat16, torch.float16):
                x = torch.randn((M, K), device="cuda").to(dt)
                clean, out = torch.empty((M, N), device="cuda", dtype=ot), torch.empty((M, N), device="cuda", dtype=ot)
                lin.forward(x, clean)
                bad = x.clone()
                bad[0, at], bad[M - 1, at] = float("inf"), -float("inf")
                lin.forward(bad, out)
                lin.check()
                assert torch.equal(out[1:M - 1], clean[1:M - 1])
                for m, s in {0: 1.0, M - 1: -1.0}.items():
                    assert torch.equal(out[m].double(), s * sign * float("inf")), (M, dt, ot, out[m])
    lin.close()
