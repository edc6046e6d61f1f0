"""Tokens near the ends of bf16's range, where an output is an ordinary number although the
sum before the global or row factor is not: the definition's values, by test_gpu_linear.py's
tolerances, whatever the number of tokens."""
import numpy as np
import pytest

import test_gpu_linear as base
import weight_quantized_swiglu_gb300 as q
from test_gpu_linear import torch  # noqa: F401 (the fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt,glob,size", [("nvfp4", 3000.0, 1e35), ("nvfp4", 1e-3, 1e-37), ("nvfp4", 2.0 ** -20, 2.0 ** -128),
                                           ("int4", 1.0, 1e36), ("int4", 1.0, 1e-36), ("nvfp4", 1e38, 1e37),
                                           ("nvfp4", 1e-38, 1e-37)])
def test_far_tokens(torch, fmt, glob, size):  # noqa: F811
    N, K = 301, 512
    a, v = base.weights(fmt, N, K, 16 if fmt == "nvfp4" else 64, 5)
    if fmt == "int4":  # weights far from one as well: the products are ordinary
        s = a["scale"].astype(np.float32) * (2.0 ** -9 if size > 1 else 2.0 ** 10)
        a["scale"] = s.astype(np.float16)
        c = np.stack((a["w"] & 15, a["w"] >> 4), -1).reshape(N, K).astype(float)
        v = (c - np.repeat(a["zero"].astype(float), 64, 1)) * np.repeat(a["scale"].astype(float), 64, 1)
    lin = q.QuantLinear(fmt, N, K, 300, global_scale=glob, **a)
    factor = float(np.float32(1.0 / np.float64(np.float32(glob))))
    for M in (1, 8, 40, 65, 300):
        x = (torch.randn((M, K), device="cuda") * size).bfloat16()
        for ot in (torch.float32, torch.bfloat16):
            out = torch.empty((M, N), device="cuda", dtype=ot)
            lin.forward(x, out)
            lin.check()
            assert out.isfinite().all()
            more = 2.0 ** -11 if M >= 65 and fmt == "int4" and ot != torch.float32 else 0.0
            base.check(torch, x, v, out, factor, more=more)
    lin.close()
