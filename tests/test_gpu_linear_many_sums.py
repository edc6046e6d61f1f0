"""Fp32 outs of the GEMM that takes 65 tokens and more: chains of 16 MMAs before a sum is
taken out of the tensor cores' accumulator.

An MMA cuts an accumulator off, on average 0.7 u of it and always downward in size: with
partial sums that grow like a root 16 x 0.7 x 2/3 = 7.5 u of a chain's sum, random in sign
from chain to chain. The n = K / 256 chains are added in fp32: a root of (n / 6) u. INT4's
second product, 2^-12 of the first, is added with half a step; the factor's product is
another: 8.5 u for K = 5120, 10 u for K = 65536, all in the relative L2 norm. Held to 16 u.
One chain over k = 17408 was 2e-5 off (330 u).

The elements as test_gpu_linear.py holds them, at sizes that leave the last tiles to be
split over k, tiles in part and rows of no multiple of four."""
import numpy as np
import pytest

import test_gpu_linear as base
import weight_quantized_swiglu_gb300 as q
from test_gpu_linear import torch  # noqa: F401 (the fixture)

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.mark.parametrize("fmt,G,N,K,M", [("nvfp4", 16, 5120, 17408, 2000), ("int4", 64, 5120, 17408, 2000),
                                         ("nvfp4", 16, 300, 65536, 300), ("int4", 128, 300, 65536, 70),
                                         ("int4", 32, 2570, 5120, 513), ("nvfp4", 16, 17408, 5120, 128),
                                         ("int4", 64, 77, 17408, 1000), ("nvfp4", 16, 1021, 1040, 65),
                                         ("int4", 32, 9000, 352, 700), ("nvfp4", 16, 20000, 2064, 600)])
def test_fp32_outs(torch, fmt, G, N, K, M):  # noqa: F811
    a, v = base.weights(fmt, N, K, G, N + K)
    bias = np.random.default_rng(1).normal(size=N).astype(np.float32) * 1e-3
    lin = q.QuantLinear(fmt, N, K, M, bias=bias, **a)
    g = torch.Generator(device="cuda").manual_seed(M)
    vd, bd = torch.tensor(v, device="cuda"), torch.tensor(bias, device="cuda").double()
    for dt in (torch.bfloat16, torch.float16):
        x = torch.randn((M, K), generator=g, device="cuda").to(dt)
        out, again = torch.full((M, N), 7.0, device="cuda"), torch.empty((M, N), device="cuda")
        lin.forward(x, out)
        lin.forward(x, again)
        lin.check()
        assert torch.equal(out, again)
        want, size = x.double() @ vd.T + bd, x.double().abs() @ vd.abs().T + bd.abs()
        err = ((out.double() - want).norm() / want.norm()).item()
        assert err <= 16 * U, err / U
        assert ((out.double() - want).abs() <= (K + 64) * U * size + 2.0 ** -38 * x.double().abs().amax(1, keepdim=True) *
                vd.abs().sum(1)).all()
    lin.close()


def test_other_types_of_out_do_not_change(torch):  # noqa: F811
    """16-bit outs are the rounded values of the fp32 ones, but for what a chain cuts off."""
    a, v = base.weights("nvfp4", 1000, 4096, 16, 3)
    lin = q.QuantLinear("nvfp4", 1000, 4096, 400, **a)
    x = torch.randn((400, 4096), device="cuda").bfloat16()
    outs = []
    for ot in (torch.float32, torch.bfloat16):
        out = torch.empty((400, 1000), device="cuda", dtype=ot)
        lin.forward(x, out)
        outs.append(out.double())
    lin.check()
    size = x.double().abs() @ torch.tensor(np.abs(v), device="cuda").T
    assert ((outs[1] - outs[0]).abs() <= 2.0 ** -8 * outs[0].abs() + 4160 * U * size).all()
    lin.close()
