"""Sums of the single projection seen closer than a bound over all of k shows them.

* Tokens that are zero but for one record of 128 k: every record, warp's share, cluster's
  share and K step alone. Products are exact and 128 of them are summed: 128 u of the
  terms' sizes, 64 u for factor, scales and the joining of shares; from 65 tokens on with a
  16-bit out an INT4 weight is rounded to fp16 (2^-11 of it).
* The relative L2 error with an fp32 out. A tensor core cuts an accumulator off, at
  most 2 u and on average 0.7 u of it a step of 16 k, always downward in size. Up to 64
  tokens chains are 8 steps or less before they are added in fp32: with partial sums that
  grow like a root, 8 x 0.7 x 2/3 = 3.7 u of a record's sum, random in sign from record to
  record, and the fp32 additions a root of (n / 6) u for n records: 8 u holds both up to n
  = 136 records one after the other. In the GEMM a chain is 16 steps: 16 u, as
  test_gpu_linear_many_sums.py derives. (What INT4's second product adds is 1e-4 of the
  result, the rounding of a weight to fp16.)
* K of less than the GEMM's step of 64."""
import numpy as np
import pytest

import test_gpu_linear as base
import weight_quantized_swiglu_gb300 as q
from test_gpu_linear import torch  # noqa: F401 (the fixture)

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def make(fmt, N, K, G, max_M):
    a, v = base.weights(fmt, N, K, G, N + K)
    return q.QuantLinear(fmt, N, K, max_M, **a), v


@pytest.mark.parametrize("fmt,G,N,K", [("nvfp4", 16, 40, 17408), ("int4", 64, 37, 17408), ("nvfp4", 16, 20, 65536),
                                       ("int4", 128, 20, 65536), ("int4", 32, 700, 5120), ("nvfp4", 16, 2500, 2048)])
@pytest.mark.parametrize("M", [1, 8, 40, 64, 130])
def test_each_record_alone(torch, fmt, G, N, K, M):  # noqa: F811
    lin, v = make(fmt, N, K, G, M)
    g = torch.Generator(device="cuda").manual_seed(M)
    recs = K // 128
    part = v.reshape(N, recs, 128)
    step = 1 if M > 1 else 7  # (one token: every seventh record, which meets every warp and CTA)
    for ot in (torch.float32, torch.bfloat16):
        half = torch.finfo(ot).eps / 2
        for r0 in range(0, recs, M * step):
            x = torch.zeros((M, K), device="cuda")
            rec = [min(r0 + m, recs - 1) for m in range(M)]
            val = torch.randn((M, 128), generator=g, device="cuda").half()
            for m, r in enumerate(rec):
                x[m, 128 * r:128 * r + 128] = val[m].float()
            out = torch.empty((M, N), device="cuda", dtype=ot)
            lin.forward(x.half(), out)
            got, xv = out.double().cpu().numpy(), val.double().cpu().numpy()
            w = part[:, rec]  # [N, M, 128]
            want = np.einsum("mk,nmk->mn", xv, w)
            size = np.einsum("mk,nmk->mn", np.abs(xv), np.abs(w))
            tol = (192 * U + (2.0 ** -11 if fmt == "int4" and M >= 65 and ot != torch.float32 else 0.0)) * size
            assert np.all(np.abs(got - want) <= tol + half * (np.abs(want) + tol)), (r0, ot)
    lin.check()
    lin.close()


@pytest.mark.parametrize("fmt,G,N,K", [("nvfp4", 16, 300, 17408), ("int4", 64, 300, 17408), ("nvfp4", 16, 2000, 5120),
                                       ("int4", 128, 640, 2048), ("nvfp4", 16, 6000, 4096)])
@pytest.mark.parametrize("M", [1, 2, 8, 9, 33, 64, 65, 300])
def test_fp32_outs_keep_their_precision(torch, fmt, G, N, K, M):  # noqa: F811
    lin, v = make(fmt, N, K, G, M)
    g = torch.Generator(device="cuda").manual_seed(M)
    for dt in (torch.bfloat16, torch.float16):
        x = torch.randn((M, K), generator=g, device="cuda").to(dt)
        out = torch.empty((M, N), device="cuda")
        lin.forward(x, out)
        want = x.double().cpu().numpy() @ v.T
        err = np.linalg.norm(out.double().cpu().numpy() - want) / np.linalg.norm(want)
        assert err <= (16 if M >= 65 else 8) * U, err / U
    lin.check()
    lin.close()


@pytest.mark.parametrize("fmt,G,K", [("nvfp4", 16, 16), ("nvfp4", 16, 48), ("nvfp4", 16, 80), ("int4", 32, 32),
                                     ("int4", 32, 96), ("int4", 64, 64)])
def test_few_inputs_and_many_tokens(torch, fmt, G, K):  # noqa: F811
    for N in (3, 264):
        lin, v = make(fmt, N, K, G, 300)
        for M in (64, 65, 257, 300):
            for dt, ot in ((torch.bfloat16, torch.float32), (torch.float16, torch.bfloat16)):
                x = torch.randn((M, K), device="cuda").to(dt)
                out = torch.full((M, N), 7.0, device="cuda", dtype=ot)
                lin.forward(x, out)
                lin.check()
                base.check(torch, x, v, out, more=2.0 ** -11 if M >= 65 and fmt == "int4" and ot != torch.float32 else 0.0)
        lin.close()
