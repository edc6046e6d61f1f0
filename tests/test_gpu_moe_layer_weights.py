"""Renormed weights where the selected experts' scores are far below fp32's smallest
number: the sum of the selected scores divides them, so the weights are ordinary numbers
by the definition (in 64 bits they are computed without that underflow).

Tolerance: a logit is off by K u of its terms' sizes at most, a renormed weight by four
times that of itself, with 32 u for the exponentials, the sum and the quotient."""
import numpy as np
import pytest

import test_gpu_moe_layer as base
import weight_quantized_swiglu_gb300 as q
from test_gpu_moe_layer import torch  # noqa: F401 (the fixture)

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("M", [1, 5, 16, 20])
@pytest.mark.parametrize("low", [-10.0, -86.0, -95.0, -200.0, -3000.0])
def test_scores_that_underflow(torch, score, M, low):  # noqa: F811
    """Sigmoid: every logit about `low`. Softmax with a bias that takes the experts with the
    large logits out of the selection: the others' scores are exp(low) of theirs."""
    E, K, topk = 40, 256, 4
    moe = base.Bank(E, K, 64, 4, 1).handle()
    g = torch.Generator(device="cuda").manual_seed(M)
    router = (torch.randn((E, K), generator=g, device="cuda") * K ** -0.5).bfloat16()
    x = torch.randn((M, K), generator=g, device="cuda").bfloat16()
    x[:, 0] = 4.0
    bias = None
    if score == "sigmoid":
        router[:, 0] = low / 4
    else:
        router[:8, 0] = -low / 4
        bias = torch.zeros(E, device="cuda")
        bias[:8] = -float("inf")
    layer = q.MoeLayer(moe, router, topk, score=score, bias=bias, max_tokens=M)
    out = torch.empty((M, K), device="cuda")
    ids, w = torch.empty((M, topk), dtype=torch.int32, device="cuda"), torch.empty((M, topk), device="cuda")
    layer.forward(x, out, ids=ids, weights=w)
    layer.check()
    xd, rd = x.double().cpu().numpy(), router.double().cpu().numpy()
    i, got = ids.cpu().numpy(), w.double().cpu().numpy()
    assert (i >= 8).all() or score == "sigmoid"
    l = np.take_along_axis(xd @ rd.T, i, 1)
    el = K * U * np.take_along_axis(np.abs(xd) @ np.abs(rd).T, i, 1).max(1, keepdims=True)
    # log of the score but for what all of a token's share
    lp = l if score == "softmax" else -np.logaddexp(0.0, -l)
    want = np.exp(lp - lp.max(1, keepdims=True))
    want /= want.sum(1, keepdims=True)
    assert np.all(np.abs(got - want) <= (4 * el + 32 * U) * want), (got, want)
    assert out.isfinite().all()
    layer.close()
    moe.close()
