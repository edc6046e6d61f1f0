"""The router's logits keep fp32's precision whatever the number of tokens and K: the
weights of a call against the scores in 64 bits of the experts that it selected.

An MMA cuts its accumulator off, on average 0.7 u of it and always downward in size. With
chains of eight MMAs or fewer warps' short ones added in fp32, a logit is off by
8 x 0.7 x 2/3 = 3.7 u of a chain's sum, random in sign from chain to chain, and a root
of (K / 128 / 6) u by the additions: 5 u of its size at K = 8192. Selected logits are of
size three at most here (unit variance, the largest of 64 to 512): 15 u, of a renormed
weight relative to the others 15 u x 1.4, and 8 u for the exponentials, the sum and the
quotient: 32 u in the relative L2 norm of all weights."""
import pytest

import test_gpu_moe_layer as base
import weight_quantized_swiglu_gb300 as q
from test_gpu_moe_layer import torch  # noqa: F401 (the fixture)

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.mark.parametrize("E,K", [(64, 256), (64, 2560), (200, 4096), (64, 8192), (512, 2560)])
@pytest.mark.parametrize("rt", ["bf16", "fp16", "fp32"])
def test_weights(torch, E, K, rt):  # noqa: F811
    topk, S = 8, 2
    T = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
    moe = base.Bank(E + S, K, 32, 4, 1).handle()
    g = torch.Generator(device="cuda").manual_seed(E + K)
    router = (torch.randn((E, K), generator=g, device="cuda") * K ** -0.5).to(T[rt])
    for score, renorm in (("softmax", True), ("softmax", False), ("sigmoid", True), ("sigmoid", False)):
        layer = q.MoeLayer(moe, router, topk, score=score, renorm=renorm, shared=S, max_tokens=130)
        for M in (1, 8, 9, 16, 17, 130):
            for dt in (torch.bfloat16, torch.float16):
                x = torch.randn((M, K), generator=g, device="cuda").to(dt)
                ids, w = torch.empty((M, topk), dtype=torch.int32, device="cuda"), torch.empty((M, topk), device="cuda")
                layer.forward(x, torch.empty((M, K), device="cuda"), ids=ids, weights=w)
                layer.check()
                logit = x.double() @ router.double().T
                p = (torch.softmax(logit, 1) if score == "softmax" else torch.sigmoid(logit)).gather(1, ids.long())
                want = p / p.sum(1, keepdim=True) if renorm else p
                err = ((w.double() - want).norm() / want.norm()).item()
                assert err <= 32 * U, (score, renorm, M, dt, err / U)
        layer.close()
    moe.close()
