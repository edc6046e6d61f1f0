"""The mixture-of-experts layer's stages keep their range and precision whatever the
number of tokens: gate, up, intermediate and each expert's output past fp16's largest
value or below its normal ones, and fp32 outs, in the grouped form (more than 16 tokens,
or x that does not fit in shared memory) as in the one-kernel form.

Two bounds. Element by element those of test_gpu_moe_layer.py for the one-kernel form,
whose arithmetic the grouped form shares: the intermediate rounded once, to fp16 times a
power of two of the token and expert (fp32 outs: to two of them). And the relative L2
error of a token's output: rounding to bf16 or fp16 is 2^-9 or 2^-12 at most, the intermediate's
rounding the same as fp16's; with an fp32 out a sum over K or I ends within 8 u (chains
of eight MMAs that lose 2 u each at most, then rounded additions of random sign), W13's
error enters twice (g, u), so 32 u for all of it."""
import numpy as np
import pytest

import test_gpu_moe_layer as base
import weight_quantized_swiglu_gb300 as q
from test_gpu_moe_layer import torch  # noqa: F401 (the fixture)

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def outputs(bank, x, ids, w):
    """fp64 outputs for a selection and its weights."""
    out = np.zeros_like(x)
    for e in np.unique(ids):
        w13, w2 = bank.weight("w13", e), bank.weight("w2", e)
        for m, r in zip(*np.nonzero(ids == e)):
            h = w13 @ x[m]
            g, u = h[:bank.I], h[bank.I:]
            out[m] += w[m, r] * (w2 @ (g * base.sigmoid(np.clip(g, -700, 700)) * u))
    return out


CASES = [  # E, S, K, I, topk, meta, x's size, x, out, tokens
    (24, 0, 256, 64, 4, 4, 1e3, "bf16", "bf16", (16, 17, 40)),
    (24, 1, 256, 64, 4, 3, 1e3, "bf16", "fp32", (16, 17, 40)),
    (24, 0, 256, 64, 4, 4, 3e5, "bf16", "bf16", (16, 17)),
    (5, 1, 320, 96, 3, 4, 3e5, "bf16", "fp32", (17, 100)),   # groups of sixteen routes
    (24, 0, 256, 64, 4, 4, 1e-4, "bf16", "bf16", (16, 17, 40)),
    (24, 0, 256, 64, 4, 3, 1e-4, "bf16", "fp32", (17, 40)),
    (6, 1, 448, 1024, 3, 3, 1.0, "fp16", "fp32", (17, 64)),
    (40, 2, 1024, 352, 14, 4, 1.0, "bf16", "fp32", (17, 33)),  # sixteen routes a token
    (40, 0, 1024, 352, 6, 4, 1.0, "fp16", "fp16", (17, 33)),
    (12, 0, 8192, 64, 3, 4, 1e3, "bf16", "fp32", (2, 12, 16)),  # past 8 tokens x does not fit
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_range_and_precision(torch, case):  # noqa: F811
    E, S, K, I, topk, meta, size, xt, ot, tokens = case
    T = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
    bank = base.Bank(E + S, K, I, meta, E + K)
    g = torch.Generator(device="cuda").manual_seed(E + K)
    # logits of size one whatever x's is
    router = (torch.randn((E, K), generator=g, device="cuda") * K ** -0.5 / size).bfloat16()
    moe = bank.handle()
    layer = q.MoeLayer(moe, router, topk, shared=S, max_tokens=max(tokens))
    f64 = lambda t: t.double().cpu().numpy()  # noqa: E731
    for M in tokens:
        x = (torch.randn((M, K), generator=g, device="cuda") * size).to(T[xt])
        out = torch.full((M, K), 9.0, device="cuda", dtype=T[ot])
        ids = torch.full((M, topk), -1, device="cuda", dtype=torch.int32)
        w = torch.empty((M, topk), device="cuda")
        layer.forward(x, out, ids=ids, weights=w)
        again = torch.empty_like(out)
        layer.forward(x, again)
        layer.check()
        assert torch.equal(out.view(torch.uint8), again.view(torch.uint8))
        i, c = ids.cpu().numpy(), f64(w)
        if S:
            i = np.concatenate((i, np.tile(np.arange(E, E + S), (M, 1))), 1)
            c = np.concatenate((c, np.ones((M, S))), 1)
        want, got = outputs(bank, f64(x), i, c), f64(out)
        assert np.isfinite(got).all(), M
        err = np.linalg.norm(got - want, axis=1) / np.linalg.norm(want, axis=1)
        assert err.max() <= (32 * U if ot == "fp32" else 2.0 ** -9 if ot == "bf16" else 2.0 ** -11), (M, err.max())
        base.verify(bank, f64(x), f64(router), None, None, dict(E=E, S=S, topk=topk, score="softmax", renorm=True,
                    rscale=1.0), ids.cpu().numpy(), f64(w), got, torch.finfo(T[ot]).eps / 2, xt == "bf16", True)
    layer.close()
    moe.close()


def test_layers_of_one_handle_share_its_workspace(torch):  # noqa: F811
    """A later layer with more routes a token, and calls of the handle itself between the
    layers' calls, whose results are those of a handle of their own."""
    E, K, I, M = 20, 256, 64, 24
    bank = base.Bank(E, K, I, 4, 7)
    moe, other = bank.handle(), bank.handle()
    g = torch.Generator(device="cuda").manual_seed(7)
    router = (torch.randn((E, K), generator=g, device="cuda") * K ** -0.5).bfloat16()
    x = torch.randn((M, K), generator=g, device="cuda").bfloat16()
    small = q.MoeLayer(moe, router, 2, max_tokens=M)
    ids, w = torch.empty((M, 2), dtype=torch.int32, device="cuda"), torch.empty((M, 2), device="cuda")
    out = torch.empty((M, K), device="cuda")
    small.forward(x, out, ids=ids, weights=w)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        small.forward(x, out)
    want = out.clone()
    large = q.MoeLayer(moe, router, 16, max_tokens=M)
    many = torch.empty_like(out)
    large.forward(x, many)
    wide = q.MoeLayer(other, router, 16, max_tokens=M)
    many2 = torch.empty_like(out)
    wide.forward(x, many2)
    assert torch.equal(many, many2)
    h1, h2 = torch.empty((M, K), dtype=torch.float16, device="cuda"), torch.empty((M, K), dtype=torch.float16, device="cuda")
    assert q.qmlp_moe_forward(moe.h, x, q.DT_BF16, ids, w, 2, M, h1) == 0
    assert q.qmlp_moe_reserve(other.h, M) == 0 and q.qmlp_moe_forward(other.h, x, q.DT_BF16, ids, w, 2, M, h2) == 0
    assert torch.equal(h1, h2)
    for run in (lambda: small.forward(x, out), graph.replay):
        out.zero_()
        run()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    for t in (small, large, wide, moe, other):
        t.close()
