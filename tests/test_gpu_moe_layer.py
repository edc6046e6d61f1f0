"""A whole mixture-of-experts layer against the definition in 64 bits.

The kernel's own selection is checked first (every selected score at least the
topk-th largest less the logits' error, largest first, no expert twice), then the
output for that selection. Bounds, from the arithmetic (u = 2^-24):
* a logit: K u of its terms' sizes; p then moves by at most twice that of itself,
  a renormed one by four times, with 32 u for exp, the quotients and the sums.
* g and u: K u of their terms' sizes, and for bf16 tokens 2^-38 of the largest |x|
  (what the scaling to fp16 leaves); act: 1.1 |u| dg + |SiLU(g)| du + 16 u |act|
  (SiLU's slope is at most 1.1), then fp16's half step, 2^-11 (two of them with an fp32
  out, 2^-22), and 2^-38 of the largest |act| of the token and expert below fp16's normal numbers.
* the sum over I and the experts: (I + 64) u of its terms' sizes.
With more than 16 tokens, or where x does not fit in shared memory, g, u, act and
each expert's y are rounded to fp16 (2^-11 of their size, at least 2^-25)."""
import numpy as np
import pytest

import weight_quantized_swiglu_gb300 as q

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.fixture(scope="module")
def torch(cuda_available):
    import torch
    from weight_quantized_swiglu_gb300 import build
    build.build()
    return torch


class Bank:
    """Random experts in the checkpoint's layout; weights in fp64 one at a time."""

    def __init__(self, B, K, I, meta, seed):
        g = np.random.default_rng(seed)
        self.B, self.K, self.I, self.meta = B, K, I, meta
        for n, N, D in (("w13", 2 * I, K), ("w2", K, I)):
            w = g.integers(0, 256, (B, N, D // 2), dtype=np.uint8)
            s = (g.uniform(0.1, 0.4, (B, N, D // 32)) * D ** -0.5).astype(np.float16)
            z = g.integers(4, 12, s.shape, dtype=np.uint8)
            bias = (-z.astype(np.float32) * s.astype(np.float32)).astype(np.float16)
            sb = s.view(np.uint8).reshape(*s.shape, 2)
            rec = np.concatenate((sb, z[..., None] if meta == 3 else bias.view(np.uint8).reshape(*s.shape, 2)), -1)
            setattr(self, n, w)
            setattr(self, n + "_m", np.ascontiguousarray(rec))
            setattr(self, n + "_s", s)
            setattr(self, n + "_b", bias)

    def weight(self, n, e):
        w, s, b = getattr(self, n)[e], getattr(self, n + "_s")[e], getattr(self, n + "_b")[e]
        c = np.stack((w & 15, w >> 4), -1).reshape(w.shape[0], -1).astype(np.float64)
        v = c * np.repeat(s.astype(float), 32, 1) + np.repeat(b.astype(float), 32, 1)
        return v.astype(np.float16).astype(np.float64)  # half_fma: one rounding of an exact sum

    def handle(self):
        return q.MoeAWQ(self.B, self.K, self.I, self.meta, self.w13, self.w13_m, self.w2, self.w2_m)


def sigmoid(t):
    return 1 / (1 + np.exp(-t))


def verify(bank, x, router, sgate, bias, cfg, ids, weights, out, half, bf16, few):
    """All in fp64; half: the output type's half step, bf16: x's type."""
    E, S, topk, M, K, I = cfg["E"], cfg["S"], cfg["topk"], x.shape[0], bank.K, bank.I
    logit = x @ router.T
    el = K * U * (np.abs(x) @ np.abs(router).T)
    p = sigmoid(logit) if cfg["score"] == "sigmoid" else np.exp(logit - logit.max(1, keepdims=True))
    if cfg["score"] == "softmax":
        p /= p.sum(1, keepdims=True)
    ep = (2 * el.max(1, keepdims=True) + 32 * U) * p
    key, ek = (p, ep) if bias is None else (p + bias, ep + 4 * U * np.abs(bias))
    for m in range(M):
        assert len(set(ids[m])) == topk and ids[m].min() >= 0 and ids[m].max() < E
        kth = np.sort(key[m])[-topk]
        err = 2 * ek[m][np.isfinite(key[m])].max()
        chosen = key[m][ids[m]]
        assert np.all(chosen >= kth - err), (m, chosen, kth)
        assert np.all(chosen[:-1] >= chosen[1:] - err)
    w = np.take_along_axis(p, ids, 1)
    ew = 2 * np.take_along_axis(ep, ids, 1)
    if cfg["renorm"]:
        w, ew = w / w.sum(1, keepdims=True), 2 * ew / w.sum(1, keepdims=True)
    w, ew = w * cfg["rscale"], ew * cfg["rscale"] + 8 * U * w * cfg["rscale"]
    assert np.all(np.abs(weights - w) <= ew)
    if S:
        sw, es = np.ones((M, S)), np.zeros((M, S))
        if sgate is not None:
            sw = sigmoid(x @ sgate.T)
            es = (K * U * (np.abs(x) @ np.abs(sgate).T) + 8 * U) * 1.0
        ids, w, ew = np.concatenate((ids, np.tile(np.arange(E, E + S), (M, 1))), 1), np.concatenate((w, sw), 1), \
            np.concatenate((ew, es), 1)
    want, tol = np.zeros((M, K)), np.zeros((M, K))
    h16 = 2.0 ** -11
    for e in np.unique(ids):
        w13, w2 = bank.weight("w13", e), bank.weight("w2", e)
        for m, r in zip(*np.nonzero(ids == e)):
            h, size = w13 @ x[m], np.abs(w13) @ np.abs(x[m])
            eh = (K + 16) * U * size
            if bf16:
                eh = eh + 2.0 ** -38 * np.abs(x[m]).max() * np.abs(w13).sum(1)
            if not few:
                eh = eh + h16 * (np.abs(h) + eh) + 2.0 ** -25
            g, u, eg, eu = h[:I], h[I:], eh[:I], eh[I:]
            silu = g * sigmoid(g)
            act = silu * u
            ea = 1.1 * eg * (np.abs(u) + eu) + np.abs(silu) * eu + 16 * U * np.abs(act)
            ha = 2.0 ** -22 if few and half < 2.0 ** -20 else h16
            ea = ea + ha * (np.abs(act) + ea) + (2.0 ** -38 * np.abs(act).max() if few else 2.0 ** -25)
            y, ey = w2 @ act, np.abs(w2) @ (ea + (I + 64) * U * np.abs(act))
            if not few:
                ey = ey + h16 * (np.abs(y) + ey) + 2.0 ** -25
            want[m] += w[m, r] * y
            tol[m] += np.abs(w[m, r]) * ey + ew[m, r] * (np.abs(y) + ey) + 32 * U * np.abs(w[m, r] * y)
    bad = np.abs(out - want) > tol + half * (np.abs(want) + tol) + 2.0 ** -25
    assert not bad.any(), (int(bad.sum()), float(np.abs(out - want).max()), float(np.abs(want).max()))


CASES = [  # E, S, K, I, topk, meta, score, bias, renorm, scale, gated, router, x, out, tokens
    (5, 0, 64, 32, 2, 4, "softmax", False, True, 1.0, False, "fp32", "bf16", "fp32", (1, 2)),
    (1, 0, 128, 64, 1, 3, "softmax", False, False, 1.0, False, "bf16", "fp16", "fp16", (1, 5)),
    (7, 1, 320, 96, 3, 4, "softmax", False, True, 1.0, True, "bf16", "bf16", "bf16", (1, 3, 8, 9)),
    (7, 2, 320, 96, 7, 3, "sigmoid", True, False, 2.5, True, "fp16", "fp16", "fp32", (1, 4, 16)),
    (40, 2, 1024, 352, 6, 3, "sigmoid", True, True, 2.5, False, "bf16", "fp16", "fp16", (16, 11)),
    (512, 1, 640, 160, 10, 4, "softmax", False, True, 1.0, True, "bf16", "bf16", "bf16", (1, 4, 16)),
    (300, 0, 256, 64, 8, 4, "softmax", True, False, 1.0, False, "fp32", "bf16", "fp32", (1, 7)),
    (1000, 0, 128, 64, 16, 3, "softmax", False, True, 1.0, False, "bf16", "bf16", "fp32", (1, 16)),
    (30, 0, 4096, 1024, 2, 4, "sigmoid", False, True, 1.0, False, "bf16", "bf16", "bf16", (16, 1)),
    (12, 1, 8192, 64, 3, 4, "softmax", False, True, 1.0, True, "bf16", "fp16", "bf16", (1, 2, 12, 16)),
    (16, 1, 256, 64, 3, 4, "softmax", False, True, 1.0, True, "bf16", "bf16", "fp32", (17, 40)),
    (16, 0, 448, 32, 4, 3, "sigmoid", True, True, 1.5, False, "fp32", "fp16", "bf16", (100, 33)),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_layer(torch, case):
    E, S, K, I, topk, meta, score, has_bias, renorm, rscale, gated, rt, xt, ot, tokens = case
    T = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
    bank = Bank(E + S, K, I, meta, E + K)
    g = torch.Generator(device="cuda").manual_seed(E * 31 + K)
    router = (torch.randn((E, K), generator=g, device="cuda") * K ** -0.5).to(T[rt])
    sgate = (torch.randn((S, K), generator=g, device="cuda") * K ** -0.5).to(T[rt]) if gated else None
    bias = torch.randn(E, generator=g, device="cuda") * 0.05 if has_bias else None
    moe = bank.handle()
    layer = q.MoeLayer(moe, router, topk, score=score, bias=bias, renorm=renorm, route_scale=rscale, shared=S,
                       shared_gate=sgate, max_tokens=max(tokens))
    f64 = lambda t: None if t is None else t.double().cpu().numpy()  # noqa: E731
    for M in tokens:
        x = torch.randn((M, K), generator=g, device="cuda").to(T[xt])
        out = torch.full((M, K), 9.0, device="cuda", dtype=T[ot])
        ids = torch.full((M, topk), -1, device="cuda", dtype=torch.int32)
        w = torch.empty((M, topk), device="cuda")
        layer.forward(x, out, ids=ids, weights=w)
        again = torch.empty_like(out)
        layer.forward(x, again)
        layer.check()
        assert torch.equal(out.view(torch.uint8), again.view(torch.uint8))
        few = M <= 16 and not (K == 8192 and M > 8)
        verify(bank, f64(x), f64(router), f64(sgate), f64(bias), dict(E=E, S=S, topk=topk, score=score, renorm=renorm,
               rscale=rscale), ids.cpu().numpy(), f64(w), f64(out), torch.finfo(T[ot]).eps / 2, xt == "bf16", few)
    layer.close()
    moe.close()


def small(torch, E=40, K=256, I=64, topk=5, S=0, max_tokens=16, seed=1, **kw):
    bank = Bank(E + S, K, I, 4, seed)
    moe = bank.handle()
    g = torch.Generator(device="cuda").manual_seed(seed)
    router = (torch.randn((E, K), generator=g, device="cuda") * K ** -0.5).to(torch.bfloat16)
    return moe, router, g


def test_ties_go_to_the_lowest_index(torch):
    for E in (40, 64, 200, 500, 1000):
        moe, router, g = small(torch, E=E)
        router[:] = router[0]
        router[E - 3:] = -router[0]
        for M in (3, 20):
            x = torch.randn((M, 256), generator=g, device="cuda").to(torch.bfloat16)
            for score, bias in (("softmax", None), ("sigmoid", None),
                                ("sigmoid", torch.zeros(E, device="cuda"))):
                layer = q.MoeLayer(moe, router, 5, score=score, bias=bias, max_tokens=M)
                ids = torch.empty((M, 5), dtype=torch.int32, device="cuda")
                layer.forward(x, torch.empty((M, 256), device="cuda"), ids=ids)
                up = (x.double() @ router[0].double()) > 0
                first = torch.arange(5, device="cuda", dtype=torch.int32)
                last = torch.tensor([E - 3, E - 2, E - 1, 0, 1], device="cuda", dtype=torch.int32)
                want = torch.where(up[:, None], first, last)
                assert torch.equal(ids, want), (E, M, score)
                layer.close()
        moe.close()


def test_experts_left_out_and_values_that_are_not_finite(torch):
    """A bias of -inf takes experts out of the selection; NaN and Inf in a token, in
    the router's row of one expert or in an expert's scales stay where they belong."""
    E, M = 40, 9
    moe, router, g = small(torch, E=E)
    bias = torch.zeros(E, device="cuda")
    bias[::2] = -float("inf")
    x = torch.randn((M, 256), generator=g, device="cuda").to(torch.bfloat16)
    layer = q.MoeLayer(moe, router, 5, score="sigmoid", bias=bias, max_tokens=40)
    ids, out = torch.empty((M, 5), dtype=torch.int32, device="cuda"), torch.empty((M, 256), device="cuda")
    layer.forward(x, out, ids=ids)
    assert (ids % 2 == 1).all()
    bad = x.clone()
    bad[4, 17], bad[6, 3] = float("nan"), float("inf")
    ids2, out2 = torch.empty_like(ids), torch.empty_like(out)
    layer.forward(bad, out2, ids=ids2)
    layer.check()
    rest = [m for m in range(M) if m not in (4, 6)]
    assert torch.equal(out2[rest], out[rest]) and torch.equal(ids2[rest], ids[rest])
    assert out2[4].isnan().all() and not out2[6].isfinite().all()
    for row in ids2.tolist():
        assert len(set(row)) == 5 and all(0 <= e < E for e in row)
    long, outl = torch.cat((bad, x, x, x)), torch.empty((36, 256), device="cuda")
    idl = torch.empty((36, 5), dtype=torch.int32, device="cuda")
    layer.forward(long, outl, ids=idl)
    assert torch.equal(idl[:9], ids2) and torch.equal(idl[9:18], ids) and torch.equal(outl[9:18], outl[27:])
    layer.close()
    moe.close()
    # an expert whose scales are infinite: only the tokens that name it
    bank = Bank(E, 256, 64, 4, 1)
    used = set(ids.flatten().tolist())
    victim = int(ids[0, 0])
    bank.w2_m[victim, :, :, 1] = 0x7C  # scale = +Inf (or NaN)
    moe = bank.handle()
    layer = q.MoeLayer(moe, router, 5, score="sigmoid", bias=bias, max_tokens=16)
    layer.forward(x, out2, ids=ids2)
    names = (ids2 == victim).any(1)
    assert torch.equal(ids2, ids) and torch.equal(out2[~names], out[~names]) and victim in used
    assert not out2[names].isfinite().any()
    layer.close()
    moe.close()


def test_captured_streams_and_two_at_once(torch):
    moe, router, g = small(torch, S=1)
    moe2, _, _ = small(torch, S=1, seed=1)
    kw = dict(shared=0, max_tokens=16)
    router41 = torch.cat((router, router[:1]))
    a, b = q.MoeLayer(moe, router41, 5, **kw), q.MoeLayer(moe2, router41, 5, **kw)
    x = torch.randn((8, 256), generator=g, device="cuda").to(torch.float16)
    out, want = torch.empty_like(x), torch.empty_like(x)
    a.forward(x, out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(3):
            a.forward(x, out)
    x.copy_(torch.randn((8, 256), generator=g, device="cuda"))
    a.forward(x, want)
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    # two layers on two streams: whole-GPU launches that must not wait for each other
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    o1, o2 = torch.empty_like(x), torch.empty_like(x)
    torch.cuda.synchronize()
    for _ in range(50):
        a.forward(x, o1, stream=s1)
        b.forward(x, o2, stream=s2)
    torch.cuda.synchronize()
    a.check()
    b.check()
    assert torch.equal(o1, want) and torch.equal(o2, want)
    for t in (a, b, moe, moe2):
        t.close()


def test_refusals(torch):
    moe, router, g = small(torch)
    with pytest.raises(ValueError):
        q.MoeLayer(moe, router[:39], 5)
    for kw in (dict(topk=17), dict(topk=0), dict(topk=41), dict(topk=5, max_tokens=0)):
        with pytest.raises(q.QmlpError) as e:
            q.MoeLayer(moe, router, **kw)
        assert e.value.status == 4
    layer = q.MoeLayer(moe, router, 5, max_tokens=4)
    x, out = torch.zeros((4, 256), device="cuda", dtype=torch.bfloat16), torch.zeros((4, 256), device="cuda")
    layer.forward(x, out)
    for bx, bo, kw in ((x.float(), out, {}), (x, out[:3], {}), (x[:, ::2], out, {}), (x, out.double(), {}),
                       (x, out, dict(ids=torch.zeros((4, 5), device="cuda"))),
                       (x, out, dict(weights=torch.zeros((4, 4), device="cuda")))):
        with pytest.raises(ValueError):
            layer.forward(bx, bo, **kw)
    with pytest.raises(q.QmlpError) as e:
        layer.forward(torch.zeros((5, 256), device="cuda", dtype=torch.bfloat16), torch.zeros((5, 256), device="cuda"))
    assert e.value.status == 4
    with pytest.raises(q.QmlpError) as e:
        layer.forward(x, x)
    assert e.value.status == 3
    layer.close()
    moe.close()
