"""One projection with 4-bit weights against the sums in 64 bits.

Tolerances, from the arithmetic (u = 2^-24). Up to 16 tokens the products are exact
(weights, or codes less zeros, and x are exact in fp16) unless x is bf16 and under
2^-29 of its row's largest value, where it is off by 2^-25 of 2^-14 of that: below
2^-38 of the largest. A sum of K terms in any order, of partial sums that the tensor
cores may cut off instead of rounding (2 u a step of 16): K u of the terms' sizes,
held against K u + 64 u for the scales', factor's and bias's own products. The
output rounds once more, by half a step of its type."""
import numpy as np
import pytest

import layer_reference as ref
import weight_quantized_swiglu_gb300 as q

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.fixture(scope="module")
def torch(cuda_available):
    import torch
    from weight_quantized_swiglu_gb300 import build
    build.build()
    return torch


def weights(fmt, N, K, G, seed, zmax=16):
    """Checkpoint arrays and the weights that they stand for, in fp64."""
    g = np.random.default_rng(seed)
    w = g.integers(0, 256, (N, K // 2), dtype=np.uint8)
    codes = np.stack((w & 15, w >> 4), -1).reshape(N, K)
    if fmt == "nvfp4":
        sc = g.integers(1, 126, (N, K // 16), dtype=np.uint8)
        e, m = sc >> 3, (sc & 7).astype(float)
        s = np.where(e > 0, (1 + m / 8) * 2.0 ** (e - 7.0), m * 2.0 ** -9)
        v = ref.E2M1[codes & 7] * np.where(codes & 8, -1.0, 1.0) * np.repeat(s, 16, 1)
        return dict(w=w, scale=sc), v
    sc = (g.uniform(0.1, 0.4, (N, K // G)) * K ** -0.5).astype(np.float16)
    z = g.integers(0, zmax, (N, K // G), dtype=np.uint8)
    v = (codes.astype(float) - np.repeat(z.astype(float), G, 1)) * np.repeat(sc.astype(float), G, 1)
    return dict(w=w, scale=sc, zero=z, group=G), v


def check(torch, x, v, out, factor=1.0, bias=None, more=0.0):
    xd = x.double().cpu().numpy()
    b = 0.0 if bias is None else bias.astype(float)
    want = xd @ v.T * factor + b
    size = np.abs(xd) @ np.abs(v).T * abs(factor) + np.abs(b)
    tol = ((x.shape[1] + 64) * U + more) * size
    if x.dtype == torch.bfloat16:  # what the scaling to fp16 leaves of the smallest values
        tol = tol + 2.0 ** -38 * np.abs(xd).max(1, keepdims=True) * np.abs(v).sum(1)[None] * abs(factor)
    half = torch.finfo(out.dtype).eps / 2
    small = 2.0 ** -25 if out.dtype == torch.float16 else 0.0  # half of fp16's smallest step
    got = out.double().cpu().numpy()
    bad = np.abs(got - want) > tol + half * (np.abs(want) + tol) + small
    assert not bad.any(), (int(bad.sum()), float(np.abs(got - want).max()))


CASES = [  # format, group, N, K, tokens, x, out, bias
    ("nvfp4", 16, 16, 16, (1, 2), "bf16", "fp32", False),
    ("nvfp4", 16, 17, 48, (1, 8, 9), "fp16", "bf16", True),
    ("nvfp4", 16, 1000, 5120, (1, 3, 16), "bf16", "bf16", False),
    ("nvfp4", 16, 5120, 1024, (1, 5, 11, 17), "bf16", "fp16", False),
    ("nvfp4", 16, 300, 17408, (1, 8, 16), "fp16", "fp32", False),
    ("nvfp4", 16, 40, 65536, (1, 16), "bf16", "fp32", False),
    ("int4", 32, 1, 32, (1, 3), "bf16", "fp32", True),
    ("int4", 32, 1001, 256, (1, 5, 16), "bf16", "bf16", True),
    ("int4", 32, 5120, 2080, (1, 7, 12, 33), "fp16", "fp16", False),
    ("int4", 64, 333, 192, (2, 10), "fp16", "fp32", False),
    ("int4", 64, 2048, 17408, (1, 8, 13), "bf16", "bf16", False),
    ("int4", 128, 17408, 640, (1, 8), "fp16", "bf16", False),
    ("int4", 128, 77, 5120, (1, 4, 15, 64), "bf16", "fp32", True),
    ("int4", 128, 20, 65536, (1, 9), "fp16", "fp32", False),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_few_tokens(torch, case):
    fmt, G, N, K, tokens, xt, ot, has_bias = case
    T = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
    a, v = weights(fmt, N, K, G, N + K)
    glob = 37.0 if fmt == "nvfp4" else 1.0
    bias = np.random.default_rng(1).normal(size=N).astype(np.float32) if has_bias else None
    lin = q.QuantLinear(fmt, N, K, max(tokens), global_scale=glob, bias=bias, **a)
    g = torch.Generator(device="cuda").manual_seed(K)
    for M in tokens:
        x = torch.randn((M, K), generator=g, device="cuda").to(T[xt])
        out = torch.full((M, N), 7.0, device="cuda", dtype=T[ot])
        lin.forward(x, out)
        again = torch.empty_like(out)
        lin.forward(x, again)
        torch.cuda.synchronize()
        assert torch.equal(out.view(torch.uint8), again.view(torch.uint8))
        check(torch, x, v, out, 1.0 / np.float64(np.float32(glob)), bias)
    lin.close()


MANY = [  # format, group, N, K, tokens, x, out, bias
    ("nvfp4", 16, 1000, 1040, (20, 64, 65, 255, 256, 300), "bf16", "bf16", True),
    ("nvfp4", 16, 256, 5120, (40, 513), "fp16", "fp32", False),
    ("int4", 32, 5120, 608, (24, 100, 257), "bf16", "fp16", False),
    ("int4", 64, 77, 17408, (33, 64, 400), "fp16", "bf16", True),
    ("int4", 128, 2050, 2048, (31, 200, 1000), "bf16", "fp32", True),
    ("int4", 32, 40, 65536, (64, 256), "bf16", "fp32", False),
    ("int4", 128, 5120, 4096, (2000,), "bf16", "bf16", False),
]


@pytest.mark.parametrize("case", MANY, ids=lambda c: "-".join(map(str, c)))
def test_many_tokens(torch, case):
    """From 65 tokens on an INT4 weight is rounded to fp16, 2^-11 of its size; with an fp32
    out nothing of it is left out."""
    fmt, G, N, K, tokens, xt, ot, has_bias = case
    T = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
    a, v = weights(fmt, N, K, G, N + K)
    bias = np.random.default_rng(1).normal(size=N).astype(np.float32) if has_bias else None
    lin = q.QuantLinear(fmt, N, K, max(tokens), global_scale=0.3 if fmt == "nvfp4" else 1.0, bias=bias, **a)
    factor = 1.0 / np.float64(np.float32(0.3)) if fmt == "nvfp4" else 1.0
    g = torch.Generator(device="cuda").manual_seed(K)
    for M in tokens:
        x = torch.randn((M, K), generator=g, device="cuda").to(T[xt])
        out = torch.full((M, N), 7.0, device="cuda", dtype=T[ot])
        lin.forward(x, out)
        again = torch.empty_like(out)
        lin.forward(x, again)
        lin.check()
        assert torch.equal(out.view(torch.uint8), again.view(torch.uint8))
        check(torch, x, v, out, factor, bias, 2.0 ** -11 if M >= 65 and fmt == "int4" and ot != "fp32" else 0.0)
    lin.close()


def test_weights_in_several_slabs(torch):
    """A projection whose images pass 1 GiB: the rows at the slabs' ends."""
    N, K, M = 70001, 8192, 300
    g = torch.Generator(device="cuda").manual_seed(1)
    w = torch.randint(0, 256, (N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    s = torch.rand((N, K // 128), generator=g, device="cuda").half() * 0.01
    z = torch.randint(0, 16, (N, K // 128), generator=g, device="cuda", dtype=torch.uint8)
    lin = q.QuantLinear("int4", N, K, M, w, s, zero=z, group=128)
    x = torch.randn((M, K), generator=g, device="cuda").to(torch.bfloat16)
    out = torch.empty((M, N), device="cuda")
    lin.forward(x, out)
    lin.check()
    rows = [*range(0, 40), *range(65500, 65600), *range(69960, 70001)]
    c = torch.stack((w[rows] & 15, w[rows] >> 4), -1).flatten(1).double()
    v = (c - z[rows].double().repeat_interleave(128, 1)) * s[rows].double().repeat_interleave(128, 1)
    check(torch, x, v.cpu().numpy(), out[:, rows].contiguous())
    lin.close()


def test_single_weights_and_any_zero(torch):
    """One-hot tokens return single weights, exactly; zeros over the whole byte."""
    for fmt, G, zmax in (("nvfp4", 16, 0), ("int4", 32, 256), ("int4", 128, 256)):
        N, K = 48, 384
        a, v = weights(fmt, N, K, G, 5, zmax)
        lin = q.QuantLinear(fmt, N, K, 16, **a)
        eye = torch.eye(K, device="cuda")
        for dt in (torch.bfloat16, torch.float16):
            got = torch.empty((K, N), device="cuda")
            for k in range(0, K, 16):
                lin.forward(eye[k:k + 16].to(dt).contiguous(), got[k:k + 16])
            assert np.array_equal(got.double().cpu().numpy(), v.T)
        lin.close()


def test_ranges_of_x(torch):
    """Tokens whose values span bf16's range, zeros, and values that are not finite,
    which stay in their own token."""
    N, K = 96, 512
    a, v = weights("int4", N, K, 64, 9)
    lin = q.QuantLinear("int4", N, K, 8, **a)
    g = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn((8, K), generator=g, device="cuda")
    x[1] *= 1e30
    x[2] *= 1e-30
    x[3] = 0
    x[4] *= torch.exp2(torch.randint(-20, 20, (K,), generator=g, device="cuda").float())
    x = x.to(torch.bfloat16)
    out = torch.empty((8, N), device="cuda")
    lin.forward(x, out)
    check(torch, x, v, out)
    bad = x.clone()
    bad[6, 3], bad[7, 100] = float("nan"), float("inf")
    got = torch.empty_like(out)
    lin.forward(bad, got)
    assert torch.equal(got[:6], out[:6]) and got[6].isnan().all() and not got[7].isfinite().any()
    lin.close()


def test_captured_and_on_a_side_stream(torch):
    N, K, M = 700, 4096, 6
    a, v = weights("nvfp4", N, K, 16, 3)
    lin = q.QuantLinear("nvfp4", N, K, M, **a)
    x = torch.randn((M, K), device="cuda").to(torch.bfloat16)
    out = torch.empty((M, N), device="cuda", dtype=torch.bfloat16)
    lin.forward(x, out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lin.forward(x, out)
    x.copy_(torch.randn((M, K), device="cuda"))
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    check(torch, x, v, out)
    side, other = torch.cuda.Stream(), torch.empty_like(out)
    side.wait_stream(torch.cuda.current_stream())
    lin.forward(x, other, stream=side)
    side.synchronize()
    assert torch.equal(out, other)
    lin.close()


def test_refusals(torch):
    a, _ = weights("int4", 64, 256, 64, 1)
    lin = q.QuantLinear("int4", 64, 256, 4, **a)
    x = torch.zeros((4, 256), device="cuda", dtype=torch.bfloat16)
    out = torch.zeros((4, 64), device="cuda")
    lin.forward(x, out)
    for bx, bo in ((x[:, :128], out), (x.float(), out), (x, out.double()), (x.t(), out), (x, out[:3]), (x.cpu(), out)):
        with pytest.raises(ValueError):
            lin.forward(bx, bo)
    with pytest.raises(q.QmlpError) as e:
        lin.forward(torch.zeros((5, 256), device="cuda", dtype=torch.bfloat16), torch.zeros((5, 64), device="cuda"))
    assert e.value.status == 4
    raw = torch.zeros(4 * 256 + 8, device="cuda", dtype=torch.bfloat16)
    with pytest.raises(q.QmlpError) as e:
        lin.forward(raw[1:1025].view(4, 256), out)
    assert e.value.status == 2
    lin.close()
