"""The operators around the quantized blocks together, as a decoder layer runs them: norms
with the residual, projections, a mixture-of-experts layer or a gated MLP between them.
Every operator's output is checked in 64 bits on the input that the one before gave it,
with that operator's own tolerances; the run is captured into a graph and replayed."""
import numpy as np
import pytest

import layer_reference as ref
import test_gpu_linear as linear
import test_gpu_moe_layer as moe_layer
import test_gpu_norm as norms
import weight_quantized_swiglu_gb300 as q
from test_gpu_norm import EPS, U, f64, torch  # noqa: F401 (the fixture)

pytestmark = pytest.mark.gpu


def check_norm(torch, z, r, wp, wr, h, y):  # noqa: F811
    """test_gpu_norm.py's tolerances; every array bf16."""
    wh, wy = ref.norm_forward(f64(z), f64(r), f64(wp), f64(wr), None, 1.0, 1.0, EPS)
    size = np.abs(f64(r)) + np.abs(wh - f64(r))
    err = 32 * U * size
    assert np.all(np.abs(f64(h) - wh) <= err + 2.0 ** -8 * (np.abs(wh) + err))
    err = 80 * U * size / ref.rms_of(wh, EPS) * np.abs(f64(wr) + 1.0)
    assert np.all(np.abs(f64(y) - wy) <= err + 2.0 ** -8 * (np.abs(wy) + err))


@pytest.mark.parametrize("M", [1, 5, 16, 40, 80])
def test_decoder_layer(torch, M):  # noqa: F811
    K, I, N, E, S, topk = 512, 96, 768, 24, 1, 4
    g = torch.Generator(device="cuda").manual_seed(M)
    w = [(torch.randn(K, generator=g, device="cuda") * 0.2).bfloat16() for _ in range(4)]
    up_a, up_v = linear.weights("nvfp4", N, K, 16, 1)
    down_a, down_v = linear.weights("int4", K, N, 64, 2)
    up = q.QuantLinear("nvfp4", N, K, M, global_scale=300.0, **up_a)
    down = q.QuantLinear("int4", K, N, M, **down_a)
    bank = moe_layer.Bank(E + S, K, I, 4, 3)
    moe = bank.handle()
    router = (torch.randn((E, K), generator=g, device="cuda") * K ** -0.5).bfloat16()
    layer = q.MoeLayer(moe, router, topk, shared=S, max_tokens=M)
    norm = q.BlockNorm(K, weight_offset=1.0)
    new = lambda n: torch.empty((M, n), device="cuda", dtype=torch.bfloat16)  # noqa: E731
    z, r = new(K), new(K)
    h1, y1, mid, z2, h2, y2, z3, h3, y3 = new(K), new(K), new(N), new(K), new(K), new(K), new(K), new(K), new(K)
    ids = torch.empty((M, topk), dtype=torch.int32, device="cuda")
    rw = torch.empty((M, topk), device="cuda")

    def step():
        norm.forward(z=z, residual=r, post_w=w[0], pre_w=w[1], residual_out=h1, out=y1)
        up.forward(y1, mid)
        down.forward(mid, z2)
        norm.forward(z=z2, residual=h1, post_w=w[2], pre_w=w[3], residual_out=h2, out=y2)
        layer.forward(y2, z3, ids=ids, weights=rw)
        norm.forward(z=z3, residual=h2, post_w=w[0], pre_w=w[1], residual_out=h3, out=y3)

    z.normal_(generator=g), r.normal_(generator=g)
    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    z.normal_(generator=g), r.normal_(generator=g)
    for t in (h1, y1, mid, z2, h2, y2, z3, h3, y3):
        t.fill_(float("nan"))
    graph.replay()
    torch.cuda.synchronize()
    for t in (up, down, layer):
        t.check()
    many = M >= 65
    check_norm(torch, z, r, w[0], w[1], h1, y1)
    linear.check(torch, y1, up_v, mid, 1.0 / np.float64(np.float32(300.0)))
    linear.check(torch, mid, down_v, z2, more=2.0 ** -11 if many else 0.0)
    check_norm(torch, z2, h1, w[2], w[3], h2, y2)
    moe_layer.verify(bank, f64(y2), f64(router), None, None,
                     dict(E=E, S=S, topk=topk, score="softmax", renorm=True, rscale=1.0), ids.cpu().numpy(), f64(rw),
                     f64(z3), 2.0 ** -8, True, M <= 16)
    check_norm(torch, z3, h2, w[0], w[1], h3, y3)
    # eagerly on another stream: the same bytes
    want = [t.clone() for t in (h3, y3, z3)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip((h3, y3, z3), want))
    for t in (up, down, layer, moe, norm):
        t.close()


@pytest.mark.parametrize("M", [24, 700])
def test_training_around_a_gated_mlp(torch, M):  # noqa: F811
    """Norm, frozen quantized MLP with an adapter, norm, and back through all three, as one
    captured step: the norms' gradients against the formulas on what they were given."""
    from test_gpu_lora import scaled_case
    K, I, r = 512, 768, 8
    g = torch.Generator(device="cuda").manual_seed(M)
    mlp = q.QuantMLP.from_case(scaled_case("nvfp4", K, I, 4), max_M=768)
    ad = q.Adapter(1.5, **{n: (torch.randn(s, generator=g, device="cuda") * s[1] ** -0.5).bfloat16()
                           for n, s in (("gate_a", (r, K)), ("gate_b", (I, r)), ("up_a", (r, K)), ("up_b", (I, r)),
                                        ("down_a", (r, I)), ("down_b", (K, r)))})
    agrads = q.Adapter(1.0, **{n: torch.empty_like(p) for n, p in ad.parts.items()})
    train = q.TrainMLP(mlp, r)
    a = norms.make(torch, M, K, torch.bfloat16, torch.bfloat16, torch.float32, "none", True, True, 1)
    norm = q.BlockNorm(K, scale=0.75, weight_dtype=torch.float32)
    e = torch.empty_like
    z, res, y2bar, h2bar = a["z"], a["residual"], a["dout"], a["dresidual_out"]
    h1, x, m, h2, y2, dm, dh1, dx, dz, dr = (e(z) for _ in range(10))
    s1, s2 = (torch.empty((M, 2), device="cuda") for _ in range(2))
    w = {"post_w": a["post_w"], "pre_w": a["pre_w"]}
    g1, g2 = ({"d" + n: e(t) for n, t in w.items()} for _ in range(2))
    saved = torch.empty(train.saved_bytes(M), dtype=torch.uint8, device="cuda")

    def step():
        norm.forward(z=z, residual=res, residual_out=h1, out=x, stats=s1, **w)
        train.forward(x, m, saved, adapter=ad)
        norm.forward(z=m, residual=h1, residual_out=h2, out=y2, stats=s2, **w)
        norm.backward(s2, z=m, residual=h1, dout=y2bar, dresidual_out=h2bar, dz=dm, dresidual=dh1, **w, **g2)
        train.backward(x, saved, dm, dx, adapter=ad, grads=agrads)
        norm.backward(s1, z=z, residual=res, dout=dx, dresidual_out=dh1, dz=dz, dresidual=dr, **w, **g1)

    step()
    first = [t.clone() for t in (y2, dz, dr, *g1.values(), *g2.values(), *agrads.parts.values())]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    graph.replay()
    torch.cuda.synchronize()
    mlp.check()
    for t, f in zip((y2, dz, dr, *g1.values(), *g2.values(), *agrads.parts.values()), first):
        assert torch.equal(t, f) and t.isfinite().all()
    for args, given, got in (((z, res), (dx, dh1), {"dz": dz, "dresidual": dr, **g1}),
                             ((m, h1), (y2bar, h2bar), {"dz": dm, "dresidual": dh1, **g2})):
        want = ref.norm_backward(f64(args[0]), f64(args[1]), f64(w["post_w"]), f64(w["pre_w"]), None, 0.75, 0.0, EPS,
                                 f64(given[0]), f64(given[1]))
        for n, t in got.items():
            v, s = want[n]
            tol = (256 + (M if n in g1 else 0)) * U * s
            assert np.all(np.abs(f64(t) - v) <= tol + torch.finfo(t.dtype).eps / 2 * (np.abs(v) + tol)), n
    for t in (train, mlp, norm):
        t.close()
