"""The norms around a block against the formulas in 64 bits.

Tolerances, from the arithmetic (u = 2^-24; each fp32 operation rounds once, a
stored value once more by half a step of its type):
* 1/rms: a row's sum of squares passes at most 16 additions in a thread, 10 in the
  shuffles and 5 over warps: 32 u, halved by the root, with the root's own 2 units
  and the mean's and eps's roundings under 24 u.
* n: that and three products: 28 u of itself. h: a product and a sum more, of the
  size |r| + |scale gate n|: 32 u of it. y: h's error times w / rms, 1/rms again,
  two products: 80 u of that size over the rms, times |w|.
* gradients: each is a sum of products of those, with one row sum whose terms'
  sizes are added up as they are: 256 u of the sizes that the reference gives.
  Sums over M tokens: any order of M additions: M u of the terms' sizes more."""
import numpy as np
import pytest

import layer_reference as ref
import weight_quantized_swiglu_gb300 as q

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
EPS = 1e-6


@pytest.fixture(scope="module")
def torch(cuda_available):
    import torch
    from weight_quantized_swiglu_gb300 import build
    build.build()
    return torch


def f64(t):
    return None if t is None else t.double().cpu().numpy()


def half_step(torch, dtype):
    return torch.finfo(dtype).eps / 2


def make(torch, M, K, dt, rdt, wdt, gate, post, pre, seed, shift=0):
    """Inputs; shift moves each array's start by that many elements."""
    g = torch.Generator(device="cuda").manual_seed(seed)

    def t(shape, std, dtype, mean=0.0):
        n = int(np.prod(shape))
        a = torch.empty(n + shift, device="cuda", dtype=dtype)[shift:].view(shape)
        a.copy_(torch.randn(shape, generator=g, device="cuda") * std + mean)
        return a

    shapes = {"none": None, "channel": (K,), "token": (M,), "full": (M, K)}
    d = {"z": t((M, K), 0.7, dt), "residual": t((M, K), 2.0, rdt), "post_w": t((K,), 0.3, wdt, 1.0) if post else None,
         "pre_w": t((K,), 0.3, wdt, 1.0) if pre else None,
         "gate": None if gate == "none" else t(shapes[gate], 0.5, wdt if gate == "channel" else dt, 0.5)}
    d["dout"] = t((M, K), 0.1, dt) if pre else None
    d["dresidual_out"] = t((M, K), 0.1, rdt)
    d["empty"] = lambda a: torch.empty(a.numel() + shift, device="cuda", dtype=a.dtype)[shift:].view(a.shape)  # noqa: E731
    return d


def wide(gate, kind):
    return None if gate is None else f64(gate)[:, None] if kind == "token" else f64(gate)


CASES = [  # M, K, types of z / residual / weights, gate, post, pre, shift, weight offset
    (1, 5120, "bf16", "bf16", "bf16", "none", True, True, 0, 0.0),
    (3, 1, "bf16", "fp32", "fp32", "full", True, True, 0, 0.0),
    (2, 7, "fp16", "fp16", "fp16", "token", True, True, 0, 1.0),
    (33, 64, "bf16", "bf16", "fp32", "channel", True, True, 0, 0.0),
    (9, 255, "fp16", "fp32", "fp16", "full", True, True, 0, 0.0),
    (17, 256, "bf16", "bf16", "bf16", "token", False, True, 0, 1.0),
    (700, 512, "fp16", "fp16", "fp32", "none", True, False, 0, 0.0),
    (41, 520, "bf16", "fp32", "bf16", "channel", True, True, 0, 0.0),
    (40, 1000, "bf16", "bf16", "bf16", "full", False, True, 3, 0.0),
    (700, 1024, "fp16", "fp32", "fp16", "channel", True, True, 0, 0.0),
    (301, 2571, "fp16", "fp32", "fp16", "token", True, True, 0, 0.0),
    (5, 4096, "bf16", "bf16", "fp32", "full", True, True, 0, 0.0),
    (1000, 5120, "bf16", "fp32", "bf16", "channel", True, True, 0, 1.0),
    (2, 8192, "fp16", "fp16", "fp16", "none", True, True, 1, 0.0),
    (2, 8200, "bf16", "bf16", "bf16", "full", True, True, 0, 0.0),
    (3, 8201, "bf16", "fp32", "fp32", "channel", True, True, 0, 0.0),
    (310, 16384, "bf16", "bf16", "bf16", "token", True, True, 0, 0.0),
    (2, 16383, "fp16", "fp32", "fp16", "none", False, False, 0, 0.0),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_forward_and_backward(torch, case):
    M, K, dt, rdt, wdt, gate, post, pre, shift, off = case
    T = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
    dt, rdt, wdt, scale = T[dt], T[rdt], T[wdt], 0.75
    d = make(torch, M, K, dt, rdt, wdt, gate, post, pre, 11 + K, shift)
    io = {n: d[n] for n in ("z", "residual", "post_w", "pre_w", "gate")}
    norm = q.BlockNorm(K, eps=EPS, weight_offset=off, scale=scale, dtype=dt, residual_dtype=rdt, weight_dtype=wdt,
                       gate=gate)
    h, y = d["empty"](d["residual"]), d["empty"](d["z"]) if pre else None
    stats = torch.empty((M, 2), device="cuda")
    norm.forward(residual_out=h, out=y, stats=stats, **io)
    grads = {"dz": d["empty"](d["z"]), "dresidual": d["empty"](d["residual"])}
    for n in ("post_w", "pre_w", "gate"):
        if d[n] is not None:
            grads["d" + n] = d["empty"](d[n])
    norm.backward(stats, dout=d["dout"], dresidual_out=d["dresidual_out"], **io, **grads)
    first = {n: t.clone() for n, t in grads.items()}
    norm.backward(stats, dout=d["dout"], dresidual_out=d["dresidual_out"], **io, **grads)
    torch.cuda.synchronize()
    for n, t in grads.items():  # the same bytes again
        assert torch.equal(t.view(torch.uint8), first[n].view(torch.uint8)), n
    norm.close()

    args = (f64(d["z"]), f64(d["residual"]), f64(d["post_w"]), f64(d["pre_w"]), wide(d["gate"], gate), scale, off, EPS)
    wh, wy = ref.norm_forward(*args)
    n = wh - args[1]
    size = np.abs(args[1]) + np.abs(n)
    err = 32 * U * size
    assert np.all(np.abs(f64(h) - wh) <= err + half_step(torch, rdt) * (np.abs(wh) + err))
    if pre:
        w = np.abs(args[3] + off)
        err = 80 * U * size / ref.rms_of(wh, EPS) * w + 2.0 ** -25 * (dt == torch.float16)  # (fp16's subnormals)
        assert np.all(np.abs(f64(y) - wy) <= err + half_step(torch, dt) * (np.abs(wy) + err))
    want = ref.norm_backward(*args, f64(d["dout"]), f64(d["dresidual_out"]))
    kinds = {"dz": dt, "dresidual": rdt, "dpost_w": wdt, "dpre_w": wdt, "dgate": wdt if gate == "channel" else dt}
    for name, t in grads.items():
        v, s = want[name]
        terms = 0
        if name == "dgate" and gate in ("channel", "token"):
            ax = 0 if gate == "channel" else 1
            v, s, terms = v.sum(ax), s.sum(ax), M if gate == "channel" else 64
        elif name in ("dpost_w", "dpre_w"):
            terms = M
        tol = (256 + terms) * U * s + 2.0 ** -25 * (kinds[name] == torch.float16)
        bad = np.abs(f64(t) - v) > tol + half_step(torch, kinds[name]) * (np.abs(v) + tol)
        assert not bad.any(), (name, int(bad.sum()))


def test_parts_of_the_operator(torch):
    """Only the norm before; a block without a residual; in place; gradients that
    are not wanted; no gradient of the stream behind."""
    M, K, dt = 37, 768, torch.bfloat16
    d = make(torch, M, K, dt, dt, dt, "none", True, True, 5)
    norm = q.BlockNorm(K, eps=EPS, dtype=dt)
    stats = torch.empty((M, 2), device="cuda")
    full, y = torch.empty_like(d["z"]), torch.empty_like(d["z"])
    z, r, wp, wr = (d[n] for n in ("z", "residual", "post_w", "pre_w"))
    norm.forward(z=z, residual=r, post_w=wp, pre_w=wr, residual_out=full, out=y)
    here, y2 = r.clone(), torch.empty_like(z)
    norm.forward(z=z, residual=here, post_w=wp, pre_w=wr, residual_out=here, out=y2, stats=stats)  # in place
    assert torch.equal(here, full) and torch.equal(y, y2)
    only = torch.empty_like(z)
    norm.forward(residual=r, pre_w=wr, out=only)
    one, _ = ref.norm_forward(np.zeros((M, K)), f64(r), None, None, None, 1.0, 0.0, EPS)
    want = one / ref.rms_of(one, EPS) * f64(wr)
    assert np.all(np.abs(f64(only) - want) <= (2.0 ** -8 + 80 * U) * np.abs(want))
    alone = torch.empty_like(z)
    norm.forward(z=z, post_w=wp, residual_out=alone)
    want, _ = ref.norm_forward(f64(z), np.zeros((M, K)), f64(wp), None, None, 1.0, 0.0, EPS)
    assert np.all(np.abs(f64(alone) - want) <= (2.0 ** -8 + 32 * U) * np.abs(want))
    # backward: dresidual in place of dresidual_out, and each gradient by itself
    g = {n: torch.empty_like(t) for n, t in (("dz", z), ("dresidual", r), ("dpost_w", wp), ("dpre_w", wr))}
    io = dict(z=z, residual=r, post_w=wp, pre_w=wr, dout=d["dout"])
    norm.backward(stats, dresidual_out=d["dresidual_out"], **io, **g)
    for n, t in g.items():
        one = torch.empty_like(t)
        norm.backward(stats, dresidual_out=d["dresidual_out"], **io, **{n: one})
        assert torch.equal(one, t), n
    run = d["dresidual_out"].clone()
    norm.backward(stats, dresidual_out=run, dresidual=run, **io)
    assert torch.equal(run, g["dresidual"])
    zero, a = torch.zeros_like(r), torch.empty_like(z)
    norm.backward(stats, dresidual_out=zero, dz=a, **io)
    b = torch.empty_like(z)
    norm.backward(stats, dz=b, **io)
    assert torch.equal(a, b)
    norm.close()


def test_values_that_are_not_finite_stay_in_their_row(torch):
    M, K = 70, 640
    for gate in ("none", "full"):
        d = make(torch, M, K, torch.bfloat16, torch.bfloat16, torch.bfloat16, gate, True, True, 3)
        io = {n: d[n] for n in ("z", "residual", "post_w", "pre_w", "gate")}
        norm = q.BlockNorm(K, dtype=torch.bfloat16, gate=gate)
        outs = []
        for bad in (None, float("nan"), float("inf")):
            if bad is not None:
                d["z"][5, 9] = bad
                d["residual"][6, 0] = bad
            d["z"][7] = 0  # a row of zeros, and all of it zeros
            d["z"][8], d["residual"][8] = 0, 0
            h, y, dz = (torch.empty_like(d["z"]) for _ in range(3))
            stats = torch.empty((M, 2), device="cuda")
            norm.forward(residual_out=h, out=y, stats=stats, **io)
            norm.backward(stats, dout=d["dout"], dresidual_out=d["dresidual_out"], dz=dz, **io)
            outs.append((h, y, dz))
        rest = [i for i in range(M) if i not in (5, 6)]
        for o in outs[1:]:
            for a, b in zip(o, outs[0]):
                assert torch.equal(a[rest], b[rest])
        assert outs[0][0][8].eq(0).all() and outs[0][1][8].eq(0).all() and outs[0][2].isfinite().all()
        assert outs[1][0][5, 9].isnan() and outs[1][1][6].isnan().all()
        norm.close()


def test_captured_and_on_a_side_stream(torch):
    M, K, dt = 130, 2048, torch.float16
    d = make(torch, M, K, dt, torch.float32, torch.float32, "channel", True, True, 8)
    io = {n: d[n] for n in ("z", "residual", "post_w", "pre_w", "gate")}
    norm = q.BlockNorm(K, dtype=dt, residual_dtype=torch.float32, weight_dtype=torch.float32, gate="channel")
    h, y, stats = torch.empty_like(d["residual"]), torch.empty_like(d["z"]), torch.empty((M, 2), device="cuda")
    g = {"dz": torch.empty_like(d["z"]), "dresidual": torch.empty_like(d["residual"])}
    g.update({"d" + n: torch.empty_like(d[n]) for n in ("post_w", "pre_w", "gate")})

    def step(stream=None):
        norm.forward(residual_out=h, out=y, stats=stats, stream=stream, **io)
        norm.backward(stats, dout=d["dout"], dresidual_out=d["dresidual_out"], stream=stream, **io, **g)

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    d["z"].mul_(1.25)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    step(side)
    side.synchronize()
    want = {n: t.clone() for n, t in dict(h=h, y=y, **g).items()}
    for t in (h, y, *g.values()):
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    for n, t in dict(h=h, y=y, **g).items():
        assert torch.equal(t, want[n]), n
    norm.close()


def test_more_than_2_31_elements(torch):
    K = 16384
    M = 2 ** 31 // K + 3
    z = torch.zeros((M, K), dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(4)
    z[-4:] = torch.randn((4, K), generator=g, device="cuda").to(torch.bfloat16)
    w = torch.randn(K, generator=g, device="cuda").to(torch.bfloat16)
    norm = q.BlockNorm(K, dtype=torch.bfloat16)
    h = torch.empty_like(z)
    stats = torch.empty((M, 2), device="cuda")
    norm.forward(z=z, post_w=w, residual_out=h, stats=stats)
    want, _ = ref.norm_forward(f64(z[-4:]), np.zeros((4, K)), f64(w), None, None, 1.0, 0.0, EPS)
    assert np.all(np.abs(f64(h[-4:]) - want) <= (2.0 ** -8 + 32 * U) * np.abs(want))
    assert h[:M - 4].count_nonzero() == 0
    dz = torch.empty_like(z)
    norm.backward(stats, z=z, post_w=w, dresidual_out=h, dz=dz)
    got = ref.norm_backward(f64(z[-4:]), np.zeros((4, K)), f64(w), None, None, 1.0, 0.0, EPS, None, f64(h[-4:]))["dz"]
    assert np.all(np.abs(f64(dz[-4:]) - got[0]) <= 2.0 ** -8 * np.abs(got[0]) + 257 * U * got[1])
    norm.close()
