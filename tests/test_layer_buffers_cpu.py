"""What BlockNorm, QuantLinear and MoeLayer refuse before anything is launched: arrays
that a kernel would read or write past their end or take for another type. Stand-ins
take the place of the CUDA tensors and of the library, so no GPU is needed; the
library's own checks of what a handle is made from are called as they are."""
import ctypes
import types

import numpy as np
import pytest
import torch

import weight_quantized_swiglu_gb300 as q

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


class Buffer:
    """What the classes ask of a tensor."""

    def __init__(self, shape, dtype=BF, cuda=True, contiguous=True):
        self.shape, self.dtype, self.is_cuda, self.contiguous = tuple(shape), dtype, cuda, contiguous

    def numel(self):
        return int(np.prod(self.shape))

    def dim(self):
        return len(self.shape)

    def element_size(self):
        return self.dtype.itemsize

    def is_contiguous(self):
        return self.contiguous

    def is_floating_point(self):
        return self.dtype.is_floating_point

    def data_ptr(self):
        return 1 << 20


@pytest.fixture
def calls(monkeypatch):
    """The calls that reach the library."""
    made = []

    def entry(name):
        return lambda *a: made.append((name, a)) or 0

    names = ("qmlp_norm_forward", "qmlp_norm_backward", "qmlp_linear_forward", "qmlp_moe_layer_forward")
    monkeypatch.setattr(q, "lib", lambda: types.SimpleNamespace(**{n: entry(n) for n in names}))
    monkeypatch.setattr(q, "_stream", lambda s: 0)
    for n in ("qmlp_norm", "qmlp_linear", "qmlp_moe_layer"):
        monkeypatch.setattr(q, n + "_create", lambda *a, **k: 1)
        monkeypatch.setattr(q, n + "_destroy", lambda h: None)
    return made


M, K = 6, 32


def norm_io(**kw):
    d = dict(z=Buffer((M, K)), residual=Buffer((M, K), F32), post_w=Buffer((K,), F32), pre_w=Buffer((K,), F32),
             residual_out=Buffer((M, K), F32), out=Buffer((M, K)), stats=Buffer((M, 2), F32))
    d.update(kw)
    return d


def test_block_norm(calls):
    for kw in (dict(gate="row"), dict(dtype=torch.float64), dict(residual_dtype=torch.int8)):
        with pytest.raises(ValueError):
            q.BlockNorm(K, **kw)
    for kind, gate in (("none", None), ("channel", Buffer((K,), F32)), ("token", Buffer((M,))), ("full", Buffer((M, K)))):
        norm = q.BlockNorm(K, residual_dtype=F32, weight_dtype=F32, gate=kind)
        io = norm_io(gate=gate)
        norm.forward(**io)
        norm.forward(**norm_io(gate=gate, z=Buffer((2, 3, K))))  # a padded batch's shape
        grads = dict(dout=Buffer((M, K)), dresidual_out=Buffer((M, K), F32), dz=Buffer((M, K)),
                     dresidual=Buffer((M, K), F32), dpost_w=Buffer((K,), F32), dpre_w=Buffer((K,), F32))
        if gate is not None:
            grads["dgate"] = Buffer(gate.shape, gate.dtype)
        back = {n: io[n] for n in ("z", "residual", "post_w", "pre_w", "gate", "stats")}
        norm.backward(**back, **grads)
        assert [c[0] for c in calls] == ["qmlp_norm_forward"] * 2 + ["qmlp_norm_backward"]
        for names, fn, good in (([n for n in io if io[n] is not None], norm.forward, io),
                                (list(grads), norm.backward, {**back, **grads})):
            for n in names:
                b = good[n]
                other = HF if b.dtype != HF else BF
                wrong = [Buffer(b.shape, other), Buffer(b.shape, b.dtype, cuda=False),
                         Buffer(b.shape, b.dtype, contiguous=False), Buffer((b.shape[0] + 1, *b.shape[1:]), b.dtype),
                         Buffer(b.shape[:-1] + (b.shape[-1] - 1,), b.dtype), Buffer((), b.dtype)]
                if n == "z":  # (M follows z)
                    wrong.pop(3)
                if len(b.shape) == 2 and b.shape[0] != b.shape[1]:
                    wrong.append(Buffer(b.shape[::-1], b.dtype))
                for w in wrong:
                    with pytest.raises(ValueError):
                        fn(**{**good, n: w})
        assert len(calls) == 3
        calls.clear()
    with pytest.raises(ValueError):
        norm.forward(gate=Buffer((M, K)), out=Buffer((M, K)))  # no M


def test_quant_linear(calls):
    N = 24
    w, s = np.zeros((N, K // 2), np.uint8), np.zeros((N, K // 16), np.uint8)
    for kw in (dict(fmt="int8", w=w, scale=s), dict(fmt="nvfp4", w=w[:, :8], scale=s), dict(fmt="nvfp4", w=w, scale=s[:3]),
               dict(fmt="nvfp4", w=w, scale=s, bias=np.zeros(N - 1, np.float32)),
               dict(fmt="int4", w=w, scale=np.zeros((N, 1), np.float16), zero=s, group=32)):
        with pytest.raises(ValueError):
            q.QuantLinear(kw.pop("fmt"), N, K, M, **kw)
    lin = q.QuantLinear("nvfp4", N, K, M, w, s)
    x, out = Buffer((M, K)), Buffer((M, N), F32)
    lin.forward(x, out)
    lin.forward(Buffer((2, 3, K), HF), out)
    assert len(calls) == 2
    for bx, bo in ((Buffer((M, K), F32), out), (Buffer((M, K), torch.int16), out), (Buffer((M, K), cuda=False), out),
                   (Buffer((M, K), contiguous=False), out), (Buffer((K, M)), out), (x, Buffer((M - 1, N), F32)),
                   (x, Buffer((N, M), F32)), (x, Buffer((M, N), torch.float64)), (x, Buffer((M, N), cuda=False)),
                   (x, Buffer((M, N), contiguous=False))):
        with pytest.raises(ValueError):
            lin.forward(bx, bo)
    with pytest.raises(ValueError):
        lin.forward(x, out, M=M + 1)
    assert len(calls) == 2


def test_moe_layer(calls):
    moe = types.SimpleNamespace(E=9, K=K, h=1)
    router, bias, sgate = torch.zeros(8, K, dtype=BF), torch.zeros(8), torch.zeros(1, K, dtype=BF)
    for r, kw in ((router[:7], {}), (router.double(), {}), (router[:, :16], {}), (router, dict(score="max")),
                  (router, dict(bias=bias[:7])), (router, dict(bias=bias.half())), (router, dict(shared_gate=sgate.half())),
                  (torch.zeros(8, 2 * K, dtype=BF)[:, ::2], {})):
        with pytest.raises(ValueError):
            q.MoeLayer(moe, r, 2, shared=1, **kw)
    layer = q.MoeLayer(moe, router, 2, shared=1, bias=bias, shared_gate=sgate)
    x, out = Buffer((M, K)), Buffer((M, K), F32)
    ids, w = Buffer((M, 2), torch.int32), Buffer((M, 2), F32)
    layer.forward(x, out)
    layer.forward(x, out, ids=ids, weights=w)
    assert len(calls) == 2
    for bx, bo, kw in ((Buffer((M, K), F32), out, {}), (x, Buffer((M - 1, K), F32), {}), (x, Buffer((K, M), F32), {}),
                       (Buffer((M, K), contiguous=False), out, {}), (x, Buffer((M, K), cuda=False), {}),
                       (x, Buffer((M, K), torch.int32), {}), (x, out, dict(ids=Buffer((M, 2), torch.int64))),
                       (x, out, dict(ids=w)), (x, out, dict(weights=ids)), (x, out, dict(weights=Buffer((M, 1), F32))),
                       (x, out, dict(ids=Buffer((M, 2), torch.int32, cuda=False))), (x, out, dict(M=M + 1))):
        with pytest.raises(ValueError):
            layer.forward(bx, bo, **kw)
    assert len(calls) == 2


def test_handles_of_the_library_refuse_bad_descriptions():
    from weight_quantized_swiglu_gb300 import build
    build.build()
    L, h = q.lib(), ctypes.c_void_p()
    bf16, f16, f32 = q.DT_BF16, q.DT_FP16, q.DT_FP32

    def norm(K=64, eps=1e-6, offset=0.0, scale=1.0, dt=bf16, rdt=f32, wdt=bf16, gate=q.GATE_NONE):
        d = q.qmlp_norm_desc(K, eps, offset, scale, dt, rdt, wdt, gate)
        return L.qmlp_norm_create(ctypes.byref(h), ctypes.byref(d), None)

    for kw in (dict(K=0), dict(K=-8), dict(dt=f32), dict(rdt=f16), dict(wdt=f16), dict(gate=9), dict(gate=-1),
               dict(eps=float("nan")), dict(eps=-1.0), dict(scale=float("inf")), dict(offset=float("nan"))):
        assert norm(**kw) in (1, 4) and not h.value, kw
    w = np.zeros(64 * 64, np.uint8)
    at = w.ctypes.data

    def linear(fmt=q.LINEAR_INT4, N=64, K=64, max_M=4, group=32, w=at, scale=at, zero=at, g=1.0, bias=None):
        d = q.qmlp_linear_desc(fmt, N, K, max_M, group, w, scale, zero, g, bias)
        return L.qmlp_linear_create(ctypes.byref(h), ctypes.byref(d), None)

    for kw in (dict(w=None), dict(scale=None), dict(zero=None), dict(fmt=7), dict(group=16), dict(group=48), dict(N=0),
               dict(K=0), dict(K=48), dict(max_M=0), dict(max_M=-1), dict(fmt=q.LINEAR_NVFP4, group=16),
               dict(fmt=q.LINEAR_NVFP4, zero=None, group=32), dict(fmt=q.LINEAR_NVFP4, zero=None, group=16, g=0.0),
               dict(fmt=q.LINEAR_NVFP4, zero=None, group=16, g=float("nan"))):
        assert linear(**kw) in (1, 4) and not h.value, kw
    d = q.qmlp_moe_layer_desc(at, bf16, None, None, 0, 2, q.SCORE_SOFTMAX, 1, 1.0, 4)
    assert L.qmlp_moe_layer_create(ctypes.byref(h), None, ctypes.byref(d), None) == 1 and not h.value
    assert L.qmlp_norm_create(None, None, None) == 1 and L.qmlp_linear_create(ctypes.byref(h), None, None) == 1
    assert L.qmlp_norm_forward(None, None, 1, None) == 1 and L.qmlp_linear_forward(None, None, bf16, 1, None, bf16, None) == 1
    assert L.qmlp_moe_layer_forward(None, None, bf16, 1, None, bf16, None, None, None) == 1
    assert L.qmlp_linear_check(None, None) == 1 and L.qmlp_moe_layer_check(None, None) == 1
    for destroy in (L.qmlp_norm_destroy, L.qmlp_linear_destroy, L.qmlp_moe_layer_destroy):
        destroy(None)
