"""The index-checking build (see test_gpu_debug_bounds.py) on the norms, the single
projection and the mixture-of-experts layer: every form of a call runs in a child
process that loads libqmlp_bounds.so; no check fails, and the outputs are the default
build's to the last bit.

Run as a script (the child): python test_gpu_debug_bounds_layer.py OUT.npz
"""
import json
import os
import subprocess
import sys

import numpy as np
import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
for p in (HERE, os.path.dirname(HERE)):
    if p not in sys.path:
        sys.path.insert(0, p)

import weight_quantized_swiglu_gb300 as q  # noqa: E402
from weight_quantized_swiglu_gb300 import build  # noqa: E402

pytestmark = pytest.mark.gpu


def _bytes(torch, *ts):
    return [t.detach().contiguous().view(-1).view(torch.uint8).cpu().numpy() for t in ts]


def _norm(torch, M, K, dt, rdt, wdt, gate, shift):
    from test_gpu_norm import make
    T = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
    d = make(torch, M, K, T[dt], T[rdt], T[wdt], gate, True, True, K, shift)
    io = {n: d[n] for n in ("z", "residual", "post_w", "pre_w", "gate")}
    norm = q.BlockNorm(K, dtype=T[dt], residual_dtype=T[rdt], weight_dtype=T[wdt], gate=gate)
    h, y, stats = d["empty"](d["residual"]), d["empty"](d["z"]), torch.empty((M, 2), device="cuda")
    g = {"dz": d["empty"](d["z"]), "dresidual": d["empty"](d["residual"])}
    g.update({"d" + n: d["empty"](d[n]) for n in ("post_w", "pre_w", "gate") if d[n] is not None})
    norm.forward(residual_out=h, out=y, stats=stats, **io)
    norm.backward(stats, dout=d["dout"], dresidual_out=d["dresidual_out"], **io, **g)
    torch.cuda.synchronize()
    norm.close()
    return _bytes(torch, h, y, *g.values())


def _linear(torch, fmt, N, K, G, tokens):
    from test_gpu_linear import weights
    a, _ = weights(fmt, N, K, G, N)
    lin = q.QuantLinear(fmt, N, K, max(tokens), **a)
    g = torch.Generator(device="cuda").manual_seed(K)
    outs = []
    for M in tokens:
        x = torch.randn((M, K), generator=g, device="cuda").bfloat16()
        out = torch.empty((M, N), device="cuda")
        lin.forward(x, out)
        outs.append(out)
    lin.check()
    lin.close()
    return _bytes(torch, *outs)


def _moe(torch, E, S, K, I, topk, meta, tokens, dtype="bf16"):
    from test_gpu_moe_layer import Bank
    moe = Bank(E + S, K, I, meta, E).handle()
    g = torch.Generator(device="cuda").manual_seed(K)
    router = (torch.randn((E, K), generator=g, device="cuda") * K ** -0.5).bfloat16()
    layer = q.MoeLayer(moe, router, topk, shared=S, max_tokens=max(tokens))
    outs = []
    for M in tokens:
        x = torch.randn((M, K), generator=g, device="cuda").bfloat16()
        out = torch.empty((M, K), device="cuda", dtype=torch.float32 if dtype == "fp32" else torch.bfloat16)
        ids = torch.empty((M, topk), dtype=torch.int32, device="cuda")
        layer.forward(x, out, ids=ids)
        outs += [out, ids]
    layer.check()
    layer.close()
    moe.close()
    return _bytes(torch, *outs)


def cases():
    out = {}
    for a in ((1, 5120, "bf16", "bf16", "bf16", "none", 0), (1300, 1024, "bf16", "bf16", "fp32", "full", 0),
              (2000, 520, "fp16", "fp32", "fp16", "channel", 0), (333, 2571, "bf16", "fp32", "bf16", "token", 0),
              (400, 8192, "bf16", "bf16", "bf16", "channel", 0), (3, 16384, "fp16", "fp16", "fp16", "full", 0),
              (50, 300, "bf16", "fp32", "fp32", "token", 3), (9, 9000, "fp16", "fp16", "fp16", "none", 1)):
        out[f"norm {a[0]} {a[1]}"] = lambda t, a=a: _norm(t, *a)
    for a in (("nvfp4", 1000, 5120, 16, (1, 5, 12, 40, 64, 65, 300)), ("int4", 333, 192, 64, (1, 8, 9, 100)),
              ("int4", 77, 17408, 128, (1, 7, 33)), ("int4", 17408, 640, 32, (1, 8, 20)),
              ("nvfp4", 17, 48, 16, (1, 8, 9))):
        out[f"linear {a[0]} {a[1]}"] = lambda t, a=a: _linear(t, *a)
    for a in ((512, 1, 640, 160, 10, 4, (1, 4, 16, 40)), (30, 0, 4096, 1024, 2, 4, (16, 1)),
              (12, 1, 8192, 64, 3, 4, (1, 12)), (7, 2, 320, 96, 7, 3, (1, 9, 17)), (40, 1, 512, 256, 6, 4, (3, 16)),
              (31, 0, 4096, 1024, 2, 4, (16, 5, 1), "fp32"), (8, 2, 320, 96, 7, 3, (1, 9, 17), "fp32")):
        out[f"moe {a[0]} {a[2]}"] = lambda t, a=a: _moe(t, *a)
    return out


def run(checking):
    import torch
    outs, reports = {}, {}
    for name, fn in cases().items():
        for i, b in enumerate(fn(torch)):
            outs[f"{name} {i}"] = b
        if checking:
            reports[name] = list(q.qmlp_debug_bounds())
    return outs, reports


def test_checking_build_is_clean_and_bit_identical(cuda_available, tmp_path):
    build.build()
    lib_check = build.build(bounds=True)
    out = str(tmp_path / "bounds.npz")
    r = subprocess.run([sys.executable, os.path.abspath(__file__), out], env=dict(os.environ, QMLP_LIB=lib_check),
                       capture_output=True, text=True, timeout=900)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-4000:]
    got = np.load(out)
    for name, rep in json.load(open(out + ".json")).items():
        assert rep == [0, 0, 0], (name, rep)
    ref, _ = run(False)
    assert set(ref) == set(got.files)
    for name, b in ref.items():
        assert np.array_equal(got[name], b), name


if __name__ == "__main__":
    assert q.qmlp_debug_bounds_enabled() == 1, "QMLP_LIB does not name a checking build"
    outs, reports = run(True)
    np.savez(sys.argv[1], **outs)
    with open(sys.argv[1] + ".json", "w") as f:
        json.dump(reports, f)
