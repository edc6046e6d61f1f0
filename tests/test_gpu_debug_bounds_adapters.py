"""The index-checking build (see test_gpu_debug_bounds.py) on the kernels of
adapters, training and AdamW: every form of a call runs in a child process that
loads libqmlp_bounds.so; no check fails, and the outputs are the default build's
to the last bit.

Run as a script (the child): python test_gpu_debug_bounds_adapters.py OUT.npz
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


def _adapter(torch, g, K, I, r):
    def part(*shape):
        return (torch.randn(shape, generator=g) * shape[1] ** -0.5).to(torch.bfloat16).cuda()
    return q.Adapter(1.5, gate_a=part(r, K), gate_b=part(I, r), up_a=part(r, K), up_b=part(I, r), down_a=part(r, I),
                     down_b=part(K, r))


def _bytes(torch, *ts):
    return [t.detach().contiguous().view(-1).view(torch.uint8).cpu().numpy() for t in ts]


def _case(fmt, K, I, seed):
    from test_gpu_lora import scaled_case
    return scaled_case(fmt, K, I, seed)


def _lora(torch, fmt, K, I, M, slots, rank, spoil=False):
    g = torch.Generator().manual_seed(M)
    mlp = q.QuantMLP.from_case(_case(fmt, K, I, 81), max_M=max(M, 17))
    lora = q.LoraMLP(mlp, slots, rank)
    ads = [_adapter(torch, g, K, I, r) for r in (rank, max(1, rank - 3), 1)]
    for s in range(slots):
        if s % 5 != 4:
            lora.set(s, ads[s % len(ads)])
    if spoil:
        ads[0].parts["gate_b"][3, 0] = float("inf")
        ads[0].parts["down_b"][5, 0] = float("nan")
        lora.set(1, ads[0])
    x = torch.randn((M, K), generator=g).to(torch.bfloat16).cuda()
    out = torch.empty_like(x)
    for k in range(2):
        ids = torch.randint(-1, slots + 1, (M,), generator=g, dtype=torch.int32).cuda()
        lora.forward(x, ids, out)
    torch.cuda.synchronize()
    mlp.check()
    lora.close()
    mlp.close()
    return _bytes(torch, out)


def _train(torch, fmt, K, I, M, r):
    g = torch.Generator().manual_seed(M + r)
    mlp = q.QuantMLP.from_case(_case(fmt, K, I, 82), max_M=max(M, 768))
    t = q.TrainMLP(mlp, max(r, 1))
    ad = _adapter(torch, g, K, I, r) if r else None
    grads = q.Adapter(1.0, **{n: torch.empty_like(p) for n, p in ad.parts.items()}) if r else None
    x, dy = (torch.randn((M, K), generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    out, dx = torch.empty_like(x), torch.empty_like(x)
    saved = torch.empty(t.saved_bytes(M), dtype=torch.uint8, device="cuda")
    t.forward(x, out, saved, adapter=ad)
    t.backward(x, saved, dy, dx, adapter=ad, grads=grads)
    torch.cuda.synchronize()
    mlp.check()
    t.close()
    mlp.close()
    return _bytes(torch, out, dx, *(grads.parts.values() if r else ()))


def _adamw(torch, eight):
    from test_gpu_adamw import HYPER, make
    d = make(torch, [1, 300, 2048 * 900 + 77, 4096], torch.bfloat16, torch.bfloat16, eight, True, 83)
    o = q.AdamW(d["params"], d["grads"], d["m"], d["v"], m_scale=d["m_scale"], v_scale=d["v_scale"],
                master=d["master"])
    o.step(**HYPER)
    torch.cuda.synchronize()
    o.close()
    return _bytes(torch, *d["params"], *d["master"], *(t.view(torch.uint8) for t in (*d["m"], *d["v"])))


def cases():
    out = {}
    for fmt, K, I, M, slots, rank in (
            ("nvfp4", 256, 512, 1, 3, 8), ("fp8", 256, 512, 6, 3, 33), ("fp8", 1280, 14592, 13, 4, 16),
            ("nvfp4", 144, 208, 30, 3, 8), ("nvfp4", 256, 512, 40, 3, 16), ("fp8", 256, 512, 200, 6, 5),
            ("nvfp4", 256, 512, 900, 1024, 4), ("nvfp4", 4096, 1024, 1333, 3, 40), ("fp8", 4096, 1024, 1000, 2, 16),
            ("nvfp4", 16384, 512, 1000, 130, 3)):
        out[f"lora {fmt} {K} {I} {M}"] = lambda t, a=(fmt, K, I, M, slots, rank): _lora(t, *a)
    out["lora not finite"] = lambda t: _lora(t, "fp8", 4096, 1024, 1000, 3, 7, spoil=True)
    for fmt, K, I, M, r in (("nvfp4", 256, 384, 20, 5), ("fp8", 256, 384, 100, 16), ("nvfp4", 2048, 5632, 50, 16),
                            ("nvfp4", 512, 1280, 700, 33), ("fp8", 512, 1280, 300, 64), ("fp8", 512, 1280, 1000, 0)):
        out[f"train {fmt} {K} {I} {M}"] = lambda t, a=(fmt, K, I, M, r): _train(t, *a)
    out["adamw 8 bit"] = lambda t: _adamw(t, True)
    out["adamw fp32"] = lambda t: _adamw(t, False)
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
