"""The norms around a block where a group of threads walks over rows, two at a time,
and where rows start behind a border of eight values: sizes at the ends of those
walks, with the tolerances of test_gpu_norm.py."""
import pytest

import test_gpu_norm as base
import weight_quantized_swiglu_gb300 as q
from test_gpu_norm import torch  # noqa: F401 (the fixture)

pytestmark = pytest.mark.gpu

CASES = [  # M, K, types of z / residual / weights, gate, post, pre, shift, weight offset
    (304, 1024, "bf16", "bf16", "bf16", "none", True, True, 0, 0.0),
    (305, 1032, "fp16", "fp32", "fp32", "full", True, True, 0, 1.0),
    (609, 520, "bf16", "fp32", "bf16", "channel", True, True, 0, 0.0),
    (1223, 640, "bf16", "bf16", "fp32", "token", True, True, 0, 0.0),
    (1999, 777, "fp16", "fp16", "fp16", "channel", True, True, 0, 1.0),
    (2500, 33, "bf16", "fp32", "bf16", "full", True, True, 0, 0.0),
    (3041, 8, "bf16", "bf16", "bf16", "token", True, True, 0, 0.0),
    (1300, 4097, "bf16", "bf16", "bf16", "token", True, True, 0, 0.0),
    (333, 5121, "fp16", "fp32", "fp16", "full", True, True, 0, 0.0),
    (1217, 6152, "bf16", "bf16", "bf16", "channel", True, True, 0, 0.0),
    (310, 8177, "bf16", "bf16", "fp32", "none", True, True, 0, 0.0),
    (160, 8192, "fp16", "fp32", "fp16", "full", True, True, 0, 0.0),
    (1216, 520, "bf16", "bf16", "bf16", "full", False, True, 0, 0.0),
    (320, 263, "fp16", "fp32", "fp32", "channel", True, False, 0, 0.0),
    (153, 1031, "bf16", "bf16", "bf16", "token", False, False, 0, 0.0),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_forward_and_backward(torch, case):  # noqa: F811
    base.test_forward_and_backward(torch, case)


@pytest.mark.parametrize("M,K,rdt", [(1300, 1024, "bf16"), (611, 1001, "fp32"), (400, 1999, "bf16")])
def test_rows_do_not_meet(torch, M, K, rdt):  # noqa: F811
    """Inf and NaN in rows that are computed beside others, share a chunk of eight values
    with them or come last; in place; and the rows are those of a shorter call."""
    rdt = {"bf16": torch.bfloat16, "fp32": torch.float32}[rdt]
    d = base.make(torch, M, K, torch.bfloat16, rdt, torch.float32, "full", True, True, 5)
    norm = q.BlockNorm(K, residual_dtype=rdt, weight_dtype=torch.float32, gate="full")
    rows = [0, 3, 152, 155, M // 2, M - 2, M - 1]
    outs = []
    for spoil in (False, True):
        io = {n: d[n].clone() for n in ("z", "residual", "post_w", "pre_w", "gate")}
        dout = d["dout"].clone()
        if spoil:
            io["z"][rows, 0], io["gate"][rows, K - 1] = float("nan"), float("inf")
            io["residual"][rows, K - 1], dout[rows, 0] = float("inf"), float("nan")
        h, y, stats = torch.empty_like(io["residual"]), torch.empty_like(io["z"]), torch.empty((M, 2), device="cuda")
        norm.forward(residual_out=h, out=y, stats=stats, **io)
        g = {"dz": torch.empty_like(y), "dresidual": torch.empty_like(h), "dgate": torch.empty_like(y)}
        norm.backward(stats, dout=dout, dresidual_out=d["dresidual_out"], **io, **g)
        here = io["residual"].clone()
        norm.forward(**{**io, "residual": here}, residual_out=here, out=torch.empty_like(y))
        assert torch.equal(here.view(torch.uint8), h.view(torch.uint8))
        outs.append((h, y, *g.values()))
    rest = torch.ones(M, dtype=torch.bool, device="cuda")
    rest[rows] = False
    for a, b in zip(*outs):
        assert torch.equal(a[rest], b[rest]) and not b[rows].isfinite().all(1).any()
    norm.close()


def test_weights_gradients_with_infinite_rows_left_out(torch):  # noqa: F811
    """Rows behind the last one (the walks' partners) add nothing: the sums over M tokens
    are those of the formula for every M beside a multiple of the walks."""
    K = 640
    for M in (304, 305, 456, 457, 607):
        base.test_forward_and_backward(torch, (M, K, "bf16", "bf16", "fp32", "channel", True, True, 0, 0.0))
        # what lies behind the arrays is never read into them
        buf = torch.full((M + 400, K), float("nan"), device="cuda", dtype=torch.bfloat16)
        d = base.make(torch, M, K, torch.bfloat16, torch.bfloat16, torch.float32, "none", True, True, 9)
        norm = q.BlockNorm(K, weight_dtype=torch.float32)
        z, dout = buf[:M], buf.clone()[:M]
        z.copy_(d["z"])
        dout.copy_(d["dout"])
        h, y, stats = torch.empty_like(z), torch.empty_like(z), torch.empty((M, 2), device="cuda")
        io = dict(z=z, residual=d["residual"], post_w=d["post_w"], pre_w=d["pre_w"])
        norm.forward(residual_out=h, out=y, stats=stats, **io)
        g = {n: torch.empty(K, device="cuda") for n in ("dpost_w", "dpre_w")}
        norm.backward(stats, dout=dout, dresidual_out=d["dresidual_out"], **io, **g)
        assert all(t.isfinite().all() for t in (h, y, *g.values()))
        norm.close()
