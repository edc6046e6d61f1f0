"""Sizes at the ends of the mixture-of-experts layer's ranges: rows of more than 8192
values, which the one-kernel form alone takes, and more tokens than eight times a grid's
second dimension."""
import pytest

import test_gpu_moe_layer as base
import weight_quantized_swiglu_gb300 as q
from test_gpu_moe_layer import torch  # noqa: F401 (the fixture)

pytestmark = pytest.mark.gpu

LONG = [  # as test_gpu_moe_layer.py's
    (10, 1, 8256, 64, 3, 4, "softmax", False, True, 1.0, True, "bf16", "bf16", "bf16", (1, 2, 8)),
    (6, 0, 12288, 32, 2, 3, "sigmoid", False, True, 1.0, False, "bf16", "fp16", "fp32", (1, 5)),
    (5, 0, 16384, 96, 2, 4, "softmax", False, False, 1.0, False, "fp32", "bf16", "fp32", (1, 3)),
]


@pytest.mark.parametrize("case", LONG, ids=lambda c: "-".join(map(str, c)))
def test_long_rows(torch, case):  # noqa: F811
    base.test_layer(torch, case)


def test_long_rows_of_too_many_tokens_are_refused(torch):  # noqa: F811
    """x of 16 tokens of 16384 values does not fit, and the grouped form does not take it."""
    moe = base.Bank(4, 16384, 32, 4, 1).handle()
    router = torch.randn((4, 16384), device="cuda").bfloat16()
    for tokens in (16, 17, 4096):
        with pytest.raises(q.QmlpError) as e:
            q.MoeLayer(moe, router, 2, max_tokens=tokens)
        assert e.value.status == 4
    moe.close()


def test_more_tokens_than_a_grids_second_dimension(torch):  # noqa: F811
    E, K, M = 6, 64, 8 * 65535 + 9
    moe = base.Bank(E, K, 32, 4, 3).handle()
    g = torch.Generator(device="cuda").manual_seed(3)
    router = torch.randn((E, K), generator=g, device="cuda").bfloat16()
    layer = q.MoeLayer(moe, router, 2, max_tokens=M)
    x = torch.randn((M, K), generator=g, device="cuda").bfloat16()
    out, ids = torch.empty((M, K), device="cuda"), torch.empty((M, 2), dtype=torch.int32, device="cuda")
    layer.forward(x, out, ids=ids)
    for at in (0, 4096, M // 2 // 8 * 8, M - 65):  # a token's result does not depend on the others
        n = min(65, M - at)
        part, pid = torch.empty((n, K), device="cuda"), torch.empty((n, 2), dtype=torch.int32, device="cuda")
        layer.forward(x[at:at + n].contiguous(), part, ids=pid)
        assert torch.equal(part, out[at:at + n]) and torch.equal(pid, ids[at:at + n])
    layer.close()
    moe.close()
