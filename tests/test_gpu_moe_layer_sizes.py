"""Rows of more than 8192 values, which the one-kernel form of the mixture-of-experts
layer alone takes."""
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
