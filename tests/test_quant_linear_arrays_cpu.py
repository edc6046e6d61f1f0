"""The arrays that QuantLinear is made from: what has another type or shape is refused
even where it has as many bytes (a bf16 scale is not an fp16 one, a transposed weight not
a weight), and every documented kind is taken. Nothing here needs a GPU: the library's
entry is replaced."""
import numpy as np
import pytest
import torch

import weight_quantized_swiglu_gb300 as q

N, K = 48, 128  # (no array has the shape of its transpose)


@pytest.fixture
def made(monkeypatch):
    """The descriptions that reach the library."""
    seen = []
    monkeypatch.setattr(q, "qmlp_linear_create", lambda d, s=None: seen.append(d) or 1)
    monkeypatch.setattr(q, "qmlp_linear_destroy", lambda h: None)
    monkeypatch.setattr(q, "lib", lambda: type("L", (), {"qmlp_linear_forward": None}))
    return seen


def nvfp4(**kw):
    return {**dict(w=np.zeros((N, K // 2), np.uint8), scale=np.zeros((N, K // 16), np.uint8),
                   bias=np.zeros(N, np.float32)), **kw}


def int4(G, **kw):
    return {**dict(w=np.zeros((N, K // 2), np.uint8), scale=np.zeros((N, K // G), np.float16),
                   zero=np.zeros((N, K // G), np.uint8), group=G, bias=np.zeros(N, np.float32)), **kw}


def test_documented_arrays_are_taken(made):
    e4m3 = torch.zeros((N, K // 16), dtype=torch.uint8).view(torch.float8_e4m3fn)
    for kw in (nvfp4(), nvfp4(scale=e4m3), nvfp4(bias=None), nvfp4(w=np.zeros((K // 2, N), np.uint8).T),
               {n: torch.from_numpy(a) for n, a in nvfp4().items()}):
        q.QuantLinear("nvfp4", N, K, 4, **kw)
    for G in (32, 64, 128):
        q.QuantLinear("int4", N, K, 4, **int4(G))
        q.QuantLinear("int4", N, K, 4, **{n: torch.from_numpy(a) if isinstance(a, np.ndarray) else a
                                          for n, a in int4(G).items()})
    q.QuantLinear("int4", N, K, 4, 1 << 20, 1 << 20, zero=1 << 20, group=32)  # raw addresses: the caller's
    assert len(made) == 12 and all(d.w and d.scale for d in made)


WRONG_NVFP4 = [
    dict(w=np.zeros((K // 2, N), np.uint8)), dict(w=np.zeros((N, K // 2), np.int8)), dict(w=np.zeros((N, K // 4), np.uint16)),
    dict(w=torch.zeros((N, K // 4), dtype=torch.bfloat16)), dict(w=torch.zeros((K // 2, N), dtype=torch.uint8).t()),
    dict(scale=np.zeros((K // 16, N), np.uint8)), dict(scale=np.zeros((N, K // 32), np.float16)),
    dict(scale=torch.zeros((N, K // 16), dtype=torch.uint8).view(torch.float8_e5m2)),
    dict(scale=torch.zeros((N, K // 16), dtype=torch.int8)), dict(bias=np.zeros(2 * N, np.float16)),
    dict(bias=np.zeros(N, np.int32)), dict(bias=np.zeros((1, N), np.float32)), dict(bias=torch.zeros(2 * N, dtype=torch.bfloat16)),
]
WRONG_INT4 = [
    dict(scale=torch.zeros((N, K // 32), dtype=torch.bfloat16)), dict(scale=np.zeros((N, K // 32), np.int16)),
    dict(scale=np.zeros((K // 32, N), np.float16)), dict(scale=np.zeros((N, K // 64), np.float32)),
    dict(scale=np.zeros((N, K // 32), np.dtype(np.float16).newbyteorder())), dict(zero=np.zeros((K // 32, N), np.uint8)),
    dict(zero=np.zeros((N, K // 32), np.int8)), dict(zero=np.zeros((N, K // 64), np.float16)), dict(group=64), dict(group=0),
    dict(w=np.zeros((K // 2, N), np.uint8)),
]


@pytest.mark.parametrize("kw", WRONG_NVFP4, ids=range(len(WRONG_NVFP4)))
def test_nvfp4_arrays_of_another_kind_are_refused(made, kw):
    with pytest.raises(ValueError, match=f"QuantLinear: {list(kw)[0]} "):
        q.QuantLinear("nvfp4", N, K, 4, **nvfp4(**kw))
    assert not made


@pytest.mark.parametrize("kw", WRONG_INT4, ids=range(len(WRONG_INT4)))
def test_int4_arrays_of_another_kind_are_refused(made, kw):
    with pytest.raises(ValueError, match="QuantLinear: "):
        q.QuantLinear("int4", N, K, 4, **int4(32, **kw))
    assert not made
