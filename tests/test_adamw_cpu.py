"""AdamW entry points: refusals that need no GPU. Addresses are made up; every
check here is host arithmetic that runs before any device call."""
import ctypes

import pytest

import weight_quantized_swiglu_gb300 as q
from weight_quantized_swiglu_gb300 import build as qbuild

OK, INVALID, ALIGN, ALIAS, SHAPE = 0, 1, 2, 3, 4
B = 1 << 32


@pytest.fixture(scope="module")
def L():
    qbuild.build()
    return q.lib()


def tensor(n=1000, **kw):
    d = dict(param=B, master=None, grad=B + 0x10000, m=B + 0x20000, v=B + 0x30000, m_scale=None, v_scale=None)
    d.update(kw)
    return q.qmlp_adamw_tensor(n, d["param"], d["master"], d["grad"], d["m"], d["v"], d["m_scale"], d["v_scale"])


def create(L, ts, pdt=q.DT_FP32, gdt=q.DT_FP32, state=q.STATE_FP32):
    h = ctypes.c_void_p()
    arr = (q.qmlp_adamw_tensor * max(1, len(ts)))(*ts)
    return L.qmlp_adamw_create(ctypes.byref(h), arr, len(ts), pdt, gdt, state, None)


def test_null_and_enums(L):
    h = ctypes.c_void_p()
    assert L.qmlp_adamw_create(None, None, 1, 3, 3, 1, None) == INVALID
    assert L.qmlp_adamw_create(ctypes.byref(h), None, 1, 3, 3, 1, None) == INVALID
    for kw in ({"pdt": q.DT_FP16}, {"gdt": q.DT_FP16}, {"state": 3}, {"pdt": 0}):
        assert create(L, [tensor()], **kw) == INVALID, kw
    assert L.qmlp_adamw_step(None, None, None) == INVALID
    L.qmlp_adamw_destroy(None)


@pytest.mark.parametrize("field", ["param", "grad", "m", "v"])
def test_a_missing_buffer(L, field):
    assert create(L, [tensor(**{field: None})]) == INVALID


def test_shapes(L):
    assert create(L, []) == SHAPE
    assert create(L, [tensor(n=0)]) == SHAPE
    assert create(L, [tensor(n=-5)]) == SHAPE
    assert create(L, [tensor(n=1 << 50)]) == SHAPE


def test_masters_and_scales(L):
    m = B + 0x40000
    assert create(L, [tensor(master=m)]) == INVALID  # beside fp32
    assert create(L, [tensor(master=m), tensor(param=B + 0x90000)], pdt=q.DT_BF16) == INVALID  # mixed
    assert create(L, [tensor()], state=q.STATE_8BIT) == INVALID  # no scales
    assert create(L, [tensor(m_scale=m, v_scale=m + 64)]) == INVALID  # scales beside fp32 states


def test_alignment(L):
    assert create(L, [tensor(param=B + 2)]) == ALIGN
    assert create(L, [tensor(grad=B + 0x10001)], gdt=q.DT_BF16) == ALIGN
    assert create(L, [tensor(m=B + 0x20002)]) == ALIGN


@pytest.mark.parametrize("a,b", [("param", "m"), ("m", "v"), ("param", "grad"), ("grad", "v")])
def test_aliases_within_a_tensor(L, a, b):
    base = {"param": B, "grad": B + 0x10000, "m": B + 0x20000, "v": B + 0x30000}
    assert create(L, [tensor(**{b: base[a] + 3996})]) == ALIAS  # the last element overlaps the first


def test_aliases_between_tensors(L):
    other = dict(param=B + 0x50000, grad=B + 0x60000, m=B + 0x70000, v=B + 0x80000)
    assert create(L, [tensor(), tensor(**{**other, "m": B + 0x20000 + 16})]) == ALIAS
    # one gradient read by two tensors is no alias: the next check needs the device
    assert create(L, [tensor(), tensor(**{**other, "grad": B + 0x10000})]) not in (OK, ALIAS)
