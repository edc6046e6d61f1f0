"""What the adapter and training classes refuse before anything is launched:
buffers that a kernel would read or write past their end. Stand-ins take the
place of the CUDA tensors and of the library, so no GPU is needed."""
import numpy as np
import pytest

import weight_quantized_swiglu_gb300 as q

K, I, M = 256, 512, 20


class Buffer:
    """What the classes ask of a tensor."""

    def __init__(self, shape, size=2, cuda=True, contiguous=True, floating=True, at=1 << 20):
        self.shape, self.size, self.is_cuda, self.contiguous, self.floating, self.at = (
            tuple(shape), size, cuda, contiguous, floating, at)

    def numel(self):
        return int(np.prod(self.shape))

    def dim(self):
        return len(self.shape)

    def element_size(self):
        return self.size

    def is_contiguous(self):
        return self.contiguous

    def is_floating_point(self):
        return self.floating

    def data_ptr(self):
        return self.at


class Block:
    K, I = K, I


@pytest.fixture
def calls(monkeypatch):
    """The calls that reach the library."""
    made = []
    for name in ("qmlp_lora_forward", "qmlp_train_forward", "qmlp_train_backward"):
        monkeypatch.setattr(q, name, lambda *a, _n=name: made.append(_n) or 0)
    monkeypatch.setattr(q, "qmlp_train_saved_bytes", lambda h, m: 1000 * m)
    return made


def handle(cls):
    h = cls.__new__(cls)
    h.mlp, h.h = Block(), None
    return h


def rows(m=M, **kw):
    return Buffer((m, K), **kw)


def saved(nbytes=1000 * M, **kw):
    return Buffer((nbytes,), size=1, **kw)


def test_saved_buffers(calls):
    t = handle(q.TrainMLP)
    for good in (saved(), saved(1000 * M + 7), Buffer((250 * M,), size=4), 1 << 20):
        t.forward(rows(), rows(), good)
        t.backward(rows(), good, rows(), rows())
    assert len(calls) == 8
    for bad in (saved(1000 * M - 1), saved(cuda=False), saved(contiguous=False), Buffer((250 * M - 1,), size=4)):
        with pytest.raises(ValueError, match="saved"):
            t.forward(rows(), rows(), bad)
        with pytest.raises(ValueError, match="saved"):
            t.backward(rows(), bad, rows(), rows())
    with pytest.raises(ValueError, match="saved"):  # M given apart from x
        t.forward(rows(), rows(), saved(), M=M + 1)
    assert len(calls) == 8


def adapter_of(rank, parts=("gate", "up", "down")):
    """An Adapter as its constructor leaves it, over stand-ins."""
    a = q.Adapter.__new__(q.Adapter)
    a.scale, a.parts = 1.0, {n: None for n in q.ADAPTER_PARTS}
    for p in parts:
        out, inp = {"gate": (I, K), "up": (I, K), "down": (K, I)}[p]
        a.parts[p + "_a"], a.parts[p + "_b"] = Buffer((rank, inp)), Buffer((out, rank))
    a.rank = rank if parts else 0
    a.c = q.qmlp_adapter(a.rank, 1.0, *[None if t is None else t.data_ptr() for t in a.parts.values()])
    return a


def test_gradients_of_another_rank(calls):
    t = handle(q.TrainMLP)
    for grads in (adapter_of(16), adapter_of(16, ("up",)), adapter_of(3, ()), None):
        t.backward(rows(), saved(), rows(), rows(), adapter=adapter_of(16), grads=grads)
    assert len(calls) == 4
    for rank in (1, 8, 15, 17, 32):
        with pytest.raises(ValueError, match="rank"):
            t.backward(rows(), saved(), rows(), rows(), adapter=adapter_of(16), grads=adapter_of(rank))
    assert len(calls) == 4


def ids(n=M, **kw):
    return Buffer((n,), **{"size": 4, "floating": False, **kw})


BAD_ROWS = [rows(M - 1), rows(cuda=False), rows(contiguous=False), rows(size=1), Buffer((K,)), Buffer((M, K // 2)),
            Buffer((M, 2 * K)), Buffer((M * K - 1,))]


def test_serving_buffers(calls):
    l = handle(q.LoraMLP)  # noqa: E741
    good = [rows(), rows(M + 5), Buffer((M * K,)), Buffer((4, M // 4, K)), Buffer((M, 2 * K), size=1), 1 << 20]
    for t in good:
        l.forward(t, ids(), rows(), M=M)
        l.forward(rows(), ids(), t)
    l.forward(rows(), ids(M + 1), rows())
    l.forward(rows(), 1 << 20, rows())
    n = 2 * len(good) + 2
    assert len(calls) == n
    for t in BAD_ROWS:
        with pytest.raises(ValueError, match="x "):
            l.forward(t, ids(), rows(), M=M)
        with pytest.raises(ValueError, match="out "):
            l.forward(rows(), ids(), t)
    with pytest.raises(ValueError, match="x "):  # one row of K values is not K tokens
        l.forward(Buffer((K,)), ids(K), rows(K))
    for t in (ids(cuda=False), ids(M - 1), ids(size=8), ids(floating=True), ids(contiguous=False)):
        with pytest.raises(ValueError, match="ids"):
            l.forward(rows(), t, rows())
    assert len(calls) == n


def test_training_buffers(calls):
    t = handle(q.TrainMLP)
    for bad in BAD_ROWS:
        with pytest.raises(ValueError, match="x "):
            t.forward(bad, rows(), saved(), M=M)
        with pytest.raises(ValueError, match="out "):
            t.forward(rows(), bad, saved())
        for at in range(3):
            a = [rows(), rows(), rows()]
            a[at] = bad
            with pytest.raises(ValueError, match=("x ", "dout ", "dx ")[at]):
                t.backward(a[0], saved(), a[1], a[2], M=M)
    assert not calls
