"""The forms that a call with adapters takes at sizes which the smaller shapes do
not reach: decode partitions over more than a hundred CTAs, FP8's 9 to 16 tokens
in one launch, long batches with more than 128 slots, a thousand slots, and
changes of slots and captured calls in the one-token and the long form. Against
the formulas in 64 bits, as test_gpu_lora.py."""
import numpy as np
import pytest

import oracle
import weight_quantized_swiglu_gb300 as q
from helpers import bits_from_dev, compare, to_dev
from test_gpu_lora import adapter, on_device, reference, run, scaled_case, weights, x_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch(cuda_available):
    import torch
    from weight_quantized_swiglu_gb300 import build
    build.build()
    return torch


_CASES = {}


def wide(fmt):
    """1280 x 14592: 114 CTAs of eight row tiles, in both formats."""
    if fmt not in _CASES:
        case = scaled_case(fmt, 1280, 14592, 71)
        _CASES[fmt] = case, weights(case)
    return _CASES[fmt]


@pytest.mark.parametrize("fmt,max_rank", [("nvfp4", 16), ("nvfp4", 64), ("fp8", 16), ("fp8", 33)])
def test_decode_on_many_ctas(torch, fmt, max_rank):
    """Every token count of the partitioned kernel (FP8: two column tiles from 9
    on), mixed ranks and parts, none, and ids out of range."""
    K, I = 1280, 14592
    rng = np.random.default_rng(max_rank)
    case, w = wide(fmt)
    mlp = q.QuantMLP.from_case(case, max_M=16)
    assert mlp.decode_ctas() >= 100
    lora = q.LoraMLP(mlp, 5, max_rank)
    ads = {0: (adapter(rng, K, I, max_rank, gain=max_rank ** -0.5), 1.5), 1: (adapter(rng, K, I, 1), 0.5),
           3: (adapter(rng, K, I, max_rank - 5, ("down", "up"), gain=0.5), -1.0),
           4: (adapter(rng, K, I, 9, ("gate",)), 1.0)}
    for s, (d, c) in ads.items():
        lora.set(s, on_device(torch, d, c))
    for M in (1, 2, 3, 4, 5, 8, 9, 11, 15, 16):
        xb, x = x_of(rng, M, K)
        ids = rng.integers(-1, 6, M) if M > 1 else np.array([0])
        out = run(torch, lora, mlp, xb, ids)
        compare(out, reference(case, w, x, ids, ads), what=f"{fmt} M={M}")
        assert np.array_equal(out, run(torch, lora, mlp, xb, ids)), M
    # a token's bytes do not depend on its place or on the others' adapters
    perm = rng.permutation(M)
    assert np.array_equal(out[perm], run(torch, lora, mlp, xb[perm], ids[perm]))
    # without adapters: the block
    want = torch.empty((M, K), dtype=torch.int16, device="cuda")
    mlp.forward(to_dev(xb), want)
    torch.cuda.synchronize()
    assert np.array_equal(run(torch, lora, mlp, xb, np.full(M, -1)), bits_from_dev(want))
    lora.close()
    mlp.close()


@pytest.mark.parametrize("fmt,M", [("fp8", 9), ("fp8", 16), ("nvfp4", 1), ("nvfp4", 8)])
def test_waits_that_run_out_on_many_ctas(torch, fmt, M):
    """A weight step that is never loaded: reported, and the next call is right."""
    K, I = 1280, 14592
    rng = np.random.default_rng(M)
    case, w = wide(fmt)
    mlp = q.QuantMLP.from_case(case, max_M=16)
    lora = q.LoraMLP(mlp, 2, 16)
    ads = {1: (adapter(rng, K, I, 16, gain=0.25), 1.0)}
    lora.set(1, on_device(torch, *ads[1]))
    xb, x = x_of(rng, M, K)
    ids = np.ones(M, dtype=np.int64)
    out = torch.empty((M, K), dtype=torch.int16, device="cuda")
    mlp.set_wait(20_000_000, True)
    lora.forward(to_dev(xb), torch.from_numpy(ids.astype(np.int32)).cuda(), out)
    with pytest.raises(q.QmlpError) as e:
        mlp.check()
    assert e.value.status == 8
    mlp.set_wait(0, False)
    compare(run(torch, lora, mlp, xb, ids), reference(case, w, x, ids, ads))
    lora.close()
    mlp.close()


@pytest.mark.parametrize("slots,M", [(127, 1000), (130, 1000), (200, 1500)])
def test_many_slots_in_long_batches(torch, slots, M):
    """Terms as steps of the GEMMs with more slots than the plan counts in one
    table (128 groups), each token another slot or runs of one, and slots of few
    tokens; the same bytes from call to call."""
    K, I = 16384, 512
    rng = np.random.default_rng(slots)
    case = scaled_case("nvfp4", K, I, 72)
    w = weights(case)
    mlp = q.QuantMLP.from_case(case, max_M=M)
    lora = q.LoraMLP(mlp, slots, 3)
    kinds = [(adapter(rng, K, I, r), c) for r, c in ((3, 1.0), (1, -0.5), (2, 2.0))]
    dev = [on_device(torch, d, c) for d, c in kinds]
    for s in range(slots):
        if s % 4 != 3:  # every fourth slot stays empty
            lora.set(s, dev[s % 4])
    xb, x = x_of(rng, M, K)
    for pattern in ("each", "runs"):
        ids = rng.integers(-1, slots + 1, M)
        if pattern == "runs":
            ids = np.sort(ids)[::-1].copy()
        kind = np.where((ids >= 0) & (ids < slots), ids % 4, -1)
        out = run(torch, lora, mlp, xb, ids)
        compare(out, reference(case, w, x, kind, dict(enumerate(kinds))), what=pattern)
        assert np.array_equal(out, run(torch, lora, mlp, xb, ids))
    lora.close()
    mlp.close()


@pytest.mark.parametrize("M", [5, 200, 900])
def test_a_thousand_slots(torch, M):
    """The most slots that a handle takes: 1025 groups of the plan."""
    K, I, slots = 256, 512, 1024
    rng = np.random.default_rng(M)
    case = scaled_case("fp8", K, I, 73)
    mlp = q.QuantMLP.from_case(case, max_M=M)
    lora = q.LoraMLP(mlp, slots, 4)
    kinds = [(adapter(rng, K, I, r), c) for r, c in ((4, 1.0), (1, -0.5))]
    dev = [on_device(torch, d, c) for d, c in kinds]
    for s in range(slots):
        lora.set(s, dev[s % 2])
    xb, x = x_of(rng, M, K)
    ids = rng.integers(-1, slots + 1, M)
    ids[:3] = (1023, 0, 1024)
    kind = np.where((ids >= 0) & (ids < slots), ids % 2, -1)
    out = run(torch, lora, mlp, xb, ids)
    compare(out, reference(case, weights(case), x, kind, dict(enumerate(kinds))))
    lora.close()
    mlp.close()


@pytest.mark.parametrize("fmt,K,I,M", [("nvfp4", 256, 512, 1), ("nvfp4", 1280, 14592, 1), ("fp8", 1280, 14592, 12),
                                       ("nvfp4", 4096, 1024, 1000), ("fp8", 4096, 1024, 1000)])
def test_changed_slots_and_captured_calls(torch, fmt, K, I, M):
    """Set, forward, set, forward on one stream without a wait; then a captured
    call whose x, ids and slot change between replays."""
    rng = np.random.default_rng(M)
    case, w = wide(fmt) if I == 14592 else (scaled_case(fmt, K, I, 74), None)
    w = weights(case) if w is None else w
    mlp = q.QuantMLP.from_case(case, max_M=M)
    lora = q.LoraMLP(mlp, 2, 8)
    d = [adapter(rng, K, I, 8, gain=0.5) for _ in range(3)]
    dev = [on_device(torch, a, 1.0) for a in d]
    xb, x = x_of(rng, M, K)
    ids = rng.integers(-1, 2, M) if M > 1 else np.array([1])
    xd, idd = to_dev(xb), torch.from_numpy(ids.astype(np.int32)).cuda()
    outs = [torch.empty((M, K), dtype=torch.int16, device="cuda") for _ in range(4)]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for k in range(4):  # slot 1 changes before every call
        if k == 0:
            lora.set(0, dev[0], stream=s)
        lora.set(1, dev[1 + k % 2], stream=s)
        lora.forward(xd, idd, outs[k], stream=s)
    torch.cuda.synchronize()
    for k in range(4):
        compare(bits_from_dev(outs[k]), reference(case, w, x, ids, {0: (d[0], 1.0), 1: (d[1 + k % 2], 1.0)}))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        lora.forward(xd, idd, outs[0], stream=s)
    for k in range(3):
        xb, x = x_of(rng, M, K)
        ids = rng.integers(-1, 2, M) if M > 1 else np.array([1])
        xd.copy_(to_dev(xb))
        idd.copy_(torch.from_numpy(ids.astype(np.int32)).cuda())
        lora.set(1, dev[k])
        g.replay()
        torch.cuda.synchronize()
        compare(bits_from_dev(outs[0]), reference(case, w, x, ids, {0: (d[0], 1.0), 1: (d[k], 1.0)}))
    mlp.check()
    lora.close()
    mlp.close()


@pytest.mark.parametrize("M", [1, 6, 12, 40, 150, 800])
def test_values_that_are_not_finite_in_short_batches(torch, M):
    """The forms without steps: an adapter of Inf and NaN, in A and in B, leaves
    every other token's bytes alone."""
    K, I = 256, 512
    rng = np.random.default_rng(75)
    for fmt in ("nvfp4", "fp8"):
        case = scaled_case(fmt, K, I, 75)
        mlp = q.QuantMLP.from_case(case, max_M=max(M, 17))
        lora = q.LoraMLP(mlp, 3, 8)
        ads = [adapter(rng, K, I, 8) for _ in range(3)]
        for s in range(3):
            lora.set(s, on_device(torch, ads[s], 1.0))
        xb, _ = x_of(rng, M, K)
        ids = rng.integers(-1, 3, M)
        own = ids == 1
        healthy = run(torch, lora, mlp, xb, ids)
        bad = {n: a.copy() for n, a in ads[1].items()}
        bad["gate_a"][0, 3] = np.inf
        bad["up_b"][7, 1] = np.nan
        bad["down_b"][9, 0] = -np.inf
        lora.set(1, on_device(torch, bad, 1.0))
        got = run(torch, lora, mlp, xb, ids)
        assert np.array_equal(got[~own], healthy[~own])
        assert not np.any(np.isfinite(oracle.bf16_bits_to_f64(got[own])))
        lora.close()
        mlp.close()


@pytest.mark.parametrize("fmt", ["nvfp4", "fp8"])
@pytest.mark.parametrize("M", [2, 40, 900])
def test_on_tensor_parallel_shards(torch, fmt, M):
    """On a shard's handle an adapter has the shard's rows and columns, and a
    rank's output is its bf16 term of the sum."""
    K, I, n = 256, 1024, 2
    rng = np.random.default_rng(M)
    case = scaled_case(fmt, K, I, 76)
    w = weights(case)
    d = adapter(rng, K, I, 8)
    xb, x = x_of(rng, M, K)
    ids = rng.integers(-1, 1, M)
    for r in range(n):
        cut = slice(r * I // n, (r + 1) * I // n)
        mlp = q.QuantMLP.from_case(case, max_M=900, shard=(r, n))
        lora = q.LoraMLP(mlp, 1, 8)
        part = {p: a[cut] if p in ("gate_b", "up_b") else a[:, cut] if p == "down_a" else a for p, a in d.items()}
        lora.set(0, on_device(torch, {p: np.ascontiguousarray(a) for p, a in part.items()}, 1.0))
        shard = type(case).__new__(type(case))
        shard.__dict__.update(case.__dict__, I=I // n)
        want = reference(shard, (w[0][cut], w[1][cut], w[2][:, cut]), x, ids, {0: (part, 1.0)})
        compare(run(torch, lora, mlp, xb, ids), want, what=f"rank {r}")
        lora.close()
        mlp.close()
