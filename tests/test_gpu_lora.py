"""Low-rank adapters of many requests beside the dense block, against the
formulas in 64 bits (weights decoded by the oracle). The reference rounds act
and out to bf16 where the operation does, so what is left are roundings that
fall the other way: the block's own tolerances (helpers.compare) hold."""
import numpy as np
import pytest

import oracle
import weight_quantized_swiglu_gb300 as q
from weight_quantized_swiglu_gb300 import inputs as gen
from helpers import bits_from_dev, compare, to_dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch(cuda_available):
    import torch
    from weight_quantized_swiglu_gb300 import build
    build.build()
    return torch


def bf16(a):
    return oracle.bf16_bits_to_f64(gen.f32_to_bf16_bits(np.asarray(a, dtype=np.float32)))


def adapter(rng, K, I, r, parts=("gate", "up", "down"), gain=1.0):
    """fp64 arrays of bf16 values."""
    shapes = {"gate": (I, K), "up": (I, K), "down": (K, I)}
    d = {}
    for p in parts:
        N, D = shapes[p]
        d[p + "_a"] = bf16(rng.standard_normal((r, D)) * D ** -0.5)
        d[p + "_b"] = bf16(rng.standard_normal((N, r)) * 0.3 * gain)
    return d


def on_device(torch, d, scale):
    return q.Adapter(scale, **{n: torch.from_numpy(a.astype(np.float32)).to(torch.bfloat16).cuda()
                               for n, a in d.items()})


def weights(case):
    w = []
    for p in (case.gate, case.up, case.down):
        f = 1.0 / np.float64(p.global_scale) if case.fmt == "nvfp4" else p.scale.astype(np.float64)[:, None]
        w.append(oracle.decode_proj(p) * f)
    return w


def reference(case, w, x, ids, adapters):
    """adapters: {slot: (fp64 arrays, scale)}"""
    K, I = case.K, case.I

    def project(z, i, name):
        y = z @ w[i].T
        for s, (d, c) in adapters.items():
            rows = np.nonzero(ids == s)[0]
            if rows.size and name + "_a" in d:
                y[rows] += c * ((z[rows] @ d[name + "_a"].T) @ d[name + "_b"].T)
        return y
    g, u = project(x, 0, "gate"), project(x, 1, "up")
    act = bf16(g / (1 + np.exp(-g)) * u)
    return gen.f32_to_bf16_bits(project(act, 2, "down").astype(np.float32))


def x_of(rng, M, K):
    b = gen.gen_x_bf16(rng, M, K)
    return b, oracle.bf16_bits_to_f64(b)


def scaled_case(fmt, K, I, seed):
    """A block whose terms and the adapters' are of one size."""
    case = gen.gen_dense_case(fmt, K, I, 1, seed)
    if fmt == "fp8":
        for p in (case.gate, case.up, case.down):
            p.scale *= np.float32(0.02)
    return case


def run(torch, lora, mlp, xb, ids):
    out = torch.full((xb.shape[0], mlp.K), 0x7FC0, dtype=torch.int16, device="cuda")
    lora.forward(to_dev(xb), torch.from_numpy(ids.astype(np.int32)).cuda(), out)
    torch.cuda.synchronize()
    mlp.check()
    return bits_from_dev(out)


SHAPES = [(256, 512), (144, 208), (1280, 2560)]  # GEMM and split; neither; a partition over many CTAs


@pytest.mark.parametrize("fmt", ["nvfp4", "fp8"])
@pytest.mark.parametrize("K,I", SHAPES)
def test_tokens_of_many_adapters(torch, fmt, K, I):
    """1 to 800 tokens, ranks 1 to 33 and an adapter of one projection alone,
    empty slots, ids out of range on both sides."""
    rng = np.random.default_rng(K + I)
    case = scaled_case(fmt, K, I, 31)
    w = weights(case)
    mlp = q.QuantMLP.from_case(case, max_M=800)
    lora = q.LoraMLP(mlp, 6, 33)
    ads = {0: (adapter(rng, K, I, 16), 2.0), 1: (adapter(rng, K, I, 1), 0.5), 3: (adapter(rng, K, I, 33), -1.0),
           4: (adapter(rng, K, I, 5, parts=("gate",)), 1.0), 5: (adapter(rng, K, I, 8, parts=("down", "up")), 1.0)}
    for s, (d, c) in ads.items():
        lora.set(s, on_device(torch, d, c))
    for M in (1, 2, 3, 7, 8, 9, 16, 17, 61, 130, 300, 800):
        xb, x = x_of(rng, M, K)
        ids = rng.integers(-2, 9, M)
        if M == 1:
            ids[:] = 3
        compare(run(torch, lora, mlp, xb, ids), reference(case, w, x, ids, ads), what=f"{fmt} {K} {I} M={M}")
    lora.close()
    mlp.close()


@pytest.mark.parametrize("M", [1, 5, 40, 800])
def test_without_adapters_it_is_the_block(torch, M):
    """Ids of no slot, empty slots and an emptied slot: the block's own result
    (to the last bit where its sums are the same)."""
    case = gen.gen_dense_case("nvfp4", 256, 512, 1, 33)
    mlp = q.QuantMLP.from_case(case, max_M=800)
    lora = q.LoraMLP(mlp, 4, 16)
    rng = np.random.default_rng(M)
    lora.set(2, on_device(torch, adapter(rng, 256, 512, 4), 1.0))
    lora.set(2, None)
    xb, _ = x_of(rng, M, 256)
    want = torch.empty((M, 256), dtype=torch.int16, device="cuda")
    mlp.forward(to_dev(xb), want)
    torch.cuda.synchronize()
    assert np.array_equal(run(torch, lora, mlp, xb, rng.choice([-1, 0, 1, 2, 3, 4, 1 << 30], M)), bits_from_dev(want))
    lora.close()
    mlp.close()


@pytest.mark.parametrize("rank", [1, 7, 16, 17, 32, 48, 64])
@pytest.mark.parametrize("M", [4, 200])
def test_ranks(torch, rank, M):
    K, I = 256, 512
    rng = np.random.default_rng(rank)
    case = scaled_case("fp8", K, I, 34)
    mlp = q.QuantMLP.from_case(case, max_M=200)
    lora = q.LoraMLP(mlp, 2, rank)
    ads = {0: (adapter(rng, K, I, rank, gain=rank ** -0.5), 1.5), 1: (adapter(rng, K, I, max(1, rank // 2)), 0.7)}
    for s, (d, c) in ads.items():
        lora.set(s, on_device(torch, d, c))
    xb, x = x_of(rng, M, K)
    ids = rng.integers(0, 2, M)
    compare(run(torch, lora, mlp, xb, ids), reference(case, weights(case), x, ids, ads), what=f"rank {rank}")
    lora.close()
    mlp.close()


def test_a_tokens_result_does_not_depend_on_the_others(torch):
    """One token's row is the same bytes wherever it stands in a batch and
    whatever the other tokens' adapters are, and from call to call."""
    K, I, M = 256, 512, 500
    rng = np.random.default_rng(35)
    case = gen.gen_dense_case("nvfp4", K, I, 1, 35)
    mlp = q.QuantMLP.from_case(case, max_M=M)
    lora = q.LoraMLP(mlp, 5, 16)
    for s in range(5):
        lora.set(s, on_device(torch, adapter(rng, K, I, 16), 1.0))
    xb, _ = x_of(rng, M, K)
    ids = rng.integers(0, 5, M)
    a = run(torch, lora, mlp, xb, ids)
    assert np.array_equal(a, run(torch, lora, mlp, xb, ids))
    perm = rng.permutation(M)
    b = run(torch, lora, mlp, xb[perm], ids[perm])
    assert np.array_equal(a[perm], b)
    lora.close()
    mlp.close()


@pytest.mark.parametrize("M", [3, 100])
def test_stream_order_graph_and_a_changed_slot(torch, M):
    """Set, forward and set again on one stream without a wait; ids and x that
    change between replays of a captured call."""
    K, I = 256, 512
    rng = np.random.default_rng(36)
    case = gen.gen_dense_case("nvfp4", K, I, 1, 36)
    w = weights(case)
    mlp = q.QuantMLP.from_case(case, max_M=M)
    lora = q.LoraMLP(mlp, 2, 8)
    d = [adapter(rng, K, I, 8) for _ in range(3)]
    dev = [on_device(torch, a, 1.0) for a in d]
    xb, x = x_of(rng, M, K)
    ids = rng.integers(0, 2, M)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    xd, idd = to_dev(xb), torch.from_numpy(ids.astype(np.int32)).cuda()
    torch.cuda.synchronize()
    outs = [torch.empty((M, K), dtype=torch.int16, device="cuda") for _ in range(2)]
    lora.set(0, dev[0], stream=s)
    lora.set(1, dev[1], stream=s)
    lora.forward(xd, idd, outs[0], stream=s)
    lora.set(1, dev[2], stream=s)
    lora.forward(xd, idd, outs[1], stream=s)
    torch.cuda.synchronize()
    for k, second in enumerate((1, 2)):
        compare(bits_from_dev(outs[k]), reference(case, w, x, ids, {0: (d[0], 1.0), 1: (d[second], 1.0)}))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        lora.forward(xd, idd, outs[0], stream=s)
    xb2, x2 = x_of(rng, M, K)
    ids2 = rng.integers(-1, 2, M)
    xd.copy_(to_dev(xb2))
    idd.copy_(torch.from_numpy(ids2.astype(np.int32)).cuda())
    g.replay()
    torch.cuda.synchronize()
    compare(bits_from_dev(outs[0]), reference(case, w, x2, ids2, {0: (d[0], 1.0), 1: (d[2], 1.0)}))
    lora.close()
    mlp.close()


@pytest.mark.parametrize("fmt,rank", [("nvfp4", 16), ("nvfp4", 40), ("fp8", 7)])
@pytest.mark.parametrize("pattern", ["runs", "each", "few", "none"])
def test_long_batches(torch, fmt, rank, pattern):
    """Enough tokens and a long enough contraction for the terms to be steps of
    the GEMMs: slots whose tokens start and end inside tiles, tiles of several
    slots and of none, and the same bytes from call to call and after other
    calls."""
    K, I, M = 4096, 1024, 1333
    rng = np.random.default_rng(rank)
    case = scaled_case(fmt, K, I, 38)
    w = weights(case)
    mlp = q.QuantMLP.from_case(case, max_M=1400)
    lora = q.LoraMLP(mlp, 3, rank)
    ads = {0: (adapter(rng, K, I, rank, gain=rank ** -0.5), 1.5), 2: (adapter(rng, K, I, max(1, rank - 3)), -0.25)}
    for s, (d, c) in ads.items():
        lora.set(s, on_device(torch, d, c))
    xb, x = x_of(rng, M, K)
    ids = {"runs": np.repeat([2, -1, 0, 1, 2], [300, 5, 640, 100, 288]), "each": rng.integers(-1, 4, M),
           "few": np.where(np.arange(M) % 400 == 7, 2, 5), "none": np.full(M, -1)}[pattern]
    out = run(torch, lora, mlp, xb, ids)
    compare(out, reference(case, w, x, ids, ads), what=f"{fmt} {pattern}")
    run(torch, lora, mlp, xb[:1000], rng.integers(0, 3, 1000))
    assert np.array_equal(out, run(torch, lora, mlp, xb, ids))
    lora.close()
    mlp.close()


@pytest.mark.parametrize("fmt,M", [("nvfp4", 1), ("nvfp4", 4), ("fp8", 3), ("nvfp4", 100), ("fp8", 800)])
def test_waits_that_run_out_are_reported(torch, fmt, M):
    """A weight step that is never loaded: the call ends by its bounded waits,
    the handle reports it, and the next call is right again."""
    K, I = 256, 512
    rng = np.random.default_rng(39)
    case = scaled_case(fmt, K, I, 39)
    mlp = q.QuantMLP.from_case(case, max_M=800)
    lora = q.LoraMLP(mlp, 2, 8)
    ads = {1: (adapter(rng, K, I, 8), 1.0)}
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
    compare(run(torch, lora, mlp, xb, ids), reference(case, weights(case), x, ids, ads))
    lora.close()
    mlp.close()


def test_ids_of_another_type_are_refused(torch):
    mlp = q.QuantMLP.from_case(gen.gen_dense_case("nvfp4", 256, 512, 1, 40), max_M=8)
    lora = q.LoraMLP(mlp, 1, 8)
    x = torch.zeros((4, 256), dtype=torch.bfloat16, device="cuda")
    for ids in (torch.zeros(4, dtype=torch.int64, device="cuda"), torch.zeros(4, device="cuda"),
                torch.zeros(8, dtype=torch.int32, device="cuda")[::2], torch.zeros(3, dtype=torch.int32, device="cuda")):
        with pytest.raises(ValueError):
            lora.forward(x, ids, torch.empty_like(x))
    lora.close()
    mlp.close()


def test_refusals(torch):
    case = gen.gen_dense_case("nvfp4", 256, 512, 1, 37)
    mlp = q.QuantMLP.from_case(case, max_M=16)
    for slots, rank in ((0, 8), (1025, 8), (4, 0), (4, 65)):
        with pytest.raises(q.QmlpError) as e:
            q.LoraMLP(mlp, slots, rank)
        assert e.value.status == 4, (slots, rank)
    lora = q.LoraMLP(mlp, 2, 8)
    rng = np.random.default_rng(0)
    ok = on_device(torch, adapter(rng, 256, 512, 8), 1.0)
    big = on_device(torch, adapter(rng, 256, 512, 9), 1.0)
    for slot, a, st in ((2, ok, 1), (-1, ok, 1), (0, big, 4)):
        with pytest.raises(q.QmlpError) as e:
            lora.set(slot, a)
        assert e.value.status == st
    half = q.qmlp_adapter(8, 1.0, ok.c.gate_a, None, None, None, None, None)
    assert q.qmlp_lora_set(lora.h, 0, half) == 1
    with pytest.raises(ValueError):
        lora.set(0, on_device(torch, adapter(rng, 512, 256, 8), 1.0))
    x = torch.zeros((17, 256), dtype=torch.bfloat16, device="cuda")
    out = torch.zeros((17, 256), dtype=torch.bfloat16, device="cuda")
    ids = torch.zeros(17, dtype=torch.int32, device="cuda")
    f = q.qmlp_lora_forward
    assert f(lora.h, x, ids, 0, out) == 4 and f(lora.h, x, ids, 17, out) == 4
    assert f(lora.h, None, ids, 1, out) == 1 and f(lora.h, x, None, 1, out) == 1 and f(lora.h, x, ids, 1, None) == 1
    assert f(None, x, ids, 1, out) == 1
    assert f(lora.h, x.data_ptr() + 2, ids, 1, out) == 2 and f(lora.h, x, ids.data_ptr() + 1, 1, out) == 2
    assert f(lora.h, x, ids, 4, x) == 3 and f(lora.h, x, out.data_ptr() + 64, 4, out) == 3
    lora.close()
    mlp.close()
