"""Forward and backward with frozen quantized weights against the formulas in
64 bits (train_reference.py, which is tested against differences).

Tolerances: a bf16 rounding is at most 2^-8 of a value, uniform: 2^-8 / sqrt(3)
in the 2-norm. out passes two (act, out); dx two (d gate and d up, dx), and with
FP8 weights a third (down's factors in the transposed weights); an adapter's
gradient two (act, or d gate and d up; the gradient itself), with FP8 a third.
So the 2-norm of a difference is under sqrt(k) 2^-8 / sqrt(3) of the result's;
single values under 2e-2 of the largest, as elsewhere."""
import numpy as np
import pytest

import oracle
import train_reference as ref
import weight_quantized_swiglu_gb300 as q
from weight_quantized_swiglu_gb300 import inputs as gen
from helpers import bits_from_dev, to_dev
from test_gpu_lora import adapter, on_device, scaled_case, weights, x_of

pytestmark = pytest.mark.gpu

ONE = 2.0 ** -8 / 3 ** 0.5
PARTS = ("gate", "up", "down")


@pytest.fixture(scope="module")
def torch(cuda_available):
    import torch
    from weight_quantized_swiglu_gb300 import build
    build.build()
    return torch


def close(got, want, k, what):
    got = got if got.dtype == np.float64 else oracle.bf16_bits_to_f64(got)
    assert np.all(np.isfinite(got)), what
    rel = np.linalg.norm(got - want) / np.linalg.norm(want)
    assert rel <= k ** 0.5 * ONE, f"{what}: rel {rel:.3e}"
    assert np.abs(got - want).max() <= 2e-2 * np.abs(want).max(), what


def step(torch, t, xb, dyb, ad=None, stream=None, want_grads=True):
    """(out, dx, grads) as they come from the device, in buffers filled with NaN."""
    M, K = xb.shape
    x, dy = to_dev(xb), to_dev(dyb)
    nan = lambda shape: torch.full(shape, 0x7FC0, dtype=torch.int16, device="cuda")  # noqa: E731
    out, dx = nan((M, K)), nan((M, K))
    saved = torch.full((t.saved_bytes(M),), 255, dtype=torch.uint8, device="cuda")
    grads = q.Adapter(1.0, **{n: nan(tuple(p.shape)).view(torch.bfloat16) for n, p in ad.parts.items()
                              if p is not None}) if ad is not None and want_grads else None
    torch.cuda.synchronize()
    t.forward(x, out, saved, adapter=ad, stream=stream)
    t.backward(x, saved, dy, dx, adapter=ad, grads=grads, stream=stream)
    torch.cuda.synchronize()
    t.mlp.check()
    g = {n: bits_from_dev(p.view(torch.int16)) for n, p in grads.parts.items() if p is not None} if grads else {}
    return bits_from_dev(out), bits_from_dev(dx), g


def compare_step(torch, t, case, w, xb, x, rng, parts, r, c):
    M, K, I = xb.shape[0], case.K, case.I
    dyb, dy = x_of(rng, M, K)
    a = adapter(rng, K, I, r, parts, gain=r ** -0.5) if r else {}
    ad = on_device(torch, a, c) if r else None
    out, dx, grads = step(torch, t, xb, dyb, ad)
    more = case.fmt == "fp8"
    close(out, ref.forward(w, x, a, c)[0], 2, f"out M={M}")
    wdx, wg = ref.backward(w, x, dy, a, c)
    close(dx, wdx, 2 + more, f"dx M={M}")
    assert set(grads) == set(wg)
    for n in grads:
        close(grads[n], wg[n], 2 + more, f"{n} M={M}")


@pytest.mark.parametrize("fmt", ["nvfp4", "fp8"])
@pytest.mark.parametrize("K,I", [(256, 384), (512, 1280)])  # the last 256-row tile of the transposed down half full
def test_step(torch, fmt, K, I):
    rng = np.random.default_rng(K)
    case = scaled_case(fmt, K, I, 51)
    w = weights(case)
    t = q.TrainMLP(q.QuantMLP.from_case(case, max_M=1100), 33)
    for M, r, parts in ((1, 4, PARTS), (2, 0, ()), (31, 16, PARTS), (64, 33, PARTS), (129, 5, ("up",)),
                        (255, 16, ("down", "gate")), (256, 1, PARTS), (300, 8, PARTS), (513, 17, PARTS),
                        (1030, 32, PARTS), (1100, 0, ())):
        xb, x = x_of(rng, M, K)
        compare_step(torch, t, case, w, xb, x, rng, parts, r, 1.3)
    t.close()
    t.mlp.close()


@pytest.mark.parametrize("rank", [1, 15, 16, 31, 33, 64])
def test_ranks(torch, rank):
    rng = np.random.default_rng(rank)
    case = scaled_case("nvfp4", 256, 512, 52)
    t = q.TrainMLP(q.QuantMLP.from_case(case, max_M=768), rank)
    xb, x = x_of(rng, 333, 256)
    compare_step(torch, t, case, weights(case), xb, x, rng, PARTS, rank, -0.8)
    t.close()
    t.mlp.close()


def test_channels_without_a_usable_factor(torch):
    """FP8 channels of gate and up whose factor is zero, negative or tiny: the
    gradients that carry the factor are never divided by it."""
    rng = np.random.default_rng(53)
    case = scaled_case("fp8", 256, 512, 53)
    for p in (case.gate, case.up):
        p.scale[::3] = 0.0
        p.scale[1::7] *= -1
        p.scale[2] = 1e-25
    t = q.TrainMLP(q.QuantMLP.from_case(case, max_M=768), 8)
    xb, x = x_of(rng, 200, 256)
    compare_step(torch, t, case, weights(case), xb, x, rng, PARTS, 8, 1.0)
    t.close()
    t.mlp.close()


def test_saturated_gates_and_zero_gradients(torch):
    """Gates far on both sides (SiLU and its derivative at their limits) stay
    finite; a zero dout gives zeros."""
    case = scaled_case("nvfp4", 256, 512, 54)
    t = q.TrainMLP(q.QuantMLP.from_case(case, max_M=768), 4)
    rng = np.random.default_rng(54)
    x = rng.standard_normal((300, 256)) * 10.0 ** rng.integers(-6, 5, (300, 1))
    xb = gen.f32_to_bf16_bits(x.astype(np.float32))
    dyb, _ = x_of(rng, 300, 256)
    ad = on_device(torch, adapter(rng, 256, 512, 4), 1.0)
    out, dx, grads = step(torch, t, xb, dyb, ad)
    for n, v in [("out", out), ("dx", dx), *grads.items()]:
        assert np.all(np.isfinite(oracle.bf16_bits_to_f64(v))), n
    out, dx, grads = step(torch, t, xb, np.zeros_like(dyb), ad)
    for n, v in [("dx", dx), *grads.items()]:
        assert not np.any(v & 0x7FFF), n
    t.close()
    t.mlp.close()


def test_forward_is_the_block_and_steps_repeat_bit_for_bit(torch):
    """Without an adapter the output is the block's own (its dequantise-once
    path) to the last bit; on another stream and in a captured graph a step
    gives the same bytes; gradients that are not asked for change nothing."""
    rng = np.random.default_rng(55)
    case = scaled_case("nvfp4", 256, 512, 55)
    mlp = q.QuantMLP.from_case(case, max_M=768)
    t = q.TrainMLP(mlp, 16)
    M = 700
    xb, _ = x_of(rng, M, 256)
    dyb, _ = x_of(rng, M, 256)
    want = torch.empty((M, 256), dtype=torch.int16, device="cuda")
    mlp.forward(to_dev(xb), want, path=q.PATH_GEMM_DQ)
    torch.cuda.synchronize()
    assert np.array_equal(step(torch, t, xb, dyb)[0], bits_from_dev(want))
    ad = on_device(torch, adapter(rng, 256, 512, 12), 1.0)
    a = step(torch, t, xb, dyb, ad)
    b = step(torch, t, xb, dyb, ad, stream=torch.cuda.Stream())
    c = step(torch, t, xb, dyb, ad, want_grads=False)
    assert np.array_equal(a[0], b[0]) and np.array_equal(a[1], b[1]) and np.array_equal(a[1], c[1])
    for n in a[2]:
        assert np.array_equal(a[2][n], b[2][n]), n
    x, dy = to_dev(xb), to_dev(dyb)
    out, dx = torch.empty_like(want), torch.empty_like(want)
    saved = torch.empty(t.saved_bytes(M), dtype=torch.uint8, device="cuda")
    grads = q.Adapter(1.0, **{n: torch.empty_like(p) for n, p in ad.parts.items()})
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        t.forward(x, out, saved, adapter=ad, stream=s)
        t.backward(x, saved, dy, dx, adapter=ad, grads=grads, stream=s)
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    assert np.array_equal(bits_from_dev(out), a[0]) and np.array_equal(bits_from_dev(dx), a[1])
    for n, p in grads.parts.items():
        assert np.array_equal(bits_from_dev(p.view(torch.int16)), a[2][n]), n
    t.close()
    mlp.close()


@pytest.mark.parametrize("M", [100, 600])
def test_waits_that_run_out_are_reported(torch, M):
    rng = np.random.default_rng(57)
    case = scaled_case("nvfp4", 256, 512, 57)
    mlp = q.QuantMLP.from_case(case, max_M=768)
    t = q.TrainMLP(mlp, 8)
    xb, x = x_of(rng, M, 256)
    dyb, _ = x_of(rng, M, 256)
    ad = on_device(torch, adapter(rng, 256, 512, 8), 1.0)
    mlp.set_wait(20_000_000, True)
    with pytest.raises(q.QmlpError) as e:
        step(torch, t, xb, dyb, ad)
    assert e.value.status == 8
    mlp.set_wait(0, False)
    compare_step(torch, t, case, weights(case), xb, x, rng, PARTS, 8, 1.0)
    t.close()
    mlp.close()


@pytest.mark.parametrize("fmt", ["nvfp4", "fp8"])
def test_split_tiles(torch, fmt):
    """Output tiles that the CTA pairs do not fill: shared over the contraction,
    with pairs left without work, and with all pairs busy before them."""
    rng = np.random.default_rng(58)
    case = scaled_case(fmt, 1024, 4096, 58)
    t = q.TrainMLP(q.QuantMLP.from_case(case, max_M=5000), 16)
    w = weights(case)
    for M, r in ((768, 16), (2049, 0), (4900, 5)):  # 12, 36 and 80 tiles of 256 x 256
        xb, x = x_of(rng, M, 1024)
        compare_step(torch, t, case, w, xb, x, rng, PARTS if r else (), r, 1.0)
    t.close()
    t.mlp.close()


def test_refusals(torch):
    small = q.QuantMLP.from_case(gen.gen_dense_case("nvfp4", 256, 512, 1, 56), max_M=100)
    odd = q.QuantMLP.from_case(gen.gen_dense_case("nvfp4", 144, 208, 1, 56), max_M=768)
    mlp = q.QuantMLP.from_case(gen.gen_dense_case("nvfp4", 256, 512, 1, 56), max_M=768)
    for m, r in ((small, 8), (odd, 8), (mlp, 0), (mlp, 65)):
        with pytest.raises(q.QmlpError) as e:
            q.TrainMLP(m, r)
        assert e.value.status == 4
    t = q.TrainMLP(mlp, 8)
    assert t.saved_bytes(0) == 0 and t.saved_bytes(769) == 0 and t.saved_bytes(768) >= 10 * 768 * 512
    rng = np.random.default_rng(0)
    ad, big = (on_device(torch, adapter(rng, 256, 512, r), 1.0) for r in (8, 9))
    one = on_device(torch, adapter(rng, 256, 512, 8, ("gate",)), 1.0)
    M = 10
    x, dy, out = (torch.zeros((M, 256), dtype=torch.bfloat16, device="cuda") for _ in range(3))
    saved = torch.zeros(t.saved_bytes(M), dtype=torch.uint8, device="cuda")
    F, B = q.qmlp_train_forward, q.qmlp_train_backward
    assert F(t.h, None, x, 0, out, saved) == 4 and F(t.h, None, x, 769, out, saved) == 4
    assert F(t.h, None, None, M, out, saved) == 1 and F(t.h, None, x, M, out, None) == 1
    assert F(t.h, big.c, x, M, out, saved) == 4
    assert F(t.h, None, x, M, x, saved) == 3 and F(t.h, None, x, M, out, x) == 3
    assert F(t.h, None, x.data_ptr() + 2, M, out, saved) == 2
    assert B(t.h, None, x, M, saved, dy, out, ad.c) == 1  # gradients of no adapter
    assert B(t.h, one.c, x, M, saved, dy, out, ad.c) == 1  # of parts that it lacks
    assert B(t.h, ad.c, x, M, saved, dy, out, ad.c) == 3  # into the adapter itself
    assert B(t.h, None, x, M, saved, dy, dy, None) == 3
    assert B(t.h, None, x, M, None, dy, out, None) == 1
    t.close()
    for m in (small, odd, mlp):
        m.close()
