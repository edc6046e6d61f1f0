"""A request's adapter that holds Inf or NaN (a fine-tune that diverged) is that
request's matter: in long batches too, where tiles of 256 tokens pass through the
images of every slot that has a token in them, all other tokens get the bytes
that they get beside a healthy adapter, and the request's own tokens get values that
are not finite where short batches, in which the slots never meet, give them such
(Inf or NaN: a product of Inf with the words of v is either)."""
import numpy as np
import pytest

import oracle
import weight_quantized_swiglu_gb300 as q
from helpers import compare
from test_gpu_lora import adapter, bf16, on_device, reference, run, scaled_case, weights, x_of

pytestmark = pytest.mark.gpu

K, I, M = 4096, 1024, 1333  # long enough a contraction for the terms to be steps of the GEMMs
SLOT = 1


@pytest.fixture(scope="module")
def torch(cuda_available):
    import torch
    from weight_quantized_swiglu_gb300 import build
    build.build()
    return torch


def handles(fmt, rank, seed, tune=None):
    case = scaled_case(fmt, K, I, seed)
    if tune:
        tune(case)
    mlp = q.QuantMLP.from_case(case, max_M=M)
    return case, mlp, q.LoraMLP(mlp, 3, rank)


def spoil(a, where):
    """(the adapter with values that are not finite, the same with zeros there)"""
    bad, zero = ({n: v.copy() for n, v in a.items()} for _ in range(2))
    last = a["gate_b"].shape[1] - 1
    spots = {"gate nan": [("gate_b", 700, 0, np.nan)], "up inf": [("up_b", 3, last, np.inf)],
             "down": [("down_b", 0, 0, np.inf), ("down_b", 1, last, -np.inf), ("down_b", K - 1, 1, np.nan),
                      ("down_b", 777, 0, np.inf), ("down_b", 777, 1, np.inf)]}
    for name, row, col, v in (sum(spots.values(), []) if where == "all" else spots[where]):
        bad[name][row, col] = v
        zero[name][row, col] = 0.0
    return bad, zero


@pytest.mark.parametrize("fmt,rank", [("nvfp4", 16), ("fp8", 7), ("nvfp4", 40)])
@pytest.mark.parametrize("where", ["gate nan", "up inf", "down", "all"])
def test_values_that_are_not_finite_stay_with_their_tokens(torch, fmt, rank, where):
    rng = np.random.default_rng(rank)
    case, mlp, lora = handles(fmt, rank, 65)
    ads = [adapter(rng, K, I, rank, gain=rank ** -0.5) for _ in range(3)]
    bad, zero = spoil(ads[SLOT], where)
    xb, _ = x_of(rng, M, K)
    ids = rng.integers(-1, 3, M)
    own = ids == SLOT
    for s in (0, 2):
        lora.set(s, on_device(torch, ads[s], 1.5))
    lora.set(SLOT, on_device(torch, zero, 1.5))
    healthy = run(torch, lora, mlp, xb, ids)
    lora.set(SLOT, on_device(torch, bad, 1.5))
    got = run(torch, lora, mlp, xb, ids)
    assert np.array_equal(got[~own], healthy[~own])
    short = np.concatenate([run(torch, lora, mlp, xb[a:a + 600], ids[a:a + 600]) for a in range(0, M, 600)])
    g, s = (oracle.bf16_bits_to_f64(b[own]) for b in (got, short))
    assert not np.all(np.isfinite(s))
    assert np.array_equal(np.isfinite(g), np.isfinite(s))
    if where == "down":  # columns without such a value are the healthy ones'
        cols = np.ones(K, dtype=bool)
        cols[[0, 1, 777, K - 1]] = False
        assert np.array_equal(got[own][:, cols], healthy[own][:, cols])
        assert not np.any(np.isfinite(g[:, ~cols]))
    else:  # a value in gate or up reaches the whole row through the down projection
        assert not np.any(np.isfinite(g))
    # a healthy adapter in the slot again, and none
    lora.set(SLOT, on_device(torch, zero, 1.5))
    assert np.array_equal(run(torch, lora, mlp, xb, ids), healthy)
    lora.set(SLOT, on_device(torch, bad, 1.5))
    lora.set(SLOT, None)
    empty = run(torch, lora, mlp, xb, ids)
    assert np.all(np.isfinite(oracle.bf16_bits_to_f64(empty)))
    lora.close()
    mlp.close()


@pytest.mark.parametrize("part", ["gate_b", "down_b"])  # (both at once: past fp32)
def test_values_past_bf16_over_their_rows_factor(torch, part):
    """FP8's images hold B over the row's factor: finite values of B that this
    takes past bf16 are right for their tokens, and nothing to the others."""
    def tune(case):
        if part == "gate_b":
            case.gate.scale[5] = 2.0 ** -58
        else:
            case.down.scale[9] = -2.0 ** -58
    rng = np.random.default_rng(66)
    case, mlp, lora = handles("fp8", 8, 66, tune)
    ads = [adapter(rng, K, I, 8) for _ in range(3)]
    big = {n: a.copy() for n, a in ads[SLOT].items()}
    zero = {n: a.copy() for n, a in big.items()}
    row, cols = (5, slice(8)) if part == "gate_b" else (9, slice(3))
    big[part][row, cols] = bf16(big[part][row, cols] * 1e28)
    zero[part][row, cols] = 0
    xb, x = x_of(rng, M, K)
    ids = rng.integers(-1, 3, M)
    own = ids == SLOT
    for s in (0, 2):
        lora.set(s, on_device(torch, ads[s], 1.0))
    lora.set(SLOT, on_device(torch, zero, 1.0))
    healthy = run(torch, lora, mlp, xb, ids)
    lora.set(SLOT, on_device(torch, big, 1.0))
    got = run(torch, lora, mlp, xb, ids)
    assert np.array_equal(got[~own], healthy[~own])
    with np.errstate(over="ignore"):
        want = reference(case, weights(case), x, ids, {s: (a, 1.0) for s, a in ((0, ads[0]), (SLOT, big), (2, ads[2]))})
    compare(got[own], want[own], what="own tokens")
    lora.close()
    mlp.close()
