"""The 64-bit reference of the operators around the blocks against differences
and by hand, on the CPU."""
import numpy as np
import pytest

import layer_reference as ref


@pytest.mark.parametrize("post,pre,gate", [(True, True, "full"), (True, False, "channel"), (False, True, "token"),
                                           (False, False, "none"), (True, True, "none")])
def test_norm_gradients_against_differences(post, pre, gate):
    g = np.random.default_rng(7)
    M, K, scale, off, eps = 3, 5, 0.7, 1.0, 1e-3
    t = {"z": g.normal(size=(M, K)), "r": g.normal(size=(M, K)), "post": 0.2 * g.normal(size=K) if post else None,
         "pre": 0.2 * g.normal(size=K) if pre else None,
         "gate": {"none": None, "channel": g.normal(size=(1, K)), "token": g.normal(size=(M, 1)),
                  "full": g.normal(size=(M, K))}[gate]}
    dh, dy = g.normal(size=(M, K)), g.normal(size=(M, K)) if pre else None

    def loss():
        h, y = ref.norm_forward(t["z"], t["r"], t["post"], t["pre"], t["gate"], scale, off, eps)
        return (h * dh).sum() + (0.0 if y is None else (y * dy).sum())

    got = ref.norm_backward(t["z"], t["r"], t["post"], t["pre"], t["gate"], scale, off, eps, dy, dh)
    names = {"z": "dz", "r": "dresidual", "post": "dpost_w", "pre": "dpre_w", "gate": "dgate"}
    step = 1e-5
    for n, a in t.items():
        if a is None:
            continue
        want = got[names[n]][0]
        if n == "gate":
            want = want.sum(0, keepdims=True) if gate == "channel" else want.sum(1, keepdims=True) if gate == "token" else want
        flat = a.reshape(-1)
        for i in range(flat.size):
            v = flat[i]
            flat[i] = v + step
            up = loss()
            flat[i] = v - step
            down = loss()
            flat[i] = v
            # central differences: step^2 times a third derivative of a few units,
            # and the loss's rounding over the step
            assert abs((up - down) / (2 * step) - want.reshape(-1)[i]) < 1e-8 * (1 + abs(want.reshape(-1)[i])), (n, i)
