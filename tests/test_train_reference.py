"""The reference of the training tests against central differences."""
import numpy as np
import pytest

import train_reference as ref


@pytest.mark.parametrize("parts", [(), ("gate", "up", "down"), ("down",), ("gate",)])
def test_gradients_are_the_differences(parts):
    rng = np.random.default_rng(5)
    K, I, M, r, c = 6, 10, 4, 3, 1.7
    w = [rng.standard_normal(s) * 0.5 for s in ((I, K), (I, K), (K, I))]
    x, dout = rng.standard_normal((M, K)), rng.standard_normal((M, K))
    shapes = {"gate": (I, K), "up": (I, K), "down": (K, I)}
    a = {}
    for p in parts:
        a[p + "_a"], a[p + "_b"] = rng.standard_normal((r, shapes[p][1])), rng.standard_normal((shapes[p][0], r))
    dx, grads = ref.backward(w, x, dout, a, c)
    assert set(grads) == set(a)

    def loss():
        return float((ref.forward(w, x, a, c)[0] * dout).sum())
    h = 1e-5
    for name, t, got in [("x", x, dx)] + [(n, a[n], grads[n]) for n in a]:
        want = np.empty_like(t)
        for i in np.ndindex(t.shape):
            keep = t[i]
            t[i] = keep + h
            up = loss()
            t[i] = keep - h
            want[i] = (up - loss()) / (2 * h)
            t[i] = keep
        # h^2 of the third derivative, and 1e-16 of the loss over h
        assert np.allclose(got, want, rtol=1e-6, atol=1e-6 * np.abs(want).max()), name
