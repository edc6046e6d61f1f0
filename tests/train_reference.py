"""The block's training step in 64 bits, with the formulas written out: used by
the GPU tests, and itself tested against differences (test_train_reference.py)."""
import numpy as np


def forward(w, x, a=None, c=1.0):
    """w = (Wg, Wu, Wd) with their factors; a: {part: array} or None. Returns
    (out, kept)."""
    wg, wu, wd = w
    a = a or {}

    def low(z, p):
        return c * ((z @ a[p + "_a"].T) @ a[p + "_b"].T) if p + "_a" in a else 0.0
    g, u = x @ wg.T + low(x, "gate"), x @ wu.T + low(x, "up")
    act = g / (1 + np.exp(-g)) * u
    return act @ wd.T + low(act, "down"), (g, u, act)


def backward(w, x, dout, a=None, c=1.0):
    """(dx, {part: gradient})"""
    wg, wu, wd = w
    a = a or {}
    _, (g, u, act) = forward(w, x, a, c)
    grads = {}

    def through(dy, z, weight, p):
        """dz of y = z W^T + c (z A^T) B^T, and the gradients of A and B."""
        dz = dy @ weight
        if p + "_a" in a:
            A, B = a[p + "_a"], a[p + "_b"]
            grads[p + "_b"] = c * dy.T @ (z @ A.T)
            grads[p + "_a"] = c * (dy @ B).T @ z
            dz = dz + c * (dy @ B) @ A
        return dz
    dact = through(dout, act, wd, "down")
    s = 1 / (1 + np.exp(-g))
    dg = dact * u * s * (1 + g * (1 - s))
    du = dact * g * s
    return through(dg, x, wg, "gate") + through(du, x, wu, "up"), grads
