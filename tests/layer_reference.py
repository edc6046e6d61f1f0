"""64-bit definitions of the operators around the quantized blocks, in plain
numpy (no code shared with the kernels)."""
import numpy as np

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def rms_of(v, eps):
    return np.sqrt((v * v).mean(1, keepdims=True) + eps)


def norm_forward(z, r, post, pre, gate, scale, offset, eps):
    """z, r [M, K]; post, pre [K] or None; gate broadcasts to [M, K] or None."""
    n = z if post is None else z / rms_of(z, eps) * (post + offset)
    h = r + scale * (1.0 if gate is None else gate) * n
    y = None if pre is None else h / rms_of(h, eps) * (pre + offset)
    return h, y


def norm_backward(z, r, post, pre, gate, scale, offset, eps, dy, dh):
    """Gradients by the formulas, and beside each the size of its terms (what
    rounding errors are relative to): {name: (gradient, size)}. dgate has the
    shape [M, K], before it is summed over what shares a value."""
    g = np.ones((1, 1)) if gate is None else gate
    rz = 1 / rms_of(z, eps) if post is not None else 1.0
    zh = z * rz
    wp = post + offset if post is not None else 1.0
    n = zh * wp
    h = r + scale * g * n
    hs = np.abs(r) + np.abs(scale * g * n)
    out = {}
    d, ds = dh.copy(), np.abs(dh)
    if pre is not None:
        rh = 1 / rms_of(h, eps)
        hh, hhs, wr = h * rh, hs * rh, pre + offset
        a = dy * wr
        d = d + rh * (a - hh * (a * hh).mean(1, keepdims=True))
        ds = ds + rh * (np.abs(a) + 3 * hhs * (np.abs(a) * hhs).mean(1, keepdims=True))
        out["dpre_w"] = ((dy * hh).sum(0), (np.abs(dy) * hhs).sum(0))
    out["dresidual"] = (d, ds)
    dn, dns = scale * g * d, np.abs(scale * g) * ds
    out["dgate"] = (scale * d * n, np.abs(scale * n) * ds)
    if post is not None:
        out["dpost_w"] = ((dn * zh).sum(0), (dns * np.abs(zh)).sum(0))
        b, bs = dn * wp, dns * np.abs(wp)
        dn = rz * (b - zh * (b * zh).mean(1, keepdims=True))
        dns = rz * (bs + 3 * np.abs(zh) * (bs * np.abs(zh)).mean(1, keepdims=True))
    out["dz"] = (dn, dns)
    return out
