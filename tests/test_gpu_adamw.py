"""AdamW over many tensors against the formulas in 64 bits.

Tolerances, from the arithmetic (u = 2^-24, each fp32 operation rounds once):
m, v: three roundings of terms of the sum's size: 4u of the terms' magnitudes.
The update: m, the root, its product, the sum, the quotient and the product
with the step round once each and the fp32 constants half a unit: 10u of its
size; p itself two more roundings of its size. bf16 parameters round once
(2^-8 of their size) from that. An 8-bit code has to be a nearest one of its
unrounded value: within half a step, plus 8u of the value."""
import numpy as np
import pytest

import weight_quantized_swiglu_gb300 as q

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HYPER = dict(lr=3e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.02, step=7, grad_scale=0.5)


@pytest.fixture(scope="module")
def torch(cuda_available):
    import torch
    from weight_quantized_swiglu_gb300 import build
    build.build()
    return torch


def make(torch, sizes, pdt, gdt, eight, master, seed, offset=0):
    """Lists of tensors; offset shifts each start by that many elements."""
    g = torch.Generator(device="cuda").manual_seed(seed)

    def buf(n, std, dt):
        t = torch.empty(n + offset, device="cuda", dtype=dt)[offset:]
        t.copy_(torch.randn(n, generator=g, device="cuda") * std)
        return t

    d = {"master": [buf(n, 0.05, torch.float32) for n in sizes] if master else None}
    d["params"] = [buf(n, 0.05, pdt) for n in sizes]
    if master:
        for p, t in zip(d["params"], d["master"]):
            p.copy_(t)
    d["grads"] = [buf(n, 1e-2, gdt) for n in sizes]
    m = [buf(n, 3e-3, torch.float32) for n in sizes]
    v = [buf(n, 1e-5, torch.float32).abs_() for n in sizes]
    d["m_scale"] = d["v_scale"] = None
    if eight:
        def code(t):
            nb = -(-t.numel() // 256)
            b = torch.nn.functional.pad(t, (0, nb * 256 - t.numel())).view(nb, 256)
            s = b.abs().amax(1) / 448
            c = (b / s[:, None]).to(torch.float8_e4m3fn).view(-1)[:t.numel()]
            out = torch.empty(t.numel() + offset, device="cuda", dtype=torch.float8_e4m3fn)[offset:]
            out.copy_(c)
            return out, s.clone()
        d["m"], d["m_scale"] = (list(x) for x in zip(*[code(t) for t in m]))
        d["v"], d["v_scale"] = (list(x) for x in zip(*[code(t.sqrt()) for t in v]))
    else:
        d["m"], d["v"] = m, v
    return d


def f64(t):
    return t.float().double().cpu().numpy()


def blocks(s, n):
    return np.repeat(f64(s), 256)[:n]


def reference(d, i, h):
    """(p, m, v, update's size) in fp64 from the tensors before the step."""
    n = d["params"][i].numel()
    p = f64(d["master"][i] if d["master"] else d["params"][i])
    g = f64(d["grads"][i]) * h["grad_scale"]
    m, v = f64(d["m"][i]), f64(d["v"][i])
    if d["m_scale"]:
        m = m * blocks(d["m_scale"][i], n)
        v = (v * blocks(d["v_scale"][i], n)) ** 2
    sm = np.abs(m) * h["beta1"] + np.abs(g) * (1 - h["beta1"])
    m = h["beta1"] * m + (1 - h["beta1"]) * g
    v = h["beta2"] * v + (1 - h["beta2"]) * g * g
    den = np.sqrt(v) / np.sqrt(1 - h["beta2"] ** h["step"]) + h["eps"]
    k = h["lr"] / (1 - h["beta1"] ** h["step"])
    return p * (1 - h["lr"] * h["weight_decay"]) - k * m / den, m, v, sm, k * sm / den


def e4m3_step(x):
    a = np.maximum(np.abs(x), 2.0 ** -6)
    return 2.0 ** (np.floor(np.log2(a)) - 3)


def check(torch, d, h):
    refs = [reference(d, i, h) for i in range(len(d["params"]))]
    opt = q.AdamW(d["params"], d["grads"], d["m"], d["v"], m_scale=d["m_scale"], v_scale=d["v_scale"],
                  master=d["master"])
    opt.step(**h)
    torch.cuda.synchronize()
    opt.close()
    for i, (p, m, v, sm, upd) in enumerate(refs):
        n = p.size
        tol = 4 * U * np.abs(p) + 12 * U * upd
        got = f64(d["params"][i])
        if d["master"]:
            assert np.all(np.abs(f64(d["master"][i]) - p) <= tol)
            assert torch.equal(d["params"][i], d["master"][i].to(torch.bfloat16))
        else:
            r = 2.0 ** -8 * np.abs(p) if d["params"][i].dtype == torch.bfloat16 else 0
            assert np.all(np.abs(got - p) <= tol + r + (2 * tol if np.ndim(r) else 0))
        if not d["m_scale"]:
            assert np.all(np.abs(f64(d["m"][i]) - m) <= 4 * U * sm)
            assert np.all(np.abs(f64(d["v"][i]) - v) <= 6 * U * v)
            continue
        for name, want, size in (("m", m, sm), ("v", np.sqrt(v), np.sqrt(v))):
            nb = -(-n // 256)
            top = np.abs(np.pad(want, (0, nb * 256 - n))).reshape(nb, 256).max(1)
            size_top = np.pad(size, (0, nb * 256 - n)).reshape(nb, 256).max(1)
            s = f64(d[name + "_scale"][i])
            assert np.all(np.abs(s - top / 448) <= 8 * U * size_top / 448)
            sb = np.repeat(s, 256)[:n]
            with np.errstate(divide="ignore", invalid="ignore"):
                qv = np.where(sb > 0, want / sb, 0.0)
                tolq = np.where(sb > 0, 8 * U * size / sb, 0.0)
            if name == "v":
                qv = np.where(qv > 0, np.maximum(qv, 2.0 ** -9), qv)
            c = f64(d[name][i])
            assert np.all(np.abs(c - np.clip(qv, -448, 448)) <= e4m3_step(qv) / 2 + tolq + 8 * U * np.abs(qv))
            if name == "v":
                assert np.all(c[want > 0] > 0)  # a root above zero keeps a code


SIZES = [1, 7, 8, 255, 256, 257, 2047, 2048, 2049, 5000, 70001]


@pytest.mark.parametrize("eight", [False, True])
@pytest.mark.parametrize("pdt,gdt,master", [("float32", "float32", False), ("float32", "bfloat16", False),
                                            ("bfloat16", "bfloat16", True), ("bfloat16", "float32", True),
                                            ("bfloat16", "bfloat16", False), ("bfloat16", "float32", False)])
def test_types_and_odd_sizes(torch, pdt, gdt, master, eight):
    d = make(torch, SIZES, getattr(torch, pdt), getattr(torch, gdt), eight, master, 11)
    check(torch, d, HYPER)


@pytest.mark.parametrize("eight", [False, True])
def test_tensors_that_start_anywhere(torch, eight):
    """Starts that rule out the wide loads, and guard elements around them."""
    d = make(torch, [300, 2048, 4096, 4099], torch.float32, torch.bfloat16, eight, False, 12, offset=1)
    before = [t._base[0].clone() for ts in (d["params"], d["m"], d["v"]) for t in ts]
    check(torch, d, HYPER)
    after = [t._base[0] for ts in (d["params"], d["m"], d["v"]) for t in ts]
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(
        [x.reshape(1) for x in before], [x.reshape(1) for x in after]))


@pytest.mark.parametrize("offset", [0, 8])
@pytest.mark.parametrize("pdt,gdt,master", [("float32", "bfloat16", False), ("bfloat16", "float32", True)])
def test_more_chunks_than_the_gpu_holds_at_a_time(torch, pdt, gdt, master, offset):
    """Many chunks, short ones among them; offset 8: 8-bit states that start on
    8 bytes and not on 16."""
    sizes = [2048 * 700 + 5] + [17, 4096, 3] * 40 + [2048 * 100 + 1031]
    d = make(torch, sizes, getattr(torch, pdt), getattr(torch, gdt), True, master, 19, offset=offset)
    assert offset == 0 or any(t.data_ptr() % 16 for t in d["m"])
    check(torch, d, HYPER)


def test_the_wide_and_the_narrow_path_agree_bit_for_bit(torch):
    n = 4096
    a = make(torch, [n], torch.float32, torch.float32, True, False, 13)
    b = {k: ([torch.cat([t.new_zeros(1) if t.dtype.itemsize > 1 else t[:1], t])[1:] for t in ts]
             if ts and not k.endswith("scale") else ([t.clone() for t in ts] if ts else None))
         for k, ts in a.items()}
    for d in (a, b):
        o = q.AdamW(d["params"], d["grads"], d["m"], d["v"], m_scale=d["m_scale"], v_scale=d["v_scale"])
        o.step(**HYPER)
        torch.cuda.synchronize()
        o.close()
    for k in ("params", "m", "v", "m_scale", "v_scale"):
        assert torch.equal(a[k][0].view(torch.uint8), b[k][0].contiguous().clone().view(torch.uint8)), k


@pytest.mark.parametrize("eight", [False, True])
def test_first_step_from_zero_states_and_zero_gradients(torch, eight):
    d = make(torch, [1000, 300], torch.float32, torch.float32, eight, False, 14)
    for ts in (d["m"], d["v"], d["m_scale"] or [], d["v_scale"] or []):
        for t in ts:
            t.view(torch.uint8).zero_()
    d["grads"][1].zero_()  # all zero: only the decay acts
    d["grads"][0][5] = 0
    p1 = d["params"][1].clone()
    h = {**HYPER, "step": 1}
    check(torch, d, h)
    decay = torch.tensor(1 - h["lr"] * h["weight_decay"], dtype=torch.float32, device="cuda")
    assert torch.equal(d["params"][1], p1 * decay)


def test_small_roots_keep_a_code_and_the_next_update_stays_small(torch):
    """One gradient 2^20 times the others of its block: their roots are under
    the smallest code of the block's scale, and still do not become zero."""
    d = make(torch, [256], torch.float32, torch.float32, True, False, 15)
    for t in d["m"] + d["v"] + d["m_scale"] + d["v_scale"]:
        t.view(torch.uint8).zero_()
    d["grads"][0].fill_(1e-6)
    d["grads"][0][17] = 1.0
    o = q.AdamW(d["params"], d["grads"], d["m"], d["v"], m_scale=d["m_scale"], v_scale=d["v_scale"])
    p0 = d["params"][0].clone()
    for t in (1, 2, 3):
        o.step(lr=1e-3, weight_decay=0.0, step=t)
    torch.cuda.synchronize()
    assert (d["v"][0].float() > 0).all()
    assert ((d["params"][0] - p0).abs() <= 3 * 1.2e-3).all()
    o.close()


@pytest.mark.parametrize("scale", [3e-38, 1e-38, 1e-39, 1e-40, 1e-42])
def test_momenta_that_have_decayed_to_subnormal_scales(torch, scale):
    """Without gradients m decays by beta1 a step, through scales whose
    reciprocal is past fp32's range. Zeros stay zeros and the others keep nearest
    codes: m rounds twice and the scale once more to a subnormal's step 2^-149."""
    n = 512
    d = make(torch, [n], torch.float32, torch.float32, True, False, 18)
    d["grads"][0].zero_()
    d["m"][0][::3] = 0
    d["m_scale"][0].copy_(torch.tensor([scale, 5e-3 / 448], dtype=torch.float32))
    m = (f64(d["m"][0]) * blocks(d["m_scale"][0], n)) * HYPER["beta1"]
    o = q.AdamW(d["params"], d["grads"], d["m"], d["v"], m_scale=d["m_scale"], v_scale=d["v_scale"])
    o.step(**HYPER)
    torch.cuda.synchronize()
    o.close()
    tiny = 2.0 ** -149
    c, s = f64(d["m"][0]), f64(d["m_scale"][0])
    top = np.abs(m).reshape(2, 256).max(1)
    assert np.all(np.abs(s - top / 448) <= 8 * U * top / 448 + tiny)
    sb = np.repeat(s, 256)
    with np.errstate(divide="ignore", invalid="ignore"):
        qv = np.where(sb > 0, m / sb, 0.0)
        tol = np.where(sb > 0, (4 * U * np.abs(m) + 2 * tiny) / sb, 0.0)
    qv = np.clip(qv, -448, 448)
    assert np.all(c[m == 0] == 0)
    assert np.all(np.abs(c - qv) <= e4m3_step(qv) / 2 + tol + 8 * U * np.abs(qv))
    assert torch.isfinite(d["params"][0]).all()


def test_not_finite_gradients_are_not_hidden(torch):
    d = make(torch, [512], torch.float32, torch.float32, True, False, 16)
    for t in d["m"] + d["v"] + d["m_scale"] + d["v_scale"]:
        t.view(torch.uint8).zero_()
    d["grads"][0].zero_()
    d["grads"][0][3] = float("nan")
    o = q.AdamW(d["params"], d["grads"], d["m"], d["v"], m_scale=d["m_scale"], v_scale=d["v_scale"])
    o.step(**HYPER)
    torch.cuda.synchronize()
    assert torch.isnan(d["params"][0][3]) and torch.isfinite(d["params"][0][4:]).all()
    assert torch.isnan(d["m"][0].float()[3]) and torch.isnan(d["v"][0].float()[3])
    o.close()


def test_steps_repeat_bit_for_bit_and_replay_in_a_graph(torch):
    runs = []
    for graph in (False, False, True):
        d = make(torch, [4097, 100], torch.bfloat16, torch.bfloat16, True, True, 17)
        o = q.AdamW(d["params"], d["grads"], d["m"], d["v"], m_scale=d["m_scale"], v_scale=d["v_scale"],
                    master=d["master"])
        if graph:
            s = torch.cuda.Stream()
            s.wait_stream(torch.cuda.current_stream())
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=s):
                o.step(**HYPER)
            g.replay()
            g.replay()
        else:
            o.step(**HYPER)
            o.step(**HYPER)
        torch.cuda.synchronize()
        runs.append([t.clone().view(torch.uint8) for k in ("params", "master", "m", "v", "m_scale", "v_scale")
                     for t in d[k]])
        o.close()
    for other in runs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(runs[0], other))


def test_refusals(torch):
    d = make(torch, [64], torch.float32, torch.float32, False, False, 18)
    o = q.AdamW(d["params"], d["grads"], d["m"], d["v"])
    before = d["params"][0].clone()
    for bad in ({"step": 0}, {"beta1": 1.0}, {"beta2": -0.1}, {"lr": float("nan")}, {"eps": float("inf")}):
        with pytest.raises(q.QmlpError) as e:
            o.step(**{**HYPER, **bad})
        assert e.value.status == 1
    torch.cuda.synchronize()
    assert torch.equal(before, d["params"][0])
    o.close()
    with pytest.raises(ValueError):
        q.AdamW(d["params"], d["grads"], d["m"], [d["v"][0][:63]])
    with pytest.raises(ValueError):
        q.AdamW(d["params"], d["grads"], [d["m"][0].half()], [d["v"][0].half()])
    with pytest.raises(q.QmlpError) as e:
        q.AdamW(d["params"], d["grads"], d["m"], d["m"])
    assert e.value.status == 3
