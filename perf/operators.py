"""Measured cases of the adapter operators of the weight-quantized SwiGLU MLP.

Three operators, each in a plain form (elementary torch operations in 32
bits) and through the package's public calls:

* lora:  the MLP block with low-rank adapters of many requests at once; every
         token names the adapter it uses (or none);
* train: the block's training forward and its backward through the frozen
         quantized weights: out, dx and the gradients of one adapter;
* adamw: an AdamW step over many tensors at once, states in 32 or in 8 bits.
"""
import math
import random

import torch

own = False  # true: the package's calls; false: the plain form

DEV = "cuda"
BLOCK = 256  # elements that share a scale in an 8-bit state


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # a chat request decoding one token on the 27B-class block
        {"name": "lora decode 1 nvfp4", "op": "lora", "fmt": "nvfp4", "K": 5120, "I": 17408, "M": 1, "slots": 8,
         "rank": 16, "ids": "each"},
        # eight requests decoding together, each with an adapter of its own, some with none
        {"name": "lora decode 8 fp8", "op": "lora", "fmt": "fp8", "K": 5120, "I": 17408, "M": 8, "slots": 32,
         "rank": 32, "ids": "each"},
        # the smallest block, four tokens: launch latency
        {"name": "lora tiny 4 nvfp4", "op": "lora", "fmt": "nvfp4", "K": 256, "I": 512, "M": 4, "slots": 3,
         "rank": 5, "ids": "each"},
        # a serving step of many requests with one token each
        {"name": "lora batch 61 nvfp4", "op": "lora", "fmt": "nvfp4", "K": 4096, "I": 11008, "M": 61, "slots": 16,
         "rank": 8, "ids": "each"},
        # a prefill batch: the prompts of seven requests back to back
        {"name": "lora prefill 3001 fp8", "op": "lora", "fmt": "fp8", "K": 5120, "I": 17408, "M": 3001, "slots": 7,
         "rank": 64, "ids": "runs"},
        # a fine-tuning step on one long batch of the 27B-class block
        {"name": "train 8192 nvfp4", "op": "train", "fmt": "nvfp4", "K": 5120, "I": 17408, "M": 8192, "rank": 16},
        # fine-tuning a smaller block with a large rank
        {"name": "train 1000 fp8", "op": "train", "fmt": "fp8", "K": 2048, "I": 5632, "M": 1000, "rank": 64},
        # one short sample, an odd rank
        {"name": "train 129 nvfp4", "op": "train", "fmt": "nvfp4", "K": 256, "I": 512, "M": 129, "rank": 5},
        # a frozen layer below an adapted one: only dx is wanted
        {"name": "train 2048 frozen nvfp4", "op": "train", "fmt": "nvfp4", "K": 5120, "I": 17408, "M": 2048,
         "rank": 0},
        # the adapters of 64 layers: bf16 copies, fp32 masters, 8-bit states
        {"name": "adamw 384 adapters 8bit", "op": "adamw", "count": 384, "sizes": "adapters", "n": 69206016,
         "param": "bf16", "grad": "bf16", "state": "8bit"},
        # a full projection and its neighbours in fp32
        {"name": "adamw 5 large fp32", "op": "adamw", "count": 5, "sizes": "large", "n": 150000000, "param": "fp32",
         "grad": "fp32", "state": "fp32"},
        # many small tensors of odd sizes
        {"name": "adamw 200 small 8bit", "op": "adamw", "count": 200, "sizes": "odd", "n": 300000, "param": "fp32",
         "grad": "bf16", "state": "8bit"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["lora", "train", "adamw"])
    if op == "adamw":
        count = _log(rng, 1, 400)
        return {"op": op, "count": count, "sizes": "odd", "n": max(count, _log(rng, 1000, 120000000)),
                "param": rng.choice(["fp32", "bf16"]), "grad": rng.choice(["fp32", "bf16"]),
                "state": rng.choice(["fp32", "8bit"])}
    K = 256 * _log(rng, 1, 20)
    K = 2816 if K == 3072 else K
    case = {"op": op, "fmt": rng.choice(["nvfp4", "fp8"]), "K": K, "I": 128 * _log(rng, 4, 136),
            "M": _log(rng, 1, 6000)}
    if case["I"] == 3072:
        case["I"] = 3200
    if op == "lora":
        case.update(slots=_log(rng, 1, 64), rank=_log(rng, 1, 64), ids=rng.choice(["each", "runs"]))
    else:
        case.update(rank=rng.choice([0, _log(rng, 1, 64), _log(rng, 1, 64)]))
    return case


def _sizes(case):
    """Tensor sizes of an adamw case."""
    n, count = case["n"], case["count"]
    if case["sizes"] == "adapters":  # r x K, r x I of gate, up and down, layer after layer
        r, K, I = 16, 5120, 17408
        return [r * K if i % 2 == (i // 4) % 2 else r * I for i in range(count)]
    if case["sizes"] == "large":  # one projection, an odd neighbour, two vectors, a square
        return [17408 * 5120, n - 17408 * 5120 - 5120 - 17408 - 4096 * 4096, 5120, 17408, 4096 * 4096][:count]
    rng = random.Random(count * 1000003 + n)
    w = [rng.expovariate(1.0) + 0.02 for _ in range(count)]
    t = sum(w)
    return [max(1, int(n * x / t)) for x in w]


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _proj(g, fmt, N, K):
    if fmt == "nvfp4":  # any codes, E4M3 group scales 2^-6 .. 2^3, a global factor
        w = torch.randint(0, 256, (N, K // 2), generator=g, device=DEV, dtype=torch.uint8)
        s = torch.randint(8, 80, (N, K // 16), generator=g, device=DEV, dtype=torch.uint8)
        return {"w": w, "scale": s, "global": float(torch.empty(1, device=DEV).uniform_(100, 1000, generator=g))}
    w = torch.randint(0, 254, (N, K), generator=g, device=DEV, dtype=torch.uint8)  # no NaN codes
    w = w + (w >= 127).to(torch.uint8)
    s = torch.empty(N, device=DEV).uniform_(2e-5, 2e-4, generator=g)
    return {"w": w, "scale": s, "global": 1.0}


def _normal(g, shape, std, dtype=torch.bfloat16):
    return (torch.randn(shape, generator=g, device=DEV) * std).to(dtype)


def _adapter(g, K, I, r):
    """A of each projection near 1/sqrt(its inputs), B as after some training."""
    return {"gate_a": _normal(g, (r, K), K ** -0.5), "gate_b": _normal(g, (I, r), 0.02),
            "up_a": _normal(g, (r, K), K ** -0.5), "up_b": _normal(g, (I, r), 0.02),
            "down_a": _normal(g, (r, I), I ** -0.5), "down_b": _normal(g, (K, r), 0.02)}


NAMES = ("gate_a", "gate_b", "up_a", "up_b", "down_a", "down_b")


def _inputs(case, seed):
    g = _gen(seed)
    if case["op"] == "adamw":
        return _inputs_adamw(case, g)
    K, I, M, r = case["K"], case["I"], case["M"], case["rank"]
    d = {"x": _normal(g, (M, K), 1.0), "gate": _proj(g, case["fmt"], I, K), "up": _proj(g, case["fmt"], I, K),
         "down": _proj(g, case["fmt"], K, I), "scale": 2.0}
    if case["op"] == "train":
        d["dout"] = _normal(g, (M, K), 1e-3)
        d["adapter"] = _adapter(g, K, I, r) if r else None
        return d
    S = case["slots"]
    d["adapters"] = [_adapter(g, K, I, r) for _ in range(S)]
    rng = random.Random(seed)
    if case["ids"] == "runs":  # prompts back to back, in any order of adapters
        cuts = sorted(rng.randrange(0, M + 1) for _ in range(S - 1))
        order = rng.sample(range(S), S)
        ids = [order[sum(m >= c for c in cuts)] for m in range(M)]
    else:  # a request a token; about one in eight uses the block as it is
        ids = [rng.randrange(S) if M == 1 or rng.random() < 0.875 else -1 for _ in range(M)]
    d["ids"] = torch.tensor(ids, dtype=torch.int32, device=DEV)
    return d


def _inputs_adamw(case, g):
    """Every kind of value in one buffer, in which each tensor starts at a
    multiple of 256 elements; what lies between two tensors is zero."""
    sizes = _sizes(case)
    room = [-(-n // BLOCK) * BLOCK for n in sizes]
    live = torch.cat([torch.arange(a, device=DEV) < n for n, a in zip(sizes, room)]).float()
    at = [0, *torch.cumsum(torch.tensor(room[:-1], dtype=torch.int64), 0).tolist()]
    pt = torch.float32 if case["param"] == "fp32" else torch.bfloat16
    gt = torch.float32 if case["grad"] == "fp32" else torch.bfloat16
    total = sum(room)
    master = _normal(g, (total,), 0.02, torch.float32) * live
    d = {"sizes": sizes, "at": at, "grad": (_normal(g, (total,), 1e-3, torch.float32) * live).to(gt),
         "master": master if pt == torch.bfloat16 else None,  # bf16 tensors keep an fp32 master
         "param": master.to(pt)}
    m = _normal(g, (total,), 3e-4, torch.float32) * live
    v = (1e-6 * torch.rand(total, generator=g, device=DEV) + 1e-8) * live
    d["ms"] = d["vs"] = None
    if case["state"] == "8bit":
        m, d["ms"] = _to8(m)
        v, d["vs"] = _to8(torch.sqrt(v))
    d["m"], d["v"] = m, v
    return d


def _to8(t):
    """A state as a program holds it in 8 bits: e4m3 values and a scale a block."""
    b = t.view(-1, BLOCK)
    s = b.abs().amax(1) * (1.0 / 448.0)
    return (b / s[:, None]).nan_to_num(0.0).to(torch.float8_e4m3fn).view(-1), s


LR, B1, B2, EPS, WD, STEP = 2e-4, 0.9, 0.999, 1e-8, 0.01, 100


def prepare(case, seed):
    d = _inputs(case, seed)
    d["case"] = dict(case)
    if case["op"] == "adamw":
        if own:
            import weight_quantized_swiglu_gb300 as q
            cut = lambda t: t if t is None else [t[a:a + n] for a, n in zip(d["at"], d["sizes"])]  # noqa: E731
            cut8 = lambda t: t if t is None else [t[a // BLOCK:-(-(a + n) // BLOCK)]  # noqa: E731
                                                  for a, n in zip(d["at"], d["sizes"])]
            d["opt"] = q.AdamW(cut(d["param"]), cut(d["grad"]), cut(d["m"]), cut(d["v"]), m_scale=cut8(d["ms"]),
                               v_scale=cut8(d["vs"]), master=cut(d["master"]))
        return d
    K, I, M = case["K"], case["I"], case["M"]
    if case["op"] == "lora":
        if own:
            import types

            import weight_quantized_swiglu_gb300 as q
            p = [types.SimpleNamespace(w=w["w"], scale=w["scale"], global_scale=w["global"])
                 for w in (d["gate"], d["up"], d["down"])]
            d["mlp"] = q.QuantMLP(case["fmt"], K, I, M, *p)
            d["lora"] = q.LoraMLP(d["mlp"], case["slots"], case["rank"])
            for s, a in enumerate(d["adapters"]):
                d["lora"].set(s, q.Adapter(d["scale"], **a))
            d["out"] = torch.empty((M, K), dtype=torch.bfloat16, device=DEV)
        else:  # the adapters of all slots as one matrix a projection, as a plain program keeps them
            d["stack"] = {n: torch.cat([a[n] for a in d["adapters"]], 0 if n.endswith("_a") else 1) for n in NAMES}
        d.pop("adapters")
        return d
    if own:
        import types

        import weight_quantized_swiglu_gb300 as q
        p = [types.SimpleNamespace(w=w["w"], scale=w["scale"], global_scale=w["global"])
             for w in (d["gate"], d["up"], d["down"])]
        d["mlp"] = q.QuantMLP(case["fmt"], K, I, max(M, 768), *p)
        d["train"] = q.TrainMLP(d["mlp"], max(case["rank"], 1))
        d["saved"] = torch.empty(d["train"].saved_bytes(M), dtype=torch.uint8, device=DEV)
        d["out"] = torch.empty((M, K), dtype=torch.bfloat16, device=DEV)
        d["dx"] = torch.empty((M, K), dtype=torch.bfloat16, device=DEV)
        if d["adapter"]:
            d["grads"] = {n: torch.empty_like(t) for n, t in d["adapter"].items()}
            d["own_adapter"] = q.Adapter(d["scale"], **d["adapter"])
            d["own_grads"] = q.Adapter(1.0, **d["grads"])
        else:
            d["grads"], d["own_adapter"], d["own_grads"] = {}, None, None
    return d


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(state):
    return {"lora": _run_lora, "train": _run_train, "adamw": _run_adamw}[state["case"]["op"]](state)


E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)


def _weight(p, fmt):
    """A projection's weights in fp32."""
    w = p["w"]
    if fmt == "fp8":
        return w.view(torch.float8_e4m3fn).float() * p["scale"][:, None]
    lut = torch.tensor(E2M1, device=w.device)
    c = torch.stack((w & 15, w >> 4), -1).view(w.shape[0], -1, 16).int()
    s = p["scale"].view(torch.float8_e4m3fn).float() * (1.0 / p["global"])
    return (lut[c] * s[:, :, None]).view(w.shape[0], -1)


def _run_lora(d):
    if own:
        return d["lora"].forward(d["x"], d["ids"], d["out"])
    x, S, r, st = d["x"].float(), d["case"]["slots"], d["case"]["rank"], d["stack"]
    fmt = d["case"]["fmt"]
    hot = (d["ids"][:, None] == torch.arange(S, device=x.device)[None, :]).float() * d["scale"]
    hot = hot.repeat_interleave(r, 1)  # [M, S r]: the columns of the token's own adapter
    g = x @ _weight(d["gate"], fmt).T + ((x @ st["gate_a"].float().T) * hot) @ st["gate_b"].float().T
    u = x @ _weight(d["up"], fmt).T + ((x @ st["up_a"].float().T) * hot) @ st["up_b"].float().T
    act = g / (1 + torch.exp(-g)) * u
    out = act @ _weight(d["down"], fmt).T + ((act @ st["down_a"].float().T) * hot) @ st["down_b"].float().T
    return out.to(torch.bfloat16)


def _run_train(d):
    if own:
        d["train"].forward(d["x"], d["out"], d["saved"], adapter=d["own_adapter"])
        d["train"].backward(d["x"], d["saved"], d["dout"], d["dx"], adapter=d["own_adapter"], grads=d["own_grads"])
        return {"out": d["out"], "dx": d["dx"], **d["grads"]}
    x, dout, c = d["x"].float(), d["dout"].float(), d["scale"]
    wg, wu, wd = (_weight(d[n], d["case"]["fmt"]) for n in ("gate", "up", "down"))
    a = {n: t.float() for n, t in d["adapter"].items()} if d["adapter"] else None
    g, u = x @ wg.T, x @ wu.T
    if a:
        vg, vu = c * (x @ a["gate_a"].T), c * (x @ a["up_a"].T)
        g, u = g + vg @ a["gate_b"].T, u + vu @ a["up_b"].T
    sig = 1 / (1 + torch.exp(-g))
    act = g * sig * u
    out, dact = act @ wd.T, dout @ wd
    if a:
        vd, dvd = c * (act @ a["down_a"].T), c * (dout @ a["down_b"])
        out, dact = out + vd @ a["down_b"].T, dact + dvd @ a["down_a"]
    du = dact * (g * sig)
    dg = dact * u * (sig * (1 + g * (1 - sig)))
    dx = dg @ wg + du @ wu
    got = {}
    if a:
        dvg, dvu = c * (dg @ a["gate_b"]), c * (du @ a["up_b"])
        dx = dx + dvg @ a["gate_a"] + dvu @ a["up_a"]
        got = {"gate_a": dvg.T @ x, "gate_b": dg.T @ vg, "up_a": dvu.T @ x, "up_b": du.T @ vu,
               "down_a": dvd.T @ act, "down_b": dout.T @ vd}
    got.update(out=out, dx=dx)
    return {n: t.to(torch.bfloat16) for n, t in got.items()}


def _quant(t):
    b = t.view(-1, BLOCK)
    s = b.abs().amax(1) * (1.0 / 448.0)
    return torch.where(s[:, None] > 0, b / s[:, None], 0.0), s


def _run_adamw(d):
    if own:
        d["opt"].step(lr=LR, beta1=B1, beta2=B2, eps=EPS, weight_decay=WD, step=STEP)
        return _whole(d)
    p, g, m, v = d["param"] if d["master"] is None else d["master"], d["grad"].float(), d["m"], d["v"]
    if d["ms"] is not None:
        m = (m.float().view(-1, BLOCK) * d["ms"][:, None]).view(-1)
        v = (v.float().view(-1, BLOCK) * d["vs"][:, None]).view(-1)
        v = v * v
    m = m * B1 + g * (1.0 - B1)
    v = v * B2 + (g * g) * (1.0 - B2)
    root = torch.sqrt(v)
    p = p * (1.0 - LR * WD) - (m / (root * (1.0 - B2 ** STEP) ** -0.5 + EPS)) * (LR / (1.0 - B1 ** STEP))
    d["param"].copy_(p)
    if d["master"] is not None:
        d["master"].copy_(p)
    if d["ms"] is None:
        d["m"].copy_(m)
        d["v"].copy_(v)
        return _whole(d)
    q, s = _quant(m)
    d["m"].copy_(q.view(-1))
    d["ms"].copy_(s)
    q, s = _quant(root)  # the root of the second moment never rounds to zero
    d["v"].copy_(torch.where(q > 0, q.clamp_min(2.0 ** -9), q).view(-1))
    d["vs"].copy_(s)
    return _whole(d)


def _whole(d):
    return {n: d[n] for n in ("param", "master", "m", "ms", "v", "vs") if d[n] is not None}


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    if case["op"] == "adamw":
        n = sum(_sizes(case))
        p = 8 if case["param"] == "fp32" else 10  # fp32 in and out, and the bf16 copy out
        s = 16 if case["state"] == "fp32" else 4 + 16 / BLOCK
        return {"bytes": n * (p + s + (4 if case["grad"] == "fp32" else 2)), "flops": 12 * n}
    K, I, M, r = case["K"], case["I"], case["M"], case["rank"]
    w = 3 * K * I * 9 // 16 if case["fmt"] == "nvfp4" else 3 * K * I + 4 * (K + 2 * I)
    low = 3 * r * (K + I)
    if case["op"] == "lora":
        used = min(case["slots"], M)
        return {"bytes": w + 2 * low * used + 4 * M * K + 4 * M, "flops": 6 * M * K * I + 2 * M * low}
    return {"bytes": w + 4 * low + 8 * M * K, "flops": 12 * M * K * I + 6 * M * low}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def _e4m3(b):
    """The number that an e4m3 byte stands for."""
    b = b.to(torch.int32)
    e, m = (b >> 3) & 15, (b & 7).double()
    mag = torch.where(e > 0, torch.ldexp(1 + m / 8, e - 7), m * 2.0 ** -9)
    return torch.where(b >= 128, -mag, mag)


def _exact_weight(p, fmt):
    if fmt == "fp8":
        return _e4m3(p["w"]) * p["scale"].double()[:, None]
    b = p["w"].to(torch.int32)
    c = torch.stack((b % 16, b // 16), 2).flatten(1)
    e, m = (c >> 1) & 3, (c & 1).double()
    mag = torch.where(e > 0, torch.ldexp(1 + m / 2, e - 1), m / 2)
    s = _e4m3(p["scale"]) / p["global"]
    return torch.where(c >= 8, -mag, mag) * torch.repeat_interleave(s, 16, 1)


def exact(case, seed):
    d = _inputs(case, seed)
    if case["op"] == "adamw":
        return _exact_adamw(d)
    x = d["x"].double()
    w = {n: _exact_weight(d[n], case["fmt"]) for n in ("gate", "up", "down")}
    sigmoid = lambda t: torch.reciprocal(1 + torch.exp(-t))  # noqa: E731
    if case["op"] == "lora":
        def project(z, name):
            y = z @ w[name].T
            for s, a in enumerate(d["adapters"]):
                rows = (d["ids"] == s).nonzero()[:, 0]
                if rows.numel():
                    A, B = a[name + "_a"].double(), a[name + "_b"].double()
                    y[rows] += d["scale"] * ((z[rows] @ A.T) @ B.T)
            return y
        g = project(x, "gate")
        return project(g * sigmoid(g) * project(x, "up"), "down")
    c, r, dout = d["scale"], case["rank"], d["dout"].double()
    z = torch.zeros
    f = dict(dtype=torch.float64, device=DEV)
    a = {n: t.double() for n, t in d["adapter"].items()} if r else {
        n: z((1, I) if n == "down_a" else (1, K) if n.endswith("_a") else (K, 1) if n == "down_b" else (I, 1), **f)
        for K, I in [(case["K"], case["I"])] for n in NAMES}
    low = {n: a[n + "_b"] @ a[n + "_a"] * c for n in w}  # the adapter's full matrix
    full = {n: w[n] + low[n] for n in w}
    g, u = x @ full["gate"].T, x @ full["up"].T
    s = sigmoid(g)
    act = s * g * u
    dact = dout @ full["down"]
    dg = dact * u * (s + g * s * (1 - s))
    du = dact * g * s
    got = {"out": act @ full["down"].T, "dx": dg @ full["gate"] + du @ full["up"]}
    if r:
        for n, dy, xin in (("gate", dg, x), ("up", du, x), ("down", dout, act)):
            got[n + "_a"] = c * (dy @ a[n + "_b"]).T @ xin
            got[n + "_b"] = c * dy.T @ (xin @ a[n + "_a"].T)
    return got


def _round8(q):
    """Nearest e4m3 number (ties to even) of q >= 0 or < 0."""
    a = q.abs()
    step = torch.exp2(torch.floor(torch.log2(a.clamp_min(2.0 ** -6))) - 3)
    return torch.sign(q) * (torch.round(a / step) * step).clamp_max(448.0)


def _exact_adamw(d):
    g, p = d["grad"].double(), (d["param"] if d["master"] is None else d["master"]).double()
    m, v = d["m"].double(), d["v"].double()
    if d["ms"] is not None:
        m = m * torch.repeat_interleave(d["ms"].double(), BLOCK)
        v = (v * torch.repeat_interleave(d["vs"].double(), BLOCK)).square()
    m, v = B1 * m + (1 - B1) * g, B2 * v + (1 - B2) * g.square()
    p = p - LR * WD * p - LR * (m / (1 - B1 ** STEP)) / ((v / (1 - B2 ** STEP)).sqrt() + EPS)
    out = {"param": p, "m": m, "v": v, "master": None if d["master"] is None else p, "ms": None, "vs": None}
    if d["ms"] is not None:
        for name, t in (("m", m), ("v", v.sqrt())):
            s = t.view(-1, BLOCK).abs().amax(1) / 448
            q = _round8((t / torch.repeat_interleave(s, BLOCK)).nan_to_num(0.0))
            out[name] = torch.where(t > 0, q.clamp_min(2.0 ** -9), q) if name == "v" else q
            out[name + "s"] = s
    return _whole(out)
