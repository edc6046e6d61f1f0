"""Measured cases of the operators around the quantized blocks of a decoder layer.

Three operators, each in a plain form (elementary torch operations) and
through the package's public calls:

* linear: one projection with 4-bit weights and group scales (the projections
          beside the MLP: attention's, the output head), one token to a prompt;
* norm:   the norms before and after a block with its gate, residual and
          residual scale, forward and, for training, backward;
* moe:    a whole mixture-of-experts layer for a few tokens: router, selection,
          routed and shared experts, weighted sum.
"""
import math
import random

import torch

own = False  # true: the package's calls; false: the plain form

DEV = "cuda"
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # attention's output projection, a chat request decoding one token beside the 27B-class block
        {"name": "linear 1 nvfp4 5120x5120", "op": "linear", "fmt": "nvfp4", "group": 16, "N": 5120, "K": 5120, "M": 1,
         "x": "bf16", "out": "bf16", "bias": False},
        # eight requests decoding together through a wide projection
        {"name": "linear 8 int4 17408x5120", "op": "linear", "fmt": "int4", "group": 128, "N": 17408, "K": 5120, "M": 8,
         "x": "fp16", "out": "fp16", "bias": False},
        # a small projection with a bias, five tokens, odd rows: launch latency
        {"name": "linear 5 int4 1001x256", "op": "linear", "fmt": "int4", "group": 32, "N": 1001, "K": 256, "M": 5,
         "x": "bf16", "out": "bf16", "bias": True},
        # the output head of one token: logits in fp32
        {"name": "linear 1 nvfp4 head", "op": "linear", "fmt": "nvfp4", "group": 16, "N": 128000, "K": 5120, "M": 1,
         "x": "bf16", "out": "fp32", "bias": False},
        # a prompt through a projection back to the hidden size
        {"name": "linear 2000 int4 5120x17408", "op": "linear", "fmt": "int4", "group": 64, "N": 5120, "K": 17408,
         "M": 2000, "x": "bf16", "out": "bf16", "bias": False},
        # between two blocks of one decoding token: norm after, residual, norm before
        {"name": "norm 1 bf16 5120", "op": "norm", "dir": "fwd", "M": 1, "K": 5120, "dt": "bf16", "rdt": "bf16",
         "wdt": "bf16", "offset": 0.0, "scale": 1.0, "gate": "none", "post": True, "pre": True},
        # the same for a long prompt with an fp32 residual stream and a gate for each channel
        {"name": "norm 8192 fp32 residual", "op": "norm", "dir": "fwd", "M": 8192, "K": 5120, "dt": "bf16",
         "rdt": "fp32", "wdt": "bf16", "offset": 1.0, "scale": 0.5, "gate": "channel", "post": True, "pre": True},
        # a training step of 4096 tokens with a gate for each value, weights and their gradients in fp32
        {"name": "norm train 4096", "op": "norm", "dir": "train", "M": 4096, "K": 4096, "dt": "bf16", "rdt": "bf16",
         "wdt": "fp32", "offset": 0.0, "scale": 1.0, "gate": "full", "post": True, "pre": True},
        # fine-tuning on a short sample: odd sizes, a gate for each token
        {"name": "norm train 301 odd", "op": "norm", "dir": "train", "M": 301, "K": 2571, "dt": "fp16", "rdt": "fp32",
         "wdt": "fp16", "offset": 0.0, "scale": 0.7, "gate": "token", "post": True, "pre": True},
        # one decoding token, 512 small experts, ten of them and a gated shared one
        {"name": "moe 1 of 512", "op": "moe", "M": 1, "E": 512, "K": 2560, "I": 160, "topk": 10, "shared": 1,
         "score": "softmax", "bias": False, "renorm": True, "rscale": 1.0, "sgate": True, "meta": 4, "x": "bf16",
         "out": "bf16"},
        # eight requests decoding together through the same layer
        {"name": "moe 8 of 512", "op": "moe", "M": 8, "E": 512, "K": 2560, "I": 160, "topk": 10, "shared": 1,
         "score": "softmax", "bias": False, "renorm": True, "rscale": 1.0, "sgate": True, "meta": 4, "x": "bf16",
         "out": "bf16"},
        # sixteen requests, fewer and larger experts, sigmoid scores with a selection bias, two shared experts
        {"name": "moe 16 of 64", "op": "moe", "M": 16, "E": 64, "K": 2048, "I": 704, "topk": 6, "shared": 2,
         "score": "sigmoid", "bias": True, "renorm": True, "rscale": 2.5, "sgate": False, "meta": 3, "x": "fp16",
         "out": "fp16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["linear", "norm", "moe"])
    if op == "linear":
        fmt = rng.choice(["nvfp4", "int4"])
        return {"op": op, "fmt": fmt, "group": 16 if fmt == "nvfp4" else rng.choice([32, 64, 128]),
                "N": _log(rng, 16, 17408), "K": 128 * _log(rng, 1, 136), "M": _log(rng, 1, 2000),
                "x": rng.choice(["bf16", "fp16"]), "out": rng.choice(["bf16", "fp16", "fp32"]),
                "bias": rng.random() < 0.3}
    if op == "norm":
        d = {"op": op, "dir": rng.choice(["fwd", "train"]), "K": _log(rng, 64, 8192), "dt": rng.choice(["bf16", "fp16"])}
        if rng.random() < 0.7:  # most hidden sizes are multiples of 64
            d["K"] = max(64, d["K"] // 64 * 64)
        d["M"] = _log(rng, 1, min(16384, 16777216 // d["K"]))
        d.update(rdt=rng.choice([d["dt"], "fp32"]), wdt=rng.choice([d["dt"], "fp32"]),
                 offset=rng.choice([0.0, 1.0]), scale=rng.choice([1.0, round(rng.uniform(0.1, 1.0), 2)]),
                 gate=rng.choice(["none", "channel", "token", "full"]), post=rng.random() < 0.6)
        d["pre"] = not d["post"] or rng.random() < 0.8
        return d
    d = {"op": op, "M": _log(rng, 1, 16), "E": _log(rng, 4, 512), "K": 64 * _log(rng, 4, 64), "I": 32 * _log(rng, 1, 32)}
    d.update(topk=rng.randint(1, min(10, d["E"])), shared=rng.choice([0, 0, 1, 2]),
             score=rng.choice(["softmax", "sigmoid"]), bias=rng.random() < 0.4, renorm=rng.random() < 0.7,
             rscale=rng.choice([1.0, 2.5]), meta=rng.choice([3, 4]), x=rng.choice(["bf16", "fp16"]),
             out=rng.choice(["bf16", "fp16", "fp32"]))
    d["sgate"] = d["shared"] > 0 and rng.random() < 0.5
    while work(d)["bytes"] > 2.5e8 and d["I"] > 32:  # what the largest listed cases read
        d["I"] = d["I"] // 64 * 32
    return d


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _normal(g, shape, std, dtype=torch.float32):
    return (torch.randn(shape, generator=g, device=DEV) * std).to(dtype)


def _codes(g, *shape):
    return torch.randint(0, 256, shape, generator=g, device=DEV, dtype=torch.uint8)


def _inputs(case, seed):
    g = _gen(seed)
    if case["op"] == "linear":
        N, K, M, G = case["N"], case["K"], case["M"], case["group"]
        d = {"x": _normal(g, (M, K), 1.0, DT[case["x"]]), "w": _codes(g, N, K // 2), "global": 1.0, "zero": None}
        if case["fmt"] == "nvfp4":  # any codes, E4M3 group scales 2^-6 .. 2^3, a global factor
            d["scale"] = torch.randint(8, 80, (N, K // 16), generator=g, device=DEV, dtype=torch.uint8)
            d["global"] = float(torch.empty(1, device=DEV).uniform_(100, 1000, generator=g))
        else:  # fp16 scales of weights near 1/sqrt(K), zeros about the middle
            d["scale"] = (torch.rand((N, K // G), generator=g, device=DEV) * 0.3 + 0.1).mul(K ** -0.5).half()
            d["zero"] = torch.randint(4, 12, (N, K // G), generator=g, device=DEV, dtype=torch.uint8)
        d["bias"] = _normal(g, (N,), 0.5) if case["bias"] else None
        return d
    if case["op"] == "norm":
        M, K, t, w = case["M"], case["K"], DT[case["dt"]], DT[case["wdt"]]
        spread = torch.exp(_normal(g, (K,), 0.7))  # some channels are far larger than others
        weight = lambda: (1 - case["offset"] + _normal(g, (K,), 0.2)).to(w)  # noqa: E731
        d = {"z": (_normal(g, (M, K), 0.5) * spread).to(t), "residual": (_normal(g, (M, K), 2.0) * spread).to(DT[case["rdt"]]),
             "post": weight() if case["post"] else None, "pre": weight() if case["pre"] else None}
        shape = {"none": None, "channel": (K,), "token": (M,), "full": (M, K)}[case["gate"]]
        d["gate"] = None if shape is None else torch.sigmoid(_normal(g, shape, 1.0)).to(
            w if case["gate"] == "channel" else t)
        if case["dir"] == "train":
            d["dy"] = _normal(g, (M, K), 1e-2, t) if case["pre"] else None
            d["dh"] = _normal(g, (M, K), 1e-2, DT[case["rdt"]])
        return d
    M, E, K, I, S, t = case["M"], case["E"], case["K"], case["I"], case["shared"], DT[case["x"]]
    B = E + S  # the shared experts are the last of the banks
    d = {"x": _normal(g, (M, K), 1.0, t), "router": _normal(g, (E, K), K ** -0.5, torch.bfloat16),
         "bias": _normal(g, (E,), 0.05) if case["bias"] else None,
         "sgate": _normal(g, (S, K), K ** -0.5, torch.bfloat16) if case["sgate"] else None}
    for name, N, D in (("w13", 2 * I, K), ("w2", K, I)):
        d[name] = _codes(g, B, N, D // 2)
        s = (torch.rand((B, N, D // 32), generator=g, device=DEV) * 0.3 + 0.1).mul(D ** -0.5).half()
        z = torch.randint(4, 12, s.shape, generator=g, device=DEV, dtype=torch.uint8)
        d[name + "_scale"], d[name + "_zero"] = s, z
    return d


def _records(s, z, meta):
    """The records of the expert banks: fp16 scale, then fp16 bias or u8 zero."""
    b = s.view(torch.uint8).view(*s.shape, 2)
    if meta == 3:
        return torch.cat((b, z[..., None]), -1).contiguous()
    bias = (-z.float() * s.float()).half()
    return torch.cat((b, bias.view(torch.uint8).view(*s.shape, 2)), -1).contiguous()


def prepare(case, seed):
    d = _inputs(case, seed)
    d["case"] = dict(case)
    if not own:
        return d
    import weight_quantized_swiglu_gb300 as q
    empty = lambda t: None if t is None else torch.empty_like(t)  # noqa: E731
    if case["op"] == "linear":
        d["linear"] = q.QuantLinear(case["fmt"], case["N"], case["K"], case["M"], d["w"], d["scale"], zero=d["zero"],
                                    group=case["group"], global_scale=d["global"], bias=d["bias"])
        d["out"] = torch.empty((case["M"], case["N"]), dtype=DT[case["out"]], device=DEV)
        for n in ("w", "scale", "zero"):
            d.pop(n)
    elif case["op"] == "norm":
        d["norm"] = q.BlockNorm(case["K"], eps=EPS, weight_offset=case["offset"], scale=case["scale"],
                                dtype=DT[case["dt"]], residual_dtype=DT[case["rdt"]], weight_dtype=DT[case["wdt"]],
                                gate=case["gate"])
        d["h"], d["y"] = empty(d["residual"]), empty(d["z"]) if case["pre"] else None
        if case["dir"] == "train":
            d["stats"] = torch.empty((case["M"], 2), device=DEV)
            d["grads"] = {"dz": empty(d["z"]), "dresidual": empty(d["residual"]), "dpost_w": empty(d["post"]),
                          "dpre_w": empty(d["pre"]), "dgate": empty(d["gate"])}
    else:
        banks = []
        for n in ("w13", "w2"):
            banks += [d.pop(n), _records(d.pop(n + "_scale"), d.pop(n + "_zero"), case["meta"])]
        d["moe"] = q.MoeAWQ(case["E"] + case["shared"], case["K"], case["I"], case["meta"], *banks)
        d["layer"] = q.MoeLayer(d["moe"], d["router"], case["topk"], score=case["score"], bias=d["bias"],
                                renorm=case["renorm"], route_scale=case["rscale"], shared=case["shared"],
                                shared_gate=d["sgate"], max_tokens=case["M"])
        d["out"] = torch.empty((case["M"], case["K"]), dtype=DT[case["out"]], device=DEV)
    return d


EPS = 1e-6


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(state):
    return {"linear": _run_linear, "norm": _run_norm, "moe": _run_moe}[state["case"]["op"]](state)


E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)


def _nibbles(w):
    """[..., n] bytes -> [..., 2n] codes, the low nibble first."""
    return torch.stack((w & 15, w >> 4), -1).flatten(-2)


def _run_linear(d):
    case = d["case"]
    if own:
        return d["linear"].forward(d["x"], d["out"])
    c = _nibbles(d["w"]).view(case["N"], -1, case["group"])
    if case["fmt"] == "nvfp4":
        lut = torch.tensor(E2M1, device=c.device)
        w = lut[c.int()] * d["scale"].view(torch.float8_e4m3fn).float()[:, :, None] * (1.0 / d["global"])
    else:
        w = (c.float() - d["zero"].float()[:, :, None]) * d["scale"].float()[:, :, None]
    y = d["x"].float() @ w.view(case["N"], -1).T
    if d["bias"] is not None:
        y = y + d["bias"]
    return y.to(DT[case["out"]])


def _run_norm(d):
    case, train = d["case"], d["case"]["dir"] == "train"
    if own:
        kw = {"z": d["z"], "residual": d["residual"], "post_w": d["post"], "pre_w": d["pre"], "gate": d["gate"]}
        d["norm"].forward(residual_out=d["h"], out=d["y"], stats=d["stats"] if train else None, **kw)
        out = {"h": d["h"], "y": d["y"]}
        if train:
            d["norm"].backward(stats=d["stats"], dout=d["dy"], dresidual_out=d["dh"], **kw, **d["grads"])
            out.update(d["grads"])
        return {n: t for n, t in out.items() if t is not None}
    z, r, s, off = d["z"].float(), d["residual"].float(), case["scale"], case["offset"]
    gate = 1.0 if d["gate"] is None else d["gate"].float()
    if case["gate"] == "token":
        gate = gate[:, None]
    if case["post"]:
        wp = d["post"].float() + off
        rz = torch.rsqrt((z * z).mean(-1, keepdim=True) + EPS)
        zn = z * rz
        n = zn * wp
    else:
        n = z
    h = r + s * (gate * n)
    out = {"h": h.to(DT[case["rdt"]])}
    if case["pre"]:
        wr = d["pre"].float() + off
        rh = torch.rsqrt((h * h).mean(-1, keepdim=True) + EPS)
        hn = h * rh
        out["y"] = (hn * wr).to(DT[case["dt"]])
    if not train:
        return out
    dh = d["dh"].float()
    if case["pre"]:
        dy = d["dy"].float()
        a = dy * wr
        dh = dh + rh * (a - hn * (a * hn).mean(-1, keepdim=True))
        out["dpre_w"] = (dy * hn).sum(0).to(DT[case["wdt"]])
    out["dresidual"] = dh.to(DT[case["rdt"]])
    dn = s * (gate * dh)
    if case["gate"] != "none":
        dg = s * (dh * n)
        dg = {"channel": lambda t: t.sum(0), "token": lambda t: t.sum(1), "full": lambda t: t}[case["gate"]](dg)
        out["dgate"] = dg.to(d["gate"].dtype)
    if case["post"]:
        out["dpost_w"] = (dn * zn).sum(0).to(DT[case["wdt"]])
        a = dn * wp
        dn = rz * (a - zn * (a * zn).mean(-1, keepdim=True))
    out["dz"] = dn.to(DT[case["dt"]])
    return out


def _expert(d, name, ids):
    """Weights of the experts `ids` in fp32: fp16(code * scale + bias), bias = fp16(-zero * scale)."""
    s = d[name + "_scale"][ids].float()[..., None]
    b = (-d[name + "_zero"][ids].float()[..., None] * s).half().float()
    c = _nibbles(d[name][ids]).float()
    c = c.view(*s.shape[:-1], 32)
    return (c * s + b).half().float().flatten(-2)


def _run_moe(d):
    case = d["case"]
    if own:
        return d["layer"].forward(d["x"], d["out"])
    E, S, I, topk = case["E"], case["shared"], case["I"], case["topk"]
    x = d["x"].float()
    logits = d["x"].double() @ d["router"].double().T  # which expert is chosen hangs on their order
    score = torch.sigmoid(logits) if case["score"] == "sigmoid" else torch.exp(
        logits - logits.amax(1, keepdim=True))
    if case["score"] == "softmax":
        score = score / score.sum(1, keepdim=True)
    key = score if d["bias"] is None else score + d["bias"].double()
    ids = torch.sort(key, dim=1, descending=True, stable=True)[1][:, :topk]
    w = torch.gather(score, 1, ids)
    if case["renorm"]:
        w = w / w.sum(1, keepdim=True)
    w = (w * case["rscale"]).float()
    if S:
        ids = torch.cat((ids, torch.arange(E, E + S, device=x.device).expand(len(x), S)), 1)
        sw = torch.ones((len(x), S), device=x.device)
        if d["sgate"] is not None:
            sw = torch.sigmoid(x @ d["sgate"].float().T)
        w = torch.cat((w, sw), 1)
    out = torch.empty((len(x), case["K"]), device=x.device)
    for m in range(len(x)):
        h = _expert(d, "w13", ids[m]) @ x[m]
        g, u = h[:, :I], h[:, I:]
        act = g / (1 + torch.exp(-g)) * u
        out[m] = (w[m][:, None] * (_expert(d, "w2", ids[m]) @ act[:, :, None])[:, :, 0]).sum(0)
    return out.to(DT[case["out"]])


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}


def work(case):
    if case["op"] == "linear":
        N, K, M = case["N"], case["K"], case["M"]
        meta = N * (K // case["group"]) * (1 if case["fmt"] == "nvfp4" else 3)
        return {"bytes": N * K // 2 + meta + 2 * M * K + SIZE[case["out"]] * M * N + (4 * N if case["bias"] else 0),
                "flops": 2 * M * N * K}
    if case["op"] == "norm":
        M, K, t, r, w = case["M"], case["K"], SIZE[case["dt"]], SIZE[case["rdt"]], SIZE[case["wdt"]]
        n = M * K
        ws = case["post"] + case["pre"]
        gate = {"none": 0, "channel": w * K, "token": t * M, "full": t * n}[case["gate"]]
        fwd = n * (t + 2 * r + (t if case["pre"] else 0)) + w * K * ws + gate
        if case["dir"] == "fwd":
            return {"bytes": fwd, "flops": 12 * n}
        return {"bytes": fwd + n * (t + 2 * r + (t if case["pre"] else 0)) + w * K * ws + gate, "flops": 40 * n}
    M, E, K, I, S = case["M"], case["E"], case["K"], case["I"], case["shared"]
    hit = E * (1 - (1 - case["topk"] / E) ** M) + S  # experts that the tokens name, when all are as likely
    per = 3 * K * I
    return {"bytes": int(hit * (per // 2 + per // 32 * case["meta"]) + 2 * K * (E + (S if case["sgate"] else 0)) +
                         M * K * (2 + SIZE[case["out"]])),
            "flops": 2 * M * (case["topk"] + S) * per + 2 * M * E * K}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def _e4m3(b):
    """The number that an e4m3 byte stands for."""
    b = b.to(torch.int32)
    e, m = (b >> 3) & 15, (b & 7).double()
    mag = torch.where(e > 0, torch.ldexp(1 + m / 8, e - 7), m * 2.0 ** -9)
    return torch.where(b >= 128, -mag, mag)


def _unpack(b):
    b = b.to(torch.int16)
    return torch.stack((b % 16, b // 16), b.dim()).flatten(b.dim() - 1)


def exact(case, seed):
    d = _inputs(case, seed)
    return {"linear": _exact_linear, "norm": _exact_norm, "moe": _exact_moe}[case["op"]](case, d)


def _exact_linear(case, d):
    x, rows, parts = d["x"].double(), 8192, []
    for a in range(0, case["N"], rows):
        q = _unpack(d["w"][a:a + rows])
        s = d["scale"][a:a + rows]
        if case["fmt"] == "nvfp4":
            e, m = ((q >> 1) & 3).int(), (q & 1).double()
            v = torch.where(e > 0, torch.ldexp(1 + m / 2, e - 1), m / 2)
            v = torch.where(q >= 8, -v, v) * torch.repeat_interleave(_e4m3(s), 16, 1)
            v = v / d["global"]
        else:
            z = torch.repeat_interleave(d["zero"][a:a + rows].double(), case["group"], 1)
            v = (q.double() - z) * torch.repeat_interleave(s.double(), case["group"], 1)
        parts.append(x @ v.T)
    y = torch.cat(parts, 1)
    return y if d["bias"] is None else y + d["bias"].double()


def _exact_norm(case, d):
    M, K = case["M"], case["K"]
    f = lambda t: t.double()  # noqa: E731
    rms = lambda t: torch.sqrt(t.pow(2).sum(1) / K + EPS)[:, None]  # noqa: E731
    one = torch.ones((1, 1), dtype=torch.float64, device=DEV)
    z, r = f(d["z"]), f(d["residual"])
    g = {"none": lambda t: one, "channel": lambda t: f(t)[None, :], "token": lambda t: f(t)[:, None],
         "full": f}[case["gate"]](d["gate"])
    if case["post"]:
        a, w1 = z / rms(z), f(d["post"]) + case["offset"]
        n = a * w1
    else:
        n = z
    h = r + case["scale"] * g * n
    got = {"h": h}
    if case["pre"]:
        b, w2 = h / rms(h), f(d["pre"]) + case["offset"]
        got["y"] = b * w2
    if case["dir"] == "fwd":
        return got

    def through(dv, v, unit):  # the gradient of v for that of unit = v / rms(v)
        return (dv - unit * torch.einsum("mk,mk->m", dv, unit)[:, None] / K) / rms(v)

    dh = f(d["dh"])
    if case["pre"]:
        dy = f(d["dy"])
        dh = dh + through(dy * w2, h, b)
        got["dpre_w"] = torch.einsum("mk,mk->k", dy, b)
    got["dresidual"] = dh
    if case["gate"] != "none":
        dg = case["scale"] * dh * n
        got["dgate"] = dg if case["gate"] == "full" else torch.einsum(
            "mk->k" if case["gate"] == "channel" else "mk->m", dg)
    dn = case["scale"] * g * dh
    if case["post"]:
        got["dpost_w"] = torch.einsum("mk,mk->k", dn, a)
        dn = through(dn * w1, z, a)
    got["dz"] = dn
    return got


def _exact_moe(case, d):
    E, I, S = case["E"], case["I"], case["shared"]
    x = d["x"].double()

    def weight(name, e):
        s = torch.repeat_interleave(d[name + "_scale"][e].double(), 32, 1)
        b = torch.repeat_interleave((d[name + "_zero"][e].double() * -d[name + "_scale"][e].double()).half().double(), 32, 1)
        return torch.addcmul(b, _unpack(d[name][e]).double(), s).half().double()

    def expert(e, rows):
        p = x[rows] @ weight("w13", e).T
        return (p[:, :I] * torch.reciprocal(1 + torch.exp(-p[:, :I])) * p[:, I:]) @ weight("w2", e).T

    out = torch.zeros((case["M"], case["K"]), dtype=torch.float64, device=DEV)
    t = torch.einsum("mk,ek->me", x, d["router"].double())
    score = torch.softmax(t, 1) if case["score"] == "softmax" else torch.reciprocal(1 + torch.exp(-t))
    rank = score if d["bias"] is None else score + d["bias"].double()
    order = torch.argsort(-rank, dim=1, stable=True)[:, :case["topk"]]
    chosen = torch.zeros_like(score).scatter_(1, order, 1.0) * score
    if case["renorm"]:
        chosen = chosen / chosen.sum(1)[:, None]
    chosen = chosen * case["rscale"]
    for e in torch.unique(order).tolist():
        rows = (chosen[:, e] != 0).nonzero()[:, 0]
        out[rows] += chosen[rows, e][:, None] * expert(e, rows)
    for j in range(S):
        w = 1.0 if d["sgate"] is None else torch.reciprocal(1 + torch.exp(-(x @ d["sgate"][j].double())))[:, None]
        out += w * expert(E + j, slice(None))
    return out
