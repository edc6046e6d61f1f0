"""Fine-tune low-rank adapters of a frozen quantized MLP block, then serve them.

Two adapters are trained, one after the other, to reproduce the block plus a
hidden low-rank change each (TrainMLP: forward and backward through the frozen
weights; AdamW with 8-bit states on fp32 masters). Both are then put into slots
of a LoraMLP and answer a mixed batch, in which every token names its adapter.

    python examples/adapters.py [--fmt nvfp4|fp8] [--steps 200] [--tokens 512]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import weight_quantized_swiglu_gb300 as q  # noqa: E402
from weight_quantized_swiglu_gb300 import inputs as gen  # noqa: E402

K, I, RANK = 256, 512, 8
PARTS = {"gate_a": (RANK, K), "gate_b": (I, RANK), "up_a": (RANK, K), "up_b": (I, RANK), "down_a": (RANK, I),
         "down_b": (K, RANK)}


def parts(seed, b_std):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return {n: torch.randn(s, generator=g, device="cuda") * (s[1] ** -0.5 if n.endswith("_a") else b_std)
            for n, s in PARTS.items()}


def as_adapter(p):
    return q.Adapter(1.0, **{n: t.to(torch.bfloat16) for n, t in p.items()})


def finetune(train, target, steps, tokens, seed):
    """Train an adapter towards `target` (another one); returns it and the losses."""
    dev = dict(device="cuda")
    master = parts(seed, 0.0)  # B = 0: it starts as the block itself
    bf = {n: t.to(torch.bfloat16) for n, t in master.items()}
    grad = {n: torch.empty_like(t) for n, t in bf.items()}
    adapter, grads = q.Adapter(1.0, **bf), q.Adapter(1.0, **grad)
    sizes = [t.numel() for t in bf.values()]
    codes = [[torch.zeros(n, dtype=torch.float8_e4m3fn, **dev) for n in sizes] for _ in range(2)]
    scales = [[torch.zeros(-(-n // 256), **dev) for n in sizes] for _ in range(2)]
    opt = q.AdamW(list(bf.values()), list(grad.values()), *codes, m_scale=scales[0], v_scale=scales[1],
                  master=list(master.values()))
    saved = torch.empty(train.saved_bytes(tokens), dtype=torch.uint8, **dev)
    out, want, dx = (torch.empty((tokens, K), dtype=torch.bfloat16, **dev) for _ in range(3))
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    losses = []
    for step in range(1, steps + 1):
        x = torch.randn((tokens, K), generator=g, device="cuda").to(torch.bfloat16)
        train.forward(x, want, saved, adapter=target)
        train.forward(x, out, saved, adapter=adapter)
        diff = out.float() - want.float()
        losses.append(diff.square().mean())
        dout = (2 * diff / tokens).to(torch.bfloat16)
        train.backward(x, saved, dout, dx, adapter=adapter, grads=grads)
        opt.step(lr=1e-2 * min(1.0, 2.0 - 2.0 * step / steps), weight_decay=0.0, step=step)
    losses = torch.stack(losses).tolist()
    opt.close()
    return adapter, losses


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--fmt", choices=("nvfp4", "fp8"), default="nvfp4")
    ap.add_argument("--steps", type=int, default=200)
    ap.add_argument("--tokens", type=int, default=512)
    a = ap.parse_args(argv)
    case = gen.gen_dense_case(a.fmt, K, I, 1, 7)
    if a.fmt == "fp8":
        for p in (case.gate, case.up, case.down):
            p.scale *= 0.02
    mlp = q.QuantMLP.from_case(case, max_M=max(768, a.tokens))
    train = q.TrainMLP(mlp, RANK)
    lora = q.LoraMLP(mlp, slots=2, max_rank=RANK)
    results, trained = [], []
    for slot in range(2):
        target = as_adapter(parts(100 + slot, 0.15))
        adapter, losses = finetune(train, target, a.steps, a.tokens, 10 * slot)
        print(f"adapter {slot}: mean square error {losses[0]:.4g} -> {losses[-1]:.4g} in {a.steps} steps")
        lora.set(slot, adapter)
        trained.append(adapter)
        results.append(losses)
    # a batch of both adapters' requests and of the block's own
    ids = torch.tensor([0, 1, -1, 1, 0, -1, 0], dtype=torch.int32, device="cuda")
    x = torch.randn((ids.numel(), K), device="cuda").to(torch.bfloat16)
    out = torch.empty_like(x)
    lora.forward(x, ids, out)
    saved = torch.empty(train.saved_bytes(ids.numel()), dtype=torch.uint8, device="cuda")
    alone = [train.forward(x, torch.empty_like(x), saved, adapter=ad).clone() for ad in (*trained, None)]
    want = torch.stack([alone[i][m] for m, i in enumerate(ids.tolist())])
    off = ((out.float() - want.float()).norm() / want.float().norm()).item()
    torch.cuda.synchronize()
    mlp.check()
    print(f"a mixed batch against each adapter alone: {off:.1e} apart")
    for h in (lora, train, mlp):
        h.close()
    return results, off


if __name__ == "__main__":
    main()
