"""Fine-tuning and serving several adapters over one block.

The block's second half as one GPU runs it: a projection with frozen weights
shared by all requests and a low-rank adapter for each, then the MoE expert
layer with residual dropout and the router's balance loss and z-loss:

    a = W x + B_i A_i x               moe_adapter_linear       (request i's adapter)
    y = a + D(MoE(a))                 route, dispatch, experts, combine with dropout
    loss = |y - target|^2 / 2 + balance_coef balance + z_coef z

`finetune` trains the adapters and the router by gradient descent of a fixed
step length on a batch of packed sequences of different lengths, one adapter
each, every loss term's gradient coming from the library's backward calls; `serve` then runs
single-token steps of a batch of requests over the trained adapters.

    python examples/finetune_block.py
"""
from __future__ import annotations

import sys
from dataclasses import dataclass
from pathlib import Path

import torch

sys.path.insert(0, str(Path(__file__).resolve().parents[1]))
import moe_expert_layer_topk_gb300 as m  # noqa: E402


@dataclass
class Sizes:
    lengths: tuple[int, ...] = (700, 33, 1, 512, 290)  # tokens of each packed sequence
    H: int = 512
    I: int = 256  # noqa: E741
    E: int = 32
    k: int = 4
    r: int = 16
    num_adapters: int = 3


def make(s: Sizes, seed: int = 0):
    """Frozen weights, adapters (B starts at zero, so that they start without effect) and a batch."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    rn = lambda *shape, std=1.0: torch.randn(*shape, generator=g, device="cuda") * std  # noqa: E731
    T, bf = sum(s.lengths), torch.bfloat16
    ends = torch.tensor([0, *s.lengths], device="cuda").cumsum(0).to(torch.int32)
    which = torch.arange(len(s.lengths), device="cuda", dtype=torch.int32) % s.num_adapters
    return dict(W=rn(s.H, s.H, std=s.H ** -0.5).to(bf), A=rn(s.num_adapters, s.r, s.H, std=s.H ** -0.5),
                B=torch.zeros(s.num_adapters, s.H, s.r, device="cuda"), scale=torch.full((s.num_adapters,), 2.0, device="cuda"),
                Wr=rn(s.H, s.E, std=0.05), Wg=rn(s.E, s.I, s.H, std=0.05).to(bf), Wu=rn(s.E, s.I, s.H, std=0.05).to(bf),
                Wd=rn(s.E, s.H, s.I, std=0.05).to(bf), x=rn(T, s.H).to(bf), target=rn(T, s.H), ends=ends, which=which)


def finetune(s: Sizes, d: dict, steps: int = 20, step: float = 0.2, balance_coef: float = 0.05, z_coef: float = 1e-3,
             dropout: float = 0.1):
    """Updates d's A, B and Wr; returns the (fit, balance, z) losses of every step."""
    T, n = sum(s.lengths), len(s.lengths)
    proj = m.AdapterLinear(T, s.H, s.H, s.r, s.num_adapters, n, training=True)
    layer = m.MoELayer(T, s.H, s.I, s.E, s.k, balance_coef=balance_coef, z_coef=z_coef, sequences=n, dropout=dropout, seed=7)
    dx2 = torch.empty(T, s.H, dtype=torch.bfloat16, device="cuda")
    seen = []
    for _ in range(steps):
        A, B = d["A"].bfloat16(), d["B"].bfloat16()  # fp32 masters, bf16 operands
        a = proj.forward(d["x"], d["W"], A, B, d["scale"], d["ends"], d["which"])
        y = layer.forward(a, d["Wr"], None, d["Wg"], d["Wu"], d["Wd"], residual=a, seg_offsets=d["ends"])
        diff = y.float() - d["target"]
        seen.append(torch.cat([diff.square().mean()[None] / 2, layer.loss]))
        dy = (diff / diff.numel()).bfloat16()
        da = layer.backward(dy, a, d["Wr"], d["Wg"], d["Wu"], d["Wd"])
        da = (da.float() + dy.float()).bfloat16()  # the residual's path
        proj.backward(da, d["x"], d["W"], A, B, d["scale"], d["ends"], d["which"], dx=dx2)
        layer.advance_rng()  # the next step drops other elements
        for name, grad in (("A", proj.dA), ("B", proj.dB), ("Wr", layer.dWr)):
            d[name] -= step * grad / grad.norm().clamp(min=1e-20)
    torch.cuda.synchronize()
    status = m.moe_read_device_status()
    assert status == 0, status
    return torch.stack(seen).tolist()


def serve(s: Sizes, d: dict, batch: int = 6, steps: int = 4):
    """Single-token steps of `batch` requests, every third without an adapter; returns the last outputs."""
    proj = m.AdapterLinear(batch, s.H, s.H, s.r, s.num_adapters, batch)
    layer = m.MoELayer(batch, s.H, s.I, s.E, s.k, training=False)
    A, B = d["A"].bfloat16(), d["B"].bfloat16()
    ends = torch.arange(batch + 1, dtype=torch.int32, device="cuda")
    which = torch.tensor([-1 if i % 3 == 2 else i % s.num_adapters for i in range(batch)], dtype=torch.int32, device="cuda")
    x = d["x"][:batch].clone()
    for _ in range(steps):
        a = proj.forward(x, d["W"], A, B, d["scale"], ends, which)
        x = layer.forward(a, d["Wr"], None, d["Wg"], d["Wu"], d["Wd"], residual=a).clone()
        x = (x.float() / x.float().square().mean(1, keepdim=True).sqrt()).bfloat16()
    torch.cuda.synchronize()
    return x


def main():
    s = Sizes()
    d = make(s)
    seen = finetune(s, d)
    for i in (0, len(seen) // 2, len(seen) - 1):
        print("step %2d: fit %.4f  balance %.4f  z %.4f" % (i, *seen[i]))
    print("served:", tuple(serve(s, d).shape))


if __name__ == "__main__":
    main()
