"""Training a stack of blocks whose activations are kept in 8 bits.

Each block is an MoE expert layer between its norms, gated by token, on a
residual stream in fp32:

    x <- x + s sigmoid(gate) norm(MoE(norm(x) pre)) post

`step` runs the stack forward and backward: every block computes the next
one's normed input on the way, keeps g and u in 8 bits and little else
(`checkpoint`), and shares its scratch with the others (`share`); it returns the
loss and all gradients.  `train` descends on the gains, gates and routers;
`serve` runs a few tokens through the trained stack.

    python examples/train_blocks.py
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
    T: int = 700
    H: int = 512
    I: int = 256  # noqa: E741
    E: int = 16
    k: int = 4
    blocks: int = 3


def make(s: Sizes, seed: int = 0):
    """Parameters of each block and a batch."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    rn = lambda *shape, std=1.0: torch.randn(*shape, generator=g, device="cuda") * std  # noqa: E731
    bf = torch.bfloat16
    params = [dict(pre=1 + rn(s.H, std=0.1), post=1 + rn(s.H, std=0.1), gate=rn(s.T), Wr=rn(s.H, s.E, std=0.05),
                   Wg=rn(s.E, s.I, s.H, std=s.H ** -0.5).to(bf), Wu=rn(s.E, s.I, s.H, std=s.H ** -0.5).to(bf),
                   Wd=rn(s.E, s.H, s.I, std=s.I ** -0.5).to(bf)) for _ in range(s.blocks)]
    return dict(params=params, x=rn(s.T, s.H), target=rn(s.T, s.H))


def stack(s: Sizes, T: int | None = None, training: bool = True, checkpoint: bool = True):
    blocks = []
    for i in range(s.blocks):
        blocks.append(m.MoEBlock(s.T if T is None else T, s.H, s.I, s.E, s.k, gate="token", out_scale=0.5, fp32=True,
                                 next_norm=i + 1 < s.blocks, training=training, checkpoint=checkpoint and training,
                                 share=blocks[0] if blocks and checkpoint and training else None))
    return blocks


def forward(blocks, params, x, gates):
    """The stack's output, and each block's input."""
    inputs, normed = [], None
    for i, (b, p) in enumerate(zip(blocks, params)):
        inputs.append(x)
        nxt = params[i + 1]["pre"] if i + 1 < len(blocks) else None
        x = b.forward(x, p["pre"], p["post"], p["Wr"], None, p["Wg"], p["Wu"], p["Wd"], gates[i], normed=normed, next_gain=nxt)
        normed = b.next_normed if nxt is not None else None
    return x, inputs


def step(blocks, d):
    """The loss |out - target|^2 / 2n, and the gradients of x and of every block's parameters."""
    params = d["params"]
    out, inputs = forward(blocks, params, d["x"], [p["gate"] for p in params])
    diff = out - d["target"]
    grad = diff / diff.numel()
    for b, p, x in reversed(list(zip(blocks, params, inputs))):
        grad = b.backward(grad, x, p["pre"], p["post"], p["Wr"], p["Wg"], p["Wu"], p["Wd"], p["gate"])
    grads = [dict(pre=b.d_pre_gain, post=b.d_post_gain, gate=b.d_gate, Wr=b.layer.dWr, Wg=b.layer.dWg, Wu=b.layer.dWu,
                  Wd=b.layer.dWd) for b in blocks]
    return diff.square().mean() / 2, grad, grads


def train(s: Sizes, d: dict, steps: int = 10, length: float = 0.3):
    """Updates gains, gates and routers by steps of a fixed length; returns the losses."""
    blocks = stack(s)
    seen = []
    for _ in range(steps):
        loss, _, grads = step(blocks, d)
        seen.append(loss)
        for p, g in zip(d["params"], grads):
            for name in ("pre", "post", "gate", "Wr"):
                p[name] -= length * g[name] / g[name].norm().clamp(min=1e-20)
    torch.cuda.synchronize()
    status = m.moe_read_device_status()
    assert status == 0, status
    return torch.stack(seen).tolist()


def serve(s: Sizes, d: dict, tokens: int = 3):
    """A few tokens through the stack."""
    blocks = stack(s, T=tokens, training=False)
    out, _ = forward(blocks, d["params"], d["x"][:tokens].contiguous(), [p["gate"][:tokens].contiguous() for p in d["params"]])
    torch.cuda.synchronize()
    return out.clone()


def main():
    s = Sizes()
    d = make(s)
    seen = train(s, d)
    for i in (0, len(seen) // 2, len(seen) - 1):
        print("step %2d: loss %.5f" % (i, seen[i]))
    print("served:", tuple(serve(s, d).shape))


if __name__ == "__main__":
    main()
