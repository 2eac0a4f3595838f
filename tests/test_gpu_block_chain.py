"""Blocks one after another, each handing the next its normed input: against
float64 autograd of the written-out stack, for plain blocks, checkpointed ones on
shared scratch, and stacks that mix both.

Bars.  On the longest chain to a gradient of a stack of three lie ten bf16
roundings a block (see the block's own tests), each at most 2^-8/sqrt(3) rms of
its value: thirty independent ones are sqrt(30) 2^-8/sqrt(3) = 1.24%.  A
checkpointed block adds 1.5% at most of what passes through it (g and u in 8 bits),
three of them sqrt(3) 1.5% = 2.6%: below 4% with the roundings.  Another block's
normed input in place of a block's own, which is what scratch used again would
leave, is another tensor altogether (off by more than its size).
"""
import pytest
import torch

import moe_expert_layer_topk_gb300 as m
from gpu_util import inputs

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
T, H, I, E, k = 150, 128, 64, 8, 2
EPS, A, B = 1e-5, 0.9, 0.6
PLAIN, EIGHT = 30 ** 0.5 * 2 ** -8 / 3 ** 0.5, 0.04
WEIGHTS = ("pre", "post", "gate", "Wr", "Wg", "Wu", "Wd")


def params(n):
    out = []
    for i in range(n):
        gen = torch.Generator().manual_seed(90 + i)
        p = {name: v.cuda() for name, v in inputs(T, H, I, E, k, seed=60 + i).items() if name in WEIGHTS}
        for name in ("Wg", "Wu", "Wd"):  # the layer's inputs have 0.02; larger, so that z is not all eps
            p[name] = (p[name].float() * 5).to(BF)
        p["pre"], p["post"] = (1 + 0.2 * torch.randn(H, generator=gen).cuda() for _ in range(2))
        p["gate"] = torch.randn(T, generator=gen).cuda()
        out.append(p)
    return out


def batch(seed=3):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(T, H, generator=g, device="cuda"), torch.randn(T, H, generator=g, device="cuda")


def stack(kinds, **options):
    """Blocks of the kinds (p: plain, c: checkpointed, sharing the scratch of the first of those)."""
    blocks, first = [], None
    for i, kind in enumerate(kinds):
        b = m.MoEBlock(T, H, I, E, k, gate="token", eps=EPS, res_scale=A, out_scale=B, fp32=True, next_norm=i + 1 < len(kinds),
                       checkpoint=kind == "c", share=first if kind == "c" else None, **options)
        first = b if first is None and kind == "c" else first
        blocks.append(b)
    return blocks


def args(p):
    return p["pre"], p["post"], p["Wr"]


def run(blocks, ps, x, dout, hand=lambda normed: normed, stream=None):
    """Forward and backward of the stack; hand: how a block's normed input reaches the next."""
    launch = launched(blocks, ps, x, dout, hand, stream)
    torch.cuda.synchronize()
    assert m.moe_read_device_status(reset=True) == 0
    return results(blocks, *launch)


def launched(blocks, ps, x, dout, hand=lambda normed: normed, stream=None):
    ins, normed = [], None
    for i, (b, p) in enumerate(zip(blocks, ps)):
        ins.append(x)
        nxt = ps[i + 1]["pre"] if i + 1 < len(blocks) else None
        x = b.forward(x, *args(p), None, p["Wg"], p["Wu"], p["Wd"], p["gate"], normed=normed, next_gain=nxt, stream=stream)
        normed = hand(b.next_normed) if nxt is not None else None
    out, grad = x, dout
    for b, p, x in reversed(list(zip(blocks, ps, ins))):
        grad = b.backward(grad, x, *args(p), p["Wg"], p["Wu"], p["Wd"], p["gate"], stream=stream)
    return out, grad


def results(blocks, out, grad):
    grads = [dict(pre=b.d_pre_gain, post=b.d_post_gain, gate=b.d_gate, Wr=b.layer.dWr, Wg=b.layer.dWg, Wu=b.layer.dWu, Wd=b.layer.dWd)
             for b in blocks]
    return out.clone(), grad.clone(), [{n: t.clone() for n, t in g.items()} for g in grads]


def autograd(blocks, ps, x, dout):
    """The stack in float64, its gradients by autograd; each block's routing held."""
    x0 = x.double().requires_grad_()
    leaves, x = [], x0
    for b, p in zip(blocks, ps):
        v = {n: p[n].detach().double().requires_grad_() for n in WEIGHTS}
        leaves.append(v)
        idx = b.layer.topk_idx.long()
        n = x * torch.rsqrt(x.square().mean(1, keepdim=True) + EPS) * v["pre"]
        w = torch.softmax((n @ v["Wr"]).gather(1, idx), 1)
        z = torch.zeros_like(x)
        for j in range(k):
            e = idx[:, j]
            g, u = torch.einsum("th,tih->ti", n, v["Wg"][e]), torch.einsum("th,tih->ti", n, v["Wu"][e])
            z = z + w[:, j:j + 1] * torch.einsum("ti,thi->th", torch.nn.functional.silu(g) * u, v["Wd"][e])
        z = z * torch.rsqrt(z.square().mean(1, keepdim=True) + EPS)
        x = A * x + B * torch.sigmoid(v["gate"])[:, None] * z * v["post"]
    (x * dout.double()).sum().backward()
    return x.detach(), x0.grad, [{n: t.grad for n, t in v.items()} for v in leaves]


def rel(a, b):
    a, b = a.double(), b.double()
    return ((a - b).norm() / b.norm()).item()


@pytest.mark.parametrize("hand", ["as given", "unpacked"])
@pytest.mark.parametrize("kinds", ["ppp", "ccc", "cpc", "ccp", "pcp", "cppc"])
def test_stack_against_autograd(kinds, hand):
    ps, (x, dout) = params(len(kinds)), batch()
    blocks = stack(kinds)
    out, dx, grads = run(blocks, ps, x, dout, (lambda normed: normed) if hand == "as given" else tuple)
    want, wdx, wgrads = autograd(blocks, ps, x, dout)
    bar = PLAIN if "c" not in kinds else EIGHT
    off = {"out": rel(out, want), "dx": rel(dx, wdx)}
    off.update({f"{i}.{n}": rel(g[n], w[n]) for i, (g, w) in enumerate(zip(grads, wgrads)) for n in g})
    assert off.pop("out") <= PLAIN
    assert all(v <= bar for v in off.values()), {n: v for n, v in off.items() if not v <= bar}


def same(a, b):
    return torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]) and all(torch.equal(g[n], w[n]) for g, w in zip(a[2], b[2]) for n in g)


@pytest.mark.parametrize("hand", ["as given", "unpacked"])
def test_mixed_stack_on_a_stream_and_in_a_graph(hand):
    """The same bits on another stream (as an object and as a handle) and from a graph, whose inputs change."""
    hand = (lambda normed: normed) if hand == "as given" else tuple
    ps, (x, dout) = params(3), batch()
    blocks = stack("cpc")
    want = run(blocks, ps, x, dout, hand)
    s = torch.cuda.Stream()
    for stream in (s, s.cuda_stream):
        assert same(run(stack("cpc"), ps, x, dout, hand, stream), want)
    other = [t.flip(0).contiguous() for t in (x, dout)]
    wother = run(blocks, ps, *other, hand)
    hx, hd = x.clone(), dout.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        left = launched(blocks, ps, hx, hd, hand)
    for inp, w in (((x, dout), want), (other, wother), ((x, dout), want)):
        hx.copy_(inp[0])
        hd.copy_(inp[1])
        g.replay()
        torch.cuda.synchronize()
        assert same(results(blocks, *left), w)


def test_one_eps_along_a_stack():
    """A normed input made with another eps than the block's own is refused, and nothing is left of the call."""
    ps, (x, _) = params(2), batch()
    (p, q) = ps
    for training in (True, False):
        a = m.MoEBlock(T, H, I, E, k, gate="token", eps=1e-2, fp32=True, next_norm=True, training=training)
        other, same_eps = (m.MoEBlock(T, H, I, E, k, gate="token", eps=eps, fp32=True, training=training) for eps in (1e-6, 1e-2))
        out = a.forward(x, *args(p), None, p["Wg"], p["Wu"], p["Wd"], p["gate"], next_gain=q["pre"])
        rest = (*args(q), None, q["Wg"], q["Wu"], q["Wd"], q["gate"])
        other.out.fill_(7.0)
        with pytest.raises(ValueError, match="eps"):
            other.forward(out, *rest, normed=a.next_normed)
        assert (other.out == 7).all()
        got = same_eps.forward(out, *rest, normed=a.next_normed).clone()
        assert rel(got, same_eps.forward(out, *rest)) <= 2 ** -8  # its own norm: other orders of the sum
