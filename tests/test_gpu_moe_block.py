"""The block (norms, gate, residual around the MoE layer) and the layer that
keeps its activations in 8 bits: against float64 autograd of the written-out
block, against each other, and the example end to end.

Bars.  The layer's acceptance bars (gpu_util.assert_close: bf16 intermediates)
hold for out and the gate's gradient.  On the longest chain to a gradient ten bf16 roundings
lie (n, g, u, y_perm, z, dz, dy_perm, dgu, dx_perm, dn), each off by at most half
a step: 2^-8 of the value at most, evenly spread, 2^-8/sqrt(3) rms; ten independent
ones are sqrt(10) 2^-8/sqrt(3) = 0.71% of a gradient (relative L2).  With g and u in 8 bits, each is off by at most s/2 with s =
amax/127 (1 + 2^-7) of its 32 columns; for normal columns amax is about 2.1 and
seldom over 3.5 standard deviations, so the error is at most 3.5/127/sqrt(12) =
0.8% (rms) of each, and enters dgu, h and d_w through two factors (g and u) with
derivatives of at most 1.1: below 1.1 sqrt(2) 0.8% = 1.3% of a gradient, 1.5% with
those roundings.  The bar is 2%, and 4% for gradients behind three such layers.
"""
import importlib.util
import sys
from pathlib import Path

import pytest
import torch

import moe_expert_layer_topk_gb300 as m
from gpu_util import assert_close, inputs, to_dev

ROOT = Path(__file__).resolve().parents[1]
BF, F32 = torch.bfloat16, torch.float32
EIGHT = 0.02
ROUNDINGS = 10 ** 0.5 * 2 ** -8 / 3 ** 0.5


def rel(a, b):
    a, b = a.double(), b.double()
    return ((a - b).norm() / b.norm()).item()


def test_options_that_do_not_go_together():
    for kw in (dict(training=False, checkpoint=True), dict(checkpoint_input=True), dict(share=object()), dict(training=False, share=object())):
        with pytest.raises(ValueError):
            m.MoELayer(8, 64, 64, 4, 2, **kw)
    for kw in (dict(gate="row"), dict(dropout=0.1), dict(fused_combine=True, training=False), dict(checkpoint=True, checkpoint_input=True)):
        with pytest.raises(ValueError):
            m.MoEBlock(8, 64, 64, 4, 2, **kw)


T, H, I, E, k = 150, 128, 64, 8, 2


def params(seed=31):
    inp = inputs(T, H, I, E, k, seed=seed)
    gen = torch.Generator().manual_seed(seed)
    inp["pre"], inp["post"] = 1 + 0.2 * torch.randn(H, generator=gen), 1 + 0.2 * torch.randn(H, generator=gen)
    inp["token"], inp["element"] = torch.randn(T, generator=gen), torch.randn(T, H, generator=gen).to(BF)
    for n in ("Wg", "Wu", "Wd"):  # the layer's inputs have 0.02; larger, so that z is not all eps
        inp[n] = (inp[n].float() * 5).to(BF)
    return inp


def autograd(inp, idx, gate, post_norm, eps, a, b):
    """The block in float64, its gradients by autograd; routing held."""
    v = {n: inp[n].detach().double().cpu().requires_grad_() for n in ("x", "pre", "post", "Wr", "Wg", "Wu", "Wd")}
    g = None if gate is None else inp[gate].detach().double().cpu().requires_grad_()
    x = v["x"]
    n = x * torch.rsqrt(x.square().mean(1, keepdim=True) + eps) * v["pre"]
    w = torch.softmax((n @ v["Wr"]).gather(1, idx), 1)
    z = torch.zeros_like(x)
    for j in range(k):
        e = idx[:, j]
        gg, uu = torch.einsum("th,tih->ti", n, v["Wg"][e]), torch.einsum("th,tih->ti", n, v["Wu"][e])
        z = z + w[:, j:j + 1] * torch.einsum("ti,thi->th", torch.nn.functional.silu(gg) * uu, v["Wd"][e])
    if post_norm:
        z = z * torch.rsqrt(z.square().mean(1, keepdim=True) + eps)
    G = 1.0 if g is None else torch.sigmoid(g if gate == "element" else g[:, None])
    out = a * x + b * G * z * v["post"]
    (out * inp["dy"].double().cpu()).sum().backward()
    return out.detach(), {n: t.grad for n, t in v.items()}, None if g is None else g.grad


@pytest.mark.gpu
@pytest.mark.parametrize("checkpoint", [False, True])
@pytest.mark.parametrize("fp32", [False, True])
@pytest.mark.parametrize("gate,post_norm", [(None, True), ("token", True), ("element", True), ("token", False)])
def test_block_against_autograd(gate, post_norm, fp32, checkpoint):
    inp = params()
    dt = F32 if fp32 else BF
    d = to_dev(inp)
    x, dout = d["x"].to(dt), d["dy"].to(dt)
    blk = m.MoEBlock(T, H, I, E, k, gate=gate, post_norm=post_norm, eps=1e-5, res_scale=0.9, out_scale=0.6, fp32=fp32, checkpoint=checkpoint)
    w = (d["pre"], d["post"], d["Wr"])
    gt = None if gate is None else d[gate]
    out = blk.forward(x, *w, None, d["Wg"], d["Wu"], d["Wd"], gt)
    dx = blk.backward(dout, x, *w, d["Wg"], d["Wu"], d["Wd"], gt)
    torch.cuda.synchronize()
    assert m.moe_read_device_status(reset=True) == 0
    want, grads, dg = autograd(inp, blk.layer.topk_idx.cpu().long(), gate, post_norm, 1e-5, 0.9, 0.6)
    bar = dict(max_frac=4e-2, rel=EIGHT) if checkpoint else dict(rel=ROUNDINGS)
    assert_close(out, want.numpy(), "out")
    assert_close(dx, grads["x"].numpy(), "dx", **bar)
    for name, got in (("pre", blk.d_pre_gain), ("post", blk.d_post_gain), ("Wr", blk.layer.dWr), ("Wg", blk.layer.dWg), ("Wu", blk.layer.dWu),
                      ("Wd", blk.layer.dWd)):
        assert_close(got, grads[name].numpy(), name, **bar)
    if gate:
        assert_close(blk.d_gate, dg.numpy(), "gate")
    first = {n: getattr(blk, n).clone() for n in ("d_pre_gain", "d_post_gain")}
    over = dout.clone()
    blk.backward(over, x, *w, d["Wg"], d["Wu"], d["Wd"], gt, accumulate=True, dx=over, overlap=False)  # dx over dout
    assert torch.equal(over, dx)
    for n, t in first.items():
        assert torch.allclose(getattr(blk, n), 2 * t, rtol=1e-6, atol=0)


@pytest.mark.gpu
@pytest.mark.parametrize("dropout", [0.0, 0.25])
@pytest.mark.parametrize("kept", [False, True])
def test_checkpointed_layer(kept, dropout):
    """Its output is the plain layer's, its gradients near the plain layer's; scratch that another
    layer has used in between changes nothing."""
    d = to_dev(params())
    opts = dict(balance_coef=0.5, z_coef=0.02, dropout=dropout, seed=5)
    P, L = m.MoELayer(T, H, I, E, k, **opts), m.MoELayer(T, H, I, E, k, checkpoint=True, checkpoint_input=kept, **opts)
    M = m.MoELayer(T, H, I, E, k, checkpoint=True, share=L)
    assert M.x_perm is L.x_perm and M.gu_q is not L.gu_q
    w = (d["Wr"], None, d["Wg"], d["Wu"], d["Wd"])
    back = lambda layer, x, **kw: layer.backward(d["dy"], x, d["Wr"], d["Wg"], d["Wu"], d["Wd"], **kw).clone()  # noqa: E731
    assert torch.equal(P.forward(d["x"], *w), L.forward(d["x"], *w))
    dx = back(P, d["x"])
    got = back(L, None if kept else d["x"])
    L.forward(d["x"], *w)
    M.forward(d["x"].flip(0).contiguous(), *w)
    back(M, d["x"].flip(0).contiguous())
    again = back(L, None if kept else d["x"], overlap=False)
    torch.cuda.synchronize()
    assert m.moe_read_device_status(reset=True) == 0
    assert torch.equal(got, again)
    # x in 8 bits adds its own error of the same size to the gradients that it enters
    more = 2 ** 0.5 if kept else 1.0
    assert rel(got, dx) <= EIGHT and rel(L.d_w, P.d_w) <= EIGHT
    for name in ("dWg", "dWu", "dWd", "dWr"):
        assert rel(getattr(L, name), getattr(P, name)) <= EIGHT * more, name
    old = L.dWd.clone()
    back(L, None if kept else d["x"], accumulate=True)
    assert torch.allclose(L.dWd, 2 * old, rtol=1e-5, atol=1e-9)
    if not kept:
        with pytest.raises(ValueError):
            back(L, None)
    with pytest.raises(ValueError):
        m.MoELayer(T, H, 2 * I, E, k, checkpoint=True, share=L)
    with pytest.raises(ValueError):
        m.MoELayer(T, H, I, E, k, checkpoint=True, share=P)


@pytest.mark.gpu
def test_checkpointed_layer_of_one_token():
    """One token, and experts without a row."""
    d = to_dev(inputs(1, H, I, E, k, seed=3))
    P, L = m.MoELayer(1, H, I, E, k), m.MoELayer(1, H, I, E, k, checkpoint=True)
    w = (d["Wr"], None, d["Wg"], d["Wu"], d["Wd"])
    assert torch.equal(P.forward(d["x"], *w), L.forward(d["x"], *w))
    for layer in (P, L):
        layer.backward(d["dy"], d["x"], d["Wr"], d["Wg"], d["Wu"], d["Wd"])
    for name in ("dWg", "dWu", "dWd", "dx"):
        assert rel(getattr(L, name), getattr(P, name)) <= EIGHT, name
    used = set(L.topk_idx.flatten().tolist())
    assert all((L.dWd[e] == 0).all() for e in range(E) if e not in used)


@pytest.mark.gpu
def test_next_norm_refusals_and_graph():
    d = to_dev(params())
    blk, nxt = m.MoEBlock(T, H, I, E, k, gate="token", next_norm=True), m.MoEBlock(T, H, I, E, k)
    args = (d["pre"], d["post"], d["Wr"], None, d["Wg"], d["Wu"], d["Wd"])
    out = blk.forward(d["x"], *args, d["token"], next_gain=d["post"])
    n, r = blk.next_normed
    own_n = torch.empty_like(n)
    m.moe_pre_norm(out, d["post"], blk.eps, T, H, own_n)
    assert rel(n, own_n) <= 2 ** -9  # other orders of the sum: another last bit of bf16 here and there
    a = nxt.forward(out, d["post"], d["pre"], *args[2:], normed=(own_n, r)).clone()
    assert torch.equal(a, nxt.forward(out, d["post"], d["pre"], *args[2:]))
    with pytest.raises(ValueError):
        nxt.forward(out, *args, next_gain=d["pre"])
    with pytest.raises(ValueError):
        nxt.forward(out, *args, d["token"])
    with pytest.raises(ValueError):
        blk.forward(d["x"], *args)
    with pytest.raises(ValueError):
        blk.forward(d["x"], *args, d["element"])
    torch.cuda.synchronize()
    want = blk.forward(d["x"], *args, d["token"], next_gain=d["post"]).clone()
    back = (d["dy"], d["x"], d["pre"], d["post"], d["Wr"], d["Wg"], d["Wu"], d["Wd"], d["token"])
    wdx = blk.backward(*back, overlap=False).clone()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        blk.forward(d["x"], *args, d["token"], next_gain=d["post"])
        blk.backward(*back, overlap=False)
    for _ in range(2):
        blk.out.zero_()
        blk.dx.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(blk.out, want) and torch.equal(blk.dx, wdx)


def example():
    spec = importlib.util.spec_from_file_location("train_blocks", ROOT / "examples" / "train_blocks.py")
    mod = importlib.util.module_from_spec(spec)
    sys.modules["train_blocks"] = mod
    spec.loader.exec_module(mod)
    return mod


@pytest.mark.gpu
def test_example_gradients_and_run():
    ex = example()
    s = ex.Sizes(T=200, H=128, I=64, E=8, k=2)
    d = ex.make(s)
    loss, dx, grads = ex.step(ex.stack(s), d)
    dx = dx.clone()
    ploss, pdx, pgrads = ex.step(ex.stack(s, checkpoint=False), d)
    torch.cuda.synchronize()
    assert loss == ploss
    assert rel(dx, pdx) <= 2 * EIGHT
    for g, p in zip(grads, pgrads):
        for name in g:
            assert rel(g[name], p[name]) <= 2 * EIGHT, name
    assert len(ex.train(s, d, steps=3)) == 3
    out = ex.serve(s, d)
    assert out.shape == (3, s.H) and torch.isfinite(out).all()
