"""The layer's training options (router losses, residual dropout) and the
adapters together: against float64 autograd, and the example end to end."""
import importlib.util
from pathlib import Path

import numpy as np
import pytest
import torch

import moe_expert_layer_topk_gb300 as m
import ops_ref
from gpu_util import assert_close, inputs, to_dev

ROOT = Path(__file__).resolve().parents[1]


def example():
    spec = importlib.util.spec_from_file_location("finetune_block", ROOT / "examples" / "finetune_block.py")
    mod = importlib.util.module_from_spec(spec)
    import sys
    sys.modules["finetune_block"] = mod
    spec.loader.exec_module(mod)
    return mod


def test_options_of_a_forward_only_layer_are_refused():
    for kw in (dict(balance_coef=0.1), dict(z_coef=0.1), dict(dropout=0.1)):
        with pytest.raises(ValueError):
            m.MoELayer(8, 64, 64, 4, 2, training=False, **kw)


@pytest.mark.gpu
@pytest.mark.parametrize("dropout", [0.0, 0.25])
@pytest.mark.parametrize("packed", [False, True])
def test_layer_against_autograd(dropout, packed):
    """y, dX, dWr and the losses of the whole layer against float64 autograd of
    the written-out layer with the routing held; the layer's acceptance bars
    (bf16 intermediates) hold."""
    T, H, I, E, k = 150, 128, 64, 8, 2
    a, b, p = 0.5, 0.02, dropout
    inp = inputs(T, H, I, E, k, seed=31)
    g = to_dev(inp)
    seqs = 3 if packed else 1
    off = [0, 60, 60, 140] if packed else [0, T]
    mask = (torch.arange(T) % 7 != 3).to(torch.uint8) if packed else None
    res = torch.randn(T, H, generator=torch.Generator().manual_seed(1)).bfloat16()
    L = m.MoELayer(T, H, I, E, k, balance_coef=a, z_coef=b, sequences=seqs, dropout=p, seed=99)
    y = L.forward(g["x"], g["Wr"], None, g["Wg"], g["Wu"], g["Wd"], residual=res.cuda(),
                  mask=None if mask is None else mask.cuda(),
                  seg_offsets=torch.tensor(off, dtype=torch.int32).cuda() if packed else None)
    L.backward(g["dy"], g["x"], g["Wr"], g["Wg"], g["Wu"], g["Wd"])
    torch.cuda.synchronize()
    assert m.moe_read_device_status(reset=True) == 0

    d = lambda n: inp[n].double()  # noqa: E731
    x, Wr = d("x").requires_grad_(), d("Wr").requires_grad_()
    idx = L.topk_idx.cpu().long()
    logits = x @ Wr
    w = torch.softmax(logits.gather(1, idx), 1)
    out = torch.zeros(T, H, dtype=torch.float64)
    for j in range(k):
        e = idx[:, j]
        gg, uu = torch.einsum("th,tih->ti", x, d("Wg")[e]), torch.einsum("th,tih->ti", x, d("Wu")[e])
        out = out + w[:, j:j + 1] * torch.einsum("ti,thi->th", torch.nn.functional.silu(gg) * uu, d("Wd")[e])
    keep = torch.from_numpy(ops_ref.keep(99, 0, 0, T * H, p).reshape(T, H)) if p else torch.ones(T, H, dtype=torch.bool)
    yr = res.double() + out * keep * ops_ref.factor(p)
    on = torch.ones(T, dtype=torch.bool) if mask is None else mask.bool()
    prob, lse = torch.softmax(logits, 1), torch.logsumexp(logits, 1)
    n = sum(int(on[s:e].sum()) for s, e in zip(off, off[1:]))
    bal = z = 0
    for s, e in zip(off, off[1:]):
        r = torch.arange(s, e)[on[s:e]]
        if len(r):
            c = torch.bincount(idx[r].reshape(-1), minlength=E).double()
            bal = bal + E / (k * len(r) * n) * (c * prob[r].sum(0)).sum()
            z = z + lse[r].square().sum() / n
    ((yr * d("dy")).sum() + a * bal + b * z).backward()
    assert_close(y, yr.detach().numpy(), "y")
    assert_close(L.dx, x.grad.numpy(), "dx")
    assert_close(L.dWr, Wr.grad.numpy(), "dWr")
    np.testing.assert_allclose(L.loss.cpu().numpy(), [float(bal.detach()), float(z.detach())], rtol=1e-4)


@pytest.mark.gpu
def test_without_options_the_layer_is_what_it_was():
    """The options off: the same bits as the layer's calls written out."""
    T, H, I, E, k = 200, 128, 64, 8, 2
    g = to_dev(inputs(T, H, I, E, k, seed=5))
    L, M = m.MoELayer(T, H, I, E, k), m.MoELayer(T, H, I, E, k, balance_coef=0.1)
    y = L.forward(g["x"], g["Wr"], None, g["Wg"], g["Wu"], g["Wd"])
    assert torch.equal(y, M.forward(g["x"], g["Wr"], None, g["Wg"], g["Wu"], g["Wd"]))
    zero = torch.zeros_like(y)
    assert torch.equal(y, L.forward(g["x"], g["Wr"], None, g["Wg"], g["Wu"], g["Wd"], residual=zero).clone())
    L.backward(g["dy"], g["x"], g["Wr"], g["Wg"], g["Wu"], g["Wd"])
    M.dlogits.zero_()
    M.backward(g["dy"], g["x"], g["Wr"], g["Wg"], g["Wu"], g["Wd"])
    assert torch.equal(L.dx, M.dx) and torch.equal(L.dWr, M.dWr) and torch.equal(L.dWg, M.dWg)


@pytest.mark.gpu
def test_advance_rng_changes_the_mask_and_a_replay_repeats_it():
    T, H, I, E, k = 64, 64, 64, 4, 2
    g = to_dev(inputs(T, H, I, E, k, seed=6))
    L = m.MoELayer(T, H, I, E, k, dropout=0.5, seed=3)
    run = lambda: L.forward(g["x"], g["Wr"], None, g["Wg"], g["Wu"], g["Wd"]).clone()  # noqa: E731
    first = run()
    assert torch.equal(first, run())
    L.advance_rng()
    second = run()
    assert not torch.equal(first, second)
    want = ops_ref.keep(3, T * H // 8, 0, T * H, 0.5).reshape(T, H)
    assert not second.cpu()[torch.from_numpy(~want)].any()


@pytest.mark.gpu
def test_example_trains_and_serves():
    ex = example()
    s = ex.Sizes(lengths=(90, 1, 47, 130), H=128, I=64, E=8, k=2, r=8, num_adapters=3)
    d = ex.make(s)
    untouched = d["A"].clone(), d["B"].clone()
    seen = ex.finetune(s, d, steps=12)
    assert np.all(np.isfinite(seen))
    assert seen[-1][0] < 0.97 * seen[0][0]              # the fit improves
    assert not torch.equal(d["A"], untouched[0]) and not torch.equal(d["B"], untouched[1])
    y = ex.serve(s, d)
    assert y.shape == (6, s.H) and torch.isfinite(y.float()).all()
