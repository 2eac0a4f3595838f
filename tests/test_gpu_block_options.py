"""The layer's options inside a block: rows gathered by the product, e4m3 products, and the router losses,
against the entry points called one after another and against the plain block."""
import pytest
import torch

import moe_expert_layer_topk_gb300 as m
from gpu_util import inputs, to_dev

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
T, H, I, E, k = 150, 128, 128, 8, 2  # (e4m3 products take I in steps of 128)
EPS, A, B = 1e-5, 0.9, 0.6


def parts(seed=21):
    d = to_dev(inputs(T, H, I, E, k, seed=seed))
    g = torch.Generator(device="cuda").manual_seed(seed)
    for n in ("Wg", "Wu", "Wd"):
        d[n] = (d[n].float() * 5).to(BF)
    d["pre"], d["post"], d["next"] = (1 + 0.2 * torch.randn(H, generator=g, device="cuda") for _ in range(3))
    d["gate"] = torch.randn(T, generator=g, device="cuda")
    d["x"], d["dy"] = d["x"].float(), d["dy"].float()
    return d


def block(**options):
    return m.MoEBlock(T, H, I, E, k, gate="token", eps=EPS, res_scale=A, out_scale=B, fp32=True, **options)


def e(*s, dt=F32):
    return torch.empty(*s, dtype=dt, device="cuda")


def rel(a, b):
    a, b = a.double(), b.double()
    return ((a - b).norm() / b.norm()).item()


def by_hand(d, L, weights, next_gain):
    """The block's forward through the entry points and a layer of its own."""
    n, r, out, ny, nr = e(T, H, dt=BF), e(T), e(T, H), e(T, H, dt=BF), e(T)
    m.moe_pre_norm(d["x"], d["pre"], EPS, T, H, n, r)
    L.forward(n, d["Wr"], None, *weights)
    m.moe_combine_post_norm(L.y_perm, L.topk_w, L.row_of_slot, d["x"], d["post"], 1, EPS, d["gate"], A, B, T, H, k, None, out, None, next_gain,
                            ny, nr)
    return out, ny, nr


@pytest.mark.parametrize("option", ["plain", "fused_dispatch", "fp8"])
def test_serving(option):
    d = parts()
    opts = {} if option == "plain" else {option: True}
    L = m.MoELayer(T, H, I, E, k, training=False, **opts)
    w = (L.quantize_weights(d["Wg"], d["Wu"], d["Wd"]), None, None) if option == "fp8" else (d["Wg"], d["Wu"], d["Wd"])
    blk = block(training=False, next_norm=True, **opts)
    rest = (d["pre"], d["post"], d["Wr"], None, *w, d["gate"])
    out = blk.forward(d["x"], *rest, next_gain=d["next"]).clone()
    n, r = (t.clone() for t in blk.next_normed)
    want, ny, nr = by_hand(d, L, w, d["next"])
    assert torch.equal(out, want) and torch.equal(n, ny) and torch.equal(r, nr)
    # the plain block's branch: the same to a bf16 rounding or two of its rows for gathered rows; e4m3 operands are
    # off by 2^-4/sqrt(3) = 3.6% of a value at most (rms), x and W of g and u, h (of both) and Wd: sqrt(2 * 2 + 2) 3.6% = 8.8%
    plain = block(training=False).forward(d["x"], d["pre"], d["post"], d["Wr"], None, d["Wg"], d["Wu"], d["Wd"], d["gate"])
    bar = {"plain": 0.0, "fused_dispatch": 2.0 ** -8, "fp8": 0.088}[option]
    assert rel(out - A * d["x"], plain - A * d["x"]) <= bar
    # the next block takes what this one left, in place of its own norm
    nxt = block(training=False, **opts)
    rest = (d["next"], d["post"], d["Wr"], None, *w, d["gate"])
    a = nxt.forward(out, *rest, normed=blk.next_normed).clone()
    assert rel(a, nxt.forward(out, *rest)) <= (2.0 ** -8 if option != "fp8" else 0.02)
    torch.cuda.synchronize()
    assert m.moe_read_device_status(reset=True) == 0


@pytest.mark.parametrize("checkpoint", [False, True])
@pytest.mark.parametrize("upstream", [False, True])
def test_router_losses(checkpoint, upstream):
    """Losses of masked sequences: their values, and the gradients with them, are the layer's on the normed input."""
    d = parts()
    opts = dict(balance_coef=0.5, z_coef=0.02, sequences=3, checkpoint=checkpoint)
    mask = (torch.arange(T, device="cuda") % 7 != 3).to(torch.uint8)
    seg = torch.tensor([0, 60, 60, 140], dtype=torch.int32, device="cuda")
    dloss = torch.tensor([2.0, 0.5], device="cuda") if upstream else None
    w = (d["Wg"], d["Wu"], d["Wd"])
    blk = block(**opts)
    out = blk.forward(d["x"], d["pre"], d["post"], d["Wr"], None, *w, d["gate"], mask=mask, seg_offsets=seg)
    dx = blk.backward(d["dy"], d["x"], d["pre"], d["post"], d["Wr"], *w, d["gate"], dloss=dloss)
    L = m.MoELayer(T, H, I, E, k, **opts)
    n, r, want, z, pr = e(T, H, dt=BF), e(T), e(T, H), e(T, H, dt=BF), e(T)
    m.moe_pre_norm(d["x"], d["pre"], EPS, T, H, n, r)
    L.forward(n, d["Wr"], None, *w, mask=mask, seg_offsets=seg)
    m.moe_combine_post_norm(L.y_perm, L.topk_w, L.row_of_slot, d["x"], d["post"], 1, EPS, d["gate"], A, B, T, H, k, z, want, pr)
    assert torch.equal(out, want) and torch.equal(blk.layer.loss, L.loss) and (L.loss > 0).all()
    ws = torch.empty(max(m.moe_post_norm_bwd_workspace_size(T, H), m.moe_pre_norm_bwd_workspace_size(T, H)), dtype=torch.uint8, device="cuda")
    dz, dpost, dgate, wdx, dpre = e(T, H, dt=BF), e(H), e(T), e(T, H), e(H)
    m.moe_post_norm_bwd(d["dy"], z, d["post"], 1, pr, d["gate"], B, T, H, dz, dpost, dgate, 0, ws)
    dn = L.backward(dz, n, d["Wr"], *w, dloss=dloss)
    m.moe_pre_norm_bwd(dn, d["x"], d["pre"], r, d["dy"], A, T, H, wdx, dpre, 0, ws)
    torch.cuda.synchronize()
    assert m.moe_read_device_status(reset=True) == 0
    assert torch.equal(dx, wdx) and torch.equal(blk.d_pre_gain, dpre) and torch.equal(blk.d_post_gain, dpost) and torch.equal(blk.d_gate, dgate)
    for name in ("dWr", "dWg", "dWu", "dWd"):
        assert torch.equal(getattr(blk.layer, name), getattr(L, name)), name
    # and they do count
    bare = block(checkpoint=checkpoint)
    bare.forward(d["x"], d["pre"], d["post"], d["Wr"], None, *w, d["gate"])
    bare.backward(d["dy"], d["x"], d["pre"], d["post"], d["Wr"], *w, d["gate"])
    assert not torch.equal(bare.layer.dWr, blk.layer.dWr)
