"""The layer's options through its own calls: recorded as a graph, on another
stream, with an upstream gradient of the router losses."""
import pytest
import torch

import moe_expert_layer_topk_gb300 as m
import ops_ref
from gpu_util import inputs, to_dev

pytestmark = pytest.mark.gpu

T, H, I, E, k = 150, 128, 64, 8, 2
OFF = [0, 60, 60, 140]


def parts(seed=31):
    g = to_dev(inputs(T, H, I, E, k, seed=seed))
    res = torch.randn(T, H, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    return dict(residual=res, mask=(torch.arange(T) % 7 != 3).to(torch.uint8).cuda(),
                seg_offsets=torch.tensor(OFF, dtype=torch.int32).cuda()), g


def weights(g):
    return g["Wr"], None, g["Wg"], g["Wu"], g["Wd"]


def layer(seed=99, dropout=0.25):
    return m.MoELayer(T, H, I, E, k, balance_coef=0.5, z_coef=0.02, sequences=3, dropout=dropout, seed=seed)


def test_graph_records_the_options():
    opts, g = parts()
    L, M = layer(), layer()
    graph = L.capture_forward(g["x"], *weights(g), **opts)
    seen = []
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        want = M.forward(g["x"], *weights(g), **opts)
        assert torch.equal(L.y, want)
        for name in ("loss", "dlogits", "seq_counts", "seq_tokens", "prob_sum"):
            assert torch.equal(getattr(L, name), getattr(M, name)), name
        seen.append(L.y.clone())
        L.advance_rng()
        M.advance_rng()
    assert not torch.equal(seen[0], seen[1]) and not torch.equal(seen[1], seen[2])
    # what the recorded tensors hold at a replay is what counts
    opts["residual"].zero_()
    opts["mask"].fill_(1)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(L.y, M.forward(g["x"], *weights(g), **opts)) and torch.equal(L.loss, M.loss)


def test_graph_of_a_residual_without_dropout():
    opts, g = parts()
    L, M = m.MoELayer(T, H, I, E, k), m.MoELayer(T, H, I, E, k)
    graph = L.capture_forward(g["x"], *weights(g), residual=opts["residual"])
    L.y.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(L.y, M.forward(g["x"], *weights(g), residual=opts["residual"]))


def test_advance_rng_without_dropout_is_nothing():
    _, g = parts()
    L = m.MoELayer(T, H, I, E, k, balance_coef=0.5)
    L.advance_rng()
    y = L.forward(g["x"], *weights(g)).clone()
    L.advance_rng()
    assert torch.equal(y, L.forward(g["x"], *weights(g)))


@pytest.mark.parametrize("raw", [False, True])
def test_advance_rng_on_the_calls_stream(raw):
    """Ordered after the work of that stream, not of the current one: a forward
    that a long kernel holds up still takes the words it was given."""
    opts, g = parts()
    L = layer()
    want0 = torch.from_numpy(ops_ref.keep(99, 0, 0, T * H, 0.25).reshape(T, H)).cuda()
    want1 = torch.from_numpy(ops_ref.keep(99, T * H // 8, 0, T * H, 0.25).reshape(T, H)).cuda()
    opts["residual"].zero_()
    L.forward(g["x"], *weights(g), **opts)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    big = torch.randn(4096, 4096, device="cuda")
    out = torch.empty_like(big)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        for _ in range(20):
            torch.mm(big, big, out=out)
    handle = s.cuda_stream if raw else s
    y0, y1 = torch.empty_like(L.y), torch.empty_like(L.y)
    L.forward(g["x"], *weights(g), handle, y0, **opts)
    L.advance_rng(handle)
    L.forward(g["x"], *weights(g), handle, y1, **opts)
    s.synchronize()
    assert not y0[~want0].any() and not y1[~want1].any()
    assert y0[want0].ne(0).float().mean() > 0.9 and y1[want1].ne(0).float().mean() > 0.9
    assert L.rng.tolist() == [99, T * H // 8]


@pytest.mark.parametrize("overlap", [False, True])
def test_upstream_gradient_of_the_router_losses(overlap):
    """dloss scales the two losses' parts of the gradient: the backward with it
    is the one of a layer whose coefficients are the products.  The scales are
    powers of two, so the gradients are the same to the bit."""
    opts, g = parts()
    up = torch.tensor([4.0, 0.125], device="cuda")
    L = layer()
    M = m.MoELayer(T, H, I, E, k, balance_coef=2.0, z_coef=0.0025, sequences=3, dropout=0.25, seed=99)
    args = (g["dy"], g["x"], g["Wr"], g["Wg"], g["Wu"], g["Wd"])
    for lay in (L, M):
        lay.forward(g["x"], *weights(g), **opts)
    L.backward(*args, overlap=overlap, dloss=up)
    M.backward(*args, overlap=overlap)
    torch.cuda.synchronize()
    assert torch.equal(L.dlogits, M.dlogits) and torch.equal(L.dx, M.dx) and torch.equal(L.dWr, M.dWr)
    assert torch.equal(L.dWg, M.dWg)
    # without it: the forward's own coefficients, after a backward with it as well
    ref = layer()
    ref.forward(g["x"], *weights(g), **opts)
    ref.backward(*args, overlap=overlap)
    for again in (False, True):
        if again:
            L.backward(*args, overlap=overlap, dloss=up)
            L.forward(g["x"], *weights(g), **opts)
        L.backward(*args, overlap=overlap)
        torch.cuda.synchronize()
        assert torch.equal(L.dx, ref.dx) and torch.equal(L.dWr, ref.dWr) and not torch.equal(L.dWr, M.dWr)
    assert m.moe_read_device_status(reset=True) == 0


def test_upstream_gradient_needs_the_losses():
    _, g = parts()
    L = m.MoELayer(T, H, I, E, k)
    L.forward(g["x"], *weights(g))
    with pytest.raises(ValueError):
        L.backward(g["dy"], g["x"], g["Wr"], g["Wg"], g["Wu"], g["Wd"], dloss=torch.ones(2, device="cuda"))
