"""The layer's options through its own calls: recorded as a graph."""
import pytest
import torch

import moe_expert_layer_topk_gb300 as m
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
