"""A stream given as its handle (an int, as the entry points take it) where the layer also needs torch's
events and its own operations on it."""
import pytest
import torch

import moe_expert_layer_topk_gb300 as m
from gpu_util import inputs, to_dev
from moe_expert_layer_topk_gb300.layer import _stream_of

T, H, I, E, k = 150, 128, 64, 8, 2


@pytest.mark.gpu
def test_stream_of():
    s = torch.cuda.Stream()
    dev = s.device
    assert _stream_of(s, dev) is s
    assert _stream_of(s.cuda_stream, dev).cuda_stream == s.cuda_stream
    assert _stream_of(0, dev) == torch.cuda.default_stream(dev)
    with torch.cuda.stream(s):
        assert _stream_of(None, dev) == s


@pytest.mark.gpu
@pytest.mark.parametrize("checkpoint", [False, True])
@pytest.mark.parametrize("which", ["side", "default"])
def test_backward_on_a_handle(which, checkpoint):
    """The backward on two streams, of which the caller names one by its handle."""
    d = to_dev(inputs(T, H, I, E, k, seed=4))
    w = (d["Wr"], None, d["Wg"], d["Wu"], d["Wd"])
    back = (d["dy"], d["x"], d["Wr"], d["Wg"], d["Wu"], d["Wd"])
    P, L = (m.MoELayer(T, H, I, E, k, checkpoint=checkpoint) for _ in range(2))
    y = P.forward(d["x"], *w)
    dx = P.backward(*back)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    handle = s.cuda_stream if which == "side" else 0
    got = L.forward(d["x"], *w, stream=handle)
    gdx = L.backward(*back, stream=handle)
    torch.cuda.synchronize()
    assert m.moe_read_device_status(reset=True) == 0
    assert torch.equal(got, y) and torch.equal(gdx, dx)
    for n in ("dWg", "dWu", "dWd", "dWr"):
        assert torch.equal(getattr(L, n), getattr(P, n)), n
