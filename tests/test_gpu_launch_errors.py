"""A call whose launch the runtime refuses reports it, and the next call of
the library does not report it again.  (The refusal is the host's: a launch on
the legacy stream while a blocking stream is being recorded.)"""
import ctypes

import pytest
import torch

import moe_expert_layer_topk_gb300 as m

pytestmark = pytest.mark.gpu


def runtime():
    for line in open("/proc/self/maps"):
        if "libcudart.so" in line:
            return ctypes.CDLL(line.split()[-1])
    pytest.skip("torch's CUDA runtime is not a shared library here")


def test_refused_launch_is_reported_once():
    T, K, N, r = 4, 64, 64, 8
    bf = dict(dtype=torch.bfloat16, device="cuda")
    x, W, A, B = torch.ones(T, K, **bf), torch.ones(N, K, **bf), torch.ones(1, r, K, **bf), torch.ones(1, N, r, **bf)
    off, wh = torch.tensor([0, T], dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    hid, y = torch.empty(m.moe_adapter_hidden_size(T, r), dtype=torch.uint8, device="cuda"), torch.empty(T, N, **bf)
    run = lambda stream=None: m.moe_adapter_linear(x, W, A, B, None, 1, off, wh, T, K, N, r, 1, hid, y, stream)  # noqa: E731
    run()
    n = 64
    v, out = torch.ones(n, device="cuda"), torch.empty(n, device="cuda")
    words = torch.zeros(2, dtype=torch.int64, device="cuda")
    m.moe_dropout(v, None, n, 0.0, words, out)
    torch.cuda.synchronize()
    rt = runtime()
    s, graph = ctypes.c_void_p(), ctypes.c_void_p()
    assert rt.cudaStreamCreate(ctypes.byref(s)) == 0
    assert rt.cudaStreamBeginCapture(s, 0) == 0
    try:
        with pytest.raises(m.MoEError) as e:
            run(0)
    finally:
        rt.cudaStreamEndCapture(s, ctypes.byref(graph))
        rt.cudaGetLastError()
        assert rt.cudaStreamDestroy(s) == 0
    assert "moe_adapter_linear" in str(e.value)
    m.moe_dropout(v, None, n, 0.0, words, out)  # a good call
    run()
    torch.cuda.synchronize()
    assert torch.equal(out, v) and torch.all(y == K + r * K)
