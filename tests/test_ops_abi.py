"""Host-side refusals of the balance-loss, dropout and adapter calls (no GPU)."""
import ctypes

import pytest

import moe_expert_layer_topk_gb300 as m
from moe_expert_layer_topk_gb300 import build as b

OK, INVALID, SHAPE, ALIGN, WS = 0, -1, -2, -3, -4
P = 0x10000  # never dereferenced: every call below fails host validation first


@pytest.fixture(scope="module")
def L():
    b.build()
    return m.lib()


def bal(L, T=16, E=8, k=2, S=1, off=None, logits=P, idx=P, counts=P, tokens=P, probs=P, loss=P, dl=P, ws=P, wsb=1 << 20):
    return L.moe_balance_loss(logits, idx, None, T, E, k, S, off, counts, tokens, probs, loss, 1.0, 1.0, dl, ws, wsb, None)


def test_balance(L):
    assert bal(L, T=-1) == INVALID and bal(L, E=0) == INVALID and bal(L, S=0) == INVALID
    assert bal(L, E=1025) == SHAPE and bal(L, k=9) == SHAPE and bal(L, E=64, k=33) == SHAPE
    assert bal(L, S=1025, off=P) == SHAPE
    assert bal(L, S=2) == INVALID and "seg_offsets" in L.moe_last_error_string().decode()
    for name in ("logits", "idx", "counts", "tokens", "probs", "loss", "ws"):
        assert bal(L, **{name: None}) == INVALID, name
    assert bal(L, logits=P + 4) == ALIGN and bal(L, dl=P + 8) == ALIGN and bal(L, ws=P + 8) == ALIGN
    assert bal(L, wsb=16) == WS and "workspace" in L.moe_last_error_string().decode()
    assert m.moe_balance_loss_workspace_size(8192, 128) > 0 and m.moe_balance_loss_workspace_size(-1, 8) == 0
    bwd = lambda **k: L.moe_balance_loss_bwd(*[k.get(n, d) for n, d in (("l", P), ("m", None), ("T", 16), ("E", 8), ("k", 2), ("S", 1),  # noqa: E731
                                             ("off", None), ("c", P), ("t", P), ("a", 1.0), ("b", 1.0), ("d", None), ("dl", P), ("s", None))])
    assert bwd(l=None) == INVALID and bwd(c=None) == INVALID and bwd(t=None) == INVALID and bwd(dl=None) == INVALID
    assert bwd(dl=P + 4) == ALIGN and bwd(E=2000) == SHAPE and bwd(T=0) == OK


def test_route_with_logits(L):
    def route(logits=P, chunk=P, E=8, k=2, wsb=1 << 20):
        return L.moe_route_topk_logits(P, P, None, 16, 128, E, k, 1, P, P, P, P, P, chunk, logits, P, wsb, None)
    assert route(logits=None) == INVALID and route(chunk=None) == INVALID and route(k=9) == SHAPE
    assert route(logits=P + 4) == ALIGN and route(wsb=8) == WS
    def back(dl=P, wsb=1 << 30, H=128):
        return L.moe_route_topk_logits_bwd(P, P, P, dl, P, P, P, 16, H, 8, 2, P, P, 0, P, wsb, None)
    assert back(dl=None) == INVALID and back(dl=P + 4) == ALIGN and back(H=100) == SHAPE and back(wsb=8) == WS
    assert "moe_route_topk_logits_bwd" in L.moe_last_error_string().decode()


def test_dropout(L):
    assert L.moe_dropout(P, P, -1, 0, 0.1, P, P, None) == INVALID
    assert L.moe_dropout(P, P, 8, 2, 0.1, P, P, None) == INVALID
    for p in (-0.1, 1.1, float("nan")):
        assert L.moe_dropout(P, P, 8, 0, p, P, P, None) == INVALID
        assert L.moe_combine_dropout(P, P, P, P, 4, 64, 2, p, P, P, None) == INVALID
        assert L.moe_combine_dropout_bwd(P, P, P, P, 4, 64, 2, p, P, P, P, None) == INVALID
    assert L.moe_dropout(P, P, 8, 0, 0.1, None, P, None) == INVALID
    assert L.moe_dropout(None, P, 8, 0, 0.1, P, P, None) == INVALID
    assert L.moe_dropout(P, P, 8, 0, 0.1, P, None, None) == INVALID
    assert L.moe_dropout(P + 2, None, 8, 0, 0.1, P, P, None) == ALIGN
    assert L.moe_dropout(P, P + 8, 8, 1, 0.1, P, P, None) == ALIGN
    assert L.moe_dropout(P, P, 8, 1, 0.1, P + 8, P, None) == ALIGN
    assert L.moe_dropout(P, P, 0, 0, 0.1, P, P, None) == OK
    assert L.moe_combine_dropout(P, P, P, None, 4, 100, 2, 0.1, P, P, None) == SHAPE
    assert L.moe_combine_dropout(P, P, P, None, 4, 64, 33, 0.1, P, P, None) == SHAPE
    assert L.moe_combine_dropout(P, None, P, None, 4, 64, 2, 0.1, P, P, None) == INVALID
    assert L.moe_combine_dropout(P, P, P, P + 8, 4, 64, 2, 0.1, P, P, None) == ALIGN
    assert L.moe_combine_dropout(P, P, P, None, 0, 64, 2, 0.1, P, P, None) == OK
    assert L.moe_combine_dropout_bwd(P, P, P, None, 4, 64, 2, 0.1, P, P, P, None) == INVALID
    assert L.moe_combine_dropout_bwd(P, P, P, P, 4, 64, 2, 0.1, P, P + 4, P, None) == ALIGN
    assert L.moe_combine_dropout_bwd(P, P, P, P, 0, 64, 2, 0.1, P, P, P, None) == OK


def fwd(L, T=16, K=64, N=64, r=8, nA=2, S=1, off=P, wh=P, ldx=64, ldy=64, x=P, W=P, A=P, B=P, hid=P, hb=1 << 20, y=P):
    return L.moe_adapter_linear(x, ldx, W, A, B, None, S, off, wh, T, K, N, r, nA, hid, hb, y, ldy, None)


def bwd(L, T=16, K=64, N=64, r=8, nA=2, S=1, off=P, wh=P, lddy=64, ldx=64, lddx=64, dy=P, x=P, W=P, A=P, B=P, hid=P,
        hb=1 << 20, dx=P, dA=P, dB=P, ws=P, wsb=1 << 24):
    return L.moe_adapter_linear_bwd(dy, lddy, x, ldx, W, A, B, None, hid, hb, S, off, wh, T, K, N, r, nA, dx, lddx, dA, dB,
                                    0, ws, wsb, None)


@pytest.mark.parametrize("call", [fwd, bwd])
def test_adapter(L, call):
    for kw in (dict(T=-1), dict(K=0), dict(N=-64), dict(r=0), dict(nA=0), dict(S=-1), dict(off=None), dict(wh=None)):
        assert call(L, **kw) == INVALID, kw
    for kw in (dict(K=96, ldx=96), dict(N=100, ldy=104) if call is fwd else dict(N=100, lddy=104), dict(r=12), dict(r=136),
               dict(nA=1025), dict(S=1025), dict(ldx=56), dict(ldx=68), dict(ldx=1 << 32)):
        assert call(L, **kw) == SHAPE, kw
    for name in ("x", "W", "A", "B", "hid") + (("y",) if call is fwd else ("dy", "dx", "dA", "dB", "ws")):
        assert call(L, **{name: None}) == INVALID, name
        assert call(L, **{name: P + 8}) == ALIGN, name
    assert call(L, hb=64) == WS and "hidden" in L.moe_last_error_string().decode()
    if call is fwd:
        assert fwd(L, ldy=32) == SHAPE and fwd(L, ldy=65) == SHAPE
        assert fwd(L, T=0) == OK
    else:
        assert bwd(L, lddx=56) == SHAPE and bwd(L, lddx=68) == SHAPE and bwd(L, lddy=8) == SHAPE
        assert bwd(L, wsb=128) == WS and "workspace" in L.moe_last_error_string().decode()


def test_adapter_sizes(L):
    assert m.moe_adapter_hidden_size(8192, 16) >= 8192 * 2 * 16 * 2
    assert m.moe_adapter_hidden_size(0, 16) > 0 and m.moe_adapter_hidden_size(4, 256) == 0
    assert m.moe_adapter_linear_bwd_workspace_size(8192, 2048, 2048, 16, 8) > 0
    assert m.moe_adapter_linear_bwd_workspace_size(-1, 2048, 2048, 16, 8) == 0
