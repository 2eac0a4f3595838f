"""Host-side refusals of the norm and 8-bit activation calls (no GPU)."""
import math

import pytest
import torch

import moe_expert_layer_topk_gb300 as m
from moe_expert_layer_topk_gb300 import build as b

OK, INVALID, SHAPE, ALIGN, WS = 0, -1, -2, -3, -4
P = 0x10000  # never dereferenced: every call below fails host validation first


@pytest.fixture(scope="module")
def L():
    b.build()
    return m.lib()


def caller(f, **defaults):
    return lambda **k: f(*{**defaults, **k}.values()) if set(k) <= set(defaults) else pytest.fail(str(k))


def test_pre_norm(L):
    call = caller(L.moe_pre_norm, x=P, ldx=64, fp32=0, gain=P, eps=1e-6, T=4, H=64, y=P, ldy=64, rstd=P, s=None)
    assert call(T=-1) == INVALID and call(H=0) == INVALID and call(fp32=2) == INVALID and call(T=0) == OK
    assert call(H=60) == SHAPE and call(H=8200, ldx=8200, ldy=8200) == SHAPE
    for eps in (0.0, -1.0, math.nan, math.inf):
        assert call(eps=eps) == INVALID
    assert call(x=None) == INVALID and call(y=None) == INVALID
    assert call(ldx=56) == INVALID and call(ldx=68) == INVALID and call(ldy=0) == INVALID and call(fp32=1, ldx=66) == INVALID
    assert "strides" in L.moe_last_error_string().decode()
    assert call(x=P + 2) == ALIGN and call(gain=P + 4) == ALIGN and call(y=P + 8) == ALIGN


def test_pre_norm_bwd(L):
    call = caller(L.moe_pre_norm_bwd, dy=P, lddy=64, x=P, ldx=64, fp32=0, gain=P, rstd=P, dres=P, lddres=64, a=1.0, T=4, H=64, dx=P,
                  lddx=64, dgain=P, acc=0, ws=P, wsb=1 << 20, s=None)
    assert call(T=-1) == INVALID and call(H=12) == SHAPE and call(T=0, dgain=None) == OK and call(T=0, acc=1) == OK
    for name in ("dy", "x", "rstd", "dx"):
        assert call(**{name: None}) == INVALID, name
    for name in ("lddy", "ldx", "lddres", "lddx"):
        assert call(**{name: 32}) == INVALID, name
    for name in ("dy", "x", "dres", "dx", "gain", "ws", "dgain"):
        assert call(**{name: P + 4}) == ALIGN, name
    assert call(wsb=4 * 64 * 4 - 1) == WS and call(ws=None) == WS and "workspace" in L.moe_last_error_string().decode()
    assert m.moe_pre_norm_bwd_workspace_size(4, 64) == 4 * 64 * 4 and m.moe_pre_norm_bwd_workspace_size(-1, 64) == 0
    assert m.moe_pre_norm_bwd_workspace_size(1 << 30, 8192) < 1 << 28


def test_post_norm(L):
    d = dict(z=P, res=P, fp32=0, gain=P, norm=1, eps=1e-6, kind=1, gate=P, a=1.0, b=1.0, T=4, H=64, out=P, rstd=P, ng=P, ny=P, nr=P, s=None)
    call = caller(L.moe_post_norm, **d)
    comb = caller(L.moe_combine_post_norm, y=P, w=P, rows=P, res=P, fp32=0, gain=P, norm=1, eps=1e-6, kind=1, gate=P, a=1.0, b=1.0, T=4,
                  H=64, k=2, z=P, out=P, rstd=P, ng=P, ny=P, nr=P, s=None)
    for f in (call, comb):
        assert f(T=-1) == INVALID and f(fp32=-1) == INVALID and f(norm=2) == INVALID and f(kind=3) == INVALID and f(kind=-1) == INVALID
        assert f(eps=0.0) == INVALID and f(H=8256) == SHAPE and f(T=0) == OK
        assert f(out=None) == INVALID and f(gate=None) == INVALID
        assert f(ny=None) == INVALID and f(ny=None, ng=None) == INVALID
        for name in ("res", "gain", "out", "ng", "ny"):
            assert f(**{name: P + 4}) == ALIGN, name
        assert f(kind=2, gate=P + 4) == ALIGN and f(gate=P + 2) == ALIGN
    assert call(z=None) == INVALID and call(z=P + 8) == ALIGN and call(H=36) == SHAPE
    assert comb(y=None) == INVALID and comb(w=None) == INVALID and comb(rows=None) == INVALID and comb(y=P + 8) == ALIGN and comb(z=P + 8) == ALIGN
    assert comb(k=0) == INVALID and comb(k=33) == SHAPE and comb(H=72) == SHAPE and comb(T=1 << 28, k=8) == SHAPE
    bwd = caller(L.moe_post_norm_bwd, dout=P, fp32=0, z=P, gain=P, norm=1, rstd=P, kind=1, gate=P, b=1.0, T=4, H=64, dz=P, dgain=P, dgate=P,
                 acc=0, ws=P, wsb=1 << 20, s=None)
    assert bwd(T=-1) == INVALID and bwd(norm=3) == INVALID and bwd(kind=7) == INVALID and bwd(H=20) == SHAPE
    for name in ("dout", "z", "rstd", "gate", "dz"):
        assert bwd(**{name: None}) == INVALID, name
    for name in ("dout", "z", "gain", "dz", "ws", "dgain"):
        assert bwd(**{name: P + 4}) == ALIGN, name
    assert bwd(kind=0) == INVALID and "gate" in L.moe_last_error_string().decode()
    assert bwd(kind=2, dgate=P + 4) == ALIGN and bwd(wsb=8) == WS and bwd(T=0, acc=1) == OK


def test_rows_in_8_bits(L):
    for f in (L.moe_ckpt_pack, L.moe_ckpt_unpack):
        call = caller(f, a=P, b=P, r=4, c=64, d=P, s=None) if f is L.moe_ckpt_unpack else caller(f, a=P, r=4, c=64, b=P, d=P, s=None)
        assert call(r=-1) == INVALID and call(c=0) == INVALID and call(c=48) == SHAPE and call(r=0) == OK
        for name in ("a", "b", "d"):
            assert call(**{name: None}) == INVALID and call(**{name: P + 8}) == ALIGN, name
    call = caller(L.moe_dispatch_rows, x=P, scale=P, rows=P, w=P, T=4, H=64, k=2, xp=P, rw=P, s=None)
    assert call(T=-1) == INVALID and call(H=0) == INVALID and call(k=0) == INVALID and call(T=0) == OK
    assert call(H=96) == SHAPE and call(k=33) == SHAPE and call(T=1 << 28, k=8) == SHAPE
    assert call(x=None) == INVALID and call(rows=None) == INVALID and call(xp=None) == INVALID
    assert call(w=None) == INVALID and call(rw=None) == INVALID and "together" in L.moe_last_error_string().decode()
    assert call(x=P + 8) == ALIGN and call(scale=P + 2) == ALIGN and call(xp=P + 4) == ALIGN


def test_products(L):
    fwd = caller(L.moe_grouped_gemm_swiglu_ckpt, x=P, Wg=P, Wu=P, n=8, off=P, se=None, R=16, H=128, I=64, E=8, h=P, q=P, sc=P, s=None)
    bwd = caller(L.moe_grouped_gemm_down_bwd_ckpt, dy=P, rw=P, q=P, sc=P, Wd=P, n=8, off=P, se=None, R=16, H=128, I=64, E=8, dgu=P, h=P,
                 rows=P, T=8, k=2, dw=P, ws=P, wsb=1 << 20, s=None)
    for f in (fwd, bwd):
        assert f(R=-1) == INVALID and f(n=-1) == INVALID and f(off=None) == INVALID
        assert f(H=100) == SHAPE and f(I=96) == SHAPE and f(E=2000) == SHAPE and f(n=2000) == SHAPE
        for name in ("q", "sc", "h"):
            assert f(**{name: None}) == INVALID and f(**{name: P + 8}) == ALIGN, name
    assert fwd(R=0) == OK and fwd(n=0) == OK and bwd(R=0, T=0) == OK
    for name in ("x", "Wg", "Wu"):
        assert fwd(**{name: None}) == INVALID and fwd(**{name: P + 8}) == ALIGN, name
    for name in ("dy", "Wd", "dgu"):
        assert bwd(**{name: None}) == INVALID and bwd(**{name: P + 8}) == ALIGN, name
    assert bwd(dw=None) == INVALID and bwd(ws=None) == WS and bwd(wsb=16) == WS and bwd(ws=P + 8) == ALIGN
    assert bwd(T=9) == INVALID and bwd(k=0) == INVALID and bwd(T=-1) == INVALID and bwd(k=33, T=0) == INVALID
    assert m.moe_grouped_gemm_down_bwd_ckpt_workspace_size(16, 64) == 2 * 16 * 4
    assert m.moe_grouped_gemm_down_bwd_ckpt_workspace_size(65536, 768) == 6 * 65536 * 4
    assert m.moe_grouped_gemm_down_bwd_ckpt_workspace_size(-1, 64) == 0


def test_binding_types():
    z = lambda *s, dt=torch.bfloat16: torch.zeros(*s, dtype=dt)  # noqa: E731
    with pytest.raises(ValueError):
        m._stream_type(z(2, 8), z(2, 8, dt=torch.float32))
    with pytest.raises(ValueError):
        m._stream_type(z(2, 8, dt=torch.float16))
    assert m._stream_type(z(2, 8), None) == 0 and m._stream_type(z(2, 8, dt=torch.float32)) == 1
    assert m._gate_kind(None, 2, 8) == 0 and m._gate_kind(z(2, dt=torch.float32), 2, 8) == 1 and m._gate_kind(z(2, 8), 2, 8) == 2
    for bad in (z(2), z(3, dt=torch.float32), z(2, 8, dt=torch.float32)):
        with pytest.raises(ValueError):
            m._gate_kind(bad, 2, 8)
    with pytest.raises(ValueError):
        m.moe_dispatch_rows(z(2, 64), z(2, 2), None, None, 2, 64, 1, None)
    f, b, i8 = z(8, dt=torch.float32), z(2, 64), z(2, 64, dt=torch.int8)
    for call in (lambda: m._fp32(z(8)), lambda: m._codes(b, z(2, 2)), lambda: m._codes(i8, f),
                 lambda: m.moe_grouped_gemm_swiglu_ckpt(None, None, None, 1, None, None, 2, 64, 32, 1, None, i8, f)):
        with pytest.raises(ValueError, match="fp32|8-bit"):
            call()
