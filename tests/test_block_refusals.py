"""Calls of the norms and of the 8-bit activations that could not be answered as defined, refused on
the host (no GPU)."""
import pytest

import moe_expert_layer_topk_gb300 as m
from moe_expert_layer_topk_gb300 import build as b

OK, INVALID, ALIGN = 0, -1, -3
P = 0x10000  # never dereferenced: every call below fails host validation first


@pytest.fixture(scope="module")
def L():
    b.build()
    return m.lib()


def test_dx_over_dres_with_another_row_stride(L):
    """A row of dx would be written over rows of dres that are still to be read."""
    d = dict(dy=P, lddy=64, x=P, ldx=64, fp32=0, gain=P, rstd=P, dres=P, lddres=64, a=1.0, T=4, H=64, dx=P, lddx=64, dgain=P, acc=0, ws=P,
             wsb=1 << 20, s=None)
    call = lambda **k: L.moe_pre_norm_bwd(*{**d, **k}.values())  # noqa: E731
    for k in (dict(lddx=72), dict(lddres=128), dict(fp32=1, lddx=68)):
        assert call(**k) == INVALID and "row stride" in L.moe_last_error_string().decode(), k
    # the same stride, one row, or another tensor: the check that follows is the one that fails
    for k in (dict(lddx=72, lddres=72), dict(T=1, lddx=72), dict(lddx=72, dres=2 * P)):
        assert call(gain=P + 4, **k) == ALIGN, k
