"""Calls of the norms and of the 8-bit activations that could not be answered as defined, refused on
the host (no GPU)."""
import pytest
import torch

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


# ------------------------------------------------------- types, in the binding

BF, F32, I8, I32 = torch.bfloat16, torch.float32, torch.int8, torch.int32
T, H, I, E, k = 4, 64, 64, 2, 2


class OnGpu:
    """What the binding asks of a tensor, without one on a GPU."""
    is_cuda = True

    def __init__(self, dtype, *shape):
        self.t = torch.empty(*shape, dtype=dtype)
        self.dtype, self.shape = dtype, self.t.shape

    def is_contiguous(self):
        return True

    def __getattr__(self, name):
        return getattr(self.t, name)


def bf(*s):
    return OnGpu(BF, *s)


def f32(*s):
    return OnGpu(F32, *s)


CALLS = {
    "moe_pre_norm": (dict(x=bf(T, H), gain=f32(H), eps=1e-6, T=T, H=H, y=bf(T, H), rstd=f32(T)), ["y", "rstd", "gain"]),
    "moe_pre_norm_bwd": (dict(dy=bf(T, H), x=f32(T, H), gain=f32(H), rstd=f32(T), dres=f32(T, H), res_scale=1.0, T=T, H=H, dx=f32(T, H),
                              dgain=f32(H)), ["dy", "rstd", "dres", "dx", "gain", "dgain"]),
    "moe_post_norm": (dict(z=bf(T, H), residual=f32(T, H), gain=f32(H), norm=1, eps=1e-6, gate=f32(T), res_scale=1.0, out_scale=1.0, T=T,
                           H=H, out=f32(T, H), rstd=f32(T), next_gain=f32(H), next_y=bf(T, H), next_rstd=f32(T)),
                      ["z", "residual", "out", "rstd", "next_gain", "next_y", "next_rstd"]),
    "moe_combine_post_norm": (dict(y_perm=bf(T * k, H), topk_w=f32(T, k), row_of_slot=OnGpu(I32, T, k), residual=bf(T, H), gain=f32(H),
                                   norm=1, eps=1e-6, gate=bf(T, H), res_scale=1.0, out_scale=1.0, T=T, H=H, k=k, z=bf(T, H), out=bf(T, H),
                                   rstd=f32(T), next_gain=f32(H), next_y=bf(T, H), next_rstd=f32(T)),
                              ["y_perm", "topk_w", "residual", "z", "out", "rstd", "next_y", "next_rstd"]),
    "moe_post_norm_bwd": (dict(dout=f32(T, H), z=bf(T, H), gain=f32(H), norm=1, rstd=f32(T), gate=f32(T), out_scale=1.0, T=T, H=H,
                               dz=bf(T, H), dgain=f32(H), dgate=f32(T)), ["z", "rstd", "dz", "dgain", "dgate"]),
    "moe_ckpt_pack": (dict(a=bf(T, H), rows=T, cols=H, q=OnGpu(I8, T, H), scale=bf(T, 2)), ["a", "q", "scale"]),
    "moe_ckpt_unpack": (dict(q=OnGpu(I8, T, H), scale=bf(T, 2), rows=T, cols=H, a=bf(T, H)), ["a", "q", "scale"]),
    "moe_dispatch_rows": (dict(x=OnGpu(I8, T, H), scale=bf(T, 2), row_of_slot=OnGpu(I32, T, k), topk_w=f32(T, k), T=T, H=H, k=k,
                               x_perm=bf(T * k, H), row_w=f32(T * k)), ["x", "scale", "topk_w", "x_perm", "row_w"]),
    "moe_grouped_gemm_swiglu_ckpt": (dict(x_perm=bf(T, H), Wg=bf(E, I, H), Wu=bf(E, I, H), num_seg=E, seg_offsets=OnGpu(I32, E + 1),
                                          seg_expert=None, R=T, H=H, I=I, E=E, h=bf(T, I), gu_q=OnGpu(I8, T, 2 * I), gu_scale=bf(T, 4)),
                                     ["x_perm", "Wg", "Wu", "h", "gu_q", "gu_scale"]),
    "moe_grouped_gemm_down_bwd_ckpt": (dict(dy_perm=bf(T, H), row_w=f32(T), gu_q=OnGpu(I8, T, 2 * I), gu_scale=bf(T, 4), Wd=bf(E, H, I),
                                            num_seg=E, seg_offsets=OnGpu(I32, E + 1), seg_expert=None, R=T, H=H, I=I, E=E,
                                            dgu=bf(T, 2 * I), h_w=bf(T, I), d_w=f32(T)),
                                       ["dy_perm", "row_w", "gu_q", "gu_scale", "Wd", "dgu", "h_w", "d_w"]),
}


@pytest.mark.parametrize("name", CALLS)
def test_a_tensor_of_another_type_is_refused(name, monkeypatch):
    """bf16 where fp32 is read and the other way round: refused before the call is made."""
    args, typed = CALLS[name]
    made = []
    monkeypatch.setattr(m, "_call", lambda fn, *a: made.append((fn, len(a))))
    f = getattr(m, name)
    f(**args, stream=0)
    assert made == [(name, len(m.ENTRY_POINTS[name][0]))]
    for arg in typed:
        t = args[arg]
        for other in (BF, F32, torch.float16):
            if other is not t.dtype:
                with pytest.raises(ValueError):
                    f(**{**args, arg: OnGpu(other, *t.shape)}, stream=0)
                    pytest.fail(f"{arg} as {other}")
    assert len(made) == 1
    addresses = {n: P for n in ("rstd", "row_w", "d_w", "z") if n in args}
    f(**{**args, **addresses}, stream=0)  # addresses are taken as they are
    assert len(made) == 2


def test_tokens_of_another_type():
    with pytest.raises(ValueError, match="bf16 tokens"):
        m.moe_dispatch_rows(OnGpu(torch.float16, T, H), None, None, None, T, H, k, bf(T * k, H))
