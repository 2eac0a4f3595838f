"""The root-mean-square norm where mean + eps lies at the ends of fp32's range, in every call that
computes it, and its backward on such rows.

Bounds as in the norms' own tests: a bf16 result is off by half a step (2^-8 of its
value at most), an fp32 one by 2^-24, and sums by 2^-17 of their magnitudes; an rstd
below fp32's normal numbers (2^-126) by half a step of 2^-149.
"""
import numpy as np
import pytest
import torch

import block_ref as ref
import moe_expert_layer_topk_gb300 as m
from test_gpu_norm import near, np64

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
WIDTHS = [64, 128, 256, 512, 2048, 4096, 8192]


def e(*s, dt=F32):
    return torch.empty(*s, dtype=dt, device="cuda")


def rand(seed, *s):
    return torch.randn(*s, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda")


def f32(v):
    return float(np.float32(v))


def check(x, eps, dt):
    """Every call's norm of the rows x (as a residual stream of type dt, or as a block's bf16 output)."""
    T, H = x.shape
    xs, z = x.to(dt), x.to(BF)
    y, r = e(T, H, dt=BF), e(T)
    m.moe_pre_norm(xs, None, eps, T, H, y, r)
    want, wr = ref.pre_norm(np64(xs), 1.0, f32(eps))
    near(r, wr, wr, "rstd")
    near(y, want, np.abs(want), "y")
    out, ny = e(T, H, dt=dt), e(T, H, dt=BF)
    m.moe_post_norm(z, None, None, 1, eps, None, 0.0, 1.0, T, H, out, r)
    w = ref.post_norm(np64(z), None, 1.0, 1, f32(eps), None, 0.0, 1.0)
    near(r, w["rstd"], w["rstd"], "post rstd")
    near(out, w["out"], w["out_mag"], "post out")
    one, slot = torch.ones(T, 1, device="cuda"), torch.arange(T, dtype=torch.int32, device="cuda").view(T, 1)
    m.moe_combine_post_norm(z, one, slot, None, None, 1, eps, None, 0.0, 1.0, T, H, 1, None, out, r)
    near(r, w["rstd"], w["rstd"], "combine rstd")
    near(out, w["out"], w["out_mag"], "combine out")
    m.moe_post_norm(z, xs, None, 0, eps, None, 1.0, 0.0, T, H, out, None, None, ny, r)  # the next norm, of the residual
    near(r, wr, wr, "next_rstd")
    near(ny, want, np.abs(want), "next_y")


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("H", WIDTHS)
def test_eps_beside_squares_beyond_the_range(H, dt):
    """eps counts beside a row whose squares' sum leaves fp32's range, and so does a mean whose sum with eps does."""
    x = rand(H, 9, H)
    x[1] *= 1e19
    x[3] *= 1e18
    x[5] *= 1e30
    check(x, 1e38, dt)
    y = rand(H + 1, 9, H)
    y[1] *= 6e18  # mean 3.6e37: beyond the range with eps only
    y[3] *= 1e17
    check(y, 3.4e38, dt)


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("H", WIDTHS)
def test_squares_below_the_range(H, dt):
    """Rows whose squares are below fp32's normal numbers, beside an eps that is no larger; the other rows of a
    warp keep theirs."""
    for eps in (1e-45, 1e-42, 1e-38, 1e-30):
        x = rand(H + 3, 37, H)
        for t, size in ((1, 1e-22), (3, 1e-20), (4, 1e-19), (6, 1e-15), (7, 1e-13), (9, 1e-30), (10, 3e-23)):
            x[t] *= size
        x[12] = 0
        x[20:] *= 1e-21
        check(x, eps, dt)


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("H", WIDTHS)
def test_backward_of_rows_beyond_the_range(H, dt):
    """With the rstd that the forward leaves for rows whose squares overflow; the gain's gradient takes those rows too."""
    T, eps = 24, 1e-5
    x = rand(H, T, H)
    x[5] *= 1e30
    x[7] = 3.0e38
    x[8] = -1.0e38
    x[9] *= 1e19
    x, dy, gain = x.to(dt), rand(H + 1, T, H).to(BF), 1 + 0.3 * rand(H + 2, H)
    y, r, dx, dg = e(T, H, dt=BF), e(T), e(T, H, dt=dt), e(H)
    m.moe_pre_norm(x, gain, eps, T, H, y, r)
    wr = ref.rstd(np64(x), eps)
    near(r, wr, wr + 2.0 ** -133, "rstd")
    ws = torch.empty(m.moe_pre_norm_bwd_workspace_size(T, H), dtype=torch.uint8, device="cuda")
    m.moe_pre_norm_bwd(dy, x, gain, r, None, 0.0, T, H, dx, dg, 0, ws)
    b = ref.pre_norm_bwd(np64(dy), np64(x), np64(gain), np64(r), None, 0)
    near(dx, b["dx"], b["dx_mag"], "dx")
    near(dg, b["dgain"], b["dgain_mag"], "dgain", 2.0 ** -15)
    z = x.to(BF)
    z[7] = 1.0e38
    m.moe_post_norm(z, None, gain, 1, eps, None, 0.0, 1.0, T, H, dx, r)
    dz, dout = e(T, H, dt=BF), dy.to(dt)
    m.moe_post_norm_bwd(dout, z, gain, 1, r, None, 1.0, T, H, dz, dg, None, 0, ws)
    b = ref.post_norm_bwd(np64(dout), np64(z), np64(gain), 1, np64(r), None, 1.0)
    near(dz, b["dz"], b["dz_mag"], "dz")
    near(dg, b["dgain"], b["dgain_mag"], "post dgain", 2.0 ** -15)
