"""Adapters on the wide product's other tiles, and what its parts hold.

run_wide takes 64-, 128- or 256-column tiles (the last as CTA pairs on 256
rows, whose last wave may be halves) by the waves' cost; the shapes here reach
each of them in both directions on the GB300's 152 SMs, next to the clusters
and 64-column tiles of test_gpu_adapter.py.

Tolerances (derived before the first run) as there: 2^-14 of the terms'
magnitudes for fp32 sums, plus 2^-8 of itself for a bf16 result; where a test
states another, its comment derives it.
"""
import numpy as np
import pytest
import torch

import moe_expert_layer_topk_gb300 as m
import ops_ref
from test_gpu_adapter import backward, forward, make, near, requests

pytestmark = pytest.mark.gpu

# T, K, N, r, adapters, requests, extra columns of a row: tiles of y, of dx
SHAPES = [
    (2477, 2048, 1024, 16, 5, 9, 0),      # pairs, pairs with a wave of halves
    (3001, 1280, 2048, 48, 6, 40, 64),    # pairs with a wave of halves, pairs
    (1333, 1280, 1024, 128, 4, 21, 0),    # 128, 128
    (2301, 768, 768, 24, 3, 1000, 0),     # 128, 128, a run a row or two
    (3001, 1024, 2560, 128, 4, 13, 0),    # pairs, pairs; two blocks of ranks
    (2477, 2048, 2560, 32, 7, 700, 0),    # pairs with a wave of halves, both ways
]


def check(T, K, N, r, nA, pitch, offsets, which, seed):
    d, c = make(T, K, N, r, nA, seed=seed, dy=True, pitch=pitch)
    ref = ops_ref.adapter(*(d[k].double().numpy() for k in ("x", "W", "A", "B", "scale")), offsets, which, d["dy"].double().numpy())
    y, hid = forward(c, offsets, which, T, K, N, r, nA, pitch)
    near(y, ref, "y", True)
    dx, dA, dB = backward(c, hid, offsets, which, T, K, N, r, nA, pitch=pitch)
    near(dx, ref, "dx", True)
    near(dA, ref, "dA", False)
    near(dB, ref, "dB", False)
    assert m.moe_read_device_status(reset=True) == 0


@pytest.mark.parametrize("T,K,N,r,nA,n,pitch", SHAPES)
def test_tiles_of_every_width(T, K, N, r, nA, n, pitch):
    check(T, K, N, r, nA, pitch, *requests(T, n, nA, seed=n), seed=T + r)


def one_row_each(T, nA, lo, n):
    """Rows lo .. lo+n-1 a request each, adapters in turn, between two long requests."""
    return [0, *range(lo, lo + n + 1), T], [nA - 1, *(i % nA for i in range(n)), 0]


@pytest.mark.parametrize("T,K,N", [(3001, 1280, 2048), (1333, 1280, 1024), (300, 320, 192)])
def test_adapters_in_turn_row_by_row(T, K, N):
    """Across the border of a tile of 128 and of 256 rows, several runs a step."""
    check(T, K, N, 16, 3, 0, *one_row_each(T, 3, 90, 200), seed=T)


@pytest.mark.parametrize("T,K,N,r", [(3001, 1280, 2048, 16), (3001, 1280, 2048, 72), (1333, 1280, 1024, 16), (300, 320, 192, 16)])
def test_no_request_reaches_another_row_by_row(T, K, N, r):
    """Every third row, gradient row and the adapter they use hold NaN and
    infinities: the rows between them keep their bits."""
    nA = 4
    offsets, which = one_row_each(T, 3, 90, 200)
    which = [2] + which[1:]
    _, c = make(T, K, N, r, nA, seed=T, dy=True)
    y, hid = forward(c, offsets, which, T, K, N, r, nA)
    clean = (y.clone(), *(v.clone() for v in backward(c, hid, offsets, which, T, K, N, r, nA)))
    c["A"][1], c["B"][1] = float("nan"), float("inf")
    c["A"][3], c["B"][3] = float("inf"), float("nan")
    bad = torch.zeros(T, dtype=torch.bool, device="cuda")
    bad[91:290:3] = True
    assert {which[i] for i in range(1, 201) if (i - 1) % 3 == 1} == {1}
    c["x"][bad], c["dy"][bad] = float("inf"), float("nan")
    y, hid = forward(c, offsets, which, T, K, N, r, nA)
    got = (y, *backward(c, hid, offsets, which, T, K, N, r, nA))
    for g, w in zip(got[:2], clean[:2]):
        assert torch.equal(g[~bad], w[~bad]) and not torch.isfinite(g[bad].float()).any()
    for g, w in zip(got[2:], clean[2:]):
        assert torch.equal(g[[0, 2, 3]], w[[0, 2, 3]]) and not torch.isfinite(g[1]).all()
    assert m.moe_read_device_status(reset=True) == 0


@pytest.mark.parametrize("r", [8, 24, 64, 104])
def test_gradients_keep_every_bit_of_u_and_v(r):
    """Rows with one non-zero gradient (input) element: u (v) is the fp32
    product s B (s A), rounded once, 2^-24; dA (dB) is u (v) times one bf16
    number.  Its three products are exact, their sum rounds twice: 2^-22 of
    the value holds them all, where u in two bf16 parts would be 2^-17 off."""
    T, K, N, nA = 40, 128, 192, 2
    d, c = make(T, K, N, r, nA, seed=r, dy=True)
    n0, k0 = 17, 101
    for name, at in (("x", slice(None)), ("dy", slice(None))):
        d[name][at] = 0
    g = torch.Generator().manual_seed(5)
    d["x"][3], d["dy"][3, n0] = torch.randn(K, generator=g).bfloat16(), 1.0
    d["x"][25, k0], d["dy"][25] = 1.0, torch.randn(N, generator=g).bfloat16()
    for name in ("x", "dy"):
        c[name] = d[name].cuda()
    offsets, which = [0, 20, 40], [0, 1]
    _, hid = forward(c, offsets, which, T, K, N, r, nA)
    _, dA, dB = backward(c, hid, offsets, which, T, K, N, r, nA)
    f = lambda v: v.double().numpy()  # noqa: E731
    s = f(d["scale"])
    wantA = s[0] * f(d["B"])[0, n0][:, None] * f(d["x"])[3][None, :]
    wantB = s[1] * f(d["dy"])[25][:, None] * f(d["A"])[1, :, k0][None, :]
    for got, want in ((dA[0], wantA), (dB[1], wantB)):
        assert np.all(np.abs(got.double().cpu().numpy() - want) <= 2.0 ** -22 * np.abs(want))


@pytest.mark.parametrize("T", [4, 40, 517, 1333, 3001])
@pytest.mark.parametrize("r", [8, 16, 32, 64, 128])
def test_outputs_keep_every_bit_of_u_and_v(T, r):
    """W x takes the first 16 bits of v = s away again: what is left of y is s
    less its two largest bf16 parts, a bf16 number itself, and every step to
    it is exact in fp32 (2^-8 of it allowed).  The same for dx with u."""
    K, N, nA, j = 1280, 2048 if T > 1500 else 1024, 2, r - 1
    _, c = make(1, K, N, r, nA, dy=True)
    s = np.float32(1.2345678)
    parts, rest = [], float(s)
    for _ in range(2):
        parts.append(float(torch.tensor(rest).bfloat16()))
        rest -= parts[-1]
    assert rest != 0 and abs(rest) <= 2.0 ** -16 and float(torch.tensor(rest).bfloat16()) == rest
    z = lambda *shape: torch.zeros(*shape, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    c.update(x=z(T, K), dy=z(T, N), W=z(N, K), A=z(nA, r, K), B=z(nA, N, r), scale=torch.full((nA,), float(s), device="cuda"))
    half = T // 2
    offsets, which = [0, half, T], [1, -1]
    c["x"][:, [70, 700]] = 1
    c["W"][:, 70], c["W"][:, 700] = -parts[0], -parts[1]
    c["A"][1, j, 70], c["B"][1, :, j] = 1, 1
    y, hid = forward(c, offsets, which, T, K, N, r, nA)
    assert (y[:half].double() - rest).abs().max() <= 2.0 ** -8 * abs(rest)
    assert torch.all(y[half:] == torch.tensor(-(parts[0] + parts[1])).bfloat16())
    c["dy"][:, [5, 600]] = 1
    c["W"].zero_()
    c["W"][5], c["W"][600] = -parts[0], -parts[1]
    c["B"].zero_()
    c["A"].zero_()
    c["B"][1, 5, j], c["A"][1, j] = 1, 1
    dx, _, _ = backward(c, hid, offsets, which, T, K, N, r, nA)
    assert (dx[:half].double() - rest).abs().max() <= 2.0 ** -8 * abs(rest)
    assert torch.all(dx[half:] == torch.tensor(-(parts[0] + parts[1])).bfloat16())


@pytest.mark.parametrize("T", [4, 40])
def test_largest_values_stay_finite(T):
    """v = u = 3.3999e38 is a finite fp32 number whose nearest bf16 number
    would be infinity: y and dx are v and u times 2^-100, dA and dB v and u
    times 2^-20.  2^-8 of a bf16 result, 2^-22 of an fp32 one."""
    K, N, r, nA = 64, 128, 8, 1
    big, s = float(torch.tensor(3.3895e38).bfloat16()), np.float32(1.003)
    want = float(np.float32(big) * s)
    assert np.isfinite(want) and not np.isfinite(float(torch.tensor(want).bfloat16()))
    _, c = make(1, K, N, r, nA, dy=True)
    z = lambda *shape: torch.zeros(*shape, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    c.update(x=z(T, K), dy=z(T, N), W=z(N, K), A=z(nA, r, K), B=z(nA, N, r), scale=torch.full((nA,), float(s), device="cuda"))
    offsets, which = [0, T], [0]
    c["x"][0, 3], c["A"][0, 2, 3], c["B"][0, :, 2] = 1, big, 2.0 ** -100
    y, hid = forward(c, offsets, which, T, K, N, r, nA)
    assert (y[0].double() / (want * 2.0 ** -100) - 1).abs().max() <= 2.0 ** -8
    c["dy"][0, 7] = 2.0 ** -20
    _, _, dB = backward(c, hid, offsets, which, T, K, N, r, nA)
    assert abs(float(dB[0, 7, 2]) / (want * 2.0 ** -20) - 1) <= 2.0 ** -22
    c["A"].zero_(), c["B"].zero_()
    c["dy"][0, 7], c["B"][0, 7, 2], c["A"][0, 2] = 1, big, 2.0 ** -100
    c["x"][0, 3] = 2.0 ** -20
    dx, dA, _ = backward(c, hid, offsets, which, T, K, N, r, nA)
    assert (dx[0].double() / (want * 2.0 ** -100) - 1).abs().max() <= 2.0 ** -8
    assert abs(float(dA[0, 2, 3]) / (want * 2.0 ** -20) - 1) <= 2.0 ** -22
