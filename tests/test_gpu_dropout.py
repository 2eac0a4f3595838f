"""Counter-based dropout, alone and in the weighted combine, forward and
backward, against a float64 restatement with the generator in numpy.

Tolerances (derived before the first run): which elements stay is compared
exactly.  Values: k fp32 fused multiply-adds, one product and one sum are
below (k + 2) 2^-24 of the terms' magnitudes, and a bf16 result adds 2^-8 of
itself (half an ulp is 2^-9; the fp32 error may cross a tie).  d_w is a sum
of H products over 32 lanes in order and a tree: 2^-24 (H/32 + 8) of the
magnitudes.
"""
import numpy as np
import pytest
import torch

import moe_expert_layer_topk_gb300 as m
import ops_ref

pytestmark = pytest.mark.gpu

I64 = torch.int64


def rng(seed, offset=0):
    s = seed - (1 << 64) if seed >= 1 << 63 else seed
    o = offset - (1 << 64) if offset >= 1 << 63 else offset
    return torch.tensor([s, o], dtype=I64, device="cuda")


def mask_of(n, p, seed, offset=0):
    x = torch.ones(n, device="cuda")
    out = torch.full_like(x, -3.0)
    m.moe_dropout(x, None, n, p, rng(seed, offset), out)
    v = out.cpu().numpy()
    assert np.all((v == 0) | (v == np.float32(ops_ref.factor(p))))
    return v != 0


@pytest.mark.parametrize("n", [1, 2, 7, 8, 9, 63, 4097])
@pytest.mark.parametrize("p", [0.0, 0.1, 0.5, 0.999, 1.0])
def test_mask_is_the_generator(n, p):
    for seed, offset in ((0, 0), (12345678901234567, 77), ((1 << 64) - 1, (1 << 32) - 2), (5, (1 << 64) - 3)):
        got = mask_of(n, p, seed, offset)
        want = ops_ref.keep(seed, offset, 0, n, p) if p < 1 else np.zeros(n, bool)
        assert np.array_equal(got, want), (seed, offset)


def test_share_that_stays():
    n, p = 1 << 22, 0.3
    kept = mask_of(n, p, 99).mean()
    q = 1 - ops_ref.dropped_below(p) / 65536
    assert abs(kept - q) <= 6 * np.sqrt(q * (1 - q) / n)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n", [1, 8, 1003, 100000])
@pytest.mark.parametrize("with_res", [False, True])
def test_values(dt, n, with_res):
    g = torch.Generator().manual_seed(n)
    x, r = torch.randn(n, generator=g).to(dt).cuda(), torch.randn(n, generator=g).to(dt).cuda()
    p, seed = 0.25, 42
    out = torch.full_like(x, 7.0)
    m.moe_dropout(x, r if with_res else None, n, p, rng(seed, 3), out)
    keep = ops_ref.keep(seed, 3, 0, n, p)
    xd, rd = x.double().cpu().numpy(), r.double().cpu().numpy() if with_res else np.zeros(n)
    want = rd + np.where(keep, xd * ops_ref.factor(p), 0)
    tol = 3 * 2.0 ** -24 * (np.abs(rd) + np.abs(xd) * ops_ref.factor(p)) + (2.0 ** -8 * np.abs(want) if dt == torch.bfloat16 else 0)
    assert np.all(np.abs(out.double().cpu().numpy() - want) <= tol)
    # into the residual's own memory, and the gradient: the same call on dout
    if with_res:
        again = r.clone()
        m.moe_dropout(x, again, n, p, rng(seed, 3), again)
        assert torch.equal(again, out)


def test_what_is_dropped_does_not_show():
    n, p, seed = 4096, 0.5, 7
    keep = torch.from_numpy(ops_ref.keep(seed, 0, 0, n, p)).cuda()
    x = torch.where(keep, 1.0, torch.tensor(float("nan"), device="cuda")).bfloat16()
    x[~keep & (torch.arange(n, device="cuda") % 2 == 0)] = float("inf")
    out = torch.empty_like(x)
    m.moe_dropout(x, None, n, p, rng(seed), out)
    assert torch.equal(out, torch.where(keep, 2.0, 0.0).bfloat16())


def test_more_than_2_32_elements():
    n, p, seed = (1 << 32) + 13, 0.5, 3
    x = torch.ones(n, dtype=torch.bfloat16, device="cuda")
    out = torch.empty_like(x)
    m.moe_dropout(x, None, n, p, rng(seed), out)
    for first in (0, (1 << 31) - 8, (1 << 32) - 64):
        cnt = min(200, n - first)
        want = ops_ref.keep(seed, 0, first, cnt, p)
        assert np.array_equal(out[first:first + cnt].float().cpu().numpy() != 0, want), first


def test_combine_of_more_than_2_31_elements():
    T, H, k, p, seed = (1 << 20) + 9, 2048, 1, 0.5, 11
    rows = torch.arange(T, dtype=torch.int32, device="cuda").flip(0).view(T, 1)
    y_perm = torch.ones(T, H, dtype=torch.bfloat16, device="cuda")
    w = torch.full((T, 1), 1.5, device="cuda")
    y = torch.empty_like(y_perm)
    m.moe_combine_dropout(y_perm, w, rows.contiguous(), None, T, H, k, p, rng(seed), y)
    dyp, dw = torch.empty_like(y_perm), torch.empty(T, 1, device="cuda")
    m.moe_combine_dropout_bwd(y_perm, y_perm, w, rows.contiguous(), T, H, k, p, rng(seed), dyp, dw)
    for t in (0, T // 2, T - 1):
        keep = ops_ref.keep(seed, 0, t * H, H, p)
        assert np.array_equal(y[t].float().cpu().numpy(), np.where(keep, 3.0, 0.0))
        assert np.array_equal(dyp[T - 1 - t].float().cpu().numpy(), np.where(keep, 3.0, 0.0))
        assert float(dw[t, 0]) == 2.0 * keep.sum()
    assert m.moe_read_device_status(reset=True) == 0


def combine_inputs(T, H, k, seed):
    g = torch.Generator().manual_seed(seed)
    rows = torch.randperm(T * k, generator=g).to(torch.int32).view(T, k)
    w = torch.rand(T, k, generator=g)
    return dict(y_perm=torch.randn(T * k, H, generator=g).bfloat16(), topk_w=w / w.sum(1, keepdim=True), row_of_slot=rows,
                residual=torch.randn(T, H, generator=g).bfloat16(), dy=torch.randn(T, H, generator=g).bfloat16())


SHAPES = [(1, 64, 1), (5, 64, 8), (33, 192, 3), (129, 128, 2), (40, 2048, 8), (7, 4160, 2), (300, 320, 17), (3, 64, 32)]


@pytest.mark.parametrize("T,H,k", SHAPES)
def test_combine(T, H, k):
    d = combine_inputs(T, H, k, seed=T + H)
    c = {n: v.cuda() for n, v in d.items()}
    p, seed = 0.1, 1 << 40
    keep = ops_ref.keep(seed, 9, 0, T * H, p).reshape(T, H)
    f = ops_ref.factor(p)
    yp, w = d["y_perm"].double().numpy()[d["row_of_slot"].long().numpy()], d["topk_w"].double().numpy()[:, :, None]
    s, mag = (w * yp).sum(1), (w * np.abs(yp)).sum(1)
    for res in (None, d["residual"]):
        y = torch.full((T, H), 5.0, dtype=torch.bfloat16, device="cuda")
        m.moe_combine_dropout(c["y_perm"], c["topk_w"], c["row_of_slot"], None if res is None else c["residual"], T, H, k, p,
                              rng(seed, 9), y)
        base = 0 if res is None else res.double().numpy()
        want = base + np.where(keep, s * f, 0)
        tol = 2.0 ** -8 * np.abs(want) + (k + 2) * 2.0 ** -24 * (np.abs(base) + mag * f)
        assert np.all(np.abs(y.double().cpu().numpy() - want) <= tol)
    # without dropout and residual: moe_combine's bits
    y0, y1 = torch.empty_like(y), torch.empty_like(y)
    m.moe_combine(c["y_perm"], c["topk_w"], c["row_of_slot"], T, H, k, y0)
    m.moe_combine_dropout(c["y_perm"], c["topk_w"], c["row_of_slot"], None, T, H, k, 0.0, rng(1), y1)
    assert torch.equal(y0, y1)
    assert m.moe_read_device_status(reset=True) == 0


@pytest.mark.parametrize("T,H,k", SHAPES)
def test_combine_backward(T, H, k):
    d = combine_inputs(T, H, k, seed=T + H)
    c = {n: v.cuda() for n, v in d.items()}
    p, seed = 0.25, 17
    dyp = torch.full((T * k, H), 5.0, dtype=torch.bfloat16, device="cuda")
    dw = torch.full((T, k), 5.0, device="cuda")
    m.moe_combine_dropout_bwd(c["dy"], c["y_perm"], c["topk_w"], c["row_of_slot"], T, H, k, p, rng(seed), dyp, dw)
    keep = ops_ref.keep(seed, 0, 0, T * H, p).reshape(T, H)
    g = np.where(keep, d["dy"].double().numpy() * ops_ref.factor(p), 0)
    rows, w = d["row_of_slot"].long().numpy(), d["topk_w"].double().numpy()
    yp = d["y_perm"].double().numpy()[rows]
    want = w[:, :, None] * g[:, None, :]
    got = dyp.double().cpu().numpy()[rows]
    assert np.all(np.abs(got - want) <= (2.0 ** -8 + 2.0 ** -22) * np.abs(want))
    terms = g[:, None, :] * yp
    tol = 2.0 ** -24 * (H / 32 + 8) * np.abs(terms).sum(2)
    assert np.all(np.abs(dw.double().cpu().numpy() - terms.sum(2)) <= tol)
    # without dropout: moe_combine_bwd's bits
    o = [torch.empty_like(dyp), torch.empty_like(dw), torch.empty_like(dyp), torch.empty_like(dw)]
    m.moe_combine_bwd(c["dy"], c["y_perm"], c["topk_w"], c["row_of_slot"], T, H, k, o[0], o[1])
    m.moe_combine_dropout_bwd(c["dy"], c["y_perm"], c["topk_w"], c["row_of_slot"], T, H, k, 0.0, rng(1), o[2], o[3])
    assert torch.equal(o[0], o[2]) and torch.equal(o[1], o[3])
    assert m.moe_read_device_status(reset=True) == 0


def test_combine_gradient_against_differences():
    """y is linear in y_perm and in topk_w for a given mask: with dy fixed,
    dy . (y(w + h) - y(w)) / h is d_w exactly in exact arithmetic; in fp32 sums
    of a bf16 y the difference of two roundings is 2^-8 |y| / h an element.
    h = 64 keeps that below 2^-13 of the sum's magnitude."""
    T, H, k, p, seed = 4, 128, 2, 0.5, 21
    d = combine_inputs(T, H, k, seed=1)
    c = {n: v.cuda() for n, v in d.items()}
    r = rng(seed)
    dyp = torch.empty(T * k, H, dtype=torch.bfloat16, device="cuda")
    dw = torch.empty(T, k, device="cuda")
    m.moe_combine_dropout_bwd(c["dy"], c["y_perm"], c["topk_w"], c["row_of_slot"], T, H, k, p, r, dyp, dw)

    def y(w):
        out = torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
        m.moe_combine_dropout(c["y_perm"], w, c["row_of_slot"], None, T, H, k, p, r, out)
        return out.double()

    h = 64.0
    for t in range(T):
        for j in range(k):
            w = c["topk_w"].clone()
            w[t, j] += h
            up, base = y(w), y(c["topk_w"])
            num = float((c["dy"].double() * (up - base)).sum()) / h
            tol = 2.0 ** -8 / h * float((c["dy"].double().abs() * (up.abs() + base.abs())).sum())
            assert abs(num - float(dw[t, j])) <= tol + 1e-6


def test_rows_out_of_range_are_skipped_and_reported():
    T, H, k = 9, 64, 2
    c = {n: v.cuda() for n, v in combine_inputs(T, H, k, seed=2).items()}
    c["row_of_slot"][4, 1] = T * k
    c["row_of_slot"][5, 0] = -1
    assert m.moe_read_device_status(reset=True) == 0
    y = torch.zeros(T, H, dtype=torch.bfloat16, device="cuda")
    m.moe_combine_dropout(c["y_perm"], c["topk_w"], c["row_of_slot"], None, T, H, k, 0.0, rng(1), y)
    assert m.moe_read_device_status(reset=True) == 1
    want = (c["topk_w"][4, 0] * c["y_perm"][c["row_of_slot"][4, 0].long()].float()).bfloat16()
    assert torch.equal(y[4], want)
    dyp = torch.zeros(T * k, H, dtype=torch.bfloat16, device="cuda")
    dw = torch.zeros(T, k, device="cuda")
    m.moe_combine_dropout_bwd(c["dy"], c["y_perm"], c["topk_w"], c["row_of_slot"], T, H, k, 0.0, rng(1), dyp, dw)
    assert m.moe_read_device_status(reset=True) == 1
    assert float(dw[4, 1]) == 0 and float(dw[5, 0]) == 0


def test_graph_replay_takes_the_new_counter():
    """The generator's words are read on the device: a captured call drops other
    elements when the program writes a new offset between replays."""
    n, p = 4096, 0.5
    x, r = torch.ones(n, device="cuda"), rng(5, 0)
    out = torch.empty_like(x)
    m.moe_dropout(x, None, n, p, r, out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m.moe_dropout(x, None, n, p, r, out)
    for offset in (0, n // 8, 123456789):
        r.copy_(rng(5, offset))
        graph.replay()
        torch.cuda.synchronize()
        assert np.array_equal(out.cpu().numpy() != 0, ops_ref.keep(5, offset, 0, n, p))
