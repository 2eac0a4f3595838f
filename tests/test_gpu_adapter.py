"""Shared projection with per-request adapters, forward and backward, against
a float64 restatement.

Tolerances (derived before the first run).  fp32 sums of n products on the
tensor cores: below n 2^-23 of the terms' magnitudes in the worst case, and
the tests' n <= 2048 random signs stay far below 2^-14 of them.  v and u are
kept as two bf16 parts: 2^-17 of themselves.  So an fp32 result is held to
2^-14 of the sum of its terms' magnitudes, and a bf16 result adds 2^-8 of
itself (half an ulp is 2^-9; the fp32 error may cross a tie).
"""
import numpy as np
import pytest
import torch

import moe_expert_layer_topk_gb300 as m
import ops_ref

pytestmark = pytest.mark.gpu


def make(T, K, N, r, nA, seed=0, dy=False, pitch=0):
    g = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    d = dict(x=rn(T, K).bfloat16(), W=(rn(N, K) * 0.05).bfloat16(), A=(rn(nA, r, K) / K ** 0.5).bfloat16(),
             B=(rn(nA, N, r) * 0.3).bfloat16(), scale=torch.rand(nA, generator=g) * 2 + 0.5)
    if dy:
        d["dy"] = rn(T, N).bfloat16()
    c = {n: v.cuda() for n, v in d.items()}
    for n in ("x", "dy"):
        if pitch and n in c:  # rows inside a wider buffer of NaN
            wide = torch.full((T, c[n].shape[1] + pitch), float("nan"), dtype=torch.bfloat16, device="cuda")
            wide[:, pitch // 2:pitch // 2 + c[n].shape[1]] = c[n]
            c[n] = wide[:, pitch // 2:pitch // 2 + c[n].shape[1]]
    return d, c


def tables(offsets, which):
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    return i32(offsets), i32(which)


def forward(c, offsets, which, T, K, N, r, nA, pitch=0, scale=True):
    off, wh = tables(offsets, which)
    hid = torch.full((m.moe_adapter_hidden_size(T, r),), 255, dtype=torch.uint8, device="cuda")
    wide = torch.full((T, N + pitch), 3.0, dtype=torch.bfloat16, device="cuda")
    y = wide[:, pitch // 2:pitch // 2 + N]
    m.moe_adapter_linear(c["x"], c["W"], c["A"], c["B"], c["scale"] if scale else None, len(which), off, wh, T, K, N, r, nA, hid, y)
    if pitch:
        assert torch.all(wide[:, :pitch // 2] == 3) and torch.all(wide[:, pitch // 2 + N:] == 3)
    return y, hid


def backward(c, hid, offsets, which, T, K, N, r, nA, acc=None, pitch=0):
    off, wh = tables(offsets, which)
    f32 = lambda *s: torch.full(s, 7.0, device="cuda")  # noqa: E731
    wide = torch.full((T, K + pitch), 3.0, dtype=torch.bfloat16, device="cuda")
    dx = wide[:, pitch // 2:pitch // 2 + K]
    dA, dB = (f32(nA, r, K), f32(nA, N, r)) if acc is None else (acc[0].clone(), acc[1].clone())
    ws = torch.full((m.moe_adapter_linear_bwd_workspace_size(T, K, N, r, len(which)),), 255, dtype=torch.uint8, device="cuda")
    m.moe_adapter_linear_bwd(c["dy"], c["x"], c["W"], c["A"], c["B"], c["scale"], hid, len(which), off, wh, T, K, N, r, nA,
                             dx, dA, dB, 0 if acc is None else 1, ws)
    if pitch:
        assert torch.all(wide[:, :pitch // 2] == 3) and torch.all(wide[:, pitch // 2 + K:] == 3)
    return dx, dA, dB


def near(got, ref, name, bf16):
    g, w, mag = got.double().cpu().numpy(), ref[name], ref[name + "_mag"]
    tol = 2.0 ** -14 * mag + (2.0 ** -8 * np.abs(w) if bf16 else 0) + 1e-30
    bad = ~(np.abs(g - w) <= tol)
    assert not bad.any(), (name, int(bad.sum()), np.argwhere(bad)[:5].tolist(), float(np.abs(g - w)[bad].max()))


def requests(T, n, nA, seed, none=True):
    """n ragged requests over the rows, some empty, rows left over at both ends."""
    g = np.random.RandomState(seed)
    offsets = np.sort(g.randint(T // 16, T - T // 16 + 1, n + 1)).tolist()
    if n > 3:
        offsets[2] = offsets[1]
    which = g.randint(-1 if none else 0, nA, n).tolist()
    return offsets, which


# T, K, N, r, adapters, requests, extra columns of a row
SHAPES = [
    (1, 64, 64, 8, 1, 1, 0),
    (1, 2048, 192, 16, 3, 1, 0),
    (5, 128, 320, 16, 4, 5, 32),
    (64, 512, 256, 24, 7, 20, 0),
    (127, 192, 128, 32, 2, 3, 0),
    (128, 64, 512, 8, 5, 40, 64),
    (129, 1024, 64, 40, 3, 9, 0),
    (300, 320, 192, 64, 6, 30, 0),
    (517, 768, 1024, 72, 4, 33, 192),
    (700, 256, 384, 128, 3, 11, 0),
    (1500, 512, 2048, 16, 9, 17, 0),
    (2600, 128, 2560, 48, 5, 25, 0),
]


@pytest.mark.parametrize("T,K,N,r,nA,n,pitch", SHAPES)
def test_forward_and_backward(T, K, N, r, nA, n, pitch):
    d, c = make(T, K, N, r, nA, seed=T + r, dy=True, pitch=pitch)
    offsets, which = ([0, T], [nA - 1]) if n == 1 else requests(T, n, nA, seed=T)
    ref = ops_ref.adapter(*(d[k].double().numpy() for k in ("x", "W", "A", "B", "scale")), offsets, which, d["dy"].double().numpy())
    y, hid = forward(c, offsets, which, T, K, N, r, nA, pitch)
    near(y, ref, "y", True)
    dx, dA, dB = backward(c, hid, offsets, which, T, K, N, r, nA, pitch=pitch)
    near(dx, ref, "dx", True)
    near(dA, ref, "dA", False)
    near(dB, ref, "dB", False)
    for a in set(range(nA)) - {w for w, s, e in zip(which, offsets, offsets[1:]) if e > s}:
        assert not dA[a].any() and not dB[a].any()
    # twice the same bits; a second step's gradients are added
    again, hid2 = forward(c, offsets, which, T, K, N, r, nA, pitch)
    assert torch.equal(again, y)
    dx2, dA2, dB2 = backward(c, hid2, offsets, which, T, K, N, r, nA, acc=(dA, dB), pitch=pitch)
    assert torch.equal(dx2, dx)
    assert torch.allclose(dA2, 2 * dA, rtol=1e-6, atol=0) and torch.allclose(dB2, 2 * dB, rtol=1e-6, atol=0)
    assert m.moe_read_device_status(reset=True) == 0


def test_every_row_its_own_request():
    for T, nA in ((64, 48), (200, 64), (1000, 1000)):
        K, N, r = 256, 192, 16
        d, c = make(T, K, N, r, nA, seed=T)
        which = [(7 * i) % nA if i % 5 != 4 else -1 for i in range(T)]
        offsets = list(range(T + 1))
        y, _ = forward(c, offsets, which, T, K, N, r, nA)
        ref = ops_ref.adapter(*(d[k].double().numpy() for k in ("x", "W", "A", "B", "scale")), offsets, which)
        near(y, ref, "y", True)


@pytest.mark.parametrize("T,n,r,nA,same", [(1300, 1024, 64, 1024, 0), (3000, 1000, 16, 48, 0), (3000, 1000, 40, 1, 1), (900, 70, 128, 5, 6)])
def test_gradients_of_many_requests(T, n, r, nA, same):
    """The most requests and adapters of a call; neighbours with one adapter (in groups of `same`), empty requests between."""
    K, N = 64, 128
    d, c = make(T, K, N, r, nA, seed=n + nA, dy=True)
    offsets, which = requests(T, n, nA, seed=n)
    if same:
        which = [which[i // same * same] % nA if i % 11 else which[i] for i in range(n)]
    ref = ops_ref.adapter(*(d[k].double().numpy() for k in ("x", "W", "A", "B", "scale")), offsets, which, d["dy"].double().numpy())
    y, hid = forward(c, offsets, which, T, K, N, r, nA)
    dx, dA, dB = backward(c, hid, offsets, which, T, K, N, r, nA)
    for got, name, bf16 in ((y, "y", True), (dx, "dx", True), (dA, "dA", False), (dB, "dB", False)):
        near(got, ref, name, bf16)
    assert m.moe_read_device_status(reset=True) == 0


def test_no_requests_no_adapters_no_scale():
    T, K, N, r, nA = 150, 192, 128, 16, 2
    d, c = make(T, K, N, r, nA, dy=True)
    for offsets, which in (([0], []), ([0, 70, T], [-1, -1])):
        ref = ops_ref.adapter(*(d[k].double().numpy() for k in ("x", "W", "A", "B", "scale")), offsets, which, d["dy"].double().numpy())
        y, hid = forward(c, offsets, which, T, K, N, r, nA)
        near(y, ref, "y", True)
        dx, dA, dB = backward(c, hid, offsets, which, T, K, N, r, nA)
        near(dx, ref, "dx", True)
        assert not dA.any() and not dB.any()
        dx, dA, dB = backward(c, hid, offsets, which, T, K, N, r, nA, acc=(dA + 1, dB + 2))
        assert torch.all(dA == 1) and torch.all(dB == 2)
    off, which = [0, 40, 140], [1, 0]
    y, _ = forward(c, off, which, T, K, N, r, nA, scale=False)
    ref = ops_ref.adapter(*(d[k].double().numpy() for k in ("x", "W", "A", "B")), None, off, which)
    near(y, ref, "y", True)


def test_no_rows():
    K, N, r, nA = 128, 64, 8, 2
    d, c = make(1, K, N, r, nA, dy=True)
    c["x"], c["dy"] = c["x"][:0], c["dy"][:0]
    y, hid = forward(c, [0, 0], [1], 0, K, N, r, nA)
    dx, dA, dB = backward(c, hid, [0, 0], [1], 0, K, N, r, nA)
    assert not dA.any() and not dB.any()


@pytest.mark.parametrize("T", [40, 300])
def test_one_request_does_not_reach_another(T):
    """NaN and infinities in one request's rows, gradient rows and adapter, and
    in adapters nobody uses, leave every other request's values as they were."""
    K, N, r, nA = 128, 192, 16, 4
    _, c = make(T, K, N, r, nA, dy=True)
    offsets, which = [0, T // 4 + 3, T // 4 + 10, T - 5, T], [0, 1, 0, 2]
    y, hid = forward(c, offsets, which, T, K, N, r, nA)
    clean = (y.clone(), *(v.clone() for v in backward(c, hid, offsets, which, T, K, N, r, nA)))
    c["A"][1], c["B"][1] = float("nan"), float("inf")
    c["A"][3], c["B"][3] = float("inf"), float("nan")
    lo, hi = offsets[1], offsets[2]
    c["x"][lo:hi], c["dy"][lo:hi] = float("inf"), float("nan")
    y, hid = forward(c, offsets, which, T, K, N, r, nA)
    got = (y, *backward(c, hid, offsets, which, T, K, N, r, nA))
    rows = torch.ones(T, dtype=torch.bool, device="cuda")
    rows[lo:hi] = False
    for g, w in zip(got[:2], clean[:2]):
        assert torch.equal(g[rows], w[rows]) and not torch.isfinite(g[~rows].float()).any()
    for g, w in zip(got[2:], clean[2:]):
        assert torch.equal(g[[0, 2, 3]], w[[0, 2, 3]]) and not torch.isfinite(g[1]).all()


def test_more_than_2_31_outputs():
    """Rows beyond element 2^31 of y and of dy: a few rows checked in float64."""
    T, K, N, r, nA = 1_100_003, 64, 2048, 8, 2
    d, c = make(1, K, N, r, nA, seed=3)
    g = torch.Generator(device="cuda").manual_seed(1)
    c["x"] = torch.randn(T, K, generator=g, device="cuda").bfloat16()
    offsets, which = [5, 600_000, T - 1], [1, 0]
    y, hid = forward(c, offsets, which, T, K, N, r, nA)
    c["dy"] = y
    dx, _, _ = backward(c, hid, offsets, which, T, K, N, r, nA)
    at = [0, 4, 5, 599_999, 600_000, T - 2, T - 1]
    f = lambda v: v.double().cpu().numpy()  # noqa: E731
    ref = ops_ref.adapter(f(c["x"][at]), *(d[k].double().numpy() for k in ("W", "A", "B", "scale")), [2, 4, 6], [1, 0], f(c["dy"][at]))
    near(y[at], ref, "y", True)
    near(dx[at], ref, "dx", True)
    assert m.moe_read_device_status(reset=True) == 0


def test_more_row_tiles_than_a_grid_dimension():
    """More than 65535 tiles of 128 rows: a few rows checked in float64."""
    T, K, N, r, nA = 65535 * 128 + 11_521, 64, 64, 8, 2
    d, c = make(1, K, N, r, nA, seed=7)
    g = torch.Generator(device="cuda").manual_seed(2)
    c["x"] = torch.empty(T, K, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    offsets, which = [5, 6_000_000, T - 1], [1, 0]
    y, hid = forward(c, offsets, which, T, K, N, r, nA)
    c["dy"] = y
    dx, _, _ = backward(c, hid, offsets, which, T, K, N, r, nA)
    at = [0, 4, 5, 5_999_999, 6_000_000, 65535 * 128, T - 2, T - 1]
    f = lambda v: v.double().cpu().numpy()  # noqa: E731
    ref = ops_ref.adapter(f(c["x"][at]), *(d[k].double().numpy() for k in ("W", "A", "B", "scale")), [2, 4, 7], [1, 0], f(c["dy"][at]))
    near(y[at], ref, "y", True)
    near(dx[at], ref, "dx", True)
    assert m.moe_read_device_status(reset=True) == 0


def test_gradient_against_differences():
    """y is linear in x, in A and in B (each alone): a difference of the float64
    loss sum(y dy) over a step is its derivative up to rounding."""
    T, K, N, r, nA = 60, 64, 128, 8, 3
    d, c = make(T, K, N, r, nA, dy=True)
    offsets, which = [3, 20, 41, 60], [2, 0, 2]
    _, hid = forward(c, offsets, which, T, K, N, r, nA)
    got = dict(zip(("x", "A", "B"), backward(c, hid, offsets, which, T, K, N, r, nA)))
    args = {k: d[k].double().numpy() for k in ("x", "W", "A", "B", "scale")}
    dy = d["dy"].double().numpy()
    f = lambda kw: float((ops_ref.adapter(kw["x"], kw["W"], kw["A"], kw["B"], kw["scale"], offsets, which)["y"] * dy).sum())  # noqa: E731
    g = np.random.RandomState(0)
    for name in ("x", "A", "B"):
        v = got[name].double().cpu().numpy()
        for _ in range(25):
            i = tuple(g.randint(s) for s in v.shape)
            up, dn = dict(args), dict(args)
            up[name], dn[name] = args[name].copy(), args[name].copy()
            up[name][i] += 0.5
            dn[name][i] -= 0.5
            assert abs(f(up) - f(dn) - v[i]) <= (2.0 ** -8 if name == "x" else 1e-4) * np.abs(v).max()


def test_bad_tables_are_reported():
    T, K, N, r, nA = 100, 64, 64, 8, 2
    d, c = make(T, K, N, r, nA)
    assert m.moe_read_device_status(reset=True) == 0
    y, _ = forward(c, [0, 50, 100], [0, 2], T, K, N, r, nA)       # no such adapter: none
    assert m.moe_read_device_status(reset=True) == 2
    ref = ops_ref.adapter(*(d[k].double().numpy() for k in ("x", "W", "A", "B", "scale")), [0, 50, 100], [0, -1])
    near(y, ref, "y", True)
    y, _ = forward(c, [0, 60, 40, 500], [0, 1, 1], T, K, N, r, nA)  # backwards, past the end
    assert m.moe_read_device_status(reset=True) == 2
    ref = ops_ref.adapter(*(d[k].double().numpy() for k in ("x", "W", "A", "B", "scale")), [0, 60, 60, 100], [0, 1, 1])
    near(y, ref, "y", True)


def test_other_stream_and_graph():
    T, K, N, r, nA = 333, 256, 256, 16, 4
    d, c = make(T, K, N, r, nA, dy=True)
    offsets, which = requests(T, 7, nA, seed=1)
    y, hid = forward(c, offsets, which, T, K, N, r, nA)
    want = (y.clone(), *(v.clone() for v in backward(c, hid, offsets, which, T, K, N, r, nA)))
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        y, hid = forward(c, offsets, which, T, K, N, r, nA)
        got = (y, *backward(c, hid, offsets, which, T, K, N, r, nA))
    s.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    off, wh = tables(offsets, which)
    y = torch.empty(T, N, dtype=torch.bfloat16, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m.moe_adapter_linear(c["x"], c["W"], c["A"], c["B"], c["scale"], len(which), off, wh, T, K, N, r, nA, hid, y)
    other, ow = requests(T, 7, nA, seed=2)
    off.copy_(tables(other, ow)[0])
    wh.copy_(tables(other, ow)[1])
    graph.replay()
    torch.cuda.synchronize()
    ref = ops_ref.adapter(*(d[k].double().numpy() for k in ("x", "W", "A", "B", "scale")), other, ow)
    near(y, ref, "y", True)
