"""Balance loss, z-loss, per-expert counts and the logits' gradient against a
plain float64 implementation, and their way through the router's calls.

Tolerances (derived before the first run): a softmax value is an exponential
(2 ulp, its argument off by half an ulp of up to 40), a sum over E <= 1024
values in a tree and a division, below 2^-24 * (40 + 2 + 10 + 2) = 3.3e-6
relative; sums of them (positive terms) keep that and add one rounding per
level.  So prob_sum is held to 8e-6, the losses to 1.6e-5 (two such factors),
a gradient element to 1.6e-5 of the sum of its terms' magnitudes (its two
terms may cancel), with 1e-30 for denormals.
"""
import numpy as np
import pytest
import torch

import moe_expert_layer_topk_gb300 as m
import ops_ref

pytestmark = pytest.mark.gpu

COEF = (0.7, 0.3)


def call(logits, idx, mask, offsets, k, coef=COEF, grad=True):
    T, E = logits.shape
    S = 1 if offsets is None else len(offsets) - 1
    e = lambda *s, dt=torch.float32: torch.full(s, -7, dtype=dt, device="cuda")  # noqa: E731
    o = dict(counts=e(S, E, dt=torch.int32), tokens=e(S, dt=torch.int32), prob_sum=e(S, E), loss=e(2))
    dl = e(T, E) if grad else None
    ws = torch.full((max(256, m.moe_balance_loss_workspace_size(T, E, S)),), 255, dtype=torch.uint8, device="cuda")
    off = None if offsets is None else torch.tensor(offsets, dtype=torch.int32, device="cuda")
    m.moe_balance_loss(logits, idx, mask, T, E, k, S, off, o["counts"], o["tokens"], o["prob_sum"], o["loss"], *coef, dl, ws)
    if grad:
        o["dlogits"] = dl
    return o


def compare(o, ref):
    assert np.array_equal(o["counts"].cpu().numpy(), ref["counts"])
    assert np.array_equal(o["tokens"].cpu().numpy(), ref["tokens"])
    np.testing.assert_allclose(o["prob_sum"].cpu().numpy(), ref["prob_sum"], rtol=8e-6, atol=1e-30)
    np.testing.assert_allclose(o["loss"].cpu().numpy(), ref["loss"], rtol=1.6e-5, atol=1e-30)
    if "dlogits" in o:
        err = np.abs(o["dlogits"].cpu().numpy().astype(np.float64) - ref["dlogits"])
        assert np.all(err <= 1.6e-5 * ref["mag"] + 1e-30), err.max()


def inputs(T, E, k, seed, masked=False, off_experts=0):
    g = torch.Generator().manual_seed(seed)
    l = torch.randn(T, E, generator=g) * 1.5 + torch.randn(E, generator=g)
    if off_experts:
        l[:, torch.randperm(E, generator=g)[:off_experts]] = -float("inf")
    idx = torch.topk(l, k, dim=1).indices.to(torch.int32)
    mask = (torch.rand(T, generator=g) > 0.3).to(torch.uint8) if masked else None
    if masked:  # what padding tokens hold does not matter
        junk = torch.tensor([float("nan"), float("inf"), -float("inf")])[torch.arange(T) % 3]
        l = torch.where(mask[:, None] == 0, junk[:, None], l)
        idx[mask == 0] = -99
    return l.cuda(), idx.cuda(), None if mask is None else mask.cuda()


# every lane layout: experts in fours (2 to 32 lanes a token, 1 to 8 vectors a lane) and one by one
SHAPES = [(1, 1, 1), (3, 4, 2), (257, 8, 2), (100, 16, 5), (77, 24, 3), (65, 64, 8), (513, 128, 8), (40, 256, 4),
          (33, 512, 32), (20, 1024, 8), (50, 3, 1), (129, 7, 2), (40, 30, 4), (61, 57, 8), (31, 126, 3), (45, 130, 8),
          (19, 511, 6), (17, 1023, 2)]


@pytest.mark.parametrize("T,E,k", SHAPES)
@pytest.mark.parametrize("packed", [False, True])
def test_matches_float64(T, E, k, packed):
    l, idx, mask = inputs(T, E, k, seed=T + E, masked=packed, off_experts=min(2, E // 4))
    offsets = None
    if packed:  # a gap before and after, an empty sequence, one token
        offsets = sorted([min(2, T // 4), T // 3, T // 3, T // 2, T // 2 + (T > 2), T - T // 8])
    o = call(l, idx, mask, offsets, k)
    ref = ops_ref.balance(l.cpu().numpy(), idx.cpu().numpy(), None if mask is None else mask.cpu().numpy(),
                          offsets or [0, T], k, *COEF)
    compare(o, ref)
    assert m.moe_read_device_status(reset=True) == 0


def test_many_sequences_and_chunks():
    """More chunks than CTAs fill at once, sequences shorter and longer than a chunk."""
    T, E, k = 30011, 128, 8
    g = np.random.RandomState(1)
    offsets = sorted(g.randint(0, T + 1, 200).tolist()) + [T]
    l, idx, mask = inputs(T, E, k, seed=5, masked=True)
    ref = ops_ref.balance(l.cpu().numpy(), idx.cpu().numpy(), mask.cpu().numpy(), offsets, k, *COEF)
    o = call(l, idx, mask, offsets, k)
    compare(o, ref)
    again = call(l, idx, mask, offsets, k)
    for n in o:
        assert torch.equal(o[n], again[n]), n  # bit for bit
    assert m.moe_read_device_status(reset=True) == 0


@pytest.mark.parametrize("packed", [False, True])
def test_backward_alone_and_forward_alone(packed):
    T, E, k = 300, 60, 4
    l, idx, mask = inputs(T, E, k, seed=9, masked=packed)
    offsets = [5, 90, 90, 250] if packed else None
    o = call(l, idx, mask, offsets, k, grad=False)
    full = call(l, idx, mask, offsets, k)
    assert torch.equal(o["loss"], full["loss"]) and torch.equal(o["prob_sum"], full["prob_sum"])
    dl = torch.full_like(l, 9.0)
    off = None if offsets is None else torch.tensor(offsets, dtype=torch.int32, device="cuda")
    S = o["tokens"].numel()
    m.moe_balance_loss_bwd(l, mask, T, E, k, S, off, o["counts"], o["tokens"], *COEF, None, dl)
    assert torch.equal(dl, full["dlogits"])
    up = torch.tensor([-1.5, 3.0], device="cuda")
    m.moe_balance_loss_bwd(l, mask, T, E, k, S, off, o["counts"], o["tokens"], *COEF, up, dl)
    ref = ops_ref.balance(l.cpu().numpy(), idx.cpu().numpy(), None if mask is None else mask.cpu().numpy(),
                          offsets or [0, T], k, COEF[0] * -1.5, COEF[1] * 3.0)
    err = np.abs(dl.cpu().numpy() - ref["dlogits"])
    assert np.all(err <= 1.6e-5 * ref["mag"] + 1e-30)


def test_gradient_against_differences():
    """Central differences of the float64 loss with the counts held: at step h
    their error is h^2/6 of the third derivative, below 1e-7 of the largest
    gradient element at h = 1e-4; the bound adds the kernel's own 1.6e-5."""
    T, E, k = 40, 12, 3
    l, idx, _ = inputs(T, E, k, seed=3)
    o = call(l, idx, None, [0, 25, 40], k)
    base, ix = l.cpu().numpy().astype(np.float64), idx.cpu().numpy()
    got = o["dlogits"].cpu().numpy()
    f = lambda v: float(np.dot(COEF, ops_ref.balance(v, ix, None, [0, 25, 40], k)["loss"]))  # noqa: E731
    g = np.random.RandomState(0)
    for _ in range(60):
        t, e = g.randint(T), g.randint(E)
        up, down = base.copy(), base.copy()
        up[t, e] += 1e-4
        down[t, e] -= 1e-4
        assert abs((f(up) - f(down)) / 2e-4 - got[t, e]) <= 5e-5 * np.abs(got).max()


def test_rows_at_the_ends_of_the_range():
    """A row of the type's lowest value is uniform; one huge logit takes all; a
    NaN in a token that counts shows in its row and in the loss, not elsewhere."""
    T, E, k = 6, 8, 2
    l, idx, _ = inputs(T, E, k, seed=4)
    low = torch.finfo(torch.float32).min
    l[0] = low
    l[1] = low
    l[1, 3] = 5.0
    l[2, 1:] = -float("inf")
    o = call(l, idx, None, None, k, coef=(1.0, 0.0))
    ref = ops_ref.balance(l.cpu().numpy(), idx.cpu().numpy(), None, [0, T], k, 1.0, 0.0)
    np.testing.assert_allclose(o["prob_sum"].cpu().numpy(), ref["prob_sum"], rtol=8e-6)
    assert np.all(np.isfinite(o["dlogits"].cpu().numpy()))
    l, idx, _ = inputs(T, E, k, seed=4)
    clean = call(l, idx, None, None, k)
    l[2, 5] = float("nan")
    o = call(l, idx, None, None, k)
    assert torch.isnan(o["loss"]).all() and torch.isnan(o["dlogits"][2]).all()
    rest = torch.arange(T, device="cuda") != 2
    assert torch.equal(o["dlogits"][rest], clean["dlogits"][rest])
    assert torch.equal(o["counts"], clean["counts"])


def test_nothing_counts():
    T, E, k = 50, 16, 2
    l, idx, _ = inputs(T, E, k, seed=6)
    for mask, offsets in ((torch.zeros(T, dtype=torch.uint8, device="cuda"), None), (None, [7, 7, 7])):
        o = call(l, idx, mask, offsets, k)
        for n, v in o.items():
            assert not v.any(), n
    o = call(l[:0], idx[:0], None, None, k)
    assert not any(v.any() for v in o.values())


def test_bad_tables_and_ids_are_reported():
    T, E, k = 64, 8, 2
    l, idx, _ = inputs(T, E, k, seed=8)
    assert m.moe_read_device_status(reset=True) == 0
    bad = idx.clone()
    bad[3, 1] = E
    bad[9, 0] = -1
    o = call(l, bad, None, None, k)
    assert m.moe_read_device_status(reset=True) == 1
    assert int(o["counts"].sum()) == T * k - 2
    call(l, idx, None, [0, 40, 20, 64], k)
    assert m.moe_read_device_status(reset=True) == 2
    call(l, idx, None, [0, 40, 900], k)
    assert m.moe_read_device_status(reset=True) == 2


def test_more_than_2_31_logits():
    """Two kinds of rows, so that every row's gradient is known from float64 of
    two: element offsets pass 2^31 in the logits and in their gradient."""
    T, E, k = (1 << 24) + 77, 130, 2
    kinds = torch.randn(2, E, generator=torch.Generator().manual_seed(2))
    kind = torch.arange(T, device="cuda") % 3 == 0
    l = torch.where(kind[:, None], kinds[0].cuda(), kinds[1].cuda())
    idx = torch.topk(kinds, k, dim=1).indices.to(torch.int32).cuda()[(~kind).long()]
    o = call(l, idx, None, None, k)
    n = [int(kind.sum()), T - int(kind.sum())]
    p = torch.softmax(kinds.double(), 1).numpy()
    lse = torch.logsumexp(kinds.double(), 1).numpy()
    counts = np.zeros(E)
    for q in range(2):
        counts[torch.topk(kinds, k, dim=1).indices[q].numpy()] += n[q]
    assert np.array_equal(o["counts"].cpu().numpy()[0], counts)
    np.testing.assert_allclose(o["prob_sum"].cpu().numpy()[0], n[0] * p[0] + n[1] * p[1], rtol=8e-6)
    a, b = COEF
    for q in range(2):
        mean = (p[q] * counts).sum()
        want = p[q] * (a * E / (k * T * T) * (counts - mean) + 2 * b / T * lse[q])
        mag = p[q] * (a * E / (k * T * T) * (counts + mean) + 2 * b / T * abs(lse[q]))
        for t in (q, T // 2 // 3 * 3 + q, (T - 3) // 3 * 3 + q):  # first rows, the middle, the last
            assert bool(kind[t]) == (q == 0)
            assert np.all(np.abs(o["dlogits"][t].cpu().numpy() - want) <= 1.6e-5 * mag)


def test_other_stream():
    T, E, k = 500, 128, 8
    l, idx, _ = inputs(T, E, k, seed=2)
    want = call(l, idx, None, None, k)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = call(l, idx, None, None, k)
    s.synchronize()
    for n in want:
        assert torch.equal(want[n], got[n]), n


def test_router_keeps_its_logits_and_takes_their_gradient():
    """moe_route_topk_logits: the same routing bit for bit, and logits that agree
    with float64 (H = 256 products: 2^-24 * 256 of the terms' magnitudes).
    moe_route_topk_logits_bwd: with a zero dlogits bit-identical to
    moe_route_topk_bwd; with one, dWr and dx gain x^T dlogits and dlogits Wr^T
    (operands split into two bf16 parts: 2^-15 of the terms' magnitudes, dx
    rounded to bf16: 2^-8)."""
    T, H, E, k = 150, 256, 24, 3
    g = torch.Generator().manual_seed(0)
    x = torch.randn(T, H, generator=g).bfloat16().cuda()
    Wr = (torch.randn(H, E, generator=g) * 0.05).cuda()
    L = m.MoELayer(T, H, 64, E, k, 1)
    L.route(x, Wr)
    names = ("topk_idx", "topk_w", "counts", "offsets", "rank_offsets", "chunk_prefix")
    want = {n: getattr(L, n).clone() for n in names}
    logits = torch.empty(T, E, device="cuda")
    m.moe_route_topk_logits(x, Wr, None, T, H, E, k, 1, L.topk_idx, L.topk_w, L.counts, L.offsets, L.rank_offsets,
                            L.chunk_prefix, logits, L.ws_route)
    for n in names:
        assert torch.equal(getattr(L, n), want[n]), n
    xd, wd = x.double().cpu(), Wr.double().cpu()
    assert torch.all((logits.double().cpu() - xd @ wd).abs() <= 2.0 ** -16 * (xd.abs() @ wd.abs()))
    d_w = torch.randn(T, k, generator=g).cuda()
    acc = torch.randn(T, H, generator=g).cuda()
    m.moe_route_topk_bwd(d_w, L.topk_w, L.topk_idx, x, Wr, acc, T, H, E, k, L.dWr, L.dx, 0, L.ws_route_bwd)
    base = L.dWr.clone(), L.dx.clone()
    dl = torch.zeros(T, E, device="cuda")
    m.moe_route_topk_logits_bwd(d_w, L.topk_w, L.topk_idx, dl, x, Wr, acc, T, H, E, k, L.dWr, L.dx, 0, L.ws_route_bwd)
    assert torch.equal(L.dWr, base[0]) and torch.equal(L.dx, base[1])
    dl = torch.randn(T, E, generator=g).cuda()
    m.moe_route_topk_logits_bwd(d_w, L.topk_w, L.topk_idx, dl, x, Wr, acc, T, H, E, k, L.dWr, L.dx, 0, L.ws_route_bwd)
    w64, i64, g64 = L.topk_w.double().cpu(), L.topk_idx.long().cpu(), d_w.double().cpu()
    full = dl.double().cpu().scatter_add(1, i64, w64 * (g64 - (w64 * g64).sum(1, keepdim=True)))
    want_w = xd.t() @ full
    assert torch.all((L.dWr.double().cpu() - want_w).abs() <= 2.0 ** -15 * (xd.abs().t() @ full.abs()))
    want_x = acc.double().cpu() + full @ wd.t()
    tol = 2.0 ** -8 * want_x.abs() + 2.0 ** -15 * (full.abs() @ wd.abs().t())
    assert torch.all((L.dx.double().cpu() - want_x).abs() <= tol)
    assert m.moe_read_device_status(reset=True) == 0
