"""The norms before and after a block against their float64 restatements.

Bounds.  u = 2^-24.  A bf16 output is off by half a step of its value (2^-8), an
fp32 one by u.  A row's sum of H <= 8192 terms is added in chains of at most 32
terms a lane, 5 shuffles and 8 warps (45 additions), each term with up to six
roundings before; with a gate's exponential (at most (4 + 1.2 |logit|) 2^-23) a
value is off by less than 2^-17 of the magnitudes that it is made of.  A gain's
gradient adds a lane's rows, the block's groups and the parts: fewer than 500
additions here, 2^-15 of its magnitudes.
"""
import numpy as np
import pytest
import torch

import block_ref as ref
import moe_expert_layer_topk_gb300 as m

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
EPS = 1e-5
CALC, SUMS = 2.0 ** -17, 2.0 ** -15


def e(*s, dt=F32):
    return torch.empty(*s, dtype=dt, device="cuda")


def np64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def near(got, want, mag, what, calc=CALC):
    got, half = np64(got), {BF: 2.0 ** -8, F32: 2.0 ** -24}[got.dtype]
    bound = half * np.abs(want) + calc * mag + 1e-37
    bad = ~(np.abs(got - want) <= bound)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size}, worst {np.nanmax(np.abs(got - want) / bound):.3g} of the bound"


def gen(seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return lambda *s: torch.randn(*s, generator=g, device="cuda")


def rows(rn, T, H, dt, pitch=0):
    return (rn(T, H + pitch) * torch.exp(rn(T, 1))).to(dt)[:, pitch // 2:pitch // 2 + H]


SHAPES = [(1, 8), (3, 64), (33, 72), (300, 128), (7, 136), (100, 256), (31, 264), (19, 520), (40, 1032), (1, 2048), (517, 2048),
          (9, 2056), (5, 4096), (3, 4104), (2, 8184), (37, 8192)]


@pytest.mark.parametrize("pitch", [0, 16])
@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("T,H", SHAPES)
def test_pre_norm(T, H, dt, pitch):
    rn = gen(T * 7 + H)
    x, gain = rows(rn, T, H, dt, pitch), 1 + 0.3 * rn(H)
    whole = torch.full((T, H + pitch), 7.0, dtype=BF, device="cuda")
    y, r = whole[:, pitch // 2:pitch // 2 + H], e(T)
    m.moe_pre_norm(x, gain, EPS, T, H, y, r)
    want, wr = ref.pre_norm(np64(x), np64(gain), EPS)
    near(r, wr, wr, "rstd")
    near(y, want, np.abs(want), "y")
    assert (whole[:, :pitch // 2] == 7).all() and (whole[:, pitch // 2 + H:] == 7).all()
    plain = e(T, H, dt=BF)
    m.moe_pre_norm(x, None, EPS, T, H, plain)
    near(plain, *[ref.pre_norm(np64(x), 1.0, EPS)[0]] * 2, "y without gain")


@pytest.mark.parametrize("pitch", [0, 16])
@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("T,H", SHAPES)
def test_pre_norm_bwd(T, H, dt, pitch):
    rn = gen(T * 5 + H)
    x, dy, dres, gain = rows(rn, T, H, dt, pitch), rows(rn, T, H, BF, pitch), rows(rn, T, H, dt, pitch), 1 + 0.3 * rn(H)
    r = torch.tensor(ref.rstd(np64(x), EPS), dtype=F32, device="cuda")
    whole = torch.full((T, H + pitch), 7.0, dtype=dt, device="cuda")
    dx, dgain = whole[:, pitch // 2:pitch // 2 + H], e(H).fill_(0.5)
    ws = torch.empty(max(16, m.moe_pre_norm_bwd_workspace_size(T, H)), dtype=torch.uint8, device="cuda")
    want = ref.pre_norm_bwd(np64(dy), np64(x), np64(gain), np64(r), np64(dres), 0.75)
    m.moe_pre_norm_bwd(dy, x, gain, r, dres, 0.75, T, H, dx, dgain, 0, ws)
    near(dx, want["dx"], want["dx_mag"], "dx")
    near(dgain, want["dgain"], want["dgain_mag"], "dgain", SUMS)
    assert (whole[:, :pitch // 2] == 7).all() and (whole[:, pitch // 2 + H:] == 7).all()
    first = dgain.clone()
    m.moe_pre_norm_bwd(dy, x, gain, r, dres, 0.75, T, H, dx, dgain, 1, ws)
    near(dgain, 2 * want["dgain"], 2 * want["dgain_mag"], "dgain, accumulated", SUMS)
    other, again = dres.clone(), e(H)
    m.moe_pre_norm_bwd(dy, x, gain, r, other, 0.75, T, H, other, again, 0, ws)  # dx over dres
    assert torch.equal(other, dx) and torch.equal(again, first)
    alone = e(T, H, dt=dt)
    m.moe_pre_norm_bwd(dy, x, None, r, None, 0.0, T, H, alone)  # no gain, no residual path, no gradient of the gain
    w = ref.pre_norm_bwd(np64(dy), np64(x), np.ones(H), np64(r), None, 0)
    near(alone, w["dx"], w["dx_mag"], "dx alone")


def gates(rn, kind, T, H):
    return {"none": None, "token": rn(T) * 3, "element": (rn(T, H) * 2).to(BF)}[kind]


@pytest.mark.parametrize("kind", ["none", "token", "element"])
@pytest.mark.parametrize("norm", [0, 1])
@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("T,H", [(1, 8), (33, 72), (70, 128), (31, 264), (40, 1032), (130, 2048), (3, 4104), (5, 8192)])
def test_post_norm(T, H, dt, norm, kind):
    rn = gen(T * 3 + H + norm)
    z, res, gain, ng = rows(rn, T, H, BF), rows(rn, T, H, dt), 1 + 0.3 * rn(H), 1 + 0.3 * rn(H)
    gate, dout = gates(rn, kind, T, H), rows(rn, T, H, dt)
    out, r, ny, nr = e(T, H, dt=dt), e(T), e(T, H, dt=BF), e(T)
    m.moe_post_norm(z, res, gain, norm, EPS, gate, 0.8, 0.5, T, H, out, r if norm else None, ng, ny, nr)
    want = ref.post_norm(np64(z), np64(res), np64(gain), norm, EPS, np64(gate), 0.8, 0.5)
    near(out, want["out"], want["out_mag"], "out")
    nxt, nwr = ref.pre_norm(np64(out), np64(ng), EPS)  # the next norm is of what is stored
    near(ny, nxt, np.abs(nxt), "next_y")
    near(nr, nwr, nwr, "next_rstd")
    if norm:
        near(r, want["rstd"], want["rstd"], "rstd")
    over = res.clone()
    m.moe_post_norm(z, over, gain, norm, EPS, gate, 0.8, 0.5, T, H, over)  # out over residual, nothing else asked for
    assert torch.equal(over, out)
    bare = e(T, H, dt=dt)
    m.moe_post_norm(z, None, None, norm, EPS, gate, 0.8, 0.5, T, H, bare)
    w = ref.post_norm(np64(z), None, 1.0, norm, EPS, np64(gate), 0.8, 0.5)
    near(bare, w["out"], w["out_mag"], "out alone")
    # backward
    dz, dgain, ws = e(T, H, dt=BF), e(H), torch.empty(max(16, m.moe_post_norm_bwd_workspace_size(T, H)), dtype=torch.uint8, device="cuda")
    dgate = None if gate is None else torch.empty_like(gate)
    b = ref.post_norm_bwd(np64(dout), np64(z), np64(gain), norm, np64(r), np64(gate), 0.5)
    m.moe_post_norm_bwd(dout, z, gain, norm, r if norm else None, gate, 0.5, T, H, dz, dgain, dgate, 0, ws)
    near(dz, b["dz"], b["dz_mag"], "dz")
    near(dgain, b["dgain"], b["dgain_mag"], "dgain", SUMS)
    if gate is not None:
        near(dgate, b["dgate"], b["dgate_mag"], "dgate")
    m.moe_post_norm_bwd(dout, z, gain, norm, r if norm else None, gate, 0.5, T, H, dz, dgain, None, 1, ws)
    near(dgain, 2 * b["dgain"], 2 * b["dgain_mag"], "dgain, accumulated", SUMS)
    over = z.clone()
    m.moe_post_norm_bwd(dout, over, gain, norm, r if norm else None, gate, 0.5, T, H, over)  # dz over z
    assert torch.equal(over, dz)


@pytest.mark.parametrize("kind", ["none", "token", "element"])
@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("T,H,k,norm", [(1, 64, 1, 1), (70, 128, 2, 1), (33, 320, 3, 0), (9, 576, 8, 1), (21, 1024, 12, 1), (1, 2048, 8, 1),
                                        (150, 2048, 8, 1), (17, 2112, 5, 1), (5, 4096, 9, 0), (3, 4160, 32, 1), (6, 8192, 2, 1)])
def test_combine_post_norm(T, H, k, norm, dt, kind):
    rn = gen(T * 11 + H + k)
    y, res, gain, ng, gate = rows(rn, T * k, H, BF), rows(rn, T, H, dt), 1 + 0.3 * rn(H), 1 + 0.3 * rn(H), gates(rn, kind, T, H)
    slot = torch.randperm(T * k, device="cuda").to(torch.int32).view(T, k)
    w = torch.softmax(rn(T, k), 1)
    z, out, r, ny, nr = e(T, H, dt=BF), e(T, H, dt=dt), e(T), e(T, H, dt=BF), e(T)
    m.moe_combine_post_norm(y, w, slot, res, gain, norm, EPS, gate, 0.8, 0.5, T, H, k, z, out, r if norm else None, ng, ny, nr)
    zw, zmag = ref.combine(np64(y), np64(w), slot.cpu().numpy())
    near(z, zw, zmag, "z")
    want = ref.post_norm(zw, np64(res), np64(gain), norm, EPS, np64(gate), 0.8, 0.5, zmag)
    near(out, want["out"], want["out_mag"], "out")
    if norm:
        # rstd goes by the squares: their errors are at most 2 k u of the terms' magnitudes times z
        near(r, want["rstd"], want["rstd"] * (1 + (zmag * np.abs(zw)).sum(1) / np.maximum((zw * zw).sum(1), 1e-30)), "rstd")
    nxt, nwr = ref.pre_norm(np64(out), np64(ng), EPS)
    near(ny, nxt, np.abs(nxt), "next_y")
    near(nr, nwr, nwr, "next_rstd")
    over = res.clone()
    m.moe_combine_post_norm(y, w, slot, over, gain, norm, EPS, gate, 0.8, 0.5, T, H, k, None, over)
    assert torch.equal(over, out)
    assert m.moe_read_device_status(reset=True) == 0
    bad = slot.clone()
    bad[0, 0] = T * k
    m.moe_combine_post_norm(y, w, bad, res, gain, norm, EPS, gate, 0.8, 0.5, T, H, k, z, out)
    assert m.moe_read_device_status(reset=True) == 1  # an index out of range is skipped and reported
    w0 = w.clone()
    w0[0, 0] = 0
    near(z[:1], *[v[:1] for v in ref.combine(np64(y), np64(w0), slot.cpu().numpy())], "z without the bad row")


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("H", [64, 128, 512, 2048, 8192])
def test_rows_at_the_ends_of_the_range(H, dt):
    """Zero rows, rows whose squares leave fp32, infinities and NaN: each row for itself."""
    rn = gen(H)
    T = 40
    x = rows(rn, T, H, F32)
    x[3] = 0
    x[5] *= 1e30  # squares beyond fp32
    x[7] = 3.0e38
    x[9] *= 1e-30
    x[11, H // 2] = float("inf")
    x[13, 0] = float("nan")
    x = x.to(dt)
    y, r = e(T, H, dt=BF), e(T)
    m.moe_pre_norm(x, None, EPS, T, H, y, r)
    fine = [t for t in range(T) if t not in (11, 13)]
    want, wr = ref.pre_norm(np64(x)[fine], 1.0, EPS)
    near(r[fine], wr, wr + 2.0 ** -133, "rstd")  # row 7's is below fp32's normal numbers: steps of 2^-149
    near(y[fine], want, np.abs(want), "y")
    assert (y[3] == 0).all() and torch.isnan(y[13]).all() and torch.isnan(y[11, H // 2])
    assert (y[11, :H // 2] == 0).all() and r[11] == 0
    ok = torch.tensor([t for t in fine if t not in (5, 7)], device="cuda")
    n = len(ok)
    dx, dg = e(T, H, dt=dt), e(H)
    ws = torch.empty(m.moe_pre_norm_bwd_workspace_size(T, H), dtype=torch.uint8, device="cuda")
    dy = rows(rn, T, H, BF)
    m.moe_pre_norm_bwd(dy, x, None, r, None, 0.0, T, H, dx)
    b = ref.pre_norm_bwd(np64(dy[ok]), np64(x[ok]), np.ones(H), np64(r[ok]), None, 0)
    near(dx[ok], b["dx"], b["dx_mag"], "dx")
    m.moe_pre_norm_bwd(dy[ok].contiguous(), x[ok].contiguous(), None, r[ok].contiguous(), None, 0.0, n, H, dx[:n], dg, 0, ws)
    near(dg, b["dgain"], b["dgain_mag"], "dgain", SUMS)


@pytest.mark.parametrize("logit", [0.0, 30.0, -30.0, 90.0, -90.0, float("inf"), float("-inf")])
def test_gates_at_the_ends_of_the_range(logit):
    T, H = 3, 64
    rn = gen(5)
    z, dout = rows(rn, T, H, BF), rows(rn, T, H, F32)
    for gate in (torch.full((T,), logit, device="cuda"), torch.full((T, H), logit, device="cuda", dtype=BF)):
        out, dz, dgate = e(T, H), e(T, H, dt=BF), torch.empty_like(gate)
        m.moe_post_norm(z, None, None, 0, EPS, gate, 0.0, 1.0, T, H, out)
        m.moe_post_norm_bwd(dout, z, None, 0, None, gate, 1.0, T, H, dz, None, dgate)
        g = np64(gate)
        with np.errstate(over="ignore", invalid="ignore"):
            o = ref.post_norm(np64(z), None, 1.0, 0, EPS, g, 0, 1)
            b = ref.post_norm_bwd(np64(dout), np64(z), np.ones(H), 0, None, g, 1)
        if not np.isfinite(logit):
            b["dgate"] = b["dgate_mag"] = np.zeros(g.shape)
        # below 2^-126 results are flushed or lose digits; e^-90 is 2^-130
        floor = 2.0 ** -120
        near(out, o["out"], o["out_mag"] + floor, "out", 2.0 ** -15)
        near(dz, b["dz"], b["dz_mag"] + floor, "dz", 2.0 ** -15)
        near(dgate, b["dgate"], b["dgate_mag"] + floor, "dgate", 2.0 ** -15)


def test_no_rows():
    dgain, ws = e(64).fill_(3.0), torch.empty(16, dtype=torch.uint8, device="cuda")
    x, r = e(0, 64, dt=BF), e(0)
    m.moe_pre_norm(x, None, EPS, 0, 64, x, r)
    m.moe_pre_norm_bwd(x, x, None, r, None, 0.0, 0, 64, x, dgain, 1, ws)
    assert (dgain == 3).all()
    m.moe_pre_norm_bwd(x, x, None, r, None, 0.0, 0, 64, x, dgain, 0, ws)
    assert (dgain == 0).all()
    dgain.fill_(3.0)
    m.moe_post_norm_bwd(x, x, None, 1, r, None, 1.0, 0, 64, x, dgain, None, 0, ws)
    assert (dgain == 0).all()


def test_more_than_2_31_elements():
    T, H = 300_000, 8192
    rn = gen(1)
    x = torch.empty(T, H, dtype=BF, device="cuda")
    x.view(-1)[:1 << 27] = rn(1 << 27).to(BF)
    for at in range(1 << 27, x.numel(), 1 << 27):
        x.view(-1)[at:at + (1 << 27)] = x.view(-1)[:min(1 << 27, x.numel() - at)]
    y, r = torch.empty_like(x), e(T)
    gain = 1 + 0.1 * rn(H)
    m.moe_pre_norm(x, gain, EPS, T, H, y, r)
    for at in (slice(0, 3), slice(T - 3, T)):
        want, wr = ref.pre_norm(np64(x[at]), np64(gain), EPS)
        near(y[at], want, np.abs(want), "y")
    dx = torch.empty_like(x)
    m.moe_pre_norm_bwd(y, x, gain, r, x, 1.0, T, H, dx)
    for at in (slice(0, 3), slice(T - 3, T)):
        b = ref.pre_norm_bwd(np64(y[at]), np64(x[at]), np64(gain), np64(r[at]), np64(x[at]), 1.0)
        near(dx[at], b["dx"], b["dx_mag"], "dx")


def test_streams_graphs_and_repeats():
    """The same bits on another stream, in two captured graphs that use one workspace in turn, and again."""
    T, H = 700, 2048
    rn = gen(9)
    x, dy, gain = rows(rn, T, H, BF), rows(rn, T, H, BF), 1 + 0.1 * rn(H)
    r, dx, dg = torch.rsqrt(x.float().square().mean(1) + EPS), e(T, H, dt=BF), e(H)
    ws = torch.empty(m.moe_pre_norm_bwd_workspace_size(T, H), dtype=torch.uint8, device="cuda")
    m.moe_pre_norm_bwd(dy, x, gain, r, x, 1.0, T, H, dx, dg, 0, ws)
    s = torch.cuda.Stream()
    dx2, dg2 = torch.empty_like(dx), torch.empty_like(dg)
    s.wait_stream(torch.cuda.current_stream())
    m.moe_pre_norm_bwd(dy, x, gain, r, x, 1.0, T, H, dx2, dg2, 0, ws, stream=s)
    s.synchronize()
    assert torch.equal(dx, dx2) and torch.equal(dg, dg2)
    graphs = []
    for out in ((dx, dg), (dx2, dg2)):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            m.moe_pre_norm_bwd(dy, x, gain, r, x, 1.0, T, H, out[0], out[1], 0, ws)
        graphs.append(g)
    want, wg = dx.clone(), dg.clone()
    for t in (dx, dg, dx2, dg2):
        t.zero_()
    for g in graphs * 2:
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(dx, want) and torch.equal(dx2, want) and torch.equal(dg, wg) and torch.equal(dg2, wg)
