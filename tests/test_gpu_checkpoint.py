"""Activations kept in 8 bits, and the experts' products that write and read
them, against plain restatements.

Codes and scales of bf16 rows, what they decode to, and permuted rows are exact.
A product of K terms in the tensor cores' fp32 accumulators is off by at most
K 2^-23 of the magnitudes (K <= 512 here: 2^-14); the SwiGLU's exponential and
division add less than 2^-17.  A bf16 output is off by half a step more (2^-8).
"""
import numpy as np
import pytest
import torch

import block_ref as ref
import moe_expert_layer_topk_gb300 as m

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
DOT = 2.0 ** -14


def e(*s, dt=F32):
    return torch.empty(*s, dtype=dt, device="cuda")


def np64(t):
    return t.detach().double().cpu().numpy()


def gen(seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return lambda *s: torch.randn(*s, generator=g, device="cuda")


def near(got, want, mag, what):
    got, half = np64(got), {BF: 2.0 ** -8, F32: 2.0 ** -24}[got.dtype]
    bound = half * np.abs(want) + DOT * mag + 1e-37
    bad = ~(np.abs(got - want) <= bound)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size}, worst {np.nanmax(np.abs(got - want) / bound):.3g} of the bound"


def packed(x):
    q, s = e(*x.shape, dt=torch.int8), e(x.shape[0], x.shape[1] // 32, dt=BF)
    m.moe_ckpt_pack(x, x.shape[0], x.shape[1], q, s)
    return q, s


@pytest.mark.parametrize("rows,cols", [(1, 32), (3, 96), (17, 64), (1, 2048), (333, 544), (70, 2048), (5, 8192)])
def test_pack_and_unpack(rows, cols):
    rn = gen(rows + cols)
    x = rn(rows, cols) * torch.exp(4 * rn(rows, 1))
    x[0, :32] = 0
    x[-1, -1] = 3.0e38
    x[rows // 2, :8] = torch.tensor([127.0, 63.5, -2.5, 1.5, 0.5, -0.5, 1e-40, -0.0], device="cuda")
    x = x.to(BF)
    q, s = packed(x)
    wq, wscale = ref.pack(x.float().cpu().numpy())
    assert np.array_equal(s.float().cpu().numpy(), wscale) and np.array_equal(q.cpu().numpy(), wq)
    a = e(rows, cols, dt=BF)
    m.moe_ckpt_unpack(q, s, rows, cols, a)
    assert torch.equal(a.cpu(), torch.from_numpy(ref.unpack(wq, wscale)).to(BF))
    # what comes back is off by half a scale, and half a step of bf16
    half = 0.5 * s.double().repeat_interleave(32, 1) * (1 + 2.0 ** -15)
    assert ((a.double() - x.double()).abs() <= half + 2.0 ** -8 * a.double().abs()).all()


def test_tiny_infinite_and_nan_groups():
    x = torch.zeros(2, 160, dtype=BF, device="cuda")
    x[:, :32] = 1e-39  # scales no smaller than 2^-126
    x[0, 32 + 5] = float("inf")
    x[1, 64 + 5] = float("-inf")
    x[0, 96 + 31] = float("nan")
    x[1, 128:] = 1.0
    q, s = packed(x)
    a = e(2, 160, dt=BF)
    m.moe_ckpt_unpack(q, s, 2, 160, a)
    assert (a[:, :32].float().abs() <= 2.0 ** -126).all()
    bad = torch.isnan(a)
    assert bad[0, 32:64].all() and bad[1, 64:96].all() and bad[0, 96:128].all() and bad.sum() == 96
    wq, ws = ref.pack(np.ones((1, 32), np.float32))  # s = 1/127 rounded up, 0.0079346: code 126
    assert (q[1, 128:].cpu().numpy() == wq).all() and wq[0, 0] == 126 and (a[1, 128:] == 1).all()


def test_the_largest_values_stay_finite():
    top = torch.tensor([252.0, 253.0, 254.0, 255.0], device="cuda") * 2.0 ** 120  # 255 * 2^120: bf16's largest
    x = (top[:, None] * torch.linspace(-1, 1, 64, device="cuda")).to(BF)
    assert x[3, 63] == torch.finfo(BF).max
    q, s = packed(x)
    wq, ws = ref.pack(x.float().cpu().numpy())
    assert np.array_equal(s.float().cpu().numpy(), ws) and np.array_equal(q.cpu().numpy(), wq)
    a, xp = e(4, 64, dt=BF), e(4, 64, dt=BF)
    m.moe_ckpt_unpack(q, s, 4, 64, a)
    m.moe_dispatch_rows(q, s, torch.arange(4, dtype=torch.int32, device="cuda").view(4, 1), None, 4, 64, 1, xp, None)
    half = 0.5 * s.double().repeat_interleave(32, 1) * (1 + 2.0 ** -15)
    assert torch.isfinite(a).all() and torch.equal(a, xp)
    assert ((a.double() - x.double()).abs() <= half + 2.0 ** -8 * a.double().abs()).all()


@pytest.mark.parametrize("weights", [True, False])
@pytest.mark.parametrize("codes", [True, False])
@pytest.mark.parametrize("T,H,k", [(1, 64, 1), (5, 128, 3), (300, 2048, 8), (33, 576, 32), (1, 2048, 8)])
def test_dispatch_rows(T, H, k, codes, weights):
    rn = gen(T + H + k)
    x, w = rn(T, H).to(BF), torch.rand(T, k, device="cuda")
    slot = torch.randperm(T * k, device="cuda").to(torch.int32).view(T, k)
    src, scale, val = x, None, x
    if codes:
        src, scale = packed(x)
        val = e(T, H, dt=BF)
        m.moe_ckpt_unpack(src, scale, T, H, val)
    xp, rw = e(T * k + 1, H, dt=BF).fill_(5.0), e(T * k + 1).fill_(5.0)
    m.moe_dispatch_rows(src, scale, slot, w if weights else None, T, H, k, xp, rw if weights else None)
    want = torch.empty(T * k, H, dtype=BF, device="cuda")
    want[slot.view(-1).long()] = val.repeat_interleave(k, 0)
    assert torch.equal(xp[:-1], want) and (xp[-1] == 5).all()
    if weights:
        assert torch.equal(rw[slot.long()], w) and rw[-1] == 5
    assert m.moe_read_device_status(reset=True) == 0
    slot[0, 0], missed = T * k, int(slot[0, 0])
    xp.fill_(5.0)
    m.moe_dispatch_rows(src, scale, slot, w if weights else None, T, H, k, xp, rw if weights else None)
    assert m.moe_read_device_status(reset=True) == 1 and (xp[missed] == 5).all() and (xp[-1] == 5).all()


def table(kind, R, E):
    """num_seg, offsets, seg_expert: the dispatch's layout with an empty expert; blocks of source ranks with empty
    ones, experts out of order, and rows before, between and behind the segments."""
    rng = np.random.default_rng(R + E)
    if kind == "experts":
        c = rng.multinomial(R, np.where(np.arange(E) == 1, 0, 1.0) / max(1, E - 1)) if E > 1 else np.array([R])
        off = np.concatenate([[0], np.cumsum(c)])
        return E, off, None
    if kind == "tails":  # segments of 512 rows and these
        return E, np.concatenate([[0], np.cumsum(512 + np.array(TAILS))]), None
    if kind == "ranks":  # 8 ranks' blocks of each expert: 48, 24 and 320 segments, some of an expert that is not there
        cut = np.sort(np.concatenate([[0, R], rng.integers(0, R, 8 * E - 1)]))
        se = np.tile(np.arange(E), 8)
        return 8 * E, cut, se
    cut = np.sort(rng.integers(R // 10, R - R // 10, 2 * E + 1))
    cut[3] = cut[2]
    return 2 * E, cut, np.concatenate([np.arange(E)[::-1], rng.permutation(E)])


TAILS = (1, 32, 63, 64, 65, 96, 128, 129, 255, 256)
CASES = [("experts", 7, 64, 64, 2), ("experts", 300, 128, 64, 8), ("experts", 700, 512, 320, 4), ("experts", 2500, 256, 128, 3),
         ("experts", 2600, 128, 256, 5), ("experts", 900, 64, 512, 2),
         ("ranks", 3000, 128, 256, 6), ("ranks", 40, 64, 64, 3), ("ranks", 2000, 64, 64, 40), ("ranks", 5000, 64, 1024, 30),
         ("experts", 129, 64, 192, 1), ("blocks", 400, 128, 128, 3), ("blocks", 1000, 256, 768, 5),
         ("tails", 6209, 128, 128, 10), ("tails", 6209, 64, 256, 10), ("tails", 6209, 64, 768, 10)]


def on_few_sms(call, n=3):
    """On few SMs, tiles come in many rounds, and several segments an expert in tiles of pieces."""
    prev = m.moe_set_gemm_sm_limit(n)
    try:
        call()
    finally:
        m.moe_set_gemm_sm_limit(prev)


def inputs(kind, R, H, I, E):
    rn = gen(R + H + I)
    n, off, se = table(kind, R, E)
    d = dict(n=n, off=off, se=se, segs=ref.experts(off, se), o=torch.tensor(off, dtype=torch.int32, device="cuda"),
             s=None if se is None else torch.tensor(se, dtype=torch.int32, device="cuda"))
    d["x"], d["dy"] = rn(R, H).to(BF), rn(R, H).to(BF)
    d["Wg"], d["Wu"], d["Wd"] = (rn(E, I, H) * H ** -0.5).to(BF), (rn(E, I, H) * H ** -0.5).to(BF), (rn(E, H, I) * H ** -0.5).to(BF)
    d["w"] = torch.rand(R, device="cuda")
    d["live"] = np.zeros(R, bool)
    for _, a, b in d["segs"]:
        d["live"][a:b] = True
    return d


@pytest.mark.parametrize("kind,R,H,I,E", CASES)
def test_swiglu_ckpt(kind, R, H, I, E):
    d = inputs(kind, R, H, I, E)
    h, h0, gu0 = (e(R, I, dt=BF).fill_(9.0), e(R, I, dt=BF).fill_(9.0), e(R, 2 * I, dt=BF).fill_(9.0))
    q, s = torch.full((R, 2 * I), 77, dtype=torch.int8, device="cuda"), e(R, 2 * I // 32, dt=BF).fill_(9.0)
    m.moe_grouped_gemm_swiglu(d["x"], d["Wg"], d["Wu"], d["n"], d["o"], d["s"], R, H, I, E, h0, gu0)
    m.moe_grouped_gemm_swiglu_ckpt(d["x"], d["Wg"], d["Wu"], d["n"], d["o"], d["s"], R, H, I, E, h, q, s)
    assert torch.equal(h, h0)  # the product and h are the same
    few = torch.empty_like(h).fill_(9.0), torch.full_like(q, 77), torch.empty_like(s).fill_(9.0)
    on_few_sms(lambda: m.moe_grouped_gemm_swiglu_ckpt(d["x"], d["Wg"], d["Wu"], d["n"], d["o"], d["s"], R, H, I, E, *few))
    assert torch.equal(h, few[0]) and torch.equal(q, few[1]) and torch.equal(s, few[2])
    dead = torch.tensor(~d["live"], device="cuda")
    assert (q[dead] == 77).all() and (s[dead] == 9).all()
    g, u, mag = ref.gate_up(np64(d["x"]), np64(d["Wg"]), np64(d["Wu"]), d["segs"])
    live = d["live"]
    want, off = np.concatenate([g, u], 1)[live], (DOT * np.concatenate([mag, mag], 1) + 1e-37)[live]
    sc = s.double().cpu().numpy()[live]
    top = np.abs(want).reshape(len(want), -1, 32).max(2)
    slack = off.reshape(len(want), -1, 32).max(2)
    assert (sc >= (top - slack) / 127 * (1 - 2.0 ** -20)).all()
    assert (sc <= (top + slack) / 127 * (1 + 2.0 ** -7) + 2.0 ** -126).all()  # the next bf16 number at most
    err = np.abs(ref.unpack(q.cpu().numpy()[live], sc) - want)
    assert (err <= np.repeat(sc, 32, 1) * (0.5 + 2.0 ** -16) + off).all()
    # and the codes are those of the product's own values where bf16 holds them: within one code of gu0's
    a = e(R, 2 * I, dt=BF)
    m.moe_ckpt_unpack(q, s, R, 2 * I, a)
    far = (a[~dead].double() - gu0[~dead].double()).abs()
    assert (far <= s[~dead].double().repeat_interleave(32, 1) * 0.51 + 2.0 ** -7 * gu0[~dead].double().abs()).all()


@pytest.mark.parametrize("weighted", [True, False])
@pytest.mark.parametrize("kind,R,H,I,E", CASES)
def test_down_bwd_ckpt(kind, R, H, I, E, weighted):
    d = inputs(kind, R, H, I, E)
    rn = gen(R)
    wq, wscale = ref.pack(rn(R, 2 * I).cpu().numpy())
    q, s = torch.tensor(wq, device="cuda"), torch.tensor(wscale, device="cuda").to(BF)
    dec = ref.unpack(wq, wscale)
    w = d["w"] if weighted else None
    b = ref.down_bwd(np64(d["dy"]), None if w is None else np64(w), dec[:, :I], dec[:, I:], np64(d["Wd"]), d["segs"])
    ws = torch.full((m.moe_grouped_gemm_down_bwd_ckpt_workspace_size(R, I),), 0xFF, dtype=torch.uint8, device="cuda")
    dgu, hw, dw = e(R, 2 * I, dt=BF).fill_(9.0), e(R, I, dt=BF).fill_(9.0), e(R).fill_(9.0)
    args = (d["dy"], w, q, s, d["Wd"], d["n"], d["o"], d["s"], R, H, I, E)
    m.moe_grouped_gemm_down_bwd_ckpt(*args, dgu, hw, dw, ws=ws)
    live, dead = d["live"], torch.tensor(~d["live"], device="cuda")
    near(dgu[~dead], b["dgu"][live], b["dgu_mag"][live], "dgu")
    near(hw[~dead], b["h_w"][live], np.abs(b["h_w"][live]), "h_w")
    near(dw, b["d_w"], b["d_w_mag"], "d_w")
    assert (dgu[dead] == 9).all() and (hw[dead] == 9).all() and (dw[dead] == 0).all()
    few = torch.empty_like(dgu).fill_(9.0), torch.empty_like(hw).fill_(9.0), e(R).fill_(9.0)
    ws.fill_(0xFF)
    on_few_sms(lambda: m.moe_grouped_gemm_down_bwd_ckpt(*args, *few, ws=ws))
    assert all(torch.equal(a, b) for a, b in zip((dgu, hw, dw), few))
    k = 2
    slot = torch.randperm(R, device="cuda")[:R // k * k].to(torch.int32).view(-1, k)
    dgu2, hw2, dwt = torch.empty_like(dgu).fill_(9.0), torch.empty_like(hw).fill_(9.0), e(R // k, k)
    m.moe_grouped_gemm_down_bwd_ckpt(*args, dgu2, hw2, dwt, slot, R // k, k, ws)
    assert torch.equal(dwt, dw[slot.long()]) and torch.equal(dgu, dgu2) and torch.equal(hw, hw2)
    assert m.moe_read_device_status(reset=True) == 0
    if slot.numel():
        slot[0, 0] = -1
        m.moe_grouped_gemm_down_bwd_ckpt(*args, dgu2, hw2, dwt, slot, R // k, k, ws)
        assert dwt[0, 0] == 0 and m.moe_read_device_status(reset=True) == 1


@pytest.mark.parametrize("sms", [0, 2])
def test_segments_of_no_expert(sms):
    """Rows of a segment whose expert is out of range are skipped and reported, by tiles and by pieces of tiles."""
    R, H, I, E, n = 900, 64, 128, 4, 12
    rn = gen(1)
    dy, Wd, w = rn(R, H).to(BF), (rn(E, H, I) * 0.1).to(BF), torch.rand(R, device="cuda")
    q, s = packed(rn(R, 2 * I).to(BF))
    off = np.linspace(0, R, n + 1).astype(np.int64)
    se = np.array([0, 1, 2, 3, -1, 3, 2, 4, 0, 1, 1, 1000])
    dec = ref.unpack(q.cpu().numpy(), s.float().cpu().numpy())
    b = ref.down_bwd(np64(dy), np64(w), dec[:, :I], dec[:, I:], np64(Wd), ref.experts(off, se))
    live = np.repeat((se >= 0) & (se < E), np.diff(off))
    ws = torch.full((m.moe_grouped_gemm_down_bwd_ckpt_workspace_size(R, I),), 0xFF, dtype=torch.uint8, device="cuda")
    dgu, hw, dw = e(R, 2 * I, dt=BF).fill_(9.0), e(R, I, dt=BF).fill_(9.0), e(R).fill_(9.0)
    o, t = torch.tensor(off, dtype=torch.int32, device="cuda"), torch.tensor(se, dtype=torch.int32, device="cuda")
    m.moe_read_device_status(reset=True)
    on_few_sms(lambda: m.moe_grouped_gemm_down_bwd_ckpt(dy, w, q, s, Wd, n, o, t, R, H, I, E, dgu, hw, dw, ws=ws), sms)
    assert m.moe_read_device_status(reset=True) == 2
    dead = torch.tensor(~live, device="cuda")
    near(dgu[~dead], b["dgu"][live], b["dgu_mag"][live], "dgu")
    near(hw[~dead], b["h_w"][live], np.abs(b["h_w"][live]), "h_w")
    near(dw, b["d_w"], b["d_w_mag"], "d_w")
    assert (dgu[dead] == 9).all() and (hw[dead] == 9).all() and (dw[dead] == 0).all()


def test_no_rows_or_segments():
    R, H, I, E = 5, 64, 64, 2
    x, W, h = e(R, H, dt=BF), e(E, I, H, dt=BF), e(R, I, dt=BF).fill_(9.0)
    q, s, off = torch.full((R, 2 * I), 7, dtype=torch.int8, device="cuda"), e(R, 4, dt=BF).fill_(9.0), torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    ws, dw, dgu = torch.empty(m.moe_grouped_gemm_down_bwd_ckpt_workspace_size(R, I), dtype=torch.uint8, device="cuda"), e(R).fill_(9.0), e(R, 2 * I, dt=BF).fill_(9.0)
    m.moe_grouped_gemm_down_bwd_ckpt(x, None, q, s, W, 0, None, None, R, H, I, E, dgu, h, dw, ws=ws)
    assert (dw == 0).all()
    dw.fill_(9.0)
    for n in (0, E):  # no segment, and empty ones
        m.moe_grouped_gemm_swiglu_ckpt(x, W, W, n, off, None, R, H, I, E, h, q, s)
        m.moe_grouped_gemm_down_bwd_ckpt(x, None, q, s, W, n, off, None, R, H, I, E, dgu, h, dw, ws=ws)
        assert (h == 9).all() and (q == 7).all() and (s == 9).all() and (dgu == 9).all() and (dw == 0).all()
        dw.fill_(9.0)


def test_streams_and_graphs():
    """Another stream, a captured graph and a grid of fewer SMs give the same bits."""
    R, H, I, E = 1500, 256, 256, 4
    d = inputs("experts", R, H, I, E)
    q, s = packed(gen(3)(R, 2 * I).to(BF))
    ws = torch.empty(m.moe_grouped_gemm_down_bwd_ckpt_workspace_size(R, I), dtype=torch.uint8, device="cuda")
    outs = [(e(R, 2 * I, dt=BF), e(R, I, dt=BF), e(R)) for _ in range(3)]

    def call(o, stream=None):
        m.moe_grouped_gemm_down_bwd_ckpt(d["dy"], d["w"], q, s, d["Wd"], E, d["o"], None, R, H, I, E, *o, ws=ws, stream=stream)
    call(outs[0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    prev = m.moe_set_gemm_sm_limit(7)
    try:
        call(outs[1], side)
    finally:
        m.moe_set_gemm_sm_limit(prev)
    side.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(outs[2])
    for t in outs[2]:
        t.zero_()
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    for o in outs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(o, outs[0]))


def test_more_than_2_31_elements():
    rows, cols = 1_100_000, 2048
    x = torch.zeros(rows, cols, dtype=BF, device="cuda")
    x[-2:] = gen(4)(2, cols).to(BF)
    q, s = packed(x)
    a = torch.empty_like(x)
    m.moe_ckpt_unpack(q, s, rows, cols, a)
    wq, wscale = ref.pack(x[-2:].float().cpu().numpy())
    assert np.array_equal(q[-2:].cpu().numpy(), wq) and (a[0] == 0).all()
    assert torch.equal(a[-2:].cpu(), torch.from_numpy(ref.unpack(wq, wscale)).to(BF))
    T = 300_000
    slot = torch.arange(T, dtype=torch.int32, device="cuda").flip(0).view(T, 1)
    out = torch.empty(T, 8192, dtype=BF, device="cuda")
    big = torch.zeros(T, 8192, dtype=BF, device="cuda")
    big[0], big[-1] = 1.0, 2.0
    m.moe_dispatch_rows(big, None, slot, None, T, 8192, 1, out)
    assert (out[-1] == 1).all() and (out[0] == 2).all() and (out[1] == 0).all()
