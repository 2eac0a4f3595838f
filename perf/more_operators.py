"""Cases, plain forms and exact values of the norms around a block and of activations kept in 8 bits.

Four operators, each reached through the package's entry points of the same names:

  pre     moe_pre_norm, moe_pre_norm_bwd: the norm before a block; its backward adds the residual path's gradient
  post    moe_post_norm, moe_combine_post_norm, moe_post_norm_bwd: the norm after a block with its gate, the
          residual and both scales, alone or on the weighted combine of the experts' rows, and the next norm
  rows    moe_ckpt_pack, moe_ckpt_unpack, moe_dispatch_rows: rows kept in 8 bits, and brought back, in order or
          permuted for the experts
  mlp     moe_grouped_gemm_swiglu_ckpt, moe_grouped_gemm_down_bwd_ckpt: the experts' gate/up product that keeps
          its g and u in 8 bits, and the backward through them

`run` computes the plain form (elementary torch operations in fp32, rounded once) unless `own` is
set, and then calls the package.  Formulas are stated at each plain form.
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

EPS = 1e-6
GROUP = 32  # columns that share a scale
A, B = 1.0, 0.5  # scales of the residual and of the block's output


# ------------------------------------------------------------------- the cases

def listed():
    return [
        # serving: the norm before the layer of a single token
        dict(name="pre_norm_token", op="pre", dir="fwd", T=1, H=2048, fp32=0, pitch=0),
        # norm of rows of 128 inside a wider buffer, an odd number of them
        dict(name="pre_norm_slices", op="pre", dir="fwd", T=65521, H=128, fp32=0, pitch=64),
        # one training step of the T=8192 layer: the norm's backward with the residual path's gradient
        dict(name="pre_norm_bwd", op="pre", dir="bwd", T=8192, H=2048, fp32=0, pitch=0),
        # serving: the end of the block for a single token, with the next block's norm
        dict(name="combine_norm_token", op="post", dir="combine", T=1, H=2048, k=8, fp32=0, gate="token", norm=1, next=1),
        # the end of the T=8192 training layer's block, gated by token, with the next block's norm
        dict(name="combine_norm_step", op="post", dir="combine", T=8192, H=2048, k=8, fp32=0, gate="token", norm=1, next=1),
        # backward of an element-gated block at an odd token count, residual stream in fp32
        dict(name="post_norm_bwd", op="post", dir="bwd", T=8191, H=2048, k=0, fp32=1, gate="element", norm=1, next=0),
        # a layer's input kept in 8 bits, and brought back
        dict(name="checkpoint_round_trip", op="rows", dir="round", T=8192, H=2048, k=0),
        # the experts' rows made again in the backward from tokens kept in 8 bits
        dict(name="checkpoint_dispatch", op="rows", dir="dispatch", T=8192, H=2048, k=8),
        # the smallest layer's gate/up product
        dict(name="swiglu_tiny", op="mlp", dir="fwd", T=256, H=128, I=64, E=8, k=2, ranks=1),
        # one training step of the T=8192 layer: forward and backward
        dict(name="swiglu_step", op="mlp", dir="fwd", T=8192, H=2048, I=768, E=128, k=8, ranks=1),
        dict(name="down_bwd_step", op="mlp", dir="bwd", T=8192, H=2048, I=768, E=128, k=8, ranks=1),
        # one expert-parallel rank: rows from 8 ranks for 16 experts, odd pieces
        dict(name="down_bwd_received", op="mlp", dir="bwd", T=16381, H=2048, I=768, E=16, k=1, ranks=8),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], even over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["pre", "post", "post", "rows", "mlp", "mlp"])
    if op == "pre":
        H = 8 * rng.choice([8, 16, 256, _spread(rng, 1, 512)])
        return dict(op=op, dir=rng.choice(["fwd", "bwd"]), T=_spread(rng, 1, max(1, 8192 * 2048 // max(H, 256))), H=H, fp32=rng.choice([0, 0, 1]),
                    pitch=rng.choice([0, 0, 64]))
    if op == "post":
        way = rng.choice(["combine", "fwd", "bwd"])
        H = 64 * rng.choice([2, 12, 32, _spread(rng, 1, 64)])
        return dict(op=op, dir=way, T=_spread(rng, 1, max(1, 8192 * 2048 // max(H, 2048))), H=H, k=rng.randint(1, 8) if way == "combine" else 0,
                    fp32=rng.choice([0, 0, 1]), gate=rng.choice(["none", "token", "element"]), norm=rng.choice([1, 1, 0]),
                    next=rng.choice([0, 1]) if way != "bwd" else 0)
    if op == "rows":
        way = rng.choice(["round", "dispatch", "copy"])
        H = 64 * rng.choice([2, 32, _spread(rng, 1, 32)])
        return dict(op=op, dir=way, T=_spread(rng, 1, 8192), H=H, k=rng.randint(1, 8) if way != "round" else 0)
    H, I = 64 * rng.choice([2, 32, _spread(rng, 1, 32)]), 64 * rng.choice([1, 12, _spread(rng, 1, 12)])
    E = rng.choice([8, 16, 64, 128, _spread(rng, 1, 128)])
    ranks = rng.choice([1, 1, 4])
    k = 1 if ranks > 1 else rng.randint(1, min(8, E))
    return dict(op=op, dir=rng.choice(["fwd", "bwd"]), T=_spread(rng, 1, 8192), H=H, I=I, E=min(E, 32) if ranks > 1 else E, k=k, ranks=ranks)


# ------------------------------------------------------------------ the inputs

def _segments(case):
    """Row counts of the (source rank, expert) blocks, by the sizes alone: popular and rare experts, one of them
    without a row where there are several.  Without ranks a token picks an expert at most once."""
    T, E, k, ranks = case["T"], case["E"], case["k"], case["ranks"]
    rng = np.random.default_rng(1000003 * T + 1009 * E + k)
    p = np.exp(0.5 * rng.standard_normal(E))
    if E > k + 1:
        p[rng.integers(E)] = 0.0
    if k == 1:
        pieces = [T // ranks + (r < T % ranks) for r in range(ranks)]
        return np.concatenate([rng.multinomial(n, p / p.sum()) for n in pieces])
    c = np.floor(p / p.sum() * T * k).astype(np.int64).clip(max=T)
    while c.sum() < T * k:  # the rest, to the experts that can take more
        more = np.flatnonzero((c < T) & ((p > 0) | (c.sum() + T > T * k)))
        c[more[rng.integers(len(more))]] += 1
    return c


def _experts(case, seed):
    """Rows, weights and tables of the experts' products."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    T, H, I, E, k, ranks = (case[n] for n in ("T", "H", "I", "E", "k", "ranks"))
    counts, R = _segments(case), T * k
    d = dict(cap=int(counts.max()), offsets=torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device="cuda"))
    d["seg_expert"] = torch.arange(E, dtype=torch.int32, device="cuda").repeat(ranks) if ranks > 1 else None
    if case["dir"] == "fwd":
        d["x_perm"] = rn(R, H).bfloat16()
        d["Wg"], d["Wu"] = ((torch.randn(E, I, H, generator=g, device="cuda", dtype=torch.bfloat16) * 0.02) for _ in range(2))
        return d
    d["dy_perm"] = rn(R, H).bfloat16()
    d["Wd"] = torch.randn(E, H, I, generator=g, device="cuda", dtype=torch.bfloat16) * 0.02
    d["row_w"] = torch.rand(R, generator=g, device="cuda")
    d["gu_q"], d["gu_scale"] = _encode(rn(R, 2 * I) * (0.02 * math.sqrt(H)))
    # rows of the (token, slot) pairs: any order of the rows will do; a rank gets its rows' sums in row order
    d["row_of_slot"] = torch.randperm(R, generator=g, device="cuda").to(torch.int32).view(T, k) if ranks == 1 else None
    return d


def _inputs(case, seed):
    if case["op"] == "mlp":
        return _experts(case, seed)
    g = torch.Generator(device="cuda").manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    T, H = case["T"], case["H"]
    d = {}
    if case["op"] == "rows":
        x = rn(T, H) * torch.exp(0.5 * rn(H))
        if H >= 256:
            x[:, torch.randint(0, H, (3,), generator=g, device="cuda")] *= 20.0  # the few large channels of a residual stream
        x = x.bfloat16()
        if case["dir"] == "round":
            return dict(x=x)
        d["x"], d["scale"] = (x, None) if case["dir"] == "copy" else _encode(x.float())
        d["row_of_slot"] = torch.randperm(T * case["k"], generator=g, device="cuda").to(torch.int32).view(T, -1)
        d["topk_w"] = torch.rand(T, case["k"], generator=g, device="cuda")
        return d
    stream = torch.float32 if case["fp32"] else torch.bfloat16
    d["gain"] = 1.0 + 0.2 * rn(H)
    if case["op"] == "pre":
        rows = lambda dt: (rn(T, H + case["pitch"]) * torch.exp(0.3 * rn(H + case["pitch"]))).to(dt)[:, case["pitch"] // 2:case["pitch"] // 2 + H]  # noqa: E731
        d["x"] = rows(stream)
        if case["dir"] == "bwd":
            d["dy"], d["dres"] = rows(torch.bfloat16), rows(stream)
            d["rstd"] = torch.rsqrt(d["x"].double().square().mean(1) + EPS).float()
        return d
    d["gate"] = {"none": lambda: None, "token": lambda: rn(T), "element": lambda: rn(T, H).bfloat16()}[case["gate"]]()
    if case["dir"] == "combine":
        k = case["k"]
        d["y_perm"] = (torch.randn(T * k, H, generator=g, device="cuda", dtype=torch.bfloat16) * 0.3)
        d["row_of_slot"] = torch.randperm(T * k, generator=g, device="cuda").to(torch.int32).view(T, k)
        w = torch.exp(rn(T, k))
        d["topk_w"] = (w / w.sum(1, keepdim=True)).contiguous()
    else:
        d["z"] = (rn(T, H) * 0.2).bfloat16()
    if case["dir"] == "bwd":
        d["dout"] = rn(T, H).to(stream)
        d["rstd"] = torch.rsqrt(d["z"].double().square().mean(1) + EPS).float()
    else:
        d["residual"] = rn(T, H).to(stream)
        d["next_gain"] = 1.0 + 0.2 * rn(H) if case["next"] else None
    return d


def prepare(case, seed):
    state = dict(case=case, **_inputs(case, seed))
    if own:
        state["buf"] = _buffers(case)
    return state


def run(state):
    op = state["case"]["op"]
    if own:
        return {"pre": _own_pre, "post": _own_post, "rows": _own_rows, "mlp": _own_mlp}[op](state)
    return {"pre": _plain_pre, "post": _plain_post, "rows": _plain_rows, "mlp": _plain_mlp}[op](state)


# ------------------------------------------------- the framework's own kernels

def _buffers(case):
    """The output tensors and workspaces that a training or serving program keeps."""
    import moe_expert_layer_topk_gb300 as m
    e = lambda *s, dt=torch.float32: torch.empty(*s, dtype=dt, device="cuda")  # noqa: E731
    bf, u8, i8 = torch.bfloat16, torch.uint8, torch.int8
    T, H = case["T"], case["H"]
    stream = torch.float32 if case.get("fp32") else bf
    if case["op"] == "pre":
        if case["dir"] == "fwd":
            return dict(y=e(T, H, dt=bf), rstd=e(T))
        return dict(dx=e(T, H, dt=stream), dgain=e(H), ws=e(max(256, m.moe_pre_norm_bwd_workspace_size(T, H)), dt=u8))
    if case["op"] == "post":
        if case["dir"] == "bwd":
            b = dict(dz=e(T, H, dt=bf), dgain=e(H), ws=e(max(256, m.moe_post_norm_bwd_workspace_size(T, H)), dt=u8))
            b["dgate"] = {"none": None, "token": e(T), "element": e(T, H, dt=bf)}[case["gate"]]
            return b
        b = dict(out=e(T, H, dt=stream), rstd=e(T) if case["norm"] else None, z=e(T, H, dt=bf) if case["dir"] == "combine" else None)
        b["next_y"], b["next_rstd"] = (e(T, H, dt=bf), e(T)) if case["next"] else (None, None)
        return b
    if case["op"] == "rows":
        if case["dir"] == "round":
            return dict(q=e(T, H, dt=i8), scale=e(T, H // GROUP, dt=bf), a=e(T, H, dt=bf))
        return dict(x_perm=e(T * case["k"], H, dt=bf), row_w=e(T * case["k"]))
    R, I = T * case["k"], case["I"]
    if case["dir"] == "fwd":
        return dict(h=e(R, I, dt=bf), gu_q=e(R, 2 * I, dt=i8), gu_scale=e(R, 2 * I // GROUP, dt=bf), gu=e(R, 2 * I, dt=bf))
    return dict(dgu=e(R, 2 * I, dt=bf), h_w=e(R, I, dt=bf), d_w=e(T, case["k"]) if case["ranks"] == 1 else e(R),
                ws=e(max(256, m.moe_grouped_gemm_down_bwd_ckpt_workspace_size(R, I)), dt=u8))


def _own_pre(s):
    import moe_expert_layer_topk_gb300 as m
    c, b = s["case"], s["buf"]
    if c["dir"] == "fwd":
        m.moe_pre_norm(s["x"], s["gain"], EPS, c["T"], c["H"], b["y"], b["rstd"])
        return b["y"], b["rstd"]
    m.moe_pre_norm_bwd(s["dy"], s["x"], s["gain"], s["rstd"], s["dres"], A, c["T"], c["H"], b["dx"], b["dgain"], 0, b["ws"])
    return b["dx"], b["dgain"]


def _own_post(s):
    import moe_expert_layer_topk_gb300 as m
    c, b = s["case"], s["buf"]
    T, H = c["T"], c["H"]
    if c["dir"] == "bwd":
        m.moe_post_norm_bwd(s["dout"], s["z"], s["gain"], c["norm"], s["rstd"], s["gate"], B, T, H, b["dz"], b["dgain"], b["dgate"], 0, b["ws"])
        return {n: b[n] for n in ("dz", "dgain", "dgate")}
    if c["dir"] == "combine":
        m.moe_combine_post_norm(s["y_perm"], s["topk_w"], s["row_of_slot"], s["residual"], s["gain"], c["norm"], EPS, s["gate"], A, B, T, H, c["k"],
                                b["z"], b["out"], b["rstd"], s["next_gain"], b["next_y"], b["next_rstd"])
    else:
        m.moe_post_norm(s["z"], s["residual"], s["gain"], c["norm"], EPS, s["gate"], A, B, T, H, b["out"], b["rstd"], s["next_gain"], b["next_y"],
                        b["next_rstd"])
    return {n: b[n] for n in ("out", "rstd", "z", "next_y", "next_rstd")}


def _own_rows(s):
    import moe_expert_layer_topk_gb300 as m
    c, b = s["case"], s["buf"]
    T, H = c["T"], c["H"]
    if c["dir"] == "round":
        m.moe_ckpt_pack(s["x"], T, H, b["q"], b["scale"])
        m.moe_ckpt_unpack(b["q"], b["scale"], T, H, b["a"])
        return b["a"]
    m.moe_dispatch_rows(s["x"], s["scale"], s["row_of_slot"], s["topk_w"], T, H, c["k"], b["x_perm"], b["row_w"])
    return b["x_perm"], b["row_w"]


def _own_mlp(s):
    import moe_expert_layer_topk_gb300 as m
    c, b = s["case"], s["buf"]
    T, H, I, E, k = (c[n] for n in ("T", "H", "I", "E", "k"))
    R, num_seg = T * k, E * c["ranks"]
    if c["dir"] == "fwd":
        m.moe_grouped_gemm_swiglu_ckpt(s["x_perm"], s["Wg"], s["Wu"], num_seg, s["offsets"], s["seg_expert"], R, H, I, E, b["h"], b["gu_q"], b["gu_scale"])
        m.moe_ckpt_unpack(b["gu_q"], b["gu_scale"], R, 2 * I, b["gu"])  # the values that the codes stand for
        return b["h"], b["gu"]
    m.moe_grouped_gemm_down_bwd_ckpt(s["dy_perm"], s["row_w"], s["gu_q"], s["gu_scale"], s["Wd"], num_seg, s["offsets"], s["seg_expert"], R, H, I, E,
                                     b["dgu"], b["h_w"], b["d_w"], s["row_of_slot"], T, k, b["ws"])
    return b["dgu"], b["h_w"], b["d_w"]


# -------------------------------------------------------------- the plain forms

def _plain_pre(s):
    """r_t = 1/sqrt(mean_h x_th^2 + eps), y = x r gain.  Backward, with n = x r and dn = dy gain:
      dx = A dres + r (dn - n mean_h(dn n)),   dgain_h = sum_t dy_th n_th"""
    x = s["x"].float()
    if s["case"]["dir"] == "fwd":
        r = 1.0 / torch.sqrt((x * x).mean(1) + EPS)
        return (x * r[:, None] * s["gain"]).bfloat16(), r
    dy, r = s["dy"].float(), s["rstd"][:, None]
    n, dn = x * r, dy * s["gain"]
    dx = A * s["dres"].float() + r * (dn - n * (dn * n).mean(1, keepdim=True))
    return dx.to(s["x"].dtype), (dy * n).sum(0)


def _sigmoid(gate):
    """What a gate multiplies by: 1 without one; its logits are of a token or of an element."""
    if gate is None:
        return torch.ones((), device="cuda")
    g = 1.0 / (1.0 + torch.exp(-gate.float()))
    return g[:, None] if gate.dim() == 1 else g


def _plain_post(s):
    """n = z r (norm) or z, v = n gain, g = sigmoid(gate):  out = A residual + B g v,  next = norm(out as stored) next_gain.
    combine: z_t = sum_j w_tj y_perm[row_tj].  Backward, with dv = B g dout and dn = dv gain:
      dz = r (dn - n mean_h(dn n)) or dn,  dgain_h = sum_t dv n,  dgate = B dout v g (1 - g) (summed over h for a token's gate)"""
    c, gain, g = s["case"], s["gain"], _sigmoid(s["gate"])
    if c["dir"] == "bwd":
        z, dout, r = s["z"].float(), s["dout"].float(), s["rstd"][:, None]
        n = z * r if c["norm"] else z
        dv = B * g * dout
        dn = dv * gain
        dz = r * (dn - n * (dn * n).mean(1, keepdim=True)) if c["norm"] else dn
        ds = B * dout * n * gain * (g * (1.0 - g))
        dgate = {"none": None, "token": ds.sum(1), "element": ds.bfloat16()}[c["gate"]]
        return dict(dz=dz.bfloat16(), dgain=(dv * n).sum(0), dgate=dgate)
    if c["dir"] == "combine":
        z = (s["topk_w"][:, :, None] * s["y_perm"].float()[s["row_of_slot"].long()]).sum(1)
    else:
        z = s["z"].float()
    r = 1.0 / torch.sqrt((z * z).mean(1) + EPS)
    n = z * r[:, None] if c["norm"] else z
    out = (A * s["residual"].float() + B * g * n * gain).to(s["residual"].dtype)
    res = dict(out=out, rstd=r if c["norm"] else None, z=z.bfloat16() if c["dir"] == "combine" else None, next_y=None, next_rstd=None)
    if c["next"]:
        o = out.float()
        res["next_rstd"] = 1.0 / torch.sqrt((o * o).mean(1) + EPS)
        res["next_y"] = (o * res["next_rstd"][:, None] * s["next_gain"]).bfloat16()
    return res


def _encode(a):
    """Codes and scales of fp32 rows: for each 32 columns s = max|a| / 127, rounded up to a bf16 number and at least
    2^-126, and the whole number next to a (1/s)."""
    t = a.view(a.shape[0], -1, GROUP)
    top = t.abs().amax(2) / 127.0
    s = ((top.view(torch.int32) + 0xFFFF) & -0x10000).view(torch.float32).clamp(min=2.0 ** -126)
    q = torch.round(t * (1.0 / s)[:, :, None])
    return q.to(torch.int8).view(a.shape), s.bfloat16()


def _decode(q, s):
    return (q.float().view(q.shape[0], -1, GROUP) * s.float()[:, :, None]).view(q.shape)


def _plain_rows(s):
    """round: the rows' codes and scales, and the values that they stand for.  dispatch: x_perm[row_tj] = those of token t
    (copy: bf16 tokens as they are), row_w[row_tj] = w_tj."""
    if s["case"]["dir"] == "round":
        return _decode(*_encode(s["x"].float())).bfloat16()
    x = s["x"] if s["scale"] is None else _decode(s["x"], s["scale"]).bfloat16()
    rows, k = s["row_of_slot"].reshape(-1).long(), s["case"]["k"]
    x_perm, row_w = torch.empty(rows.numel(), x.shape[1], dtype=x.dtype, device="cuda"), torch.empty(rows.numel(), device="cuda")
    x_perm[rows] = x[:, None, :].expand(-1, k, -1).reshape(rows.numel(), -1)
    row_w[rows] = s["topk_w"].reshape(-1)
    return x_perm, row_w


def _plain_mlp(s):
    """Row r of expert e.  Forward: g = Wg_e x_r, u = Wu_e x_r, h = silu(g) u; g and u are kept in 8 bits.  Backward from
    those, with dh = Wd_e^T dy_r, sg = sigmoid(g), silu = g sg and the row's weight w:
      dgu = w [dh u sg (1 + g (1 - sg)), dh silu],  h_w = w silu u,  d_w = sum_i dh silu u
    The experts' products are taken at once, each block of rows padded to the longest."""
    c = s["case"]
    R, E, dev = c["T"] * c["k"], c["E"], "cuda"
    off, S, cap = s["offsets"].long(), E * c["ranks"], s["cap"]
    row = torch.arange(R, device=dev)
    seg = torch.searchsorted(off[1:], row, right=True)
    place = seg * cap + row - off[seg]
    take = (off[:-1, None] + torch.arange(cap, device=dev)[None, :]).clamp(max=R - 1)
    of = (lambda W: W.float()) if s["seg_expert"] is None else (lambda W: W.float()[s["seg_expert"].long()])
    if c["dir"] == "fwd":
        x = s["x_perm"].float()[take]
        g, u = ((x @ of(W).transpose(1, 2)).reshape(S * cap, -1)[place] for W in (s["Wg"], s["Wu"]))
        h = (g / (1.0 + torch.exp(-g)) * u).bfloat16()
        return h, _decode(*_encode(torch.cat([g, u], 1))).bfloat16()
    dh = (s["dy_perm"].float()[take] @ of(s["Wd"])).reshape(S * cap, -1)[place]
    g, u = _decode(s["gu_q"], s["gu_scale"]).split(c["I"], 1)
    w = s["row_w"][:, None]
    sg = 1.0 / (1.0 + torch.exp(-g))
    h = g * sg * u
    d_w = (dh * h).sum(1)
    dgu = torch.cat([w * dh * u * sg * (1.0 + g * (1.0 - sg)), w * dh * g * sg], 1)
    return dgu.bfloat16(), (w * h).bfloat16(), d_w if s["row_of_slot"] is None else d_w[s["row_of_slot"].long()]


# ------------------------------------------------------------------- the bytes

def work(case):
    c = case
    T, H = c["T"], c["H"]
    if c["op"] == "pre":
        st = 4 if c["fp32"] else 2
        if c["dir"] == "fwd":
            return dict(bytes=T * H * (st + 2) + 4 * T + 4 * H, flops=4 * T * H)
        return dict(bytes=T * H * (3 * st + 2) + 4 * T + 8 * H, flops=10 * T * H)
    if c["op"] == "post":
        st, g = 4 if c["fp32"] else 2, {"none": 0, "token": 4 * T, "element": 2 * T * H}[c["gate"]]
        if c["dir"] == "bwd":
            return dict(bytes=T * H * (st + 4) + 2 * g + 4 * T * c["norm"] + 8 * H, flops=14 * T * H)
        z = 2 * T * H * (c["k"] + 1) + 8 * T * c["k"] if c["dir"] == "combine" else 2 * T * H
        more = (2 * T * H + 4 * T + 4 * H) if c["next"] else 0
        return dict(bytes=z + 2 * st * T * H + g + more + 4 * T * c["norm"] + 4 * H, flops=T * H * (2 * c["k"] + 8))
    if c["op"] == "rows":
        kept = T * H + 2 * T * (H // GROUP)
        if c["dir"] == "round":
            return dict(bytes=4 * T * H + 2 * kept, flops=4 * T * H)
        return dict(bytes=(2 * T * H if c["dir"] == "copy" else kept) + 2 * T * c["k"] * H + 12 * T * c["k"], flops=T * H)
    R, I, used = T * c["k"], c["I"], int((_segments(c).reshape(c["ranks"], -1).sum(0) > 0).sum())
    kept = 2 * R * I + 2 * R * (2 * I // GROUP)
    if c["dir"] == "fwd":  # the codes written, and read for the values that come back
        return dict(bytes=2 * R * H + 4 * used * I * H + 2 * R * I + 2 * kept + 4 * R * I, flops=4 * R * H * I)
    return dict(bytes=2 * R * H + 2 * used * I * H + kept + 6 * R * I + 8 * R, flops=2 * R * H * I)


# ----------------------------------------------------------- the exact values

def exact(case, seed):
    s = _inputs(case, seed)
    return {"pre": _exact_pre, "post": _exact_post, "rows": _exact_rows, "mlp": _exact_mlp}[case["op"]](case, s)


def _dot(a, b):
    """Sums of products along a row, in float64."""
    return torch.einsum("th,th->t", a, b)


def _exact_pre(c, s):
    x, gain = s["x"].double(), s["gain"].double()
    if c["dir"] == "fwd":
        r = (_dot(x, x) / c["H"] + EPS).rsqrt()
        return torch.einsum("th,t,h->th", x, r, gain), r
    dy, r = s["dy"].double(), s["rstd"].double()
    through = _dot(dy * gain, x) * r.pow(3) / c["H"]
    dx = s["dres"].double() * A + torch.einsum("th,h,t->th", dy, gain, r) - x * through[:, None]
    return dx, torch.einsum("th,th,t->h", dy, x, r)


def _exact_post(c, s):
    gain, H = s["gain"].double(), c["H"]
    shape = (c["T"], 1 if c["gate"] != "element" else H)
    g = torch.ones(shape, dtype=torch.float64, device="cuda") if s["gate"] is None else torch.sigmoid(s["gate"].double()).view(shape)
    if c["dir"] == "bwd":
        z, dout = s["z"].double(), s["dout"].double()
        r = s["rstd"].double() if c["norm"] else torch.ones_like(s["rstd"], dtype=torch.float64)
        dv = dout * g * B
        dz = dv * gain * r[:, None]
        if c["norm"]:
            dz -= z * (_dot(dv * gain, z) * r.pow(3) / H)[:, None]
        ds = dv * gain * z * r[:, None] * (1 - g)
        dgate = None if s["gate"] is None else ds if c["gate"] == "element" else torch.einsum("th->t", ds)
        return dict(dz=dz, dgain=torch.einsum("th,th,t->h", dv, z, r), dgate=dgate)
    if c["dir"] == "combine":
        z = torch.zeros(c["T"], H, dtype=torch.float64, device="cuda")
        for j in range(c["k"]):
            z += s["y_perm"][s["row_of_slot"][:, j].long()].double() * s["topk_w"][:, j:j + 1].double()
    else:
        z = s["z"].double()
    r = (_dot(z, z) / H + EPS).rsqrt()
    out = s["residual"].double() * A + z * (r[:, None] if c["norm"] else 1.0) * gain * g * B
    res = dict(out=out, rstd=r if c["norm"] else None, z=z if c["dir"] == "combine" else None, next_y=None, next_rstd=None)
    if c["next"]:
        o = out.to(s["residual"].dtype).double()  # the norm is of what is stored
        q = (_dot(o, o) / H + EPS).rsqrt()
        res["next_y"], res["next_rstd"] = torch.einsum("th,t,h->th", o, q, s["next_gain"].double()), q
    return res


def _exact_kept(a):
    """The values that the codes of rows a stand for, in float64."""
    t = a.double().unflatten(1, (-1, GROUP))
    s = (t.abs().amax(2, keepdim=True) / 127).float()
    up = s.bfloat16().double()
    up = torch.where(up < s.double(), torch.nextafter(s.bfloat16(), torch.full_like(s, math.inf, dtype=torch.bfloat16)).double(), up).clamp(min=2.0 ** -126)
    return ((t / up).round() * up).flatten(1)


def _exact_rows(c, s):
    if c["dir"] == "round":
        return _exact_kept(s["x"])
    x = s["x"].double() if s["scale"] is None else s["x"].double() * s["scale"].double().repeat_interleave(GROUP, 1)
    slot = torch.argsort(s["row_of_slot"].reshape(-1))
    return x[slot // c["k"]], s["topk_w"].reshape(-1)[slot].double()


def _exact_mlp(c, s):
    """Block by block, in float64."""
    R, I, off = c["T"] * c["k"], c["I"], s["offsets"].tolist()
    which = range(c["E"]) if s["seg_expert"] is None else s["seg_expert"].tolist()
    dbl = lambda *n: torch.empty(*n, dtype=torch.float64, device="cuda")  # noqa: E731
    if c["dir"] == "fwd":
        h, gu = dbl(R, I), dbl(R, 2 * I)
        for e, a, b in zip(which, off, off[1:]):
            if b > a:
                x = s["x_perm"][a:b].double()
                g, u = x @ s["Wg"][e].double().t(), x @ s["Wu"][e].double().t()
                h[a:b] = torch.nn.functional.silu(g) * u
                gu[a:b] = _exact_kept(torch.cat([g, u], 1))
        return h, gu
    dgu, h_w, d_w = dbl(R, 2 * I), dbl(R, I), dbl(R)
    for e, a, b in zip(which, off, off[1:]):
        if b > a:
            dh = s["dy_perm"][a:b].double() @ s["Wd"][e].double()
            gu = s["gu_q"][a:b].double() * s["gu_scale"][a:b].double().repeat_interleave(GROUP, 1)
            g, u, w = gu[:, :I], gu[:, I:], s["row_w"][a:b].double()
            sg = torch.sigmoid(g)
            d_w[a:b] = torch.einsum("ri,ri->r", dh, g * sg * u)
            h_w[a:b] = w[:, None] * g * sg * u
            dgu[a:b, :I] = w[:, None] * dh * u * (sg + g * sg * (1 - sg))
            dgu[a:b, I:] = w[:, None] * dh * g * sg
    return dgu, h_w, d_w if s["row_of_slot"] is None else d_w[s["row_of_slot"].long()]
