"""Cases, plain forms and exact values of the operators around the MoE layer's training and serving.

Three operators, each reached through the package's entry points of the same names:

  balance   moe_balance_loss, moe_balance_loss_bwd: the load-balance loss and the router z-loss of
            masked, packed tokens, the per-expert counts, and the gradient of the router logits
  dropout   moe_dropout, moe_combine_dropout, moe_combine_dropout_bwd: dropout whose mask is computed
            from a counter and never stored, alone and in the weighted combine of the experts' rows
  adapter   moe_adapter_linear, moe_adapter_linear_bwd: a projection shared by all requests plus a
            low-rank adapter for each request, forward and backward

`run` computes the plain form (elementary torch operations in fp32, rounded once) unless `own` is
set, and then calls the package.  Formulas are stated at each plain form.
"""
from __future__ import annotations

import math
import random

import numpy as np
import torch

own = False

VALUE_BYTES = {"bf16": 2, "fp32": 4}


# ------------------------------------------------------------------- the cases

def listed():
    return [
        # the smallest router of the layer's own workloads: launch latency is all there is
        dict(name="balance_tiny", op="balance", dir="loss_grad", T=256, E=8, k=2, segs=0, off=0, pad=0),
        # one training step of the T=8192 layer: loss and router gradient, one group of tokens
        dict(name="balance_step", op="balance", dir="loss_grad", T=8192, E=128, k=8, segs=0, off=0, pad=0),
        # a long packed batch with padding: a loss for each of 37 sequences, four experts switched off
        dict(name="balance_packed", op="balance", dir="loss_grad", T=65519, E=128, k=8, segs=37, off=4, pad=1),
        # residual dropout after a small layer
        dict(name="combine_dropout_tiny", op="dropout", dir="combine", T=256, H=128, k=2, E=8, p=0.1),
        # residual dropout after the T=8192 training layer, and its backward at an odd token count
        dict(name="combine_dropout_step", op="dropout", dir="combine", T=8192, H=2048, k=8, E=128, p=0.1),
        dict(name="combine_dropout_bwd", op="dropout", dir="combine_bwd", T=8191, H=2048, k=8, E=128, p=0.1),
        # dropout of an activation whose size is no multiple of anything
        dict(name="dropout_odd", op="dropout", dir="plain", n=16777213, dtype="bf16", p=0.25),
        # serving: one token of one request
        dict(name="adapter_token", op="adapter", dir="fwd", T=1, K=2048, N=2048, r=16, reqs=1, nA=8, kind="ones", pitch=0),
        # serving: one token each of 64 requests over 48 adapters, every fifth request without one
        dict(name="adapter_decode", op="adapter", dir="fwd", T=64, K=2048, N=2048, r=16, reqs=64, nA=48, kind="ones", pitch=0),
        # serving: prompt pieces and single tokens in one batch, rows inside a wider buffer
        dict(name="adapter_mixed", op="adapter", dir="fwd", T=517, K=768, N=2048, r=64, reqs=40, nA=12, kind="mixed", pitch=192),
        # serving: the prompts of 23 requests over 8 adapters
        dict(name="adapter_prompts", op="adapter", dir="fwd", T=16381, K=2048, N=4096, r=32, reqs=23, nA=8, kind="ragged", pitch=0),
        # fine-tuning 8 adapters at once: forward and backward of T=8192 tokens
        dict(name="adapter_train", op="adapter", dir="fwd_bwd", T=8192, K=2048, N=2048, r=16, reqs=8, nA=8, kind="ragged", pitch=0),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], even over its logarithm; never the one size this file avoids."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    v = min(hi, max(lo, v))
    return v if v != 3072 else 3071


def draw(rng):
    op = rng.choice(["balance", "dropout", "adapter", "adapter"])
    if op == "balance":
        E = rng.choice([8, 16, 60, 64, 128, 130, 256, _spread(rng, 2, 512)])
        segs = rng.choice([0, 0, 1, _spread(rng, 2, 200)])
        return dict(op=op, dir=rng.choice(["loss_grad", "loss_grad", "loss", "bwd"]), T=_spread(rng, 1, max(1, 65536 * 128 // max(E, 128))), E=E,
                    k=rng.randint(1, min(8, E)), segs=segs, off=rng.choice([0, min(2, E // 4)]), pad=rng.choice([0, 1]))
    if op == "dropout":
        p = rng.choice([0.0, 0.05, 0.1, 0.25, 0.5])
        way = rng.choice(["combine", "combine_bwd", "plain"])
        if way == "plain":
            return dict(op=op, dir=way, n=_spread(rng, 1, 16777216), dtype=rng.choice(["bf16", "fp32"]), p=p)
        H = 64 * _spread(rng, 1, 32)
        E = rng.choice([4, 8, 64, 128])
        k = rng.randint(1, min(8, E))
        return dict(op=op, dir=way, T=_spread(rng, 1, 8192), H=H, k=k, E=E, p=p)
    K, N = (64 * rng.choice([_spread(rng, 1, 32), 12, 32]) for _ in range(2))
    r = 8 * rng.choice([1, 2, 2, 3, 4, 8, _spread(rng, 1, 16)])
    nA = rng.randint(1, max(1, min(48, 1024 // r)))
    way = rng.choice(["fwd", "fwd", "fwd_bwd"])
    kind = rng.choice(["ones", "ragged", "mixed"]) if way == "fwd" else "ragged"
    if kind == "ones":
        T = _spread(rng, 1, 256)
        reqs = T
    else:
        T = _spread(rng, 2, 8192)
        reqs = min(T, _spread(rng, 1, 64))
    return dict(op=op, dir=way, T=T, K=K, N=N, r=r, reqs=reqs, nA=nA, kind=kind, pitch=rng.choice([0, 0, 64]))


# ------------------------------------------------------------------ the inputs

def _cuts(T, n, kind):
    """Ends of n pieces of T rows, by the sizes alone: single rows, ragged pieces (one of them empty
    where there are several), or a batch in which most pieces are single rows."""
    rng = random.Random(1000003 * T + n)
    if kind == "ones":
        sizes = [1] * T
    elif kind == "mixed":
        ones = min(n - 1, T - 1) * 3 // 4
        sizes = _cuts_sizes(rng, T - ones, n - ones) + [1] * ones
    else:
        sizes = _cuts_sizes(rng, T, n)
    ends, at = [0], 0
    for s in sizes:
        at += s
        ends.append(at)
    return ends


def _cuts_sizes(rng, T, n):
    if n <= 1:
        return [T]
    marks = sorted(rng.randint(0, T) for _ in range(n - 1))
    if n > 2:
        marks[1] = marks[0]  # an empty piece
    marks = [0] + marks + [T]
    return [b - a for a, b in zip(marks, marks[1:])]


def _which(case):
    """The adapter of each request; every fifth request of a serving batch has none."""
    n = len(_cuts(case["T"], case["reqs"], case["kind"])) - 1
    none = case["dir"] == "fwd" and n > 4
    return [-1 if none and i % 5 == 4 else (i * 7) % case["nA"] for i in range(n)]


def _inputs(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    d = {}
    if case["op"] == "balance":
        T, E, k = case["T"], case["E"], case["k"]
        logits = rn(T, E) * 0.9 + rn(E) * 0.7  # x.Wr of the layer's inputs, some experts more popular
        if case["off"]:
            logits[:, torch.randperm(E, generator=g, device="cuda")[:case["off"]]] = -math.inf
        d["topk_idx"] = torch.topk(logits, k, dim=1).indices.to(torch.int32).contiguous()
        d["mask"] = None
        if case["pad"]:  # padding tokens hold whatever was in the buffer
            d["mask"] = (torch.rand(T, generator=g, device="cuda") > 0.1).to(torch.uint8)
        d["ends"] = None
        if case["segs"]:
            ends = _cuts(T - T // 50, case["segs"], "ragged")  # the last fiftieth belongs to no sequence
            d["ends"] = torch.tensor(ends, dtype=torch.int32, device="cuda")
            if case["pad"] and case["segs"] > 3:
                d["mask"][ends[-2]:ends[-1]] = 0  # a sequence of padding alone
        if case["pad"]:
            junk = torch.tensor([math.nan, math.inf, 3.0e38], device="cuda")
            off = d["mask"] == 0
            logits = torch.where(off[:, None], junk[torch.arange(T, device="cuda") % 3][:, None], logits)
        d["logits"] = logits.contiguous()
        if case["dir"] == "bwd":
            d["dloss"] = torch.rand(2, generator=g, device="cuda") + 0.5
    elif case["op"] == "dropout":
        words = torch.randint(0, 1 << 62, (1,), generator=g, device="cuda")
        d["rng"] = torch.cat([words, words % 100003 + (1 << 33)])  # seed, counter offset
        if case["dir"] == "plain":
            dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
            d["x"], d["residual"] = rn(case["n"]).to(dt), rn(case["n"]).to(dt)
        else:
            T, H, k, E = case["T"], case["H"], case["k"], case["E"]
            idx = torch.topk(rn(T, E) + rn(E) * 0.5, k, dim=1).indices
            order = torch.sort(idx.reshape(-1), stable=True).indices
            rows = torch.empty(T * k, dtype=torch.int32, device="cuda")
            rows[order] = torch.arange(T * k, dtype=torch.int32, device="cuda")
            d["row_of_slot"] = rows.view(T, k)
            w = torch.exp(rn(T, k))
            d["topk_w"] = (w / w.sum(1, keepdim=True)).contiguous()
            d["y_perm"] = (rn(T * k, H) * 0.3).bfloat16()
            d["residual" if case["dir"] == "combine" else "dy"] = rn(T, H).bfloat16()
    else:
        T, K, N, r, nA = (case[n] for n in ("T", "K", "N", "r", "nA"))
        wide = rn(T, K + case["pitch"]).bfloat16()
        d["x"] = wide[:, case["pitch"] // 2:case["pitch"] // 2 + K]
        d["W"] = (rn(N, K) * 0.02).bfloat16()
        d["A"] = (rn(nA, r, K) / math.sqrt(K)).bfloat16()
        d["B"] = (rn(nA, N, r) * 0.1).bfloat16()
        d["scale"] = 16.0 / r * (1.0 + torch.arange(nA, device="cuda") % 3)
        if case["dir"] == "fwd_bwd":
            d["dy"] = rn(T, N).bfloat16()
        d["ends"] = torch.tensor(_cuts(T, case["reqs"], case["kind"]), dtype=torch.int32, device="cuda")
        d["which"] = torch.tensor(_which(case), dtype=torch.int32, device="cuda")
    return d


def prepare(case, seed):
    state = dict(case=case, **_inputs(case, seed))
    if own:
        state["buf"] = _buffers(case)
    return state


def run(state):
    op = state["case"]["op"]
    if op == "balance":
        return _own_balance(state) if own else _plain_balance(state)
    if op == "dropout":
        return _own_dropout(state) if own else _plain_dropout(state)
    return _own_adapter(state) if own else _plain_adapter(state)


COEF = (0.01, 0.001)  # of the balance loss and of the z-loss in the logits' gradient


# ------------------------------------------------- the framework's own kernels

def _buffers(case):
    """The output tensors and workspaces that a training or serving program keeps."""
    import moe_expert_layer_topk_gb300 as m
    e = lambda *s, dt=torch.float32: torch.empty(*s, dtype=dt, device="cuda")  # noqa: E731
    bf, u8, i32 = torch.bfloat16, torch.uint8, torch.int32
    if case["op"] == "balance":
        T, E, S = case["T"], case["E"], max(1, case["segs"])
        return dict(counts=e(S, E, dt=i32), tokens=e(S, dt=i32), prob_sum=e(S, E), loss=e(2), dlogits=e(T, E),
                    ws=e(max(256, m.moe_balance_loss_workspace_size(T, E, S)), dt=u8))
    if case["op"] == "dropout":
        if case["dir"] == "plain":
            return dict(out=e(case["n"], dt=bf if case["dtype"] == "bf16" else torch.float32))
        T, H, k = case["T"], case["H"], case["k"]
        return dict(y=e(T, H, dt=bf)) if case["dir"] == "combine" else dict(dy_perm=e(T * k, H, dt=bf), d_w=e(T, k))
    T, K, N, r, nA = (case[n] for n in ("T", "K", "N", "r", "nA"))
    S = len(_which(case))
    b = dict(y=e(T, N, dt=bf), hidden=e(m.moe_adapter_hidden_size(T, r), dt=u8))
    if case["dir"] == "fwd_bwd":
        b.update(dx=e(T, K, dt=bf), dA=e(nA, r, K), dB=e(nA, N, r),
                 ws=e(m.moe_adapter_linear_bwd_workspace_size(T, K, N, r, S), dt=u8))
    return b


def _own_balance(s):
    import moe_expert_layer_topk_gb300 as m
    c, b = s["case"], s["buf"]
    T, E, k, S = c["T"], c["E"], c["k"], max(1, c["segs"])
    grad = c["dir"] == "loss_grad"
    m.moe_balance_loss(s["logits"], s["topk_idx"], s["mask"], T, E, k, S, s["ends"], b["counts"], b["tokens"], b["prob_sum"],
                       b["loss"], COEF[0], COEF[1], b["dlogits"] if grad else None, b["ws"])
    if c["dir"] == "bwd":
        m.moe_balance_loss_bwd(s["logits"], s["mask"], T, E, k, S, s["ends"], b["counts"], b["tokens"], COEF[0], COEF[1],
                               s["dloss"], b["dlogits"])
    out = {n: b[n] for n in ("counts", "tokens", "prob_sum", "loss")}
    if c["dir"] != "loss":
        out["dlogits"] = b["dlogits"]
    return out


def _own_dropout(s):
    import moe_expert_layer_topk_gb300 as m
    c, b = s["case"], s["buf"]
    if c["dir"] == "plain":
        m.moe_dropout(s["x"], s["residual"], c["n"], c["p"], s["rng"], b["out"])
        return b["out"]
    T, H, k = c["T"], c["H"], c["k"]
    if c["dir"] == "combine":
        m.moe_combine_dropout(s["y_perm"], s["topk_w"], s["row_of_slot"], s["residual"], T, H, k, c["p"], s["rng"], b["y"])
        return b["y"]
    m.moe_combine_dropout_bwd(s["dy"], s["y_perm"], s["topk_w"], s["row_of_slot"], T, H, k, c["p"], s["rng"], b["dy_perm"], b["d_w"])
    return b["dy_perm"], b["d_w"]


def _own_adapter(s):
    import moe_expert_layer_topk_gb300 as m
    c, b = s["case"], s["buf"]
    T, K, N, r, nA, S = c["T"], c["K"], c["N"], c["r"], c["nA"], s["which"].numel()
    m.moe_adapter_linear(s["x"], s["W"], s["A"], s["B"], s["scale"], S, s["ends"], s["which"], T, K, N, r, nA, b["hidden"], b["y"])
    if c["dir"] == "fwd":
        return b["y"]
    m.moe_adapter_linear_bwd(s["dy"], s["x"], s["W"], s["A"], s["B"], s["scale"], b["hidden"], S, s["ends"], s["which"],
                             T, K, N, r, nA, b["dx"], b["dA"], b["dB"], 0, b["ws"])
    return {n: b[n] for n in ("y", "dx", "dA", "dB")}


# -------------------------------------------------------------- the plain forms

def _plain_balance(s):
    """Token t of sequence q (mask m_t): p_t = softmax(l_t); n_q = sum m_t; c_qe = its slots routed to
    e; P_qe = sum m_t p_te; n = sum n_q.
      balance = 1/n sum_q E/(k n_q) sum_e c_qe P_qe,   z = 1/n sum_t m_t lse(l_t)^2
      dl_te = m_t p_te ( a E/(k n_q n) (c_qe - sum_j c_qj p_tj) + 2 b/n lse(l_t) )"""
    c = s["case"]
    T, E, k = c["T"], c["E"], c["k"]
    dev = s["logits"].device
    if s["ends"] is None:
        seq, S, live = torch.zeros(T, dtype=torch.long, device=dev), 1, torch.ones(T, dtype=torch.bool, device=dev)
    else:
        S = c["segs"]
        seq = torch.searchsorted(s["ends"], torch.arange(T, dtype=torch.int32, device=dev), right=True) - 1
        live = seq < S
        seq = torch.where(live, seq, 0)
    if s["mask"] is not None:
        live = live & (s["mask"] != 0)
    l = torch.where(live[:, None], s["logits"], 0.0)
    top = l.amax(1, keepdim=True)
    ex = torch.exp(l - top)
    tot = ex.sum(1, keepdim=True)
    p, lse = ex / tot, (top + torch.log(tot))[:, 0]
    in_seq = (seq[None, :] == torch.arange(S, device=dev)[:, None]) & live[None, :]
    tokens = in_seq.sum(1).to(torch.int32)
    counts = torch.zeros(S * E, dtype=torch.int32, device=dev)
    counts.index_add_(0, (seq[:, None] * E + s["topk_idx"]).reshape(-1), live[:, None].expand(T, k).reshape(-1).to(torch.int32))
    counts = counts.view(S, E)
    prob_sum = in_seq.float() @ p
    n = tokens.sum().clamp(min=1).float()
    per = E / (k * tokens.clamp(min=1).float() * n)
    cf = counts.float()
    loss = torch.stack([(per * (cf * prob_sum).sum(1)).sum(), torch.where(live, lse * lse, 0.0).sum() / n])
    out = dict(counts=counts, tokens=tokens, prob_sum=prob_sum, loss=loss)
    if c["dir"] != "loss":
        a, b = COEF
        if c["dir"] == "bwd":
            a, b = a * s["dloss"][0], b * s["dloss"][1]
        ct = cf[seq]
        mean = (ct * p).sum(1, keepdim=True)
        dl = p * ((a * per)[seq][:, None] * (ct - mean) + (2.0 * b / n * lse)[:, None])
        out["dlogits"] = torch.where(live[:, None], dl, 0.0)
    return out


def _mul32(m, v):
    """High and low 32 bits of the product of the constant m and v (both below 2^32, in int64)."""
    t = m * (v & 0xFFFF)
    u = m * (v >> 16) + (t >> 16)
    return u >> 16, ((u & 0xFFFF) << 16) | (t & 0xFFFF)


def _keep(rng, n, p):
    """Which of n elements stay.  Philox4x32-10 (Salmon, Moraes, Dror, Shaw, "Parallel random numbers: as
    easy as 1, 2, 3", 2011) under the key rng[0] at the 64-bit counter rng[1] + i/8 gives elements
    8(i/8) .. 8(i/8)+7 sixteen bits each, lowest first; element i stays when they are at least p 2^16."""
    ctr = rng[1] + torch.arange((n + 7) // 8, device=rng.device)
    c0, c1 = ctr & 0xFFFFFFFF, (ctr >> 32) & 0xFFFFFFFF
    c2 = c3 = torch.zeros_like(c0)
    k0, k1 = rng[0] & 0xFFFFFFFF, (rng[0] >> 32) & 0xFFFFFFFF
    for _ in range(10):
        h0, l0 = _mul32(0xD2511F53, c0)
        h1, l1 = _mul32(0xCD9E8D57, c2)
        c0, c1, c2, c3 = h1 ^ c1 ^ k0, l1, h0 ^ c3 ^ k1, l0
        k0, k1 = (k0 + 0x9E3779B9) & 0xFFFFFFFF, (k1 + 0xBB67AE85) & 0xFFFFFFFF
    words = torch.stack([c0, c1, c2, c3], 1)
    halves = torch.stack([words & 0xFFFF, words >> 16], 2).reshape(-1)[:n]
    return halves >= _threshold(p)


def _threshold(p):
    return int(math.floor(p * 65536 + 0.5))


def _factor(p):
    t = _threshold(p)
    return 65536.0 / (65536 - t) if t < 65536 else 0.0


def _plain_dropout(s):
    """D(v)_i = keep_i v_i 65536/(65536 - p 2^16).  plain: out = residual + D(x).  combine:
    y_t = residual_t + D(sum_j w_tj y_perm[row_tj]).  combine_bwd: g = D(dy), dy_perm[row_tj] = w_tj g_t,
    d_w_tj = g_t . y_perm[row_tj]."""
    c = s["case"]
    f = _factor(c["p"])
    if c["dir"] == "plain":
        keep = _keep(s["rng"], c["n"], c["p"])
        return (s["residual"].float() + torch.where(keep, s["x"].float() * f, 0.0)).to(s["x"].dtype)
    T, H, k = c["T"], c["H"], c["k"]
    keep = _keep(s["rng"], T * H, c["p"]).view(T, H)
    rows = s["row_of_slot"].long()
    yp = s["y_perm"].float()[rows]
    w = s["topk_w"][:, :, None]
    if c["dir"] == "combine":
        return (s["residual"].float() + torch.where(keep, (w * yp).sum(1) * f, 0.0)).bfloat16()
    g = torch.where(keep, s["dy"].float() * f, 0.0)[:, None, :]
    dy_perm = torch.empty(T * k, H, dtype=torch.bfloat16, device=rows.device)
    dy_perm[rows.reshape(-1)] = (w * g).reshape(T * k, H).bfloat16()
    return dy_perm, (g * yp).sum(2)


def _plain_adapter(s):
    """Row t of a request with adapter a (none: the second term is left out):
      y_t = W x_t + s_a B_a (A_a x_t)
      dx_t = W^T dy_t + A_a^T u_t with u_t = s_a B_a^T dy_t,  dA_a = sum_t u_t x_t^T,  dB_a = sum_t s_a dy_t (A_a x_t)^T
    The adapters' products are taken for all adapters at once and each row's own is chosen."""
    c = s["case"]
    T, K, N, r, nA = (c[n] for n in ("T", "K", "N", "r", "nA"))
    dev = s["W"].device
    x, W, A, B = s["x"].float(), s["W"].float(), s["A"].float().view(nA * r, K), s["B"].float()
    Bt = B.transpose(0, 1).reshape(N, nA * r)
    row = torch.searchsorted(s["ends"], torch.arange(T, dtype=torch.int32, device=dev), right=True) - 1
    ad = s["which"][row.clamp(max=s["which"].numel() - 1)]
    mine = (ad[:, None] == torch.arange(nA, dtype=torch.int32, device=dev)[None, :])[:, :, None]
    chosen = lambda v: torch.where(mine, v.view(T, nA, r) * s["scale"][None, :, None], 0.0).view(T, nA * r)  # noqa: E731
    v = chosen(x @ A.t())
    y = (x @ W.t() + v @ Bt.t()).bfloat16()
    if c["dir"] == "fwd":
        return y
    dy = s["dy"].float()
    u = chosen(dy @ Bt)
    return dict(y=y, dx=(dy @ W + u @ A).bfloat16(), dA=(u.t() @ x).view(nA, r, K),
                dB=(dy.t() @ v).view(N, nA, r).transpose(0, 1).contiguous())


# ------------------------------------------------------------------- the bytes

def work(case):
    c = case
    if c["op"] == "balance":
        T, E, k, S = c["T"], c["E"], c["k"], max(1, c["segs"])
        b = 4 * T * E * (1 if c["dir"] == "loss" else 2) + 4 * T * k + (T if c["pad"] else 0) + 8 * S * E
        return dict(bytes=b, flops=8 * T * E)
    if c["op"] == "dropout":
        if c["dir"] == "plain":
            return dict(bytes=3 * c["n"] * VALUE_BYTES[c["dtype"]], flops=3 * c["n"])
        T, H, k = c["T"], c["H"], c["k"]
        if c["dir"] == "combine":
            return dict(bytes=2 * T * H * (k + 2) + 8 * T * k, flops=2 * T * H * k)
        return dict(bytes=2 * T * H * (2 * k + 1) + 12 * T * k, flops=4 * T * H * k)
    T, K, N, r = (c[n] for n in ("T", "K", "N", "r"))
    ends, which = _cuts(T, c["reqs"], c["kind"]), _which(c)
    live = sum(b - a for a, b, w in zip(ends, ends[1:], which) if w >= 0)
    used = len({w for a, b, w in zip(ends, ends[1:], which) if w >= 0 and b > a})
    b = 2 * (T * K + N * K + T * N + used * r * (K + N))
    f = 2 * T * K * N + 2 * live * r * (K + N)
    if c["dir"] == "fwd_bwd":  # x, W, A and B again, dy; dx, and dA, dB in fp32
        b += 2 * (T * K + N * K + T * N + used * r * (K + N) + T * K) + 4 * c["nA"] * r * (K + N)
        f += 2 * T * K * N + 6 * live * r * (K + N)
    return dict(bytes=b, flops=f)


# ----------------------------------------------------------- the exact values

def exact(case, seed):
    s = _inputs(case, seed)
    return {"balance": _exact_balance, "dropout": _exact_dropout, "adapter": _exact_adapter}[case["op"]](case, s)


def _exact_balance(c, s):
    """Sequence by sequence, in float64."""
    T, E, k = c["T"], c["E"], c["k"]
    ends = [0, T] if s["ends"] is None else s["ends"].tolist()
    S = len(ends) - 1
    on = torch.ones(T, dtype=torch.bool, device="cuda") if s["mask"] is None else s["mask"].bool()
    counts = torch.zeros(S, E, dtype=torch.float64, device="cuda")
    probs, lse = torch.zeros_like(counts), []
    rows = [torch.arange(a, b, device="cuda")[on[a:b]] for a, b in zip(ends, ends[1:])]
    n = max(1, sum(x.numel() for x in rows))
    dl = torch.zeros(T, E, dtype=torch.float64, device="cuda")
    a, b = COEF
    if c["dir"] == "bwd":
        a, b = a * s["dloss"][0].item(), b * s["dloss"][1].item()
    bal = z = 0.0
    for q, at in enumerate(rows):
        if not at.numel():
            continue
        l = s["logits"][at].double()
        p, ls = torch.softmax(l, 1), torch.logsumexp(l, 1)
        counts[q] = torch.bincount(s["topk_idx"][at].reshape(-1).long(), minlength=E).double()
        probs[q] = p.sum(0)
        per = E / (k * at.numel() * n)
        bal += per * torch.dot(counts[q], probs[q]).item()
        z += ls.square().sum().item() / n
        dl[at] = p * (a * per * (counts[q] - p @ counts[q][:, None]) + 2 * b / n * ls[:, None])
    out = dict(counts=counts.to(torch.int32), tokens=torch.tensor([x.numel() for x in rows], dtype=torch.int32, device="cuda"), prob_sum=probs,
               loss=torch.tensor([bal, z], dtype=torch.float64, device="cuda"))
    if c["dir"] != "loss":
        out["dlogits"] = dl
    return out


def _exact_keep(rng, n, p):
    """The same generator on the host, in unsigned 64-bit arithmetic."""
    key, off = (int(v) for v in rng.tolist())
    ctr = np.arange((n + 7) // 8, dtype=np.uint64) + np.uint64(off)
    low, w = np.uint64(0xFFFFFFFF), np.uint64(32)
    x = [ctr & low, ctr >> w, np.zeros_like(ctr), np.zeros_like(ctr)]
    ka, kb = key & 0xFFFFFFFF, key >> 32
    for _ in range(10):
        a, b = x[0] * np.uint64(0xD2511F53), x[2] * np.uint64(0xCD9E8D57)
        x = [(b >> w) ^ x[1] ^ np.uint64(ka), b & low, (a >> w) ^ x[3] ^ np.uint64(kb), a & low]
        ka, kb = (ka + 0x9E3779B9) & 0xFFFFFFFF, (kb + 0xBB67AE85) & 0xFFFFFFFF
    bits = np.stack([v.astype(np.uint32) for v in x], 1).view(np.uint16).reshape(-1)[:n]
    return torch.from_numpy(bits >= p * 65536 - 0.5).cuda() if p < 1 else torch.zeros(n, dtype=torch.bool, device="cuda")


def _exact_dropout(c, s):
    n = c["n"] if c["dir"] == "plain" else c["T"] * c["H"]
    keep = _exact_keep(s["rng"], n, c["p"])
    f = 65536 / (65536 - round(c["p"] * 65536))
    if c["dir"] == "plain":
        return s["residual"].double() + s["x"].double() * keep * f
    T, H, k = c["T"], c["H"], c["k"]
    keep = keep.view(T, H)
    rows, w = s["row_of_slot"].long(), s["topk_w"].double()
    if c["dir"] == "combine":
        y = torch.zeros(T, H, dtype=torch.float64, device="cuda")
        for j in range(k):
            y += w[:, j:j + 1] * s["y_perm"][rows[:, j]].double()
        return s["residual"].double() + y * keep * f
    g = s["dy"].double() * keep * f
    dy_perm, d_w = torch.empty(T * k, H, dtype=torch.float64, device="cuda"), torch.empty(T, k, dtype=torch.float64, device="cuda")
    for j in range(k):
        dy_perm[rows[:, j]] = w[:, j:j + 1] * g
        d_w[:, j] = (g * s["y_perm"][rows[:, j]].double()).sum(1)
    return dy_perm, d_w


def _exact_adapter(c, s):
    """Request by request, in float64."""
    T, K, N, r, nA = (c[n] for n in ("T", "K", "N", "r", "nA"))
    ends, which = s["ends"].tolist(), s["which"].tolist()
    x, W = s["x"].double(), s["W"].double()
    y = x @ W.t()
    if c["dir"] == "fwd_bwd":
        dy = s["dy"].double()
        dx = dy @ W
        dA = torch.zeros(nA, r, K, dtype=torch.float64, device="cuda")
        dB = torch.zeros(nA, N, r, dtype=torch.float64, device="cuda")
    for a, b, w in zip(ends, ends[1:], which):
        if w < 0 or a == b:
            continue
        A, B, f = s["A"][w].double(), s["B"][w].double(), s["scale"][w].double()
        v = f * (x[a:b] @ A.t())
        y[a:b] += v @ B.t()
        if c["dir"] == "fwd_bwd":
            u = f * (dy[a:b] @ B)
            dx[a:b] += u @ A
            dA[w] += u.t() @ x[a:b]
            dB[w] += dy[a:b].t() @ v
    return y if c["dir"] == "fwd" else dict(y=y, dx=dx, dA=dA, dB=dB)
