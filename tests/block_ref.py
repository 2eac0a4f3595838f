"""Plain float64 restatements of the norms around a block and of activations
kept in 8 bits, on the CPU (numpy), for the GPU parity tests.

They are written from the definitions in include/moe_topk.h and share no code
with the package.  Next to a result stands `<name>_mag`, its formula with every
term's magnitude added, for error bounds.
"""
from __future__ import annotations

import numpy as np

f64 = lambda v: np.asarray(v, np.float64)  # noqa: E731


def rstd(x, eps):
    x = f64(x)
    return 1.0 / np.sqrt((x * x).mean(1) + eps)


def pre_norm(x, gain, eps):
    r = rstd(x, eps)
    return f64(x) * r[:, None] * f64(gain), r


def _norm_bwd(dn, n, r):
    """r (dn - n mean(dn n)), and its magnitude."""
    dx = r[:, None] * (dn - n * (dn * n).mean(1, keepdims=True))
    mag = np.abs(r)[:, None] * (np.abs(dn) + np.abs(n) * np.abs(dn * n).mean(1, keepdims=True))
    return dx, mag


def pre_norm_bwd(dy, x, gain, r, dres, a):
    dy, x, r = f64(dy), f64(x), f64(r)
    n = x * r[:, None]
    dx, mag = _norm_bwd(dy * f64(gain), n, r)
    if dres is not None:
        dx, mag = dx + a * f64(dres), mag + np.abs(a * f64(dres))
    return dict(dx=dx, dx_mag=mag, dgain=(dy * n).sum(0), dgain_mag=np.abs(dy * n).sum(0))


def gate_value(gate, shape):
    """sigmoid of no gate, of a token's or of an element's logit, and its derivative."""
    if gate is None:
        return np.ones(shape), np.zeros(shape)
    s = f64(gate)
    s = np.broadcast_to(s[:, None] if s.ndim == 1 else s, shape)
    g = 1.0 / (1.0 + np.exp(-s))
    return g, g / (1.0 + np.exp(s))


def combine(y_perm, w, rows):
    y, w = f64(y_perm), f64(w)
    return (w[:, :, None] * y[rows]).sum(1), (np.abs(w)[:, :, None] * np.abs(y[rows])).sum(1)


def post_norm(z, residual, gain, norm, eps, gate, a, b, z_mag=None):
    z = f64(z)
    r = rstd(z, eps) if norm else np.ones(len(z))
    G, _ = gate_value(gate, z.shape)
    out = b * G * z * r[:, None] * f64(gain)
    mag = np.abs(b * G * (np.abs(z) if z_mag is None else z_mag) * r[:, None] * f64(gain))
    if residual is not None:
        out, mag = out + a * f64(residual), mag + np.abs(a * f64(residual))
    return dict(out=out, out_mag=mag, rstd=r)


def post_norm_bwd(dout, z, gain, norm, r, gate, b):
    dout, z, gain = f64(dout), f64(z), f64(gain)
    r = f64(r) if norm else np.ones(len(z))
    n = z * r[:, None]
    G, dG = gate_value(gate, z.shape)
    dv = b * G * dout
    dn = dv * gain
    dz, mag = _norm_bwd(dn, n, r) if norm else (dn, np.abs(dn))
    ds = b * dout * n * gain * dG
    if gate is not None and np.asarray(gate).ndim == 1:
        dgate, gmag = ds.sum(1), np.abs(ds).sum(1)
    else:
        dgate, gmag = ds, np.abs(ds)
    return dict(dz=dz, dz_mag=mag, dgain=(dv * n).sum(0), dgain_mag=np.abs(dv * n).sum(0), dgate=dgate, dgate_mag=gmag)


# --------------------------------------------------------- 8-bit activations

def bf16_up(v):
    """The smallest bf16 number that is at least the fp32 value v >= 0."""
    u = np.asarray(v, np.float32).view(np.uint32)
    return ((u + np.uint32(0xFFFF)) & np.uint32(0xFFFF0000)).view(np.float32)


def pack(a):
    """Codes int8 [rows, cols] and scales fp32 [rows, cols/32] of fp32 values."""
    g = np.asarray(a, np.float32).reshape(len(a), -1, 32)
    s = np.maximum(bf16_up(np.abs(g).max(2) / np.float32(127)), np.float32(2.0 ** -126))
    s[s > 2.0 ** 121] = 2.125 * 2.0 ** 120
    q = np.rint(g * (np.float32(1) / s)[:, :, None])
    assert np.abs(q).max(initial=0) <= 127
    return q.astype(np.int8).reshape(np.shape(a)), s


def unpack(q, s):
    """The values that codes and scales stand for, exactly (15 bits at most)."""
    return (f64(q).reshape(len(q), -1, 32) * f64(s)[:, :, None]).reshape(np.shape(q))


def experts(offsets, seg_expert=None):
    return [(s if seg_expert is None else int(seg_expert[s]), int(a), int(b)) for s, (a, b) in enumerate(zip(offsets, offsets[1:]))]


def gate_up(x_perm, Wg, Wu, segs):
    x = f64(x_perm)
    I = np.shape(Wg)[1]
    g, u, mag = (np.zeros((len(x), I)) for _ in range(3))
    for e, a, b in segs:
        if 0 <= e < len(Wg):
            g[a:b], u[a:b] = x[a:b] @ f64(Wg[e]).T, x[a:b] @ f64(Wu[e]).T
            mag[a:b] = np.maximum(np.abs(x[a:b]) @ np.abs(f64(Wg[e])).T, np.abs(x[a:b]) @ np.abs(f64(Wu[e])).T)
    return g, u, mag


def down_bwd(dy_perm, w, g, u, Wd, segs):
    """dgu, h_w and d_w of every row (0 outside the segments)."""
    dy, g, u = f64(dy_perm), f64(g), f64(u)
    w = np.ones(len(dy)) if w is None else f64(w)
    R, I = g.shape
    out = {n: np.zeros((R, 2 * I) if n.startswith("dgu") else ((R, I) if n == "h_w" else R)) for n in ("dgu", "dgu_mag", "h_w", "d_w", "d_w_mag")}
    sg = 1.0 / (1.0 + np.exp(-g))
    h = g * sg * u
    fg, fu = u * sg * (1.0 + g * (1.0 - sg)), g * sg
    for e, a, b in segs:
        if 0 <= e < len(Wd) and b > a:
            W = f64(Wd[e])
            dh, mag, ww = dy[a:b] @ W, np.abs(dy[a:b]) @ np.abs(W), w[a:b, None]
            out["dgu"][a:b] = ww * np.concatenate([dh * fg[a:b], dh * fu[a:b]], 1)
            out["dgu_mag"][a:b] = np.abs(ww) * np.concatenate([mag * np.abs(u[a:b] * sg[a:b]) * (1 + np.abs(g[a:b])), mag * np.abs(fu[a:b])], 1)
            out["h_w"][a:b] = ww * h[a:b]
            out["d_w"][a:b] = (dh * h[a:b]).sum(1)
            out["d_w_mag"][a:b] = (mag * np.abs(h[a:b])).sum(1)
    return out
