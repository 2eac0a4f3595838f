"""Plain float64 restatements of the balance loss, the counter-based dropout
and the per-request adapters, on the CPU (numpy), for the GPU parity tests.

They are written from the definitions in include/moe_topk.h, sequence by
sequence and request by request, and share no code with the package.
"""
from __future__ import annotations

import numpy as np


# -------------------------------------------------------------- balance loss

def balance(logits, idx, mask, offsets, k, a=0.0, b=0.0):
    """counts, tokens, prob_sum, loss, dlogits of a loss[0] + b loss[1]; also
    `mag`, dlogits' formula with every term's magnitude added (for error bounds)."""
    l = np.asarray(logits, np.float64)
    T, E = l.shape
    S = len(offsets) - 1
    on = np.ones(T, bool) if mask is None else np.asarray(mask) != 0
    counts, tokens = np.zeros((S, E), np.int64), np.zeros(S, np.int64)
    P, z = np.zeros((S, E)), 0.0
    rows = [np.flatnonzero(on[s:e]) + s for s, e in zip(offsets, offsets[1:])]
    n = max(1, sum(len(r) for r in rows))
    dl, mag = np.zeros((T, E)), np.zeros((T, E))
    bal = 0.0
    for q, r in enumerate(rows):
        if not len(r):
            continue
        top = l[r].max(1, keepdims=True)
        ex = np.exp(l[r] - top)
        p = ex / ex.sum(1, keepdims=True)
        lse = (top + np.log(ex.sum(1, keepdims=True)))[:, 0]
        tokens[q] = len(r)
        np.add.at(counts[q], np.asarray(idx)[r].reshape(-1), 1)
        P[q] = p.sum(0)
        per = E / (k * len(r) * n)
        bal += per * (counts[q] * P[q]).sum()
        z += (lse * lse).sum() / n
        mean = p @ counts[q][:, None]
        dl[r] = p * (a * per * (counts[q] - mean) + 2 * b / n * lse[:, None])
        mag[r] = p * (abs(a) * per * (counts[q] + mean) + 2 * abs(b) / n * np.abs(lse)[:, None])
    return dict(counts=counts, tokens=tokens, prob_sum=P, loss=np.array([bal, z]), dlogits=dl, mag=mag)


# ------------------------------------------------------------------- dropout

def philox4x32(ctr, key, rounds=10):
    """ctr [n,4], key (2 words) -> [n,4] (uint32), Philox4x32 of Salmon et al. 2011."""
    c = [np.asarray(ctr)[:, i].astype(np.uint64) for i in range(4)]
    k = [int(key[0]), int(key[1])]
    low, w = np.uint64(0xFFFFFFFF), np.uint64(32)
    for _ in range(rounds):
        p0, p1 = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(p1 >> w) ^ c[1] ^ np.uint64(k[0]), p1 & low, (p0 >> w) ^ c[3] ^ np.uint64(k[1]), p0 & low]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return np.stack(c, 1).astype(np.uint32)


def dropped_below(p):
    return int(np.floor(p * 65536 + 0.5))


def keep(seed, offset, first, n, p):
    """Which of elements first .. first+n-1 stay (first a multiple of 8)."""
    assert first % 8 == 0
    blocks = np.array([(offset + first // 8 + i) % (1 << 64) for i in range((n + 7) // 8)], dtype=object)
    ctr = np.zeros((len(blocks), 4), np.uint64)
    ctr[:, 0] = [int(v) & 0xFFFFFFFF for v in blocks]
    ctr[:, 1] = [int(v) >> 32 for v in blocks]
    seed %= 1 << 64
    words = philox4x32(ctr, (seed & 0xFFFFFFFF, seed >> 32))
    bits = np.stack([words & 0xFFFF, words >> 16], 2).reshape(-1)[:n]
    return bits >= dropped_below(p)


def factor(p):
    d = dropped_below(p)
    return 65536.0 / (65536 - d) if d < 65536 else 0.0


# ------------------------------------------------------------------ adapters

def adapter(x, W, A, B, scale, offsets, which, dy=None):
    """y (and with dy: dx, dA, dB) in float64; each with the sum of its terms'
    magnitudes as <name>_mag (for error bounds)."""
    f = lambda v: np.asarray(v, np.float64)  # noqa: E731
    x, W, A, B = f(x), f(W), f(A), f(B)
    sc = np.ones(len(A)) if scale is None else f(scale)
    out = dict(y=x @ W.T, y_mag=np.abs(x) @ np.abs(W).T)
    if dy is not None:
        dy = f(dy)
        out.update(dx=dy @ W, dx_mag=np.abs(dy) @ np.abs(W), dA=np.zeros_like(A), dB=np.zeros_like(B),
                   dA_mag=np.zeros_like(A), dB_mag=np.zeros_like(B))
    for s, e, w in zip(offsets, offsets[1:], which):
        if w < 0 or e <= s:
            continue
        a, b, c = A[w], B[w], sc[w]
        v, va = c * (x[s:e] @ a.T), abs(c) * (np.abs(x[s:e]) @ np.abs(a).T)
        out["y"][s:e] += v @ b.T
        out["y_mag"][s:e] += va @ np.abs(b).T
        if dy is not None:
            u, ua = c * (dy[s:e] @ b), abs(c) * (np.abs(dy[s:e]) @ np.abs(b))
            out["dx"][s:e] += u @ a
            out["dx_mag"][s:e] += ua @ np.abs(a)
            out["dA"][w] += u.T @ x[s:e]
            out["dA_mag"][w] += ua.T @ np.abs(x[s:e])
            out["dB"][w] += dy[s:e].T @ v
            out["dB_mag"][w] += np.abs(dy[s:e]).T @ va
    return out
