"""fp64 gradient of block / full-utterance attention, from the definition
(test infrastructure only; numpy).

All arrays are float64 [frames, heads, 64]; `segments` lists (first frame,
frames) of every block or utterance.  `out` is the forward's output as the
caller holds it (rounded to bf16 in training), since the gradient is defined
through delta_i = sum_d dout_id out_id."""
from __future__ import annotations

import numpy as np


def segments(cu, block_frames: int = 0):
    """(first, frames) of every block, or (block_frames = 0) utterance, that has frames."""
    segs = []
    for a, b in zip(cu[:-1], cu[1:]):
        step = block_frames or max(int(b - a), 1)
        segs += [(f, min(step, int(b) - f)) for f in range(int(a), int(b), step)]
    return segs


def forward(q, k, v, segs, scale=0.125):
    """(out, lse [heads, frames])."""
    out, lse = np.zeros_like(q), np.zeros((q.shape[1], q.shape[0]))
    for a, n in segs:
        s = np.einsum("ihd,jhd->hij", q[a:a + n], k[a:a + n]) * scale
        m = s.max(-1, keepdims=True)
        p = np.exp(s - m)
        l = p.sum(-1, keepdims=True)
        out[a:a + n] = np.einsum("hij,jhd->ihd", p / l, v[a:a + n])
        lse[:, a:a + n] = (m + np.log(l))[..., 0]
    return out, lse


def backward(dout, q, k, v, out, segs, scale=0.125, bounds=False, rel=2.0 ** -8 + 2.0 ** -12, absd=2.0 ** -17):
    """(dq, dk, dv), and with `bounds` also elementwise bounds of what a kernel
    may be off that rounds P and dS once to bf16 (`rel` of each term, with the
    fp32 error of P's exponent), forms D = dO.v and delta in fp32 (`absd` of
    the sums of absolute products) and rounds the result once (2^-8)."""
    g = [np.zeros_like(q) for _ in range(3)]
    tol = [np.zeros_like(q) for _ in range(3)] if bounds else None
    for a, n in segs:
        sl = slice(a, a + n)
        for h in range(q.shape[1]):
            qq, kk, vv, do, o = (x[sl, h] for x in (q, k, v, dout, out))
            s = qq @ kk.T * scale
            s -= s.max(-1, keepdims=True)
            p = np.exp(s)
            p /= p.sum(-1, keepdims=True)
            ds = p * (do @ vv.T - (do * o).sum(-1, keepdims=True))
            g[0][sl, h], g[1][sl, h], g[2][sl, h] = scale * ds @ kk, scale * ds.T @ qq, p.T @ do
            if bounds:
                ads = rel * np.abs(ds) + absd * p * (np.abs(do) @ np.abs(vv).T + np.abs(do * o).sum(-1, keepdims=True))
                tol[0][sl, h] = scale * ads @ np.abs(kk) + 2.0 ** -8 * np.abs(g[0][sl, h])
                tol[1][sl, h] = scale * ads.T @ np.abs(qq) + 2.0 ** -8 * np.abs(g[1][sl, h])
                tol[2][sl, h] = rel * p.T @ np.abs(do) + 2.0 ** -8 * np.abs(g[2][sl, h])
    return (*g, *tol) if bounds else tuple(g)
