"""fp64 definition of the per-head RMS norm with rotary positions and of its
gradient (test infrastructure only; numpy).

x: [frames, heads, 64] values; pos: [frames]; inv_freq: [rot_dim / 2]; w: [64]
or None.  Pairs are (j, j + rot_dim/2), or (2j, 2j + 1) when interleaved.  The
rotation is applied as one 64 x 64 matrix per frame, so the gradient is its
transpose by construction."""
from __future__ import annotations

import numpy as np


def rotation(pos: float, inv_freq, interleaved: bool = False, rot_scale: float = 1.0, d: int = 64) -> np.ndarray:
    """The matrix R(pos) with y = R z."""
    m = len(inv_freq)
    r = np.eye(d)
    for j in range(m):
        a, b = (2 * j, 2 * j + 1) if interleaved else (j, j + m)
        t = float(pos) * float(inv_freq[j])
        c, s = rot_scale * np.cos(t), rot_scale * np.sin(t)
        r[a, a], r[a, b], r[b, a], r[b, b] = c, -s, s, c
    return r


def rotations(pos, inv_freq, interleaved=False, rot_scale=1.0) -> np.ndarray:
    return np.stack([rotation(p, inv_freq, interleaved, rot_scale) for p in pos]) if len(pos) else np.zeros((0, 64, 64))


def norm(x, w, eps: float):
    """(z, n, r): z = w n, n = x r, r = 1 / sqrt(mean(x^2) + eps)."""
    x = np.asarray(x, np.float64)
    if w is None:
        return x, None, None
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    return x * r * np.asarray(w, np.float64), x * r, r


def norm_rope(x, w, pos, inv_freq, eps=1e-6, interleaved=False, rot_scale=1.0) -> np.ndarray:
    z, _, _ = norm(x, w, eps)
    return np.einsum("fab,fhb->fha", rotations(pos, inv_freq, interleaved, rot_scale), z)


def norm_rope_bwd(dy, x, w, pos, inv_freq, eps=1e-6, interleaved=False, rot_scale=1.0):
    """(dx, dw, dz): gradient of x, of w (None without) and the rotated-back
    gradient dz = R^T dy (of z)."""
    dz = np.einsum("fab,fha->fhb", rotations(pos, inv_freq, interleaved, rot_scale), np.asarray(dy, np.float64))
    if w is None:
        return dz, None, dz
    _, n, r = norm(x, w, eps)
    g = dz * np.asarray(w, np.float64)
    dx = r * (g - n * (g * n).mean(-1, keepdims=True))
    return dx, (dz * n).sum((0, 1)), dz


def positions(cu) -> np.ndarray:
    """Index of every frame of [cu[0], cu[-1]) inside its utterance."""
    cu = np.asarray(cu, np.int64)
    return np.concatenate([np.arange(b - a) for a, b in zip(cu[:-1], cu[1:])] or [np.zeros(0, np.int64)])
