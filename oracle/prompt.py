"""Rotary axes, head norms with rotation and the attention of many queries in 64 bits
(NumPy): what mkv_rope_multi, mkv_norm_rope, mkv_prefill and mkv_paged_attend are
tested against.  Written from the definitions; shares no code with the library."""
from __future__ import annotations

import math

import numpy as np

from oracle import paged as P


def axes_of(sections, order):
    """Axis of each pair."""
    if order == "blocks":
        return np.repeat(np.arange(len(sections)), sections)
    # in rounds: in round k every axis with more than k pairs gets one
    return np.array([a for k in range(max(sections)) for a, n in enumerate(sections) if n > k])


def axes_frequencies(sections, order, restart, base, **scaling):
    axis = axes_of(sections, order)
    if not restart:
        return axis, *P.rope_frequencies(2 * len(axis), base, **scaling)
    f = np.zeros(len(axis))
    for a, n in enumerate(sections):
        f[axis == a], mult = P.rope_frequencies(2 * n, base, **scaling)
    return axis, f, mult


def spin(x, pos, axis, freq, mult=1.0, interleaved=False, transposed=False):
    """x [batch, tokens, heads, dim], pos [axes, batch, tokens]."""
    rot = 2 * len(freq)
    th = np.moveaxis(pos[axis].astype(np.float64), 0, -1)[..., None, :] * freq
    z = mult * np.exp((-1j if transposed else 1j) * th)
    x = x.astype(np.float64)
    y = x.copy()
    a, b = ((slice(0, rot, 2), slice(1, rot, 2)) if interleaved
            else (slice(0, rot // 2), slice(rot // 2, rot)))
    w = (x[..., a] + 1j * x[..., b]) * z
    y[..., a], y[..., b] = w.real, w.imag
    return y


def norm(x, weight, eps):
    """(x r, x r weight, r)."""
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    return x * r, x * r * weight, r


def norm_grad(u, x, weight, eps):
    """Gradients of x and of the weight, from u = R^T dy."""
    n, _, r = norm(x, weight, eps)
    e = u * weight
    dx = r * (e - n * (e * n).mean(-1, keepdims=True))
    return dx, (u * n).reshape(-1, x.shape[-1]).sum(0)


def visible(n, m, causal=True, window=0, prefix=None, docs=None):
    """[n, m]: which of m keys the n queries see, the last query at the last key."""
    p = np.arange(m - n, m)[:, None]
    j = np.arange(m)[None]
    see = np.ones((n, m), dtype=bool)
    if causal:
        see &= (j <= p) | (j < (0 if prefix is None else prefix))
    if window:
        see &= p - j < window
        if not causal:
            see &= j - p < window
    if docs is not None:
        see &= (p >= 0) & (docs[np.maximum(p, 0)] == docs[None, :m])
    return see


def tree_places(rows, base):
    """(places of the new tokens, [new, new]: which sees which) of a tree's rows (integers)."""
    m = len(rows)
    sees = np.array([[r >> j & 1 for j in range(m)] for r in rows], dtype=bool).reshape(m, m)
    depth = (sees & ~np.eye(m, dtype=bool)).sum(1)
    return base + depth, sees


def attend(q, k, v, see, place, at, scale=None, cap=0.0, slopes=None):
    """q [n, Hq, D] at `place` [n], k, v [H, m, D] at `at` [m], see [n, m].  Returns (out, lse, and
    for tolerances: sum of weights times |v|, largest scale sum |q k| of a row, mean |v| sum)."""
    n, hq, d = q.shape
    h = k.shape[0]
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    out, lse = np.zeros((n, hq, d)), np.full((n, hq), -np.inf)
    spread, size, total = np.zeros((n, hq, d)), np.zeros((n, hq)), np.zeros((n, hq, d))
    if k.shape[1] == 0:
        return out, lse, spread, size, total
    for i in range(hq):
        kk, vv = k[i * h // hq], v[i * h // hq]
        z = scale * (q[:, i] @ kk.T)
        a = scale * (np.abs(q[:, i]) @ np.abs(kk).T)
        if cap:
            z = cap * np.tanh(z / cap)
        if slopes is not None:
            far = slopes[i] * np.abs(place[:, None] - at[None])
            z = z - far
            a = a + far
        z = np.where(see, z, -np.inf)
        top = z.max(-1, keepdims=True)
        w = np.exp(z - np.where(np.isinf(top), 0.0, top))
        s = w.sum(-1, keepdims=True)
        with np.errstate(divide="ignore"):
            lse[:, i] = (np.where(np.isinf(top), 0.0, top) + np.log(s))[:, 0]
        w = w / np.where(s > 0, s, 1.0)
        out[:, i] = w @ vv
        spread[:, i] = w @ np.abs(vv)
        size[:, i] = np.where(see, a, 0.0).max(-1)
        total[:, i] = see.astype(np.float64) @ np.abs(vv)
    return out, lse, spread, size, total
