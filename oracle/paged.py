"""Rotary positions and the paged cache in 64 bits (NumPy): what the library's
mkv_rope and mkv_paged_* calls are tested against.  Written from the
definitions; shares no code with the library."""
from __future__ import annotations

import math

import numpy as np


def rope_frequencies(rot, base, scaling="none", factor=1.0, original=0.0, low_freq=1.0,
                     high_freq=4.0, beta_fast=32.0, beta_slow=1.0):
    """(radians per position of every pair, factor on rotated vectors)."""
    f, mult = [], 1.0
    for i in range(rot // 2):
        w = base ** (-2.0 * i / rot)
        if scaling == "linear":
            w /= factor
        elif scaling == "ntk":
            w = (base * factor ** (rot / (rot - 2))) ** (-2.0 * i / rot)
        elif scaling == "yarn":
            # index of the pair with `turns` turns over the original context
            at = lambda turns: rot * math.log(original / (2 * math.pi * turns)) / (2 * math.log(base))
            lo, hi = max(0, math.floor(at(beta_fast))), min(rot - 1, math.ceil(at(beta_slow)))
            part = min(1.0, max(0.0, (i - lo) / max(0.001, hi - lo)))
            w = w * (1 - part) + w / factor * part
            mult = 0.1 * math.log(factor) + 1.0
        elif scaling == "banded":
            length = 2 * math.pi / w
            if length > original / low_freq:
                w /= factor
            elif length >= original / high_freq:
                part = (original / length - low_freq) / (high_freq - low_freq)
                w = (1 - part) * w / factor + part * w
        f.append(w)
    return np.array(f), mult


def rope(x, pos, freq, mult=1.0, interleaved=False, transposed=False):
    """x [..., heads, dim], pos [...]."""
    rot = 2 * len(freq)
    th = pos[..., None, None].astype(np.float64) * freq
    if transposed:
        th = -th
    z = mult * np.exp(1j * th)
    x = x.astype(np.float64)
    y = x.copy()
    if interleaved:
        w = (x[..., 0:rot:2] + 1j * x[..., 1:rot:2]) * z
        y[..., 0:rot:2], y[..., 1:rot:2] = w.real, w.imag
    else:
        w = (x[..., : rot // 2] + 1j * x[..., rot // 2:rot]) * z
        y[..., : rot // 2], y[..., rot // 2:rot] = w.real, w.imag
    return y


def gather(pages, table, n, scale=None):
    """Rows 0..n-1 of one sequence, [heads, n, dim], from pages [n_pages, heads, size, dim]."""
    size = pages.shape[2]
    x = np.concatenate([pages[table[i]] for i in range(-(-n // size))], axis=1)[:, :n] if n else \
        np.zeros((pages.shape[1], 0, pages.shape[3]))
    x = x.astype(np.float64)
    return x if scale is None else x * scale[:, None, None]


def decode(q, k, v, scale=None):
    """One sequence: q [q_heads, dim], k, v [heads, n, dim].  (out [q_heads, dim], lse [q_heads],
    weights [heads, n] summed over the group, weights' absolute value sum p |v|)."""
    h, n, d = k.shape
    g = q.shape[0] // h
    scale = d ** -0.5 if scale is None else scale
    out, lse = np.zeros(q.shape), np.full(q.shape[0], -np.inf)
    mass, size = np.zeros((h, n)), np.zeros(q.shape)
    if n:
        for i in range(q.shape[0]):
            z = scale * (k[i // g] @ q[i].astype(np.float64))
            top = z.max()
            p = np.exp(z - top)
            lse[i] = top + math.log(p.sum())
            p /= p.sum()
            out[i], size[i] = p @ v[i // g], p @ np.abs(v[i // g])
            mass[i // g] += p
    return out, lse, mass, size


def evict(acc, pos, next_pos, budget, sink=0, recent=0):
    """One stream of n tokens: src [min(n, budget)], the slot each kept token comes from."""
    n = len(acc)
    if n <= budget:
        return np.arange(n)
    safe = (pos < sink) | (pos.astype(np.int64) >= int(next_pos) - recent)
    a = np.where(np.nan_to_num(acc, nan=0.0, posinf=np.inf) > 0, acc, 0.0).astype(np.float64)
    a[safe] = np.inf
    keep = np.zeros(n, bool)
    keep[np.lexsort((np.arange(n), -a, ~safe))[:budget]] = True
    src = np.arange(budget)
    src[~keep[:budget]] = budget + np.nonzero(keep[budget:])[0]
    return src
