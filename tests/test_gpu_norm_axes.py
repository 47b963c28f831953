"""Norms of heads with rotations of several axes, and their gradients, against the 64-bit oracle:
every form of a unit (vectors of half pairs, of interleaved pairs, elements, two units a lane) with
blocks and cyclic axes.  Tolerances as derived in test_gpu_prompt.py (norm, grad)."""
import numpy as np
import pytest
import torch

from oracle import paged as P
from oracle import prompt as O
from test_gpu_prompt import BF16, DEV, F16, F32, HALF, M, U, f64, i32, near, pair_length, rnd  # noqa: F401

pytestmark = pytest.mark.gpu

PLANS = [  # sections, order, restart, head_dim, interleaved
    ((16, 24, 24), "blocks", False, 128, False), ((16, 24, 24), "cyclic", True, 128, False),
    ((16, 24, 24), "cyclic", False, 128, True), ((20, 20), "blocks", True, 80, True),
    ((64, 32, 32), "blocks", False, 256, False), ((40, 44, 44), "cyclic", True, 256, True),
    ((8, 8, 16), "cyclic", False, 256, False), ((4, 8, 4), "blocks", True, 256, True),
    ((5, 1, 7, 3), "cyclic", True, 40, False), ((3, 9), "cyclic", False, 29, True), ((6, 5, 5), "blocks", False, 33, False),
    ((1,), "blocks", False, 2, True), ((2, 2), "cyclic", False, 8, True)]
SHAPES = [(1, 1, 1, 0), (2, 19, 5, 2), (1, 130, 28, 4)]


def inputs(shape, dim, dtype, seed):
    b, t, h, kv = shape
    proj = rnd((b, t, h + kv + 1, dim), dtype, seed, 1.5)
    return proj[:, :, :h], proj[:, :, h:h + kv] if kv else None


def grad_near(dx, dw, u, x, weight, eps, rot, inter, dtype):
    d = x.shape[-1]
    want, want_w = O.norm_grad(u, f64(x), weight, eps)
    n, _, r = O.norm(f64(x), weight, eps)
    e = pair_length(u, rot, inter) * np.abs(weight)
    en = (e * np.abs(n)).mean(-1, keepdims=True)
    tol = r * U * ((d / 2 + 24) * e + (2.5 * d + 48) * np.abs(n) * en) + HALF[dtype] * np.abs(want) * 1.01
    near(f64(dx), want, tol + (2.0**-25 if dtype == F16 else 0.0))
    if dw is not None:
        terms = (pair_length(u, rot, inter) * np.abs(n)).reshape(-1, d)
        near(f64(dw), want_w, (d / 2 + 20 + len(terms)) * U * terms.sum(0))


@pytest.mark.parametrize("dtype,wtype", [(F16, F32), (BF16, BF16), (F32, F32)])
@pytest.mark.parametrize("sections,order,restart,dim,inter", PLANS)
@pytest.mark.parametrize("shape", SHAPES)
def test_norm_and_gradient(M, sections, order, restart, dim, inter, shape, dtype, wtype):
    b, t, h, kv = shape
    q, k = inputs(shape, dim, dtype, dim + t)
    w = [rnd((dim,), wtype, s, 0.3) for s in (1, 2)]
    pos = np.random.default_rng(t).integers(-5, 1 << 20, (len(sections), b, t))
    plan = M.mkv_rope_axes_plan(dim, sections, order=order, restart=restart, base=5000.0, interleaved=inter)
    axis, freq, mult = O.axes_frequencies(sections, order, restart, 5000.0)
    rot = 2 * len(axis)
    kw = dict(eps=1e-5, weight_offset=0.5, k=k, k_weight=w[1] if kv else None)
    got = M.mkv_norm_rope(plan, q, w[0], i32(pos), **kw)
    for x, y, weight in zip((q, k), got if kv else (got,), w):
        n = O.norm(f64(x), f64(weight) + 0.5, 1e-5)[1]
        want = O.spin(n, pos, axis, freq, mult, inter)
        tol = (dim / 2 + 20) * U * pair_length(n, rot, inter) + HALF[dtype] * np.abs(want) * 1.01
        near(f64(y), want, tol + (2.0**-25 if dtype == F16 else 0.0))
    dy = [rnd(x.shape, dtype, 7) if x is not None else None for x in (q, k)]
    got = M.mkv_norm_rope_grad(plan, dy[0], q, w[0], i32(pos), dk=dy[1], **kw)
    dxs, dws = (got[:2], got[2:]) if kv else (got[:1], got[1:])
    for x, g, weight, dx, dw in zip((q, k), dy, w, dxs, dws):
        grad_near(dx, dw, O.spin(f64(g), pos, axis, freq, mult, inter, True), x, f64(weight) + 0.5, 1e-5, rot, inter, dtype)


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("dim,rot,inter", [(128, 128, False), (256, 64, True), (33, 16, False)])
def test_gradient_from_a_first_position_without_weights_and_over_its_input(M, dtype, dim, rot, inter):
    """Positions first_pos + token; no weights, to which no offset is added; out = x and out = grad."""
    q, k = inputs((2, 37, 3, 2), dim, dtype, dim)
    g, gk = rnd(q.shape, dtype, 7), rnd(k.shape, dtype, 8)
    plan = M.mkv_rope_plan(dim, rot_dim=rot, interleaved=inter)
    freq, mult = P.rope_frequencies(rot, 10000.0)
    pos = np.tile(900000 + np.arange(37), (2, 1))
    n = O.norm(f64(q), 1.0, 1e-6)[1]
    want = P.rope(n, pos, freq, mult, inter)
    tol = (dim / 2 + 20) * U * pair_length(n, rot, inter) + HALF[dtype] * np.abs(want) * 1.01
    near(f64(M.mkv_norm_rope(plan, q, first_pos=900000, weight_offset=0.5)), want, tol + (2.0**-25 if dtype == F16 else 0.0))
    kw = dict(first_pos=900000, weight_offset=0.5)
    dq, dk, dw, dkw = M.mkv_norm_rope_grad(plan, g, q, dk=gk, k=k, **kw)
    assert dw is None and dkw is None
    for x, dy, dx in ((q, g, dq), (k, gk, dk)):
        grad_near(dx, None, P.rope(f64(dy), pos, freq, mult, inter, True), x, np.ones(dim), 1e-6, rot, inter, dtype)
    w = rnd((dim,), F32, 3, 0.3)
    want = M.mkv_norm_rope_grad(plan, g, q, w, dk=gk, k=k, **kw)          # k has no weight
    assert want[3] is None
    x, y = q.clone(), g.clone()
    got = M.mkv_norm_rope_grad(plan, g, x, w, dq_out=x, **kw)
    assert got[0] is x and torch.equal(x, want[0]) and torch.equal(got[1], want[2])
    got = M.mkv_norm_rope_grad(plan, y, q, w, dq_out=y, **kw)
    assert got[0] is y and torch.equal(y, want[0]) and torch.equal(got[1], want[2])
