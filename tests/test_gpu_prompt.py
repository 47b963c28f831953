"""Rotary axes, head norms with rotation and the attention of many queries on the GPU
against the 64-bit oracle.

Tolerances, derived here once (u = 2^-24, e(t) = the half step of the output type):

multi    As one axis: 12 u of a pair's length, the output's rounding, and 2^-25 below
         fp16's normal range.
norm     A sum of D squares and its root are within (D / 2 + 4) u of r, the products with
         r and the weight add 3 u, the rotation 12 u: (D / 2 + 20) u of a pair's length, then
         the output's rounding.
grad     u = R^T dy within 12 u of the pair's length, n within (D / 2 + 6) u.  e = u w: (14 u)
         of the pair.  mean(e n): a sum of D products whose terms are off by (D / 2 + 20) u:
         (3 D / 2 + 24) u mean|e n|.  So dx within r u ((D / 2 + 24) |e| + (5 D / 2 + 48) |n|
         mean|e n|), |e| the length of its pair, and the output's rounding.  dw: N terms, each
         off by (D / 2 + 20) u of its size, and N u for their sum.
scores   A sum of D exact products in fp32 by matrix steps: (D / 16 + 4) 2^-22 A, A = scale
         sum |q k| (and the taken-off slope times distance, twice rounded).  tanh: 2^-21 of
         the cap.  d: their sum.
attend   Weights off by 2 d + 2^-16 relative, and by the 16-bit rounding's e; sums of n terms by
         n u: out within (2 d + 2^-16 + e + (n + 64) u) sum p |v| + e |o|.  fp16 weights carry
         a factor 2^8 and are off by up to 2^-25 below the normal range, so by 2^-33 sum |v|
         more.  lse within d + (n + 64) u + 2^-22 |lse| + 2^-21.
"""
import math

import numpy as np
import pytest
import torch

from oracle import paged as P
from oracle import prompt as O

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
U = 2.0**-24
HALF = {torch.float16: 2.0**-11, torch.bfloat16: 2.0**-8, torch.float32: U}
F16, BF16, F32, E4M3 = torch.float16, torch.bfloat16, torch.float32, torch.float8_e4m3fn


@pytest.fixture(scope="module")
def M():
    from two_compressed_kv_gb300 import mkv
    return mkv


def f64(t):
    return t.detach().to(torch.float32).cpu().numpy().astype(np.float64)


def rnd(shape, dtype, seed, size=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * size).to(dtype).to(DEV)


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


def near(got, want, tol):
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (np.argwhere(bad)[:4].tolist(), int(bad.sum()),
                           float(np.nanmax(np.where(bad, np.abs(got - want) / np.maximum(tol, 1e-300), 0))))


# ---- axes ---------------------------------------------------------------------------------------

def pair_length(x, rot, interleaved):
    x = np.abs(x)
    out = x.copy()
    if interleaved:
        out[..., 0:rot:2] = out[..., 1:rot:2] = np.hypot(x[..., 0:rot:2], x[..., 1:rot:2])
    else:
        r = np.hypot(x[..., :rot // 2], x[..., rot // 2:rot])
        out[..., :rot] = np.concatenate([r, r], -1)
    return out


AXES = [  # sections, order, restart, dim, interleaved
    ((8, 12, 12), "blocks", False, 64, False), ((16, 24, 24), "cyclic", False, 128, False),
    ((20, 20), "blocks", True, 80, True), ((1,), "blocks", False, 2, True),
    ((5, 1, 7, 3), "cyclic", True, 40, False), ((64, 32, 32), "blocks", False, 256, False),
    ((3, 9), "cyclic", False, 24, True)]


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("sections,order,restart,dim,inter", AXES)
@pytest.mark.parametrize("batch,tokens,heads", [(1, 1, 1), (2, 37, 5), (3, 130, 28)])
def test_multi(M, dtype, sections, order, restart, dim, inter, batch, tokens, heads):
    x = rnd((batch, tokens, heads, dim), dtype, dim + tokens)
    rng = np.random.default_rng(tokens)
    pos = rng.integers(-5, 1 << 20, (len(sections), batch, tokens))
    plan = M.mkv_rope_axes_plan(dim, sections, order=order, restart=restart, base=5000.0, interleaved=inter)
    axis, freq, mult = O.axes_frequencies(sections, order, restart, 5000.0)
    rot = 2 * len(axis)
    for back in (False, True):
        want = O.spin(f64(x), pos, axis, freq, mult, inter, back)
        tol = 12 * U * pair_length(f64(x), rot, inter) + HALF[dtype] * np.abs(want) * 1.01
        tol += 2.0**-25 if dtype == F16 else 0.0
        near(f64(M.mkv_rope_multi(plan, x, i32(pos), transposed=back)), want, tol)


def test_multi_strides_in_place_and_shared_positions(M):
    """Odd strides take the element form; a broadcast picture of positions; in place."""
    sections, dim = (6, 5, 5), 33
    big = rnd((2, 19, 4, 40), BF16, 1)
    x = big[..., 1:34]
    pos = i32(np.arange(3 * 19).reshape(3, 1, 19) * 7).expand(3, 2, 19)
    plan = M.mkv_rope_axes_plan(dim, sections)
    axis, freq, _ = O.axes_frequencies(sections, "blocks", False, 10000.0)
    want = O.spin(f64(x), pos.cpu().numpy(), axis, freq)
    tol = 12 * U * pair_length(f64(x), 32, False) + HALF[BF16] * np.abs(want) * 1.01
    rest = big[..., 34:].clone()
    out = M.mkv_rope_multi(plan, x, pos, out=x)
    assert out is x
    near(f64(x), want, tol)
    assert torch.equal(big[..., 34:], rest)


def test_multi_of_one_axis_is_rope(M):
    x = rnd((2, 65, 3, 96), BF16, 9)
    pos = i32(np.arange(130).reshape(2, 65) * 31)
    one = M.mkv_rope(M.mkv_rope_plan(96, rot_dim=64), x, pos)
    assert torch.equal(one, M.mkv_rope_multi(M.mkv_rope_axes_plan(96, (32,)), x, pos[None]))
    three = M.mkv_rope_multi(M.mkv_rope_axes_plan(96, (8, 12, 12), order="cyclic"), x, pos.expand(3, 2, 65))
    assert torch.equal(one, three)


# ---- norms --------------------------------------------------------------------------------------

NORM = [  # batch, tokens, heads, kv heads, dim, rot, interleaved
    (1, 1, 1, 0, 128, 128, False), (2, 1, 32, 8, 128, 128, False), (3, 33, 5, 2, 64, 64, True),
    (1, 300, 3, 3, 80, 80, False), (2, 17, 4, 1, 96, 64, True), (1, 40, 2, 2, 256, 256, False),
    (1, 40, 2, 2, 256, 64, True), (2, 9, 3, 1, 256, 128, False), (1, 21, 2, 1, 30, 10, True),
    (2, 5, 1, 3, 33, 16, False), (1, 3, 2, 2, 8, 8, True), (1, 130, 28, 4, 128, 64, False)]


def norm_inputs(shape, dtype, seed, views=True):
    b, t, h, kv, d, _, _ = shape
    proj = rnd((b, t, h + kv + 1, d), dtype, seed, 1.5)
    q, k = proj[:, :, :h], proj[:, :, h:h + kv]
    return (q, k if kv else None) if views else (q.contiguous(), k.contiguous() if kv else None)


@pytest.mark.parametrize("dtype,wtype", [(F16, F16), (BF16, F32), (F32, F32), (BF16, BF16)])
@pytest.mark.parametrize("shape", NORM)
def test_norm(M, shape, dtype, wtype):
    b, t, h, kv, d, rot, inter = shape
    q, k = norm_inputs(shape, dtype, 3 * d + t)
    w = [rnd((d,), wtype, s, 0.3) for s in (1, 2)]
    pos = np.random.default_rng(t).integers(0, 1 << 20, (b, t))
    plan = M.mkv_rope_plan(d, rot_dim=rot, interleaved=inter)
    freq, mult = P.rope_frequencies(rot, 10000.0)
    got = M.mkv_norm_rope(plan, q, w[0], i32(pos), k=k, k_weight=w[1] if kv else None, eps=1e-5, weight_offset=1.0)
    for x, y, weight in zip((q, k), got if kv else (got,), w):
        n = O.norm(f64(x), f64(weight) + 1.0, 1e-5)[1]
        want = P.rope(n, pos, freq, mult, inter)
        tol = (d / 2 + 20) * U * pair_length(n, rot, inter) + HALF[dtype] * np.abs(want) * 1.01
        near(f64(y), want, tol + (2.0**-25 if dtype == F16 else 0.0))


@pytest.mark.parametrize("dtype,wtype", [(F16, F32), (BF16, BF16), (F32, F32)])
@pytest.mark.parametrize("shape", NORM + [(2, 700, 16, 4, 128, 128, False)])
def test_norm_grad(M, shape, dtype, wtype):
    b, t, h, kv, d, rot, inter = shape
    q, k = norm_inputs(shape, dtype, 5 * d + t)
    w = [rnd((d,), wtype, s, 0.3) for s in (1, 2)]
    pos = np.random.default_rng(t).integers(0, 1 << 20, (b, t))
    plan = M.mkv_rope_plan(d, rot_dim=rot, interleaved=inter)
    freq, mult = P.rope_frequencies(rot, 10000.0)
    dy = [rnd(x.shape, dtype, 7) if x is not None else None for x in (q, k)]
    got = M.mkv_norm_rope_grad(plan, dy[0], q, w[0], i32(pos), dk=dy[1], k=k, k_weight=w[1] if kv else None,
                               eps=1e-5, weight_offset=0.5)
    dxs, dws = (got[:2], got[2:]) if kv else (got[:1], got[1:])
    for x, g, weight, dx, dw in zip((q, k), dy, w, dxs, dws):
        weight = f64(weight) + 0.5
        u = P.rope(f64(g), pos, freq, mult, inter, True)
        want, want_w = O.norm_grad(u, f64(x), weight, 1e-5)
        n, _, r = O.norm(f64(x), weight, 1e-5)
        e = pair_length(u, rot, inter) * np.abs(weight)
        en = (e * np.abs(n)).mean(-1, keepdims=True)
        tol = r * U * ((d / 2 + 24) * e + (2.5 * d + 48) * np.abs(n) * en) + HALF[dtype] * np.abs(want) * 1.01
        near(f64(dx), want, tol + (2.0**-25 if dtype == F16 else 0.0))
        terms = (pair_length(u, rot, inter) * np.abs(n)).reshape(-1, d)
        near(f64(dw), want_w, (d / 2 + 20 + len(terms)) * U * terms.sum(0))


def test_norm_grad_against_differences(M):
    """The gradient of a weighted sum of the forward call's fp32 outputs, by central differences:
    their own error is a step's square (1e-4) and rounding over the step."""
    d, shape = 64, (1, 3, 2, 64)
    x, g, w = rnd(shape, F32, 1), rnd(shape, F32, 2), rnd((d,), F32, 3, 0.3) + 1.0
    pos = i32([[5, 900, 77]])
    plan = M.mkv_rope_plan(d)
    f = lambda x, w: float((M.mkv_norm_rope(plan, x, w, pos).double() * g.double()).sum())
    dx, dw = M.mkv_norm_rope_grad(plan, g, x, w, pos)
    for seed in range(3):
        to, tw, step = rnd(shape, F32, 10 + seed), rnd((d,), F32, 20 + seed), 2.0**-6
        num = (f(x + step * to, w) - f(x - step * to, w)) / (2 * step)
        assert abs(num - float((dx * to).sum())) <= 2e-2
        num = (f(x, w + step * tw) - f(x, w - step * tw)) / (2 * step)
        assert abs(num - float((dw * tw).sum())) <= 2e-3


def test_norm_axes_in_place_and_no_weight(M):
    q = rnd((2, 50, 4, 128), BF16, 4)
    pos = i32(np.random.default_rng(0).integers(0, 5000, (3, 2, 50)))
    plan = M.mkv_rope_axes_plan(128, (16, 24, 24))
    axis, freq, _ = O.axes_frequencies((16, 24, 24), "blocks", False, 10000.0)
    n = O.norm(f64(q), 1.0, 1e-6)[1]
    want = O.spin(n, pos.cpu().numpy(), axis, freq)
    out = M.mkv_norm_rope(plan, q, None, pos, q_out=q)
    assert out is q
    near(f64(q), want, 84 * U * pair_length(n, 128, False) + HALF[BF16] * np.abs(want) * 1.01)


def test_norm_grad_in_place_repeats_and_empty(M):
    q, g, w = rnd((2, 300, 8, 128), BF16, 4), rnd((2, 300, 8, 128), BF16, 5), rnd((128,), F32, 6)
    plan = M.mkv_rope_plan(128)
    dx, dw = M.mkv_norm_rope_grad(plan, g, q, w)
    again = M.mkv_norm_rope_grad(plan, g, q, w)
    assert torch.equal(dx, again[0]) and torch.equal(dw, again[1])
    out, dw2 = M.mkv_norm_rope_grad(plan, g, q, w, dq_out=g)
    assert out is g and torch.equal(g, dx) and torch.equal(dw2, dw)
    none = torch.empty((0, 3, 8, 128), dtype=BF16, device=DEV)
    dx, dw = M.mkv_norm_rope_grad(plan, none, none, w)
    assert dx.numel() == 0 and not dw.any()


# ---- prompts ------------------------------------------------------------------------------------

def score_error(d, size, cap):
    return (d / 16 + 4) * 2.0**-22 * size + (2.0**-21 * cap if cap else 0.0)


def attend_near(got, lse, ref, dtype, n, cap=0.0, what=""):
    out, want_lse, spread, size, total = ref
    d = score_error(out.shape[-1], size, cap)[..., None]
    e = HALF[dtype]
    tol = (2 * d + 2.0**-16 + e + (n + 64) * U) * spread + e * np.abs(out) * 1.01
    tol = tol + (2.0**-33 * total + 2.0**-25 if dtype == F16 else 0.0)
    near(got, out, tol)
    if lse is not None:
        live = np.isfinite(want_lse)
        assert np.array_equal(np.isfinite(lse), live) and (lse[~live] == -np.inf).all()
        near(lse[live], want_lse[live], (d[..., 0] + (n + 64) * U + 2.0**-22 * np.abs(want_lse) + 2.0**-21)[live])


def prefill_check(M, dtype, b, nq, nk, heads, kv, d, seed=0, q_lens=None, kv_lens=None, prefix=None, docs=None,
                  cap=0.0, slopes=None, scale=0.0, size=1.0, head_major=False, causal=True, window=0, stray=None):
    q = rnd((b, nq, heads, d), dtype, seed + 1, size)
    k, v = rnd((b, nk, kv, d), dtype, seed + 2, size), rnd((b, nk, kv, d), dtype, seed + 3)
    kl = [nk] * b if kv_lens is None else [int(x) for x in kv_lens]
    ql = [nq] * b if q_lens is None else [int(x) for x in q_lens]
    if stray is not None:        # what lies behind a sequence's keys and queries
        for i in range(b):
            k[i, kl[i]:] = stray
            v[i, kl[i]:] = stray
            q[i, ql[i]:] = stray
    if head_major:
        q, k, v = (x.transpose(1, 2).contiguous().transpose(1, 2) for x in (q, k, v))
    out = torch.full_like(q, 7.0)
    lse = torch.full((b, nq, heads), 7.0, device=DEV)
    back = M.mkv_prefill(q, k, v, out=out, lse=lse, causal=causal, window=window,
                         prefix=None if prefix is None else i32(prefix), docs=None if docs is None else i32(docs),
                         q_lens=None if q_lens is None else i32(q_lens),
                         kv_lens=None if kv_lens is None else i32(kv_lens), scale=scale, cap=cap,
                         slopes=None if slopes is None else torch.tensor(slopes, dtype=F32, device=DEV))
    assert back is out
    for i in range(b):
        n, m = ql[i], kl[i]
        see = O.visible(n, m, causal, window, None if prefix is None else prefix[i],
                        None if docs is None else np.asarray(docs[i]))
        ref = O.attend(f64(q[i, :n]), f64(k[i, :m]).transpose(1, 0, 2), f64(v[i, :m]).transpose(1, 0, 2), see,
                       np.arange(m - n, m), np.arange(m), scale or None, cap, slopes)
        attend_near(f64(out[i, :n]), f64(lse[i, :n]), ref, dtype, m, cap)
        assert (out[i, n:] == 7.0).all() and (lse[i, n:] == 7.0).all()


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("nq,nk", [(1, 1), (1, 2), (2, 2), (1, 300), (17, 17), (63, 200), (64, 64), (65, 65),
                                   (127, 127), (128, 128), (129, 129), (130, 257), (300, 300), (255, 513)])
def test_prefill_lengths(M, dtype, d, nq, nk):
    prefill_check(M, dtype, 2, nq, nk, 4, 2, d)


@pytest.mark.parametrize("heads,kv", [(1, 1), (3, 1), (8, 8), (7, 1), (28, 4), (16, 1), (40, 2), (128, 1), (65, 1)])
@pytest.mark.parametrize("causal", [True, False])
def test_prefill_heads(M, heads, kv, causal):
    prefill_check(M, BF16, 1, 70, 150, heads, kv, 128, causal=causal)


MASKS = [dict(causal=False), dict(window=2**31 - 1), dict(window=2**31 - 1, causal=False), dict(window=1), dict(window=50), dict(window=200, causal=False), dict(window=1, causal=False),
         dict(prefix=[100, 0]), dict(prefix=[3, 1000]), dict(prefix=[260, 130], window=70),
         dict(docs="blocks"), dict(docs="mixed"), dict(docs="mixed", causal=False), dict(docs="blocks", window=40),
         dict(docs="blocks", prefix=[90, 200]), dict(docs="own"), dict(cap=2.0), dict(cap=30.0, size=4.0),
         dict(cap=0.5, size=6.0), dict(slopes=True), dict(slopes=True, causal=False),
         dict(slopes=True, cap=5.0, window=90), dict(scale=0.7), dict(size=8.0)]


@pytest.mark.parametrize("d,heads,kv", [(128, 6, 2), (64, 4, 4), (256, 4, 1)])
@pytest.mark.parametrize("kw", MASKS)
def test_prefill_masks(M, d, heads, kv, kw):
    kw = dict(kw)
    n = 290
    if kw.get("slopes"):
        kw["slopes"] = [2.0**(-8.0 * (i + 1) / heads) for i in range(heads)]
    if "docs" in kw:
        at = np.arange(n)
        kw["docs"] = {"blocks": np.stack([(at >= 31) * 5 + (at >= 160), (at >= 128) * 1 - (at >= 250)]),
                      "mixed": np.stack([at % 3, (at // 7) % 2]), "own": np.stack([at, -at])}[kw["docs"]]
    prefill_check(M, BF16, 2, n, n, heads, kv, d, **kw)
    prefill_check(M, F16, 2, 133, n, heads, kv, d, seed=40, **kw)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("stray", [float("nan"), float("inf"), 60000.0])
def test_prefill_ragged(M, d, causal, stray):
    """Empty sequences, more queries than keys (some see nothing), garbage behind the lengths."""
    prefill_check(M, F16, 6, 140, 270, 4, 2, d, q_lens=[0, 1, 140, 100, 37, 140], kv_lens=[0, 1, 270, 40, 0, 131],
                  causal=causal, stray=stray, head_major=True)
    prefill_check(M, BF16, 3, 140, 140, 2, 2, d, q_lens=[129, 64, 3], kv_lens=[129, 64, 3], causal=causal,
                  stray=float("nan"), docs=[[0] * 70 + [1] * 70] * 3)


def test_prefill_queries_that_see_nothing(M):
    prefill_check(M, BF16, 2, 200, 60, 2, 1, 128)
    prefill_check(M, BF16, 2, 200, 60, 2, 1, 128, prefix=[5, 0])
    prefill_check(M, BF16, 1, 30, 60, 2, 1, 128, q_lens=[30], kv_lens=[0])


def test_prefill_long_few_rows(M):
    """One part of a prompt over many cached tokens, and a long window that starts late."""
    prefill_check(M, BF16, 1, 3, 9001, 8, 2, 128)
    prefill_check(M, F16, 2, 40, 5000, 4, 4, 64, window=300)
    prefill_check(M, BF16, 1, 2, 4099, 2, 1, 256, kv_lens=[4099], docs=[[0] * 4000 + [1] * 99])


def test_prefill_scores_far_apart(M):
    """A row whose maximum grows in every block, and one that only falls."""
    d, n = 128, 700
    q = torch.zeros((1, n, 2, d), dtype=F16, device=DEV)
    q[..., 0] = 16.0
    k = torch.zeros((1, n, 1, d), dtype=F16, device=DEV)
    for up in (True, False):
        ramp = torch.linspace(-60, 60, n) * (1 if up else -1)
        k[0, :, 0, 0] = ramp.to(F16).to(DEV)
        v = rnd((1, n, 1, d), F16, 5)
        out = M.mkv_prefill(q, k, v, causal=False)
        ref = O.attend(f64(q[0]), f64(k[0]).transpose(1, 0, 2), f64(v[0]).transpose(1, 0, 2),
                       np.ones((n, n), bool), np.arange(n), np.arange(n))
        attend_near(f64(out[0]), None, ref, F16, n)


@pytest.mark.parametrize("d,heads,kv", [(64, 24, 24), (128, 48, 16), (256, 24, 24)])
@pytest.mark.parametrize("kw", [dict(), dict(window=100), dict(docs=True), dict(cap=10.0, causal=False)])
def test_prefill_many_pieces(M, d, heads, kv, kw):
    """More pieces of work than the GPU runs at once, of unequal lengths, some without any."""
    kw = dict(kw)
    n = 700
    if kw.get("docs"):
        kw["docs"] = np.sort(np.random.default_rng(3).integers(0, 9, (8, n)), 1)
    lens = [700, 1, 0, 333, 64, 650, 129, 511]
    prefill_check(M, BF16, 8, n, n, heads, kv, d, q_lens=lens, kv_lens=lens, stray=float("nan"), **kw)


@pytest.mark.parametrize("ctype,qtype", [(F16, F16), (E4M3, BF16)])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("m", [1, 40])
def test_attend_many_pieces(M, ctype, qtype, d, m):
    rng = np.random.default_rng(m)
    lens = [int(x) for x in rng.integers(0, 700, 40)]
    new = [min(m, n) if i % 3 else min(1, n) for i, n in enumerate(lens)]
    attend_check(M, ctype, qtype, lens, m, 8, 5, d, 48, new=new, tree=[random_tree(rng, m) for _ in lens])


def test_prefill_strided_views_and_streams(M):
    """q, k and v as views of one projection, the result into a view, on another stream."""
    proj = rnd((2, 150, 4 + 2 + 2, 128), BF16, 3)
    q, k, v = proj[:, :, :4], proj[:, :, 4:6], proj[:, :, 6:]
    out = torch.zeros((2, 4, 200, 128), dtype=BF16, device=DEV)
    want = M.mkv_prefill(q.contiguous(), k.contiguous(), v.contiguous())
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    M.mkv_prefill(q, k, v, out=out[:, :, 20:170].transpose(1, 2), stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(out[:, :, 20:170].transpose(1, 2), want)
    assert not out[:, :, :20].any() and not out[:, :, 170:].any()
    assert torch.equal(want, M.mkv_prefill(q, k, v))


def test_prefill_empty_calls(M):
    q = rnd((2, 0, 4, 64), F16, 1)
    assert M.mkv_prefill(q, rnd((2, 5, 4, 64), F16, 1), rnd((2, 5, 4, 64), F16, 1)).numel() == 0
    q = rnd((2, 3, 4, 64), F16, 1)
    none = rnd((2, 0, 4, 64), F16, 1)
    lse = torch.zeros((2, 3, 4), device=DEV)
    assert not M.mkv_prefill(q, none, none, lse=lse).any() and (lse == -np.inf).all()


# ---- new tokens over pages ----------------------------------------------------------------------

def make_cache(M, ctype, b, h, d, ps, per, seed, scales=True, extra=2):
    n = b * per + extra
    g = torch.Generator().manual_seed(seed)
    table = torch.randperm(n, generator=g)[:b * per].view(b, per).to(torch.int32).to(DEV)
    kp, vp = (rnd((n, h, ps, d), F32, seed + s).to(ctype) for s in (1, 2))
    ks = vs = None
    if ctype == E4M3 and scales:
        ks, vs = ((torch.rand(h, generator=g) + 0.5).to(DEV) for _ in range(2))
    return M.MkvPaged(kp, vp, table, k_scale=ks, v_scale=vs)


def rows_of(cache, which, b, n):
    pages, scale = ((cache.k_pages, cache.k_scale), (cache.v_pages, cache.v_scale))[which]
    x = pages.to(F32).cpu().numpy().astype(np.float64)
    ps = x.shape[2]
    table = cache.page_table[b].cpu().numpy()
    rows = np.concatenate([x[table[i]] for i in range(-(-n // ps))], 1)[:, :n] if n else x[0][:, :0]
    return rows if scale is None else rows * f64(scale)[:, None, None]


def random_tree(rng, m):
    rows = []
    for i in range(m):
        rows.append((rows[rng.integers(max(0, i - 5), i)] if i else 0) | 1 << i)
    return rows


def signed(rows):
    return [r - (1 << 64) if r >> 63 else r for r in rows]


def attend_check(M, ctype, qtype, lens, m, h, g, d, ps, tree=None, new=None, cap=0.0, slopes=None, window=0, seed=0,
                 max_len=0, scale=0.0, cache=None, size=1.0):
    b = len(lens)
    per = max(1, -(-max(lens) // ps))
    cache = cache or make_cache(M, ctype, b, h, d, ps, per, seed)
    q = rnd((b, m, h * g, d), qtype, seed + 9, size)
    out = torch.full((b, m, h * g, d), 7.0, dtype=qtype, device=DEV)
    lse = torch.full((b, m, h * g), 7.0, device=DEV)
    M.mkv_paged_attend(cache, q, i32(lens), new_lens=None if new is None else i32(new), out=out, lse=lse,
                       tree=None if tree is None else torch.tensor([signed(r) for r in tree], dtype=torch.int64, device=DEV),
                       cap=cap, window=window, max_len=max_len, scale=scale,
                       slopes=None if slopes is None else torch.tensor(slopes, dtype=F32, device=DEV))
    for i, n in enumerate(lens):
        mm = min(m if new is None else new[i], n)
        base = n - mm
        if tree is None:
            place, sees = base + np.arange(mm), np.tril(np.ones((mm, mm), bool))
        else:
            place, sees = O.tree_places([r & ((1 << mm) - 1) for r in tree[i][:mm]], base)
        at = np.concatenate([np.arange(base), place])
        see = np.concatenate([np.ones((mm, base), bool), sees], 1)
        if window:
            see = see & (place[:, None] - at[None] < window)
        ref = O.attend(f64(q[i, :mm]), rows_of(cache, 0, i, n), rows_of(cache, 1, i, n), see, place, at, scale or None,
                       cap, slopes)
        # fp16 carries the weights of an 8-bit cache
        attend_near(f64(out[i, :mm]), f64(lse[i, :mm]), ref, qtype, n, cap)
        assert (out[i, mm:] == 7.0).all() and (lse[i, mm:] == 7.0).all()
    assert cache.check() == M.MKV_OK


TYPES = [(F16, F16), (BF16, BF16), (E4M3, F16), (E4M3, BF16)]


@pytest.mark.parametrize("ctype,qtype", TYPES)
@pytest.mark.parametrize("d,ps", [(64, 16), (128, 48), (256, 64)])
@pytest.mark.parametrize("m", [1, 5, 64])
def test_attend_types(M, ctype, qtype, d, ps, m):
    rng = np.random.default_rng(m)
    lens = [m, 300, 64, 129 + m]
    attend_check(M, ctype, qtype, lens, m, 2, 4, d, ps, seed=d)
    attend_check(M, ctype, qtype, lens, m, 2, 4, d, ps, tree=[random_tree(rng, m) for _ in lens], seed=d + 50)


@pytest.mark.parametrize("h,g", [(1, 1), (2, 3), (1, 7), (3, 8), (1, 16), (1, 40), (1, 128)])
@pytest.mark.parametrize("m", [1, 9, 33])
def test_attend_heads(M, h, g, m):
    attend_check(M, BF16, BF16, [200, 65], m, h, g, 128, 16)
    attend_check(M, E4M3, F16, [200, 65], m, h, g, 64, 32)


@pytest.mark.parametrize("ctype,qtype", [(BF16, BF16), (E4M3, F16)])
@pytest.mark.parametrize("kw", [dict(cap=3.0, size=4.0), dict(cap=30.0), dict(slopes=True), dict(window=1), dict(window=7),
                                dict(window=130), dict(window=2**31 - 1), dict(slopes=True, cap=4.0, window=60), dict(scale=0.5)])
def test_attend_scores(M, ctype, qtype, kw):
    kw = dict(kw)
    if kw.get("slopes"):
        kw["slopes"] = [2.0**-(i + 1) for i in range(6)]
    rng = np.random.default_rng(5)
    lens = [260, 12, 131]
    attend_check(M, ctype, qtype, lens, 12, 2, 3, 128, 32, **kw)
    attend_check(M, ctype, qtype, lens, 12, 2, 3, 128, 32, tree=[random_tree(rng, 12) for _ in lens], **kw)
    attend_check(M, ctype, qtype, [70, 1, 0, 200], 1, 2, 3, 64, 16, **kw)


def test_attend_ragged_new_tokens(M):
    rng = np.random.default_rng(8)
    lens, new = [0, 1, 400, 64, 90], [0, 1, 20, 3, 0]
    attend_check(M, F16, F16, lens, 20, 2, 4, 128, 16, new=new)
    attend_check(M, E4M3, BF16, lens, 20, 2, 4, 256, 48, new=new, tree=[random_tree(rng, 20) for _ in lens])


@pytest.mark.parametrize("ctype,qtype", [(F16, F16), (BF16, BF16), (E4M3, BF16)])
@pytest.mark.parametrize("m,g", [(2, 4), (3, 3), (8, 4), (11, 3), (9, 7), (16, 4), (13, 5), (64, 1)])
def test_attend_few_rows(M, ctype, qtype, m, g):
    """Rows of a KV head around 8, 32 and 64, with sequences that have fewer of them or none."""
    rng = np.random.default_rng(m)
    lens = [500, m, 1, 0, 90, 2222]
    new = [m, min(m, 5), 1, 0, 0, max(1, m // 2)]
    tree = [random_tree(rng, m) for _ in lens]
    for d, ps in ((64, 32), (128, 16), (256, 80)):
        attend_check(M, ctype, qtype, lens, m, 2, g, d, ps, new=new, seed=m)
        attend_check(M, ctype, qtype, lens, m, 2, g, d, ps, new=new, tree=tree, seed=m, cap=5.0, window=300,
                     slopes=[2.0**-(i + 1) for i in range(2 * g)])


def test_attend_rows_that_see_nothing_and_odd_trees(M):
    """A row of zeros, one that does not see itself, bits of tokens that are not there, one that
    sees later ones."""
    tree = [[0, 1, 0b101, (1 << 64) - 1, 0b0100, 1 << 20]]
    attend_check(M, BF16, BF16, [6], 6, 2, 2, 64, 16, tree=tree)
    attend_check(M, BF16, BF16, [100], 6, 2, 2, 64, 16, tree=tree, slopes=[0.5, 0.1, 0.02, 0.9], window=9)
    attend_check(M, E4M3, F16, [4], 6, 2, 2, 64, 16, tree=tree, new=[4])


def test_attend_chain_is_prefill(M):
    """A prompt's later part over pages, longer than a tree, against the oracle."""
    attend_check(M, BF16, BF16, [700, 333], 210, 2, 2, 128, 64)
    attend_check(M, E4M3, BF16, [300, 210], 210, 1, 3, 128, 64, window=100)


@pytest.mark.parametrize("ctype", [F16, E4M3])
def test_attend_long(M, ctype):
    attend_check(M, ctype, F16, [20000, 1, 7001], 3, 2, 4, 128, 64)
    attend_check(M, ctype, F16, [12345], 1, 1, 8, 64, 16, window=5000, max_len=12345)


def test_attend_matches_decode(M):
    """One new token without options: mkv_paged_decode's result but for the weights' rounding."""
    cache = make_cache(M, BF16, 3, 4, 128, 32, 40, 3)
    q = rnd((3, 1, 8, 128), BF16, 4)
    lens = i32([1280, 77, 500])
    a = M.mkv_paged_attend(cache, q, lens)[:, 0]
    b = M.mkv_paged_decode(cache, q[:, 0], lens)
    assert (a.float() - b.float()).abs().max() <= 2.0**-6 * b.float().abs().max()


@pytest.mark.parametrize("ctype,stray", [(F16, float("nan")), (BF16, float("inf")), (F16, 65504.0)])
def test_attend_garbage_behind_the_sequence(M, ctype, stray):
    cache = make_cache(M, ctype, 2, 2, 128, 32, 6, 5)
    lens = [70, 33]
    for b, n in enumerate(lens):
        for t in range(n, 192):
            page = int(cache.page_table[b, t // 32])
            cache.k_pages[page, :, t % 32] = stray
            cache.v_pages[page, :, t % 32] = stray
    attend_check(M, ctype, ctype, lens, 4, 2, 4, 128, 32, cache=cache)


def test_attend_reports_what_lies_outside(M):
    cache = make_cache(M, BF16, 2, 2, 64, 16, 8, 5)
    q = rnd((2, 3, 4, 64), BF16, 1)
    for lens, new in (([200, 50], None), ([-1, 50], None), ([50, 50], [4, 1]), ([2, 50], [3, 3])):
        M.mkv_paged_attend(cache, q, i32(lens), new_lens=None if new is None else i32(new))
        assert cache.check() == M.MKV_ERR_DEVICE_CHECK, (lens, new)
        assert cache.check() == M.MKV_OK
    table = cache.page_table.clone()
    cache.page_table[0, 1] = 1 << 20
    cache.page_table[1, 0] = -3
    lens = [40, 40]
    out = M.mkv_paged_attend(cache, q, i32(lens))
    assert cache.check() == M.MKV_ERR_DEVICE_CHECK
    cache.page_table.copy_(table)
    for b, gone in ((0, range(16, 32)), (1, range(0, 16))):
        keep = [t for t in range(40) if t not in gone]
        see = O.visible(3, 40)[:, keep]
        ref = O.attend(f64(q[b]), rows_of(cache, 0, b, 40)[:, keep], rows_of(cache, 1, b, 40)[:, keep], see,
                       np.arange(37, 40), np.array(keep))
        attend_near(f64(out[b]), None, ref, BF16, 40)


# ---- together -----------------------------------------------------------------------------------

def test_a_layer_from_projection_to_drafts(M):
    """Norm and rotation of a prompt's projection, attention of the prompt, its rows into pages, then
    a tree of drafts over them, all captured into a graph and replayed with other inputs."""
    b, t, h, kv, d, m = 2, 150, 8, 2, 128, 7
    plan = M.mkv_rope_plan(d)
    rng = np.random.default_rng(3)
    trees = [random_tree(rng, m) for _ in range(b)]
    tree = torch.tensor([signed(r) for r in trees], dtype=torch.int64, device=DEV)
    depth = np.stack([O.tree_places(r, 0)[0] for r in trees])
    proj, draft = (torch.zeros((b, n, h + 2 * kv, d), dtype=BF16, device=DEV) for n in (t, m))
    w = rnd((d,), F32, 2, 0.2) + 1.0
    pool = [torch.zeros((16, kv, 32, d), dtype=BF16, device=DEV) for _ in range(2)]
    table = torch.randperm(16, generator=torch.Generator().manual_seed(1))[:12].view(b, 6).to(torch.int32).to(DEV)
    cache = M.MkvPaged(*pool, table)
    lens = i32([t + m] * b)
    seq = i32(np.repeat(np.arange(b), t))
    slot = i32(np.tile(np.arange(t), b))
    dseq, dslot = i32(np.repeat(np.arange(b), m)), i32(np.tile(t + np.arange(m), b))
    dpos = i32(t + depth)

    def layer():
        q, k = M.mkv_norm_rope(plan, proj[:, :, :h], w, None, k=proj[:, :, h:h + kv], k_weight=w)
        o = M.mkv_prefill(q, k, proj[:, :, h + kv:], cap=20.0)
        M.mkv_paged_append(cache, k.view(b * t, kv, d), proj[:, :, h + kv:].reshape(b * t, kv, d), slot, seq=seq)
        dq, dk = M.mkv_norm_rope(plan, draft[:, :, :h], w, dpos, k=draft[:, :, h:h + kv], k_weight=w)
        M.mkv_paged_append(cache, dk.view(b * m, kv, d), draft[:, :, h + kv:].reshape(b * m, kv, d), dslot, seq=dseq)
        return q, k, o, dq, dk, M.mkv_paged_attend(cache, dq, lens, tree=tree, cap=20.0, max_len=t + m)

    layer()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        made = layer()
    for seed in (1, 2):
        proj.copy_(rnd(proj.shape, BF16, seed))
        draft.copy_(rnd(draft.shape, BF16, seed + 10))
        graph.replay()
        torch.cuda.synchronize()
        q, k, o, dq, dk, do = (f64(x) for x in made)
        freq, mult = P.rope_frequencies(d, 10000.0)
        n = O.norm(f64(proj[:, :, :h]), f64(w), 1e-6)[1]
        want = P.rope(n, np.tile(np.arange(t), (b, 1)), freq, mult)
        near(q, want, 84 * U * pair_length(n, d, False) + HALF[BF16] * np.abs(want) * 1.01)
        for i in range(b):
            v, dv = f64(proj[i, :, h + kv:]).transpose(1, 0, 2), f64(draft[i, :, h + kv:]).transpose(1, 0, 2)
            kk, dkk = k[i].transpose(1, 0, 2), dk[i].transpose(1, 0, 2)
            ref = O.attend(q[i], kk, v, O.visible(t, t), np.arange(t), np.arange(t), None, 20.0)
            attend_near(o[i], None, ref, BF16, t, 20.0)
            place, sees = O.tree_places(trees[i], t)
            see = np.concatenate([np.ones((m, t), bool), sees], 1)
            ref = O.attend(dq[i], np.concatenate([kk, dkk], 1), np.concatenate([v, dv], 1), see, place,
                           np.concatenate([np.arange(t), place]), None, 20.0)
            attend_near(do[i], None, ref, BF16, t + m, 20.0)
    assert cache.check() == M.MKV_OK


def test_prompt_keys_into_the_compressed_cache(M):
    """Normed and rotated keys written head-major are what mkv_compress takes."""
    b, t, h, d = 1, 128, 2, 128
    proj = rnd((b, t, h, d), F16, 3)
    keys = torch.empty((b, h, t, d), dtype=F16, device=DEV)
    k_view = keys.transpose(1, 2)
    M.mkv_norm_rope(M.mkv_rope_plan(d), proj, rnd((d,), F16, 1), q_out=k_view)
    assert torch.equal(k_view, M.mkv_norm_rope(M.mkv_rope_plan(d), proj, rnd((d,), F16, 1)))
    cfg = M.make_config(b, h, 4, t, 64, 40, 0.85, 48)
    with M.Mkv(cfg) as m:
        m.compress(keys, keys)
        assert m.stats()["ctx_len"] == t


def test_calls_on_two_streams_at_once(M):
    """Each call's own workspace: results do not depend on what runs beside it."""
    cache = make_cache(M, BF16, 2, 2, 128, 64, 160, 3)
    q = [rnd((2, 8, 8, 128), BF16, s) for s in (1, 2)]
    lens = i32([10000, 9000])
    want = [M.mkv_paged_attend(cache, x, lens) for x in q]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in q]
    for _ in range(5):
        got = [M.mkv_paged_attend(cache, x, lens, stream=s) for x, s in zip(q, streams)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_workspaces_of_the_caller(M):
    """A tensor of as many bytes as the call names is enough, and one byte less is refused."""
    def room(n):
        return torch.full((n,), 0xff, dtype=torch.uint8, device=DEV)

    def check(call, n, outs):
        want = call(None)
        assert n > 0
        assert all(torch.equal(a, b) for a, b in zip(outs(want), outs(call(room(n)))))
        with pytest.raises(M.MkvError):
            call(room(n - 1))

    q, k, v = rnd((1, 3, 8, 64), BF16, 1), rnd((1, 5000, 2, 64), BF16, 2), rnd((1, 5000, 2, 64), BF16, 3)
    docs = torch.zeros((1, 5000), dtype=torch.int32, device=DEV)
    check(lambda w: M.mkv_prefill(q, k, v, docs=docs, workspace=w),
          M.mkv_prefill_workspace(1, 3, 5000, 8, 2, 64, docs=True), lambda o: [o])
    lens = i32([5000, 4000])
    for ctype, m in ((F16, 3), (E4M3, 1), (E4M3, 40)):
        cache = make_cache(M, ctype, 2, 2, 64, 64, 80, 3)
        x = rnd((2, m, 8, 64), F16, 4)
        check(lambda w: M.mkv_paged_attend(cache, x, lens, workspace=w),
              M.mkv_paged_attend_workspace(cache, m, 8), lambda o: [o])
    plan, w32 = M.mkv_rope_plan(64), rnd((64,), F32, 5)
    g = rnd((1, 3, 8, 64), BF16, 6)
    check(lambda w: M.mkv_norm_rope_grad(plan, g, q, w32, workspace=w), M.mkv_norm_rope_grad_workspace(plan), list)
    assert M.mkv_prefill_workspace(2, 4096, 4096, 16, 16, 128) == 0   # many rows: no parts
    with pytest.raises(M.MkvError):
        M.mkv_prefill_workspace(1, 3, 5000, 8, 3, 64)


def test_offsets_past_32_bits(M):
    """Two keys stand out of 2^25 and more whose rows take 2^32 elements, in a tensor and in pages:
    the output is the mean of their values, up to the roundings of weights (bf16: half a step, 2^-9
    with the two weights' ratio, 2^-9 with the output) and e^-30 times the others' number."""
    n, d, page = 2**25 + 64 * 9, 128, 64
    k = torch.zeros((1, n, 1, d), dtype=BF16, device=DEV)
    v = torch.ones((1, n, 1, d), dtype=BF16, device=DEV)
    q = torch.zeros((1, 1, 4, d), dtype=BF16, device=DEV)
    q[..., 0] = 1.0
    two = [77, n - 3]
    for t in two:
        k[0, t, 0, 0] = 30.0
    v[0, two] = rnd((2, 1, d), BF16, 1, 4.0)
    want = v[0, two].float().mean(0)
    size = float(v[0, two].float().abs().max()) + 1.0
    bound = size * (2.0**-8 + 2.0**-9 + n * float(np.exp(-30.0)) + 2.0**-16)
    got = M.mkv_prefill(q, k, v, scale=1.0)
    assert (got[0, 0].float() - want).abs().max() <= bound
    table = torch.arange(n // page, dtype=torch.int32, device=DEV).view(1, -1)
    cache = M.MkvPaged(k.view(n // page, 1, page, d), v.view(n // page, 1, page, d), table)
    got = M.mkv_paged_attend(cache, q, i32([n]), scale=1.0)
    assert (got[0, 0].float() - want).abs().max() <= bound and cache.check() == M.MKV_OK


def test_many_sequences(M):
    """As many sequences as a call takes: each sees its own one to three keys."""
    b, d = 65535, 64
    q, k, v = rnd((b, 1, 2, d), F16, 1), rnd((b, 3, 1, d), F16, 2), rnd((b, 3, 1, d), F16, 3)
    lens = torch.arange(b, dtype=torch.int32, device=DEV) % 3 + 1
    got = M.mkv_prefill(q, k, v, kv_lens=lens)
    z = torch.einsum("bqhd,bkud->bhqk", q.double(), k.double()) / 8.0
    z.masked_fill_(torch.arange(3, device=DEV).view(1, 1, 1, 3) >= lens.view(b, 1, 1, 1), -np.inf)
    want = torch.einsum("bhqk,bkud->bqhd", torch.softmax(z, -1), v.double())
    # scores of 64 products in fp32 (2^-18 of their size, here up to 2^6), weights and output half a step of fp16 each
    bound = 2.0**-11 * (want.abs() + v.double().abs().amax((1, 2, 3), keepdim=True)) + 2.0**-11
    assert ((got.double() - want).abs() <= bound).all()
    w = rnd((d,), F32, 4)
    y = M.mkv_norm_rope(M.mkv_rope_plan(d), q, w, first_pos=5)
    assert torch.equal(y[-3:], M.mkv_norm_rope(M.mkv_rope_plan(d), q[-3:], w, first_pos=5))
