"""Rotary axes and argument checks of the prompt calls, without a GPU.

The refusals come before any CUDA call, so made-up addresses are never touched."""
import ctypes
import math

import numpy as np
import pytest

from oracle import paged as P
from oracle import prompt as O

FAKE = 1 << 20          # an aligned address that is never touched


@pytest.fixture(scope="module")
def M():
    import os
    from two_compressed_kv_gb300 import build_lib
    if not os.path.exists(build_lib.LIB):
        build_lib.build()
    from two_compressed_kv_gb300 import mkv
    return mkv


# ---- axes ---------------------------------------------------------------------------------------

SCALINGS = [dict(), dict(scaling="linear", factor=4.0), dict(scaling="ntk", factor=8.0),
            dict(scaling="yarn", factor=16.0, original=8192), dict(scaling="banded", factor=8.0, original=8192)]


@pytest.mark.parametrize("kw", SCALINGS)
@pytest.mark.parametrize("sections", [(16, 24, 24), (4, 4), (30,), (2, 2, 2, 2), (5, 20, 3)])
@pytest.mark.parametrize("order", ["blocks", "cyclic"])
@pytest.mark.parametrize("restart", [False, True])
def test_axes_match_definition(M, kw, sections, order, restart):
    made = M.mkv_rope_axes_plan(256, sections, order=order, restart=restart, base=500000.0, **kw)
    axis, freq, mult = O.axes_frequencies(sections, order, restart, 500000.0, **kw)
    n = len(axis)
    assert list(made.axes.axis[:n]) == list(axis) and made.axes.n_axes == len(sections)
    assert made.plan.rot_dim == 2 * n and made.plan.head_dim == 256
    got = np.array([made.plan.turn[i] for i in range(n)], dtype=np.float64) / 2.0**64 * 2 * math.pi
    assert np.allclose(got, freq, rtol=16 * 2.0**-53, atol=2 * math.pi * 2.0**-64)
    assert abs(made.plan.mult - mult) <= 2.0**-24 * mult * 1.01


def test_axes_by_hand(M):
    """Six pairs dealt to axes of 3, 1 and 2; the second round passes over the axis that is full."""
    made = M.mkv_rope_axes_plan(12, (3, 1, 2), order="cyclic")
    assert list(made.axes.axis[:6]) == [0, 1, 2, 0, 2, 0]
    assert list(M.mkv_rope_axes_plan(12, (3, 1, 2)).axes.axis[:6]) == [0, 0, 0, 1, 2, 2]
    own = M.mkv_rope_axes_plan(12, (3, 1, 2), order="cyclic", restart=True)
    one = M.mkv_rope_plan(6)
    assert [own.plan.turn[i] for i in (0, 3, 5)] == [one.turn[i] for i in range(3)]


def test_one_axis_is_the_plan(M):
    made, plan = M.mkv_rope_axes_plan(128, (64,)), M.mkv_rope_plan(128)
    assert bytes(made.plan) == bytes(plan)


@pytest.mark.parametrize("args,kw", [
    (((),), dict(rot_dim=8)), (((1, 1, 1, 1, 1),), dict()), (((4, 0),), dict()), (((4, -1),), dict(rot_dim=6)),
    (((4, 4),), dict(rot_dim=12)), (((1, 3),), dict(scaling="ntk", factor=2.0, restart=True)), (((100, 100),), dict())])
def test_axes_refusals(M, args, kw):
    with pytest.raises(M.MkvError) as e:
        M.mkv_rope_axes_plan(128, *args, **kw)
    assert e.value.status == M.MKV_ERR_INVALID_ARG


def test_unknown_order(M):
    with pytest.raises(ValueError):
        M.mkv_rope_axes_plan(128, (64,), order="other")


def _rope_args(M, **kw):
    a = M.mkv_rope_args(x=FAKE, out=2 * FAKE, pos=3 * FAKE, tokens=5, batch=2, heads=3, dtype=M.MKV_DT_F16)
    a.x_stride[:] = a.out_stride[:] = [5 * 3 * 128, 3 * 128, 128]
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("kw", [dict(x=None), dict(out=None), dict(pos=None), dict(dtype=3), dict(tokens=-1), dict(transposed=2)])
def test_multi_refusals(M, kw):
    made = M.mkv_rope_axes_plan(128, (16, 24, 24))
    a = _rope_args(M, **kw)
    assert M.lib.mkv_rope_multi(made.address, made.axes_address, ctypes.byref(a), 10, None) == M.MKV_ERR_INVALID_ARG
    assert "mkv_rope" in M.mkv_last_error_string()


def test_multi_wants_axes_of_its_plan(M):
    made, a = M.mkv_rope_axes_plan(128, (16, 24, 24)), _rope_args(M)
    call = lambda plan, axes: M.lib.mkv_rope_multi(plan, axes, ctypes.byref(a), 10, None)
    assert call(made.address, None) == call(None, made.axes_address) == M.MKV_ERR_INVALID_ARG
    made.axes.axis[63] = 3
    assert call(made.address, made.axes_address) == M.MKV_ERR_INVALID_ARG
    made.axes.axis[63] = 2
    made.axes.n_axes = 5
    assert call(made.address, made.axes_address) == M.MKV_ERR_INVALID_ARG
    made.axes.n_axes = 3
    a.tokens = 0
    assert call(made.address, made.axes_address) == M.MKV_OK


# ---- norms --------------------------------------------------------------------------------------

def _norm_args(M, **kw):
    a = M.mkv_norm_rope_args(tokens=5, batch=2, dtype=M.MKV_DT_BF16, weight_dtype=M.MKV_DT_F32, eps=1e-6,
                             workspace=9 * FAKE, workspace_bytes=1 << 30)
    for s in range(2):
        a.x[s], a.out[s], a.grad[s], a.weight[s] = FAKE, 2 * FAKE, 3 * FAKE, 4 * FAKE
        a.weight_grad[s] = 5 * FAKE
        a.heads[s] = 3
        for t in (a.x_stride, a.out_stride, a.grad_stride):
            t[s][:] = [5 * 3 * 128, 3 * 128, 128]
    for k, v in kw.items():
        if isinstance(v, tuple):
            getattr(a, k)[v[0]] = v[1]
        else:
            setattr(a, k, v)
    return a


BOTH = [dict(x=(0, None)), dict(out=(1, None)), dict(dtype=3), dict(weight_dtype=0), dict(batch=-1), dict(heads=(1, -1)),
        dict(tokens=-1), dict(batch=65536), dict(heads=(0, 65536)), dict(eps=-1.0), dict(eps=float("nan")),
        dict(eps=float("inf")), dict(weight_offset=float("nan")), dict(x=(0, FAKE + 1)), dict(weight=(1, FAKE + 2)),
        dict(first_pos=2**31 - 2), dict(x=(0, 2 * FAKE), x_stride=(0, (ctypes.c_int64 * 3)(1920, 128, 640)))]


@pytest.mark.parametrize("kw", BOTH)
def test_norm_refusals(M, kw):
    plan, a = M.mkv_rope_plan(128), _norm_args(M, **kw)
    for call in (M.lib.mkv_norm_rope, M.lib.mkv_norm_rope_grad):
        assert call(plan.address, None, ctypes.byref(a), None) == M.MKV_ERR_INVALID_ARG
        assert "mkv_norm_rope" in M.mkv_last_error_string()


@pytest.mark.parametrize("kw", [dict(grad=(1, None)), dict(weight=(0, None)), dict(grad=(0, FAKE + 1))])
def test_norm_grad_refusals(M, kw):
    plan, a = M.mkv_rope_plan(128), _norm_args(M, **kw)
    assert M.lib.mkv_norm_rope_grad(plan.address, None, ctypes.byref(a), None) == M.MKV_ERR_INVALID_ARG


def test_norm_sizes(M):
    big, plan, a = M.mkv_rope_plan(512, rot_dim=64), M.mkv_rope_plan(128), _norm_args(M)
    assert M.lib.mkv_norm_rope(big.address, None, ctypes.byref(a), None) == M.MKV_ERR_INVALID_ARG
    assert M.lib.mkv_norm_rope(None, None, ctypes.byref(a), None) == M.MKV_ERR_INVALID_ARG
    assert M.lib.mkv_norm_rope(plan.address, None, None, None) == M.MKV_ERR_INVALID_ARG
    made = M.mkv_rope_axes_plan(128, (32, 32))
    a.pos = None
    assert M.lib.mkv_norm_rope(made.address, made.axes_address, ctypes.byref(a), None) == M.MKV_ERR_INVALID_ARG
    a = _norm_args(M, tokens=0)
    assert M.lib.mkv_norm_rope(plan.address, None, ctypes.byref(a), None) == M.MKV_OK
    a = _norm_args(M)
    a.weight_grad[0] = a.weight_grad[1] = None
    assert M.lib.mkv_norm_rope_grad_workspace(plan.address, ctypes.byref(a)) == 0


# ---- attention ----------------------------------------------------------------------------------

def _prefill_args(M, **kw):
    a = M.mkv_prefill_args(q=FAKE, k=2 * FAKE, v=3 * FAKE, out=4 * FAKE, q_tokens=7, kv_tokens=9, batch=2, n_q_heads=4,
                           n_kv_heads=2, head_dim=128, dtype=M.MKV_DT_BF16, causal=1)
    for t, h, n in ((a.q_stride, 4, 7), (a.k_stride, 2, 9), (a.v_stride, 2, 9), (a.out_stride, 4, 7)):
        t[:] = [n * h * 128, h * 128, 128]
    for k, v in kw.items():
        if isinstance(v, list):
            getattr(a, k)[:] = v
        else:
            setattr(a, k, v)
    return a


BAD_SIZES = [dict(batch=-1), dict(batch=65536), dict(n_q_heads=3), dict(n_q_heads=0), dict(n_kv_heads=0),
             dict(n_q_heads=258, n_kv_heads=2), dict(head_dim=96), dict(head_dim=0), dict(dtype=2), dict(dtype=3),
             dict(q_tokens=-1), dict(kv_tokens=-1), dict(q_tokens=(1 << 30) + 1), dict(causal=2), dict(window=-1),
             dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")), dict(cap=-1.0),
             dict(cap=float("inf")), dict(cap=float("nan")), dict(causal=0, prefix=FAKE),
             dict(q_tokens=1 << 30, n_q_heads=8)]


@pytest.mark.parametrize("kw", BAD_SIZES)
def test_prefill_sizes(M, kw):
    a = _prefill_args(M, **kw)
    assert M.lib.mkv_prefill(ctypes.byref(a), None) == M.MKV_ERR_INVALID_ARG
    assert "mkv_prefill" in M.mkv_last_error_string()
    assert M.lib.mkv_prefill_workspace(ctypes.byref(a)) == 2**64 - 1


@pytest.mark.parametrize("kw", [
    dict(q=None), dict(k=None), dict(v=None), dict(out=None), dict(q=FAKE + 2), dict(out=FAKE + 8), dict(k=FAKE + 4),
    dict(q_stride=[7 * 512, 508, 128]), dict(k_stride=[9 * 256, 256, 0]), dict(v_stride=[-8, 256, 128]),
    dict(out_stride=[0, 512, 128]), dict(out=FAKE), dict(out=2 * FAKE), dict(out=3 * FAKE)])
def test_prefill_pointers_and_strides(M, kw):
    a = _prefill_args(M, **kw)
    assert M.lib.mkv_prefill(ctypes.byref(a), None) == M.MKV_ERR_INVALID_ARG
    assert "mkv_prefill" in M.mkv_last_error_string()


def test_prefill_nothing_to_do(M):
    for kw in (dict(batch=0), dict(q_tokens=0)):
        a = _prefill_args(M, q=None, out=None, **kw)
        assert M.lib.mkv_prefill(ctypes.byref(a), None) == M.MKV_OK
    assert M.lib.mkv_prefill(None, None) == M.MKV_ERR_INVALID_ARG


def _cache(M, **kw):
    c = M.mkv_paged_cache(k_pages=FAKE, v_pages=2 * FAKE, page_table=3 * FAKE, table_stride=8, dtype=M.MKV_DT_F16,
                          batch=2, n_kv_heads=2, head_dim=128, page_size=64, n_pages=16, max_pages=8)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def _attend_args(M, **kw):
    a = M.mkv_paged_attend_args(q=FAKE, out=2 * FAKE, seq_lens=3 * FAKE, workspace=4 * FAKE, workspace_bytes=1 << 30, n=5,
                                n_q_heads=4, q_dtype=M.MKV_DT_F16)
    a.q_stride[:] = [5 * 4 * 128, 4 * 128, 128]
    for k, v in kw.items():
        if isinstance(v, list):
            getattr(a, k)[:] = v
        else:
            setattr(a, k, v)
    return a


@pytest.mark.parametrize("kw", [
    dict(n=-1), dict(n=65536), dict(n=65, tree=FAKE), dict(n_q_heads=3), dict(n_q_heads=0), dict(n_q_heads=260),
    dict(q_dtype=1), dict(q_dtype=2), dict(max_len=-1), dict(max_len=513), dict(window=-1), dict(scale=-0.5),
    dict(scale=float("nan")), dict(cap=-1.0), dict(cap=float("inf"))])
def test_attend_sizes(M, kw):
    c, a = _cache(M), _attend_args(M, **kw)
    assert M.lib.mkv_paged_attend(ctypes.byref(c), ctypes.byref(a), None) == M.MKV_ERR_INVALID_ARG
    assert "mkv_paged_attend" in M.mkv_last_error_string()
    assert M.lib.mkv_paged_attend_workspace(ctypes.byref(c), ctypes.byref(a)) == 2**64 - 1


@pytest.mark.parametrize("kw", [dict(q=None), dict(out=None), dict(seq_lens=None), dict(q=FAKE + 2), dict(out=FAKE + 8),
                                dict(q_stride=[2560, 512, 100]), dict(q_stride=[2560, 0, 128]), dict(out=FAKE)])
def test_attend_pointers_and_strides(M, kw):
    c, a = _cache(M), _attend_args(M, **kw)
    assert M.lib.mkv_paged_attend(ctypes.byref(c), ctypes.byref(a), None) == M.MKV_ERR_INVALID_ARG
    assert "mkv_paged_attend" in M.mkv_last_error_string()


@pytest.mark.parametrize("kw", [dict(head_dim=96), dict(dtype=2), dict(k_scale=FAKE), dict(page_size=8)])
def test_attend_refuses_a_bad_cache(M, kw):
    c, a = _cache(M, **kw), _attend_args(M)
    assert M.lib.mkv_paged_attend(ctypes.byref(c), ctypes.byref(a), None) == M.MKV_ERR_INVALID_ARG


def test_attend_nothing_to_do(M):
    c, a = _cache(M), _attend_args(M, n=0, q=None, out=None)
    assert M.lib.mkv_paged_attend(ctypes.byref(c), ctypes.byref(a), None) == M.MKV_OK
    assert M.lib.mkv_paged_attend(ctypes.byref(c), None, None) == M.MKV_ERR_INVALID_ARG
    assert M.lib.mkv_paged_attend(None, ctypes.byref(a), None) == M.MKV_ERR_INVALID_ARG


# ---- the oracle ---------------------------------------------------------------------------------

def test_oracle_attention_by_hand():
    """Two keys, scores 0 and ln 3 after the slope: weights 1/4 and 3/4."""
    q = np.array([[[1.0]]])
    k = np.array([[[math.log(3.0) + 0.5], [0.0]]])
    v = np.array([[[8.0], [4.0]]])
    see = np.ones((1, 2), bool)
    out, lse, *_ = O.attend(q, k, v, see, np.array([1]), np.arange(2), 1.0, 0.0, [0.5])
    assert np.allclose(out, 7.0) and np.allclose(lse, math.log(4.0))
    out, lse, *_ = O.attend(q, k * 1e6, v, see, np.array([1]), np.arange(2), 1.0, math.log(3.0))
    assert np.allclose(out, 7.0)
    out, lse, *_ = O.attend(q, k, v, ~see, np.array([1]), np.arange(2))
    assert not out.any() and lse[0, 0] == -np.inf


def test_oracle_visibility_by_hand():
    see = O.visible(3, 5, window=2, prefix=1)
    assert see.astype(int).tolist() == [[0, 1, 1, 0, 0], [0, 0, 1, 1, 0], [0, 0, 0, 1, 1]]
    see = O.visible(2, 4, causal=False, window=2, docs=np.array([1, 1, 0, 0]))
    assert see.astype(int).tolist() == [[0, 0, 1, 1], [0, 0, 1, 1]]
    place, sees = O.tree_places([0b1, 0b11, 0b101, 0b1101], 10)
    assert place.tolist() == [10, 11, 11, 12]
    assert sees[3].tolist() == [True, False, True, True]


def test_oracle_norm_gradient_by_differences():
    rng = np.random.default_rng(0)
    x, u, w = rng.normal(size=(2, 3, 8)), rng.normal(size=(2, 3, 8)), rng.normal(size=8)
    f = lambda x, w: float((O.norm(x, w, 1e-3)[1] * u).sum())
    dx, dw = O.norm_grad(u, x, w, 1e-3)
    t, s, h = rng.normal(size=x.shape), rng.normal(size=8), 1e-5
    assert abs((f(x + h * t, w) - f(x - h * t, w)) / (2 * h) - (dx * t).sum()) < 1e-8
    assert abs((f(x, w + h * s) - f(x, w - h * s)) / (2 * h) - (dw * s).sum()) < 1e-8


def test_oracle_axes_reduce_to_one():
    rng = np.random.default_rng(1)
    x, pos = rng.normal(size=(2, 5, 3, 16)), rng.integers(0, 999, (2, 5))
    axis, f, mult = O.axes_frequencies((2, 3, 1), "cyclic", False, 1000.0)
    want = P.rope(x, pos, *P.rope_frequencies(12, 1000.0))
    assert np.allclose(O.spin(x, np.stack([pos] * 3), axis, f, mult), want)


@pytest.mark.parametrize("name", ["scale", "cap"])
def test_factors_that_overflow_are_refused(M, name):
    """Scores are formed in the log2 domain: a factor of 1.4427 has to fit. 2^127 does."""
    for x in (1.8e38, 2.4e38, 3.4e38):
        a = _prefill_args(M, **{name: x})
        assert M.lib.mkv_prefill(ctypes.byref(a), None) == M.MKV_ERR_INVALID_ARG
        assert name in M.mkv_last_error_string()
        assert M.lib.mkv_prefill_workspace(ctypes.byref(a)) == 2**64 - 1
        c, a = _cache(M), _attend_args(M, **{name: x})
        assert M.lib.mkv_paged_attend(ctypes.byref(c), ctypes.byref(a), None) == M.MKV_ERR_INVALID_ARG
        assert name in M.mkv_last_error_string()
    a = _prefill_args(M, q=None, out=None, batch=0, **{name: 2.0**127})
    assert M.lib.mkv_prefill(ctypes.byref(a), None) == M.MKV_OK
    c, a = _cache(M), _attend_args(M, n=0, q=None, out=None, **{name: 2.0**127})
    assert M.lib.mkv_paged_attend(ctypes.byref(c), ctypes.byref(a), None) == M.MKV_OK
