"""Rotary plans, argument checks and the oracle of the paged cache, without a GPU.

The refusals come before any CUDA call, so made-up addresses are never touched."""
import ctypes
import math

import numpy as np
import pytest

from oracle import paged as P


@pytest.fixture(scope="module")
def M():
    import os
    from two_compressed_kv_gb300 import build_lib
    if not os.path.exists(build_lib.LIB):
        build_lib.build()
    from two_compressed_kv_gb300 import mkv
    return mkv


SCALINGS = [dict(), dict(scaling="linear", factor=4.0), dict(scaling="ntk", factor=8.0),
            dict(scaling="yarn", factor=16.0, original=8192),
            dict(scaling="yarn", factor=2.5, original=500, beta_fast=4.0, beta_slow=4.0),
            dict(scaling="banded", factor=8.0, original=8192)]


@pytest.mark.parametrize("kw", SCALINGS)
@pytest.mark.parametrize("rot,base", [(2, 10000.0), (64, 10000.0), (128, 500000.0), (256, 1.5)])
def test_plan_matches_definition(M, kw, rot, base):
    if kw.get("scaling") == "ntk" and rot < 4:
        pytest.skip("NTK scaling divides by rot_dim - 2")
    plan = M.mkv_rope_plan(256, rot_dim=rot, base=base, **kw)
    freq, mult = P.rope_frequencies(rot, base, **kw)
    got = np.array([plan.turn[i] for i in range(rot // 2)], dtype=np.float64) / 2.0**64 * 2 * math.pi
    # pow, two products and a quotient in 64 bits: a few 2^-53 relative; the cut to whole
    # units of the phase adds 2^-64 of a turn
    assert np.allclose(got, freq, rtol=16 * 2.0**-53, atol=2 * math.pi * 2.0**-64)
    assert abs(plan.mult - mult) <= 2.0**-24 * mult * 1.01
    assert plan.rot_dim == rot and plan.head_dim == 256


def test_phase_is_exact_at_far_positions(M):
    """position * turn modulo 2^64 is the phase to 2^-53 of the frequency's own error."""
    plan = M.mkv_rope_plan(128, base=500000.0)
    for pos in (1, 131071, 1048575, 2**31 - 1, -5, -2**31):
        for i in (0, 1, 40, 63):
            phase = (pos * plan.turn[i]) % 2**64 / 2.0**64
            want = (pos * (500000.0 ** (-2.0 * i / 128)) / (2 * math.pi)) % 1.0
            d = abs(phase - want)
            assert min(d, 1 - d) <= abs(pos) * 2.0**-51, (pos, i)


def test_attn_factor_overrides(M):
    assert M.mkv_rope_plan(64, scaling="yarn", factor=16, original=4096, attn_factor=1.0).mult == 1.0
    assert M.mkv_rope_plan(64, attn_factor=0.5).mult == 0.5


@pytest.mark.parametrize("kw", [
    dict(rot_dim=3), dict(rot_dim=0), dict(rot_dim=130), dict(base=1.0), dict(base=float("nan")),
    dict(base=float("inf")), dict(scaling="linear", factor=0.5), dict(scaling="ntk", factor=2.0, rot_dim=2),
    dict(scaling="yarn", factor=2.0), dict(scaling="yarn", factor=2.0, original=100, beta_fast=1, beta_slow=2),
    dict(scaling="banded", factor=2.0, original=100, low_freq=4.0, high_freq=4.0),
    dict(scaling="banded", factor=2.0, original=-1.0), dict(attn_factor=-1.0),
    dict(attn_factor=float("inf")), dict(head_dim=0), dict(head_dim=5000)])
def test_plan_refusals(M, kw):
    with pytest.raises(M.MkvError) as e:
        M.mkv_rope_plan(**{"head_dim": 128, **kw})
    assert e.value.status == M.MKV_ERR_INVALID_ARG and "mkv_rope_plan_init:" in str(e.value)


def test_unknown_scaling(M):
    with pytest.raises(ValueError):
        M.mkv_rope_plan(128, scaling="other")


FAKE = 1 << 20          # an aligned address that is never touched


def _rope_args(M, **kw):
    a = M.mkv_rope_args(x=FAKE, out=2 * FAKE, tokens=5, batch=2, heads=3, dtype=M.MKV_DT_F16)
    a.x_stride[:] = a.out_stride[:] = [5 * 3 * 128, 3 * 128, 128]
    for k, v in kw.items():
        if k.endswith("stride") and isinstance(v, list):
            getattr(a, k)[:] = v
        else:
            setattr(a, k, v)
    return a


@pytest.mark.parametrize("kw", [
    dict(x=None), dict(out=None), dict(dtype=3), dict(batch=-1), dict(heads=-1),
    dict(tokens=-1), dict(batch=65536), dict(transposed=2), dict(x=FAKE + 1),
    dict(out_stride=[0, 384, 128]), dict(out_stride=[1920, -384, 128]),
    dict(out=FAKE, out_stride=[1920, 128, 640]), dict(first_pos=2**31 - 2)])
def test_rope_refusals(M, kw):
    plan = M.mkv_rope_plan(128)
    a = _rope_args(M, **kw)
    assert M.lib.mkv_rope(ctypes.byref(plan), ctypes.byref(a), None) == M.MKV_ERR_INVALID_ARG
    assert "mkv_rope" in M.mkv_last_error_string()


def test_rope_nothing_to_do(M):
    plan = M.mkv_rope_plan(128)
    for kw in (dict(batch=0), dict(heads=0), dict(tokens=0)):
        a = _rope_args(M, x=None, out=None, **kw)
        assert M.lib.mkv_rope(ctypes.byref(plan), ctypes.byref(a), None) == M.MKV_OK
    assert M.lib.mkv_rope(None, ctypes.byref(a), None) == M.MKV_ERR_INVALID_ARG
    broken = M.MkvRopePlan()
    a = _rope_args(M)
    assert M.lib.mkv_rope(ctypes.byref(broken), ctypes.byref(a), None) == M.MKV_ERR_INVALID_ARG


def _cache(M, **kw):
    c = M.mkv_paged_cache(k_pages=FAKE, v_pages=2 * FAKE, page_table=3 * FAKE, table_stride=8,
                          dtype=M.MKV_DT_F16, batch=2, n_kv_heads=2, head_dim=128, page_size=64,
                          n_pages=16, max_pages=8)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


BAD_CACHES = [
    dict(k_pages=None), dict(v_pages=FAKE + 8), dict(page_table=None), dict(dtype=2), dict(dtype=9),
    dict(k_scale=FAKE), dict(batch=0), dict(batch=65536), dict(n_kv_heads=0), dict(head_dim=96),
    dict(page_size=8), dict(page_size=40), dict(page_size=272), dict(n_pages=0), dict(max_pages=0),
    dict(table_stride=7), dict(max_pages=1 << 25, table_stride=1 << 25),
    dict(n_pages=1 << 30)]


@pytest.mark.parametrize("kw", BAD_CACHES)
def test_cache_refusals(M, kw):
    c = _cache(M, **kw)
    bad = M.MKV_ERR_INVALID_ARG
    assert M.lib.mkv_paged_validate(ctypes.byref(c)) == bad
    assert "paged cache" in M.mkv_last_error_string()
    assert M.lib.mkv_paged_decode(ctypes.byref(c), ctypes.byref(_decode_args(M)), None) == bad
    assert M.lib.mkv_paged_append(ctypes.byref(c), None, ctypes.byref(_append_args(M)), None) == bad
    assert M.lib.mkv_paged_evict(ctypes.byref(c), ctypes.byref(_evict_args(M)), None) == bad
    assert M.lib.mkv_paged_validate(ctypes.byref(_cache(M))) == M.MKV_OK


def _append_args(M, **kw):
    a = M.mkv_paged_append_args(k=FAKE, v=FAKE, slot=FAKE, n=2, in_dtype=M.MKV_DT_F16)
    a.k_stride[:] = a.v_stride[:] = [256, 128]
    for k, v in kw.items():
        if isinstance(v, list):
            getattr(a, k)[:] = v
        else:
            setattr(a, k, v)
    return a


@pytest.mark.parametrize("kw", [
    dict(k=None), dict(v=None), dict(slot=None), dict(n=-1), dict(n=3), dict(k=FAKE + 2),
    dict(in_dtype=1), dict(in_dtype=2), dict(q=FAKE, n_q_heads=4), dict(q=FAKE, q_out=FAKE),
    dict(k_stride=[252, 128]), dict(v_stride=[256, 4]), dict(acc=FAKE), dict(pos_meta=FAKE),
    dict(q=FAKE, q_out=2 * FAKE, n_q_heads=4, q_stride=[512, 128], q_out_stride=[0, 128]),
    dict(q=FAKE, q_out=FAKE, n_q_heads=4, q_stride=[512, 128], q_out_stride=[1024, 128])])
def test_append_refusals(M, kw):
    st = M.lib.mkv_paged_append(ctypes.byref(_cache(M)), None, ctypes.byref(_append_args(M, **kw)), None)
    assert st == M.MKV_ERR_INVALID_ARG and "mkv_paged_append" in M.mkv_last_error_string()


def test_append_plan_refusals(M):
    for plan in (M.mkv_rope_plan(64), M.mkv_rope_plan(128, rot_dim=24), M.mkv_rope_plan(128, rot_dim=20, interleaved=True)):
        st = M.lib.mkv_paged_append(ctypes.byref(_cache(M)), ctypes.byref(plan),
                                    ctypes.byref(_append_args(M)), None)
        assert st == M.MKV_ERR_INVALID_ARG
    assert M.lib.mkv_paged_append(ctypes.byref(_cache(M)), None,
                                  ctypes.byref(_append_args(M, n=0, k=None)), None) == M.MKV_OK


def _decode_args(M, **kw):
    a = M.mkv_paged_decode_args(q=FAKE, out=FAKE, seq_lens=FAKE, workspace=FAKE,
                                workspace_bytes=1 << 40, n_q_heads=8)
    a.q_stride[:] = [8 * 128, 128]
    for k, v in kw.items():
        if isinstance(v, list):
            getattr(a, k)[:] = v
        else:
            setattr(a, k, v)
    return a


@pytest.mark.parametrize("kw", [
    dict(q=None), dict(out=None), dict(seq_lens=None), dict(q=FAKE + 4), dict(out=FAKE + 4),
    dict(n_q_heads=7), dict(n_q_heads=0), dict(n_q_heads=34), dict(q_dtype=1), dict(q_dtype=2),
    dict(out_dtype=1), dict(max_len=-1), dict(max_len=513), dict(scale=-1.0),
    dict(scale=float("nan")), dict(scale=float("inf")), dict(q_stride=[1024, 127]),
    dict(workspace=None), dict(workspace=FAKE + 8), dict(acc=FAKE, acc_stride=511),
    dict(acc=FAKE, acc_stride=99, max_len=100)])
def test_decode_refusals(M, kw):
    st = M.lib.mkv_paged_decode(ctypes.byref(_cache(M)), ctypes.byref(_decode_args(M, **kw)), None)
    assert st == M.MKV_ERR_INVALID_ARG and "mkv_paged_decode" in M.mkv_last_error_string()


def _evict_args(M, **kw):
    a = M.mkv_paged_evict_args(acc=FAKE, pos=FAKE, acc_out=2 * FAKE, pos_out=2 * FAKE, seq_lens=FAKE,
                               next_pos=FAKE, lens_out=FAKE, src=FAKE, workspace=FAKE,
                               workspace_bytes=1 << 40, meta_stride=512, out_stride=100, budget=100,
                               sink=4, recent=50)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("kw", [
    dict(acc=None), dict(pos=None), dict(acc_out=None), dict(pos_out=None), dict(seq_lens=None),
    dict(next_pos=None), dict(lens_out=None), dict(src=None), dict(workspace=None),
    dict(workspace=FAKE + 8), dict(workspace_bytes=100), dict(meta_stride=511), dict(out_stride=99),
    dict(budget=0), dict(sink=-1), dict(recent=-1), dict(recent=97), dict(max_len=-1),
    dict(max_len=513), dict(acc_out=FAKE), dict(pos_out=FAKE)])
def test_evict_refusals(M, kw):
    st = M.lib.mkv_paged_evict(ctypes.byref(_cache(M)), ctypes.byref(_evict_args(M, **kw)), None)
    assert st == M.MKV_ERR_INVALID_ARG and "mkv_paged_evict" in M.mkv_last_error_string()


def test_binding_refuses_host_tensors_and_types(M):
    import torch
    plan = M.mkv_rope_plan(128)
    x = torch.zeros((1, 2, 3, 128), dtype=torch.float16)
    with pytest.raises(ValueError, match="CUDA"):
        M.mkv_rope(plan, x)
    with pytest.raises(TypeError):
        M.mkv_rope(plan, [1.0])
    with pytest.raises(ValueError, match="CUDA"):
        M.MkvPaged(x, x, torch.zeros((1, 1), dtype=torch.int32))


def test_struct_sizes_match_the_header(M, tmp_path):
    import os
    import subprocess
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    names = ["mkv_rope_config", "mkv_rope_plan", "mkv_rope_args", "mkv_paged_cache",
             "mkv_paged_append_args", "mkv_paged_decode_args", "mkv_paged_evict_args"]
    classes = [M.mkv_rope_config, M.MkvRopePlan, M.mkv_rope_args, M.mkv_paged_cache,
               M.mkv_paged_append_args, M.mkv_paged_decode_args, M.mkv_paged_evict_args]
    body = "".join(f'printf("%zu\\n", sizeof({n}));' for n in names)
    for n, c in zip(names, classes):
        body += "".join(f'printf("%zu\\n", offsetof({n}, {f[0]}));' for f in c._fields_)
    src = tmp_path / "s.c"
    src.write_text(f'#include <stdio.h>\n#include "mkv.h"\nint main(void) {{ {body} return 0; }}\n')
    exe = str(tmp_path / "s")
    subprocess.check_call(["gcc", "-I", os.path.join(root, "include"), str(src), "-o", exe])
    got = [int(v) for v in subprocess.check_output([exe]).split()]
    want = [ctypes.sizeof(c) for c in classes]
    for c in classes:
        want += [getattr(c, f[0]).offset for f in c._fields_]
    assert got == want


# ---- the oracle against closed forms ------------------------------------------------------------

def test_oracle_rope_is_a_rotation():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((7, 3, 16))
    freq, _ = P.rope_frequencies(12, 100.0)
    pos = np.arange(7) * 1000
    for inter in (False, True):
        y = P.rope(x, pos, freq, interleaved=inter)
        assert np.allclose((y**2).sum(-1), (x**2).sum(-1))
        assert np.allclose(y[..., 12:], x[..., 12:]) and np.allclose(y[0], x[0])
        assert np.allclose(P.rope(y, pos, freq, interleaved=inter, transposed=True), x)
        # scores depend on the difference of positions alone
        z = P.rope(x, pos + 77, freq, interleaved=inter)
        assert np.allclose(np.einsum("thd,shd->hts", y, y), np.einsum("thd,shd->hts", z, z))
    # a quarter turn by hand
    q = P.rope(np.array([[1.0, 2.0, 3.0, 4.0]]), np.array(1), np.array([math.pi / 2, math.pi]))
    assert np.allclose(q, [[-3.0, -2.0, 1.0, -4.0]])


def test_oracle_decode_closed_forms():
    v = np.array([[[1.0, 2.0], [3.0, 6.0]]])
    out, lse, mass, _ = P.decode(np.zeros((2, 2)), np.ones((1, 2, 2)), v)
    assert np.allclose(out, [[2.0, 4.0]] * 2) and np.allclose(lse, math.log(2)) and np.allclose(mass, 1.0)
    out, lse, _, _ = P.decode(np.zeros((1, 2)), np.ones((1, 0, 2)), np.ones((1, 0, 2)))
    assert (out == 0).all() and lse[0] == -np.inf


def test_oracle_evict_by_hand():
    acc = np.array([0.5, 0.1, 0.9, 0.1, 0.7, 0.1], dtype=np.float32)
    pos = np.arange(6)
    assert P.evict(acc, pos, 6, 6).tolist() == [0, 1, 2, 3, 4, 5]
    assert P.evict(acc, pos, 6, 3).tolist() == [0, 4, 2]
    assert P.evict(acc, pos, 6, 4).tolist() == [0, 1, 2, 4]            # tie of the 0.1s: slot 1
    assert P.evict(acc, pos, 6, 3, sink=2).tolist() == [0, 1, 2]
    assert P.evict(acc, pos, 6, 3, recent=2).tolist() == [4, 5, 2]
    assert P.evict(np.array([np.nan, -1.0, 2.0], np.float32), np.arange(3), 9, 2).tolist() == [0, 2]



# ---- the marshalling module ---------------------------------------------------------------------

def test_missing_marshalling_module_names_the_build(M, monkeypatch):
    import sys

    import two_compressed_kv_gb300 as package
    monkeypatch.setattr(M, "_M", None)
    monkeypatch.delattr(package, "_marshal", raising=False)
    monkeypatch.setitem(sys.modules, "two_compressed_kv_gb300._marshal", None)
    with pytest.raises(ImportError, match="two_compressed_kv_gb300.build_lib"):
        M.mkv_rope(M.mkv_rope_plan(128), None)


# ---- strides of extents of 1 --------------------------------------------------------------------
# The calls below are refused for a later reason, so that nothing is launched anywhere.

@pytest.mark.parametrize("cache,kw", [
    (dict(batch=1), dict(q_stride=[1, 128])), (dict(n_kv_heads=1), dict(q_stride=[128, 3], n_q_heads=1)),
    (dict(batch=1, n_kv_heads=1), dict(q_stride=[-5, 77], n_q_heads=1))])
def test_decode_ignores_strides_of_extents_of_1(M, cache, kw):
    a = _decode_args(M, acc=FAKE, acc_stride=511, **kw)
    assert M.lib.mkv_paged_decode(ctypes.byref(_cache(M, **cache)), ctypes.byref(a), None) == M.MKV_ERR_INVALID_ARG
    assert "acc_stride" in M.mkv_last_error_string()
    # the stride of an extent of 2 still counts
    a = _decode_args(M, acc=FAKE, acc_stride=511, q_stride=[1, 77], n_q_heads=2)
    assert M.lib.mkv_paged_decode(ctypes.byref(_cache(M, **cache)), ctypes.byref(a), None) == M.MKV_ERR_INVALID_ARG
    assert "strides" in M.mkv_last_error_string()


@pytest.mark.parametrize("cache,kw", [
    (dict(), dict(n=1, k_stride=[252, 128], v_stride=[1, 128])),
    (dict(n_kv_heads=1), dict(k_stride=[256, 1], v_stride=[256, 77])),
    (dict(), dict(n=1, q=FAKE, q_out=2 * FAKE, n_q_heads=4, q_stride=[5, 128], q_out_stride=[0, 128])),
    (dict(), dict(q=FAKE, q_out=2 * FAKE, n_q_heads=1, q_stride=[512, 3], q_out_stride=[512, -3])),
    (dict(), dict(n=1, q=FAKE, q_out=FAKE, n_q_heads=4, q_stride=[512, 128], q_out_stride=[1024, 128]))])
def test_append_ignores_strides_of_extents_of_1(M, cache, kw):
    a = _append_args(M, acc=FAKE, **kw)
    assert M.lib.mkv_paged_append(ctypes.byref(_cache(M, **cache)), None, ctypes.byref(a), None) == M.MKV_ERR_INVALID_ARG
    assert "meta_stride" in M.mkv_last_error_string()
