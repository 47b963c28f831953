"""Scores of the attention of many queries where their forms meet: caps of any size, against
the 64-bit oracle.

Tolerances, derived here once (u = 2^-24, e(t), scores, attend as in test_gpu_prompt.py):

capped   A capped score is within 2^-20 of itself: up to half the cap z times a polynomial that is
         within 2^-25 of tanh(t) / t, with 8 roundings; beyond it 1 - 2 / (x + 1) with t > 1/2: the
         argument's rounding, 2^-23 t (1 - tanh^2) / tanh <= 2^-23, of the exponential 2^-22, worth
         (1 - tanh^2) / (2 tanh) <= 0.86 of it, of the reciprocal 2^-23, worth 2 r / tanh <= 1.2, two
         roundings more: less than 2.5 2^-22.  So 2^-20 A in place of test_gpu_prompt.py's 2^-21 cap: it
         does not grow with the cap.
"""
import numpy as np
import pytest
import torch

from oracle import prompt as O
from test_gpu_prompt import (BF16, DEV, E4M3, F16, HALF, M, U, f64, i32, make_cache, near, rnd, rows_of)  # noqa: F401

pytestmark = pytest.mark.gpu


def capped_near(got, lse, ref, dtype, n):
    out, want_lse, spread, size, total = ref
    d = ((out.shape[-1] / 16 + 4) * 2.0**-22 + 2.0**-20) * size
    e = HALF[dtype]
    tol = (2 * d[..., None] + 2.0**-16 + e + (n + 64) * U) * spread + e * np.abs(out) * 1.01
    near(got, out, tol + (2.0**-33 * total + 2.0**-25 if dtype == F16 else 0.0))
    near(lse, want_lse, d + (n + 64) * U + 2.0**-22 * np.abs(want_lse) + 2.0**-21)


def pages_check(M, ctype, qtype, n, m, g, d, cap, q=None, scale=0.0, slopes=None, seed=0):
    """One sequence of n slots, its last m new in a chain, over one KV head."""
    cache = make_cache(M, ctype, 1, 1, d, 32, -(-n // 32), seed)
    q = rnd((1, m, g, d), qtype, seed + 9) if q is None else q
    lse = torch.empty((1, m, g), device=DEV)
    out = M.mkv_paged_attend(cache, q, i32([n]), lse=lse, cap=cap, scale=scale,
                             slopes=None if slopes is None else torch.tensor(slopes, dtype=torch.float32, device=DEV))
    ref = O.attend(f64(q[0]), rows_of(cache, 0, 0, n), rows_of(cache, 1, 0, n), O.visible(m, n), np.arange(n - m, n),
                   np.arange(n), scale or None, cap, slopes)
    capped_near(f64(out[0]), f64(lse[0]), ref, qtype, n)


CAPS = [0.01, 1.0, 20.0, 1e3, 1e4, 1e5, 1e6, 1e8, 1e18, 1e30, 1e37, 2.0**127]


@pytest.mark.parametrize("cap", CAPS)
@pytest.mark.parametrize("ctype,qtype", [(E4M3, F16), (E4M3, BF16), (F16, F16), (BF16, BF16)])
def test_pages_caps_of_any_size(M, ctype, qtype, cap):
    for m, g, d in ((1, 8, 128), (2, 4, 64), (1, 3, 256), (3, 3, 128), (12, 4, 64)):
        pages_check(M, ctype, qtype, 300, m, g, d, cap, seed=d)
    pages_check(M, ctype, qtype, 300, 2, 4, 128, cap, slopes=[0.5, 0.1, 0.02, 0.004])


@pytest.mark.parametrize("ctype,qtype", [(E4M3, F16), (E4M3, BF16), (F16, F16), (BF16, BF16)])
@pytest.mark.parametrize("m,g", [(4, 2), (9, 2)])
def test_pages_scores_above_a_large_cap_beside_small_ones(M, ctype, qtype, m, g):
    """One new token's scores reach the cap, the others' are a millionth of it."""
    q = rnd((1, m, g, 128), qtype, 3, 0.01)
    q[:, 0] *= 3e5
    pages_check(M, ctype, qtype, 300, m, g, 128, 1e6, q=q, scale=100.0)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("cap", CAPS)
def test_prompt_caps_of_any_size(M, dtype, d, cap):
    n = 200
    q, k, v = rnd((1, n, 3, d), dtype, 1), rnd((1, n, 1, d), dtype, 2), rnd((1, n, 1, d), dtype, 3)
    lse = torch.empty((1, n, 3), device=DEV)
    out = M.mkv_prefill(q, k, v, lse=lse, cap=cap)
    ref = O.attend(f64(q[0]), f64(k[0]).transpose(1, 0, 2), f64(v[0]).transpose(1, 0, 2), O.visible(n, n), np.arange(n),
                   np.arange(n), None, cap)
    capped_near(f64(out[0]), f64(lse[0]), ref, dtype, n)
