"""Scores of the attention of many queries where their forms meet: caps of any size against
the 64-bit oracle, capped calls that repeat bit for bit, and sums over very many keys.

Tolerances, derived here once (u = 2^-24, e(t), scores, attend as in test_gpu_prompt.py):

capped   A capped score is within 2^-20 of itself: up to half the cap z times a polynomial that is
         within 2^-25 of tanh(t) / t, with 8 roundings; beyond it 1 - 2 / (x + 1) with t > 1/2: the
         argument's rounding, 2^-23 t (1 - tanh^2) / tanh <= 2^-23, of the exponential 2^-22, worth
         (1 - tanh^2) / (2 tanh) <= 0.86 of it, of the reciprocal 2^-23, worth 2 r / tanh <= 1.2, two
         roundings more: less than 2.5 2^-22.  So 2^-20 A in place of test_gpu_prompt.py's 2^-21 cap: it
         does not grow with the cap.  Caps up to 128 ln 2 = 88.7 (128 in the log2 domain) may take the second
         form for all scores of a block: its sum 1 - 2 r is off by 2^-23 for the reciprocal, 2^-23 for the
         exponential and 2^-24 more, together below 2^-21 of the cap, which comes on top.
pages    8-bit caches have fp16 weights whatever the queries' type is, so the 2^-33 sum |v| of such
         weights below the normal range (attend) holds for bf16 queries too: one key of weight 1 whose
         value is 0 leaves an output of 1e-9, of the other keys, where 2^-33 sum |v| is 1.4e-8.
long     The products' sums are cut off by less than 2 u of themselves in each of the 1024 steps of 16384
         keys; those of several times 16384 are added with u each, and the sum of weights, a block of 64
         or 128 keys at a time, by u of itself: (2048 + n / 16384 + n / 64) u in place of n u.  Capped
         or biased scores: 2048 steps of 32768 keys.
"""
import numpy as np
import pytest
import torch

from oracle import prompt as O
from test_gpu_prompt import (BF16, DEV, E4M3, F16, HALF, M, U, f64, i32, make_cache, near, rnd, rows_of)  # noqa: F401

pytestmark = pytest.mark.gpu


def capped_near(got, lse, ref, dtype, n, cap, fp16_weights=False):
    out, want_lse, spread, size, total = ref
    d = ((out.shape[-1] / 16 + 4) * 2.0**-22 + 2.0**-20) * size + (2.0**-21 * cap if cap <= 88.7 else 0.0)
    e = HALF[dtype]
    tol = (2 * d[..., None] + 2.0**-16 + e + (n + 64) * U) * spread + e * np.abs(out) * 1.01
    tol = tol + (2.0**-33 * total if dtype == F16 or fp16_weights else 0.0)
    near(got, out, tol + (2.0**-25 if dtype == F16 else 0.0))
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
    capped_near(f64(out[0]), f64(lse[0]), ref, qtype, n, cap, ctype == E4M3)


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
    capped_near(f64(out[0]), f64(lse[0]), ref, dtype, n, cap)


@pytest.mark.parametrize("cap", [2.0, 50.0, 88.0, 90.0, 200.0])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_scores_past_the_cap(M, dtype, cap):
    """Scores of some 45 in size, so that caps of any of the forms are reached."""
    for d, heads, kv in ((128, 4, 1), (64, 5, 1), (256, 2, 1)):
        n = 200
        q, k, v = rnd((1, n, heads, d), dtype, 1), rnd((1, n, kv, d), dtype, 2), rnd((1, n, kv, d), dtype, 3)
        lse = torch.empty((1, n, heads), device=DEV)
        scale = 45.0 / d**0.5
        out = M.mkv_prefill(q, k, v, lse=lse, cap=cap, scale=scale)
        ref = O.attend(f64(q[0]), f64(k[0]).transpose(1, 0, 2), f64(v[0]).transpose(1, 0, 2), O.visible(n, n),
                       np.arange(n), np.arange(n), scale, cap)
        capped_near(f64(out[0]), f64(lse[0]), ref, dtype, n, cap)
    for ctype in (dtype, E4M3):
        for m, g in ((2, 4), (12, 4), (40, 4)):
            pages_check(M, ctype, dtype, 300, m, g, 128, cap, scale=4.0)


TINY = [1e-3, 1e-4, 1e-6, 1e-8, 1e-20, 1e-37, 2.0**-149]


@pytest.mark.parametrize("cap", TINY)
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_tiny_caps(M, dtype, cap):
    """Queries of zeros, of which every score is 0, beside ones whose scores reach the cap."""
    for d, heads, kv in ((128, 2, 1), (64, 5, 1), (256, 2, 1)):
        n = 150
        q, k, v = rnd((1, n, heads, d), dtype, 1), rnd((1, n, kv, d), dtype, 2), rnd((1, n, kv, d), dtype, 3)
        q[:, :70] = 0.0
        lse = torch.empty((1, n, heads), device=DEV)
        out = M.mkv_prefill(q, k, v, lse=lse, cap=cap)
        ref = O.attend(f64(q[0]), f64(k[0]).transpose(1, 0, 2), f64(v[0]).transpose(1, 0, 2), O.visible(n, n),
                       np.arange(n), np.arange(n), None, cap)
        capped_near(f64(out[0]), f64(lse[0]), ref, dtype, n, cap)
    for ctype in (dtype, E4M3):
        for m, g in ((2, 4), (12, 4)):
            q = rnd((1, m, g, 128), dtype, 3)
            q[:, :m // 2] = 0.0
            pages_check(M, ctype, dtype, 300, m, g, 128, cap, q=q)


def prompt_call(M, d, heads, kv, cap, stray, slopes=None, dtype=BF16, nq=150, nk=333):
    """A padded batch whose rows behind the lengths hold `stray`: (out, lse) of the rows that are there."""
    q_lens, kv_lens = [150, 41, 7], [333, 300, 64]
    q, k, v = rnd((3, nq, heads, d), dtype, 1), rnd((3, nk, kv, d), dtype, 2), rnd((3, nk, kv, d), dtype, 3)
    for i in range(3):
        q[i, q_lens[i]:] = stray
        k[i, kv_lens[i]:] = stray
        v[i, kv_lens[i]:] = stray
    out, lse = torch.zeros_like(q), torch.zeros((3, nq, heads), device=DEV)
    M.mkv_prefill(q, k, v, out=out, lse=lse, cap=cap, q_lens=i32(q_lens), kv_lens=i32(kv_lens),
                  slopes=None if slopes is None else torch.tensor(slopes, dtype=torch.float32, device=DEV))
    return out, lse


@pytest.mark.parametrize("slopes", [False, True])
@pytest.mark.parametrize("d,heads,kv", [(128, 7, 1), (128, 28, 4), (64, 3, 1), (256, 6, 2), (64, 40, 2)])
def test_capped_prompts_do_not_depend_on_what_is_not_there(M, d, heads, kv, slopes):
    """The same bits whatever lies behind the lengths, and whatever calls ran before: rows of a tile
    that no query fills are what an earlier call left."""
    slopes = [2.0**-(i % 8 + 1) for i in range(heads)] if slopes else None
    want = prompt_call(M, d, heads, kv, 9.0, 0.0, slopes)
    loud = [rnd((2, 500, 8, x), BF16, 5, 50.0) for x in (64, 128, 256)]
    for stray in (0.0, 1e3, float("nan"), -1e30):
        for x in loud:
            M.mkv_prefill(x, x[:, :, :2], x[:, :, :2])
        assert all(torch.equal(a, b) for a, b in zip(want, prompt_call(M, d, heads, kv, 9.0, stray, slopes)))


@pytest.mark.parametrize("ctype,qtype", [(BF16, BF16), (E4M3, F16)])
@pytest.mark.parametrize("m,g", [(1, 1), (5, 3), (9, 3), (4, 7), (20, 7)])
def test_capped_pages_do_not_depend_on_what_is_not_there(M, ctype, qtype, m, g):
    q = rnd((2, m, 2 * g, 128), qtype, 4)
    lens, new = i32([300, 77]), i32([m, max(1, m // 2)])
    loud = rnd((2, 500, 8, 128), qtype, 5, 50.0)
    want = None
    for stray in (0.0, 1.0, 400.0, -400.0):
        cache = make_cache(M, ctype, 2, 2, 128, 32, 10, 3)
        for b, n in enumerate((300, 77)):
            for t in range(n, 320):
                page = int(cache.page_table[b, t // 32])
                cache.k_pages[page, :, t % 32] = stray
                cache.v_pages[page, :, t % 32] = stray
        x = q.clone()
        x[1, max(1, m // 2):] = 10 * stray
        M.mkv_prefill(loud, loud[:, :, :2], loud[:, :, :2])
        out, lse = torch.zeros_like(x), torch.zeros((2, m, 2 * g), device=DEV)
        M.mkv_paged_attend(cache, x, lens, new_lens=new, out=out, lse=lse, cap=9.0)
        want = want or (out, lse)
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


def test_capped_prompts_repeat(M):
    q, k, v = rnd((1, 3000, 28, 128), BF16, 1), rnd((1, 3000, 4, 128), BF16, 2), rnd((1, 3000, 4, 128), BF16, 3)
    want = M.mkv_prefill(q, k, v, cap=50.0)
    loud = rnd((2, 700, 14, 128), BF16, 5, 50.0)
    for _ in range(5):
        M.mkv_prefill(loud, loud[:, :, :2], loud[:, :, :2])
        assert torch.equal(want, M.mkv_prefill(q, k, v, cap=50.0))


def test_windows_both_ways_are_split_for_what_they_reach(M):
    """Without the causal mask a window of w sees as many keys as one of 2 w with it, and with a
    prefix any number: the parts of the keys, and the workspace, go by that."""
    sizes = (1, 4, 1 << 17, 8, 2, 128)
    both, one = (M.mkv_prefill_workspace(*sizes, window=w, causal=c, prefix=False)
                 for w, c in ((4096, False), (8192, True)))
    assert both == one != M.mkv_prefill_workspace(*sizes, window=4096, causal=True, prefix=False)
    assert M.mkv_prefill_workspace(*sizes, window=4096, prefix=True) == M.mkv_prefill_workspace(*sizes)
    assert M.mkv_prefill_workspace(*sizes, window=4096) == M.mkv_prefill_workspace(*sizes)
    q, k, v = rnd((1, 4, 8, 128), BF16, 1), rnd((1, 30000, 2, 128), BF16, 2), rnd((1, 30000, 2, 128), BF16, 3)
    for kw in (dict(window=4096, causal=False), dict(window=300, causal=False), dict(window=4096), dict(window=700, prefix=[9000])):
        kw = dict(kw)
        prefix = kw.pop("prefix", None)
        room = torch.empty(M.mkv_prefill_workspace(1, 4, 30000, 8, 2, 128, window=kw["window"], causal=kw.get("causal", True),
                                                   prefix=prefix is not None), dtype=torch.uint8, device=DEV)
        lse = torch.empty((1, 4, 8), device=DEV)
        out = M.mkv_prefill(q, k, v, lse=lse, prefix=None if prefix is None else i32(prefix), workspace=room, **kw)
        see = O.visible(4, 30000, kw.get("causal", True), kw["window"], None if prefix is None else prefix[0])
        ref = O.attend(f64(q[0]), f64(k[0]).transpose(1, 0, 2), f64(v[0]).transpose(1, 0, 2), see,
                       np.arange(29996, 30000), np.arange(30000))
        capped_near(f64(out[0]), f64(lse[0]), ref, BF16, 30000, 0.0)


def long_check(got, q, k, v, rows, base, cap=0.0, steps=1024):
    """Outputs of some rows of queries at places base + row, over keys and values [n, kv heads, d], against
    64 bits, and the mean of their relative errors where values have one sign."""
    n, hk, d = k.shape
    g = q.shape[1] // hk
    e, lost = HALF[got.dtype], []
    for h in range(q.shape[1]):
        kk, vv, qq = k[:, h // g].double(), v[:, h // g].double(), q[rows, h].double()
        z = qq @ kk.T / d**0.5
        size = (qq.abs() @ kk.abs().T / d**0.5).amax(-1, keepdim=True)
        z = cap * torch.tanh(z / cap) if cap else z
        z.masked_fill_(torch.arange(n, device=DEV)[None] > base + rows[:, None], -np.inf)
        w = torch.softmax(z, -1)
        want, spread = w @ vv, w @ vv.abs()
        # the roundings of the weights and of values held in 16 bits, and of the output
        tol = (2 * (d / 16 + 4) * 2.0**-22 * size + 2.0**-16 + e + (2 * steps + n / 16 / steps + n / 64 + 64) * U) * spread
        tol = tol + e * want.abs() * 1.01 + 2.0**-25
        assert ((got[rows, h].double() - want).abs() <= tol).all()
        lost.append((got[rows, h].double() / want - 1).flatten())
    return float(torch.cat(lost).mean())


def many(shape, dtype, seed, size=1.0, mean=0.0):
    """As rnd(), drawn on the GPU."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    return (torch.randn(shape, generator=g, device=DEV) * size + mean).to(dtype)


def ramp(n, hk, d, dtype, seed, size):
    """Keys whose scores with a first channel of 1 grow by `size` over all places."""
    k = many((1, n, hk, d), dtype, seed, 0.5)
    k[..., 0] = (torch.linspace(0, size * d**0.5, n, device=DEV)[:, None]).to(dtype)
    return k


@pytest.mark.parametrize("d,nq,heads,kv", [(256, 4096, 8, 4), (128, 8192, 16, 4), (64, 8192, 16, 4), (128, 3, 8, 2),
                                           (256, 1, 4, 1), (64, 20, 4, 1)])
@pytest.mark.parametrize("size", [0.0, 25.0])
def test_long_walks_lose_nothing(M, d, nq, heads, kv, size):
    """Values of one sign over many keys, scores nearly equal or growing all the way."""
    n = (1 << 21) + 77 if nq < 100 else (1 << 17) + 77
    q = rnd((1, nq, heads, d), F16, 1, 0.25)
    q[..., 0] = 1.0
    k = ramp(n, kv, d, F16, 2, size)
    v = many((1, n, kv, d), F16, 3, 0.25, 1.5)
    out = M.mkv_prefill(q, k, v)
    lost = long_check(out[0], q[0], k[0], v[0], torch.arange(0, nq, max(1, nq // 16), device=DEV), n - nq)
    # 1024 steps cut off by less than 2 u, blocks of the sum of weights u each, and the mean of roundings
    # of which there are thousands: six deviations of a step of 2^-11 over the square root of their number
    parts = n if nq >= 100 else n / 64
    assert abs(lost) <= (2048 + parts / 64) * U + 6 * 2.0**-11 / (3 * 16 * d) ** 0.5


@pytest.mark.parametrize("d,nq,heads,kv", [(256, 4096, 8, 4), (128, 8192, 16, 4)])
@pytest.mark.parametrize("size", [0.0, 25.0])
def test_long_capped_walks_lose_little(M, d, nq, heads, kv, size):
    n = (1 << 19) + 77
    q = rnd((1, nq, heads, d), F16, 1, 0.25)
    q[..., 0] = 1.0
    k = ramp(n, kv, d, F16, 2, size)
    v = many((1, n, kv, d), F16, 3, 0.25, 1.5)
    out = M.mkv_prefill(q, k, v, cap=30.0)
    lost = long_check(out[0], q[0], k[0], v[0], torch.arange(0, nq, nq // 16, device=DEV), n - nq, 30.0, 2048)
    assert abs(lost) <= (4096 + n / 64) * U + 6 * 2.0**-11 / (3 * 16 * d) ** 0.5


@pytest.mark.parametrize("ctype,qtype", [(F16, F16), (E4M3, F16)])
@pytest.mark.parametrize("m,g", [(512, 4), (40, 4), (4, 4)])
@pytest.mark.parametrize("size", [0.0, 25.0])
def test_long_walks_over_pages_lose_nothing(M, ctype, qtype, m, g, size):
    n, kv, d, ps = (1 << 17) * (4 if m < 512 else 1), 8 if m == 512 else 1, 128, 128
    q = rnd((1, m, kv * g, d), qtype, 1, 0.25)
    q[..., 0] = 1.0
    k = ramp(n, kv, d, F16, 2, size).to(ctype)
    v = many((1, n, kv, d), F16, 3, 0.25, 1.5).to(ctype)
    pages = [x.view(n // ps, ps, kv, d).view(torch.uint8 if ctype == E4M3 else ctype).transpose(1, 2).contiguous().view(ctype)
             for x in (k, v)]
    cache = M.MkvPaged(*pages, torch.arange(n // ps, dtype=torch.int32, device=DEV).view(1, -1))
    out = M.mkv_paged_attend(cache, q, i32([n]))
    long_check(out[0], q[0], k[0].float(), v[0].float(), torch.arange(0, m, max(1, m // 16), device=DEV), n - m)
    assert cache.check() == M.MKV_OK


def test_long_walks_with_options(M):
    """Biased scores walk from the last key down; capped ones; documents and windows skip blocks."""
    n, nq = 40000, 4096
    q, k = rnd((1, nq, 8, 128), BF16, 1), rnd((1, n, 2, 128), BF16, 2)
    v = (rnd((1, n, 2, 128), torch.float32, 3, 0.25) + 1.5).to(BF16)
    rows = [0, 1234, nq - 1]
    docs = ((torch.arange(n, device=DEV)[None] // 3000) % 2).int()
    for kw in (dict(slopes=[1e-4 * (i + 1) for i in range(8)]), dict(cap=5.0), dict(docs=docs), dict(window=20000),
               dict(window=12000, causal=False), dict(slopes=[-1e-4] * 8, cap=9.0)):
        call = dict(kw)
        if "slopes" in kw:
            call["slopes"] = torch.tensor(kw["slopes"], dtype=torch.float32, device=DEV)
        lse = torch.empty((1, nq, 8), device=DEV)
        out = M.mkv_prefill(q, k, v, lse=lse, **call)
        see = O.visible(nq, n, kw.get("causal", True), kw.get("window", 0), None,
                        docs[0].cpu().numpy() if "docs" in kw else None)[rows]
        ref = O.attend(f64(q[0, rows]), f64(k[0]).transpose(1, 0, 2), f64(v[0]).transpose(1, 0, 2), see,
                       n - nq + np.array(rows), np.arange(n), None, kw.get("cap", 0.0), kw.get("slopes"))
        capped_near(f64(out[0, rows]), f64(lse[0, rows]), ref, BF16, 4096 + n / 64, kw.get("cap", 0.0))


@pytest.mark.parametrize("m,g", [(1, 4), (2, 4), (3, 3), (4, 8), (12, 5), (40, 4)])
@pytest.mark.parametrize("d,ps", [(64, 16), (128, 32), (256, 48)])
@pytest.mark.parametrize("kw", [{}, dict(cap=9.0), dict(slopes=True)])
def test_nan_behind_a_sequence_of_8_bit_pages(M, d, ps, m, g, kw):
    """Slots from the length on may hold anything, NaN too, which e4m3 has (0x7f, 0xff)."""
    lens = [300, 33 + m, m]
    clean = make_cache(M, E4M3, 3, 2, d, ps, -(-320 // ps), 5)
    q = rnd((3, m, 2 * g, d), F16, 4)
    call = dict(kw)
    if "slopes" in kw:
        call["slopes"] = torch.tensor([2.0**-(i % 6 + 1) for i in range(2 * g)], dtype=torch.float32, device=DEV)
    got = []
    for stray in (0x00, 0x7f, 0xff):
        for b, n in enumerate(lens):
            for t in range(n, clean.page_table.shape[1] * ps):
                page = int(clean.page_table[b, t // ps])
                for pool in (clean.k_pages, clean.v_pages):
                    pool.view(torch.uint8)[page, :, t % ps] = stray
        lse = torch.empty((3, m, 2 * g), device=DEV)
        got.append((M.mkv_paged_attend(clean, q, i32(lens), lse=lse, **call), lse))
    assert clean.check() == M.MKV_OK
    for out, lse in got:
        assert torch.isfinite(out.float()).all() and torch.equal(out, got[0][0]) and torch.equal(lse, got[0][1])
    for i, n in enumerate(lens):
        ref = O.attend(f64(q[i]), rows_of(clean, 0, i, n), rows_of(clean, 1, i, n), O.visible(m, n), np.arange(n - m, n),
                       np.arange(n), None, kw.get("cap", 0.0), f64(call["slopes"]) if "slopes" in kw else None)
        capped_near(f64(got[1][0][i]), f64(got[1][1][i]), ref, F16, n, kw.get("cap", 0.0))


def test_the_status_word_of_prompts(M):
    """Left as it is where every wait was over in time, whatever the lengths, and not needed."""
    q, k = rnd((2, 140, 4, 128), BF16, 1), rnd((2, 300, 2, 128), BF16, 2)
    want = M.mkv_prefill(q, k, k, q_lens=i32([140, 500]), kv_lens=i32([300, -4]))
    for word in (0, 64):
        status = i32([word])
        got = M.mkv_prefill(q, k, k, q_lens=i32([140, 500]), kv_lens=i32([300, -4]), status=status)
        assert torch.equal(got, want) and int(status) == word
    with pytest.raises((TypeError, ValueError)):
        M.mkv_prefill(q, k, k, status=torch.zeros(1, dtype=torch.int64, device=DEV))


@pytest.mark.parametrize("cap", [0.0, 30.0])
def test_long_walks_captured_and_on_two_streams(M, cap):
    """The sums of a call lie in its own workspace: a replayed graph and calls side by side give the
    same bits, whatever the workspace held before."""
    q = [many((1, 4096, 8, 128), BF16, s) for s in (1, 2)]
    k, v = many((1, 40000, 2, 128), BF16, 3), many((1, 40000, 2, 128), BF16, 4)
    need = M.mkv_prefill_workspace(1, 4096, 40000, 8, 2, 128, capped=cap > 0)
    assert need > 0
    want = [M.mkv_prefill(x, k, v, cap=cap) for x in q]
    torch.cuda.synchronize()
    room = torch.full((need,), 0xff, dtype=torch.uint8, device=DEV)
    x = torch.zeros_like(q[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = M.mkv_prefill(x, k, v, cap=cap, workspace=room)
    for i in (0, 1, 0):
        x.copy_(q[i])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[i])
    streams = [torch.cuda.Stream() for _ in q]
    for _ in range(3):
        got = [M.mkv_prefill(y, k, v, cap=cap, stream=s) for y, s in zip(q, streams)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    with pytest.raises(M.MkvError):
        M.mkv_prefill(q[0], k, v, cap=cap, workspace=room[:-1])
