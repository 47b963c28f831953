"""Rotary positions and the paged cache on the GPU against the 64-bit oracle.

Tolerances, derived here once (u = 2^-24, the half step of fp32 relative to a
value; e(t) = the half step of the output type):

rope     The phase is exact; read as an fp32 fraction of a half turn below 1 it is
         off by 2^-25, pi times that in radians: 1.6 u.  sincospif is within 2 units
         in the last place (4 u), its product with the factor 1 u (the factor's own
         rounding 1 u), two products and a sum 2 u on a pair of length r: at most
         10 u r, then the output's rounding.  Taken: 12 u r + e(t) |y| + the
         smallest half step (2^-25 for fp16).
decode   A score is a sum of D exact products, accumulated in fp32 by D / 16 matrix
         steps and rounded by the scaling: at most d = (D / 16 + 4) 2^-22 A with A =
         scale sum |q_i k_i| (a step may truncate: 2^-23 of the partial sums, twice
         for the order inside).  Each weight is then off by 2 d + 2^-16 relative
         (maximum and sum share d; exp2f 2 u; bf16 halves leave 2^-18), sums of n
         terms by n u: out within (2 d + 2^-16 + (n + 64) u) sum p |v| + e(t) |o|.
         8-bit caches: the products of scales add 4 u, inside 2^-16.
         fp16 weights (F16 and E4M3 caches) are 2^12 p / max p as a sum of two fp16
         numbers; below 2^-14 their steps are 2^-24, the second cannot refine the
         first, and they are off by up to 2^-25, so p by 2^-37: 2^-37 sum |v| more.
         lse within d + (n + 64) u + 2^-22 |lse| + 2^-21.  Accumulated weights
         within (2 d + 2^-16 + (n + 64) u) w + u acc.
append   16-bit rows as rope; 8-bit rows half a step of e4m3 (2^-4 of the value, 2^-10
         below the normal range) more than the rope error over the scale.
evict    exact.
"""
import math

import numpy as np
import pytest
import torch

from oracle import paged as P

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


# ---- rope ---------------------------------------------------------------------------------------

def rope_close(got, want, x, rot, interleaved, mult, dtype):
    x = np.abs(x)
    pair = x.copy()
    if interleaved:
        r = np.hypot(x[..., 0:rot:2], x[..., 1:rot:2])
        pair[..., 0:rot:2] = pair[..., 1:rot:2] = r
    else:
        r = np.hypot(x[..., : rot // 2], x[..., rot // 2:rot])
        pair[..., :rot] = np.concatenate([r, r], -1)
    pair[..., rot:] = 0.0
    low = 2.0**-25 if dtype == F16 else 0.0
    tol = 12 * U * pair * mult + HALF[dtype] * np.abs(want) * (1 + 2.0**-8) + low
    tol[..., rot:] = 0.0
    bad = np.abs(got - want) > tol
    assert not bad.any(), (np.argwhere(bad)[:3], np.abs(got - want).max())


ROPE_SHAPES = [
    # batch, tokens, heads, dim, rot
    (1, 1, 1, 2, 2), (1, 1, 32, 128, 128), (3, 5, 2, 64, 64), (2, 33, 3, 80, 80), (1, 257, 5, 96, 64),
    (2, 7, 28, 128, 32), (1, 19, 8, 256, 256), (2, 3, 4, 128, 24), (1, 6, 2, 100, 50), (1, 4, 3, 4096, 256),
    (5, 1, 1, 17, 16)]


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("shape", ROPE_SHAPES)
def test_rope(M, shape, interleaved, dtype):
    b, t, h, d, rot = shape
    for n, kw in enumerate([dict(), dict(scaling="yarn", factor=8.0, original=64)]):
        base = 1000.0 if n else 500000.0
        x = rnd((b, t, h, d), dtype, 3 + n, 4.0)
        pos = torch.randint(-5, 1 << 20, (b, t), dtype=torch.int32, generator=torch.Generator().manual_seed(n))
        pos[0, 0] = 2**31 - 1
        plan = M.mkv_rope_plan(d, rot_dim=rot, base=base, interleaved=interleaved, **kw)
        freq, mult = P.rope_frequencies(rot, base, **kw)
        for back in (False, True):
            got = M.mkv_rope(plan, x, pos.to(DEV), transposed=back)
            want = P.rope(f64(x), pos.numpy(), freq, mult, interleaved, back)
            rope_close(f64(got), want, f64(x), rot, interleaved, mult, dtype)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_strides_layouts_and_in_place(M, interleaved):
    b, t, h, d = 2, 37, 3, 64
    plan = M.mkv_rope_plan(d, interleaved=interleaved)
    freq, _ = P.rope_frequencies(d, 10000.0)
    big = rnd((b, t, 3 * h, d + 8), F16, 1)
    pos = torch.arange(1000, 1000 + b * t, dtype=torch.int32).view(b, t)
    wide = torch.full((b, t + 5), -3, dtype=torch.int32, device=DEV)
    wide[:, :t] = pos.to(DEV)
    for first in (0, 1):                       # aligned and unaligned starts of a head
        x = big[:, :, h:2 * h, first:first + d]
        before = big.clone()
        want = P.rope(f64(x), pos.numpy(), freq, interleaved=interleaved)
        # token-major in, head-major out
        out = torch.full((b, h, t, d), 7.0, dtype=F16, device=DEV)
        got = M.mkv_rope(plan, x, wide[:, :t], out=out.transpose(1, 2))
        rope_close(f64(got), want, f64(x), d, interleaved, 1.0, F16)
        assert torch.equal(got, M.mkv_rope(plan, x.contiguous(), pos.to(DEV)))
        assert torch.equal(before, big)
        # in place in the larger tensor: nothing around it changes
        M.mkv_rope(plan, x, pos.to(DEV), out=x)
        assert torch.equal(x, got)
        rest = torch.ones_like(big, dtype=torch.bool)
        rest[:, :, h:2 * h, first:first + d] = False
        assert torch.equal(big[rest], before[rest])
    # a broadcast input, and positions that count from first_pos
    one = rnd((1, 1, 1, d), F16, 2)
    got = M.mkv_rope(plan, one.expand(2, 9, 4, d), first_pos=70)
    want = P.rope(f64(one.expand(2, 9, 4, d)), np.broadcast_to(np.arange(70, 79), (2, 9)), freq, interleaved=interleaved)
    rope_close(f64(got), want, f64(one.expand(2, 9, 4, d)), d, interleaved, 1.0, F16)
    with pytest.raises(M.MkvError):
        M.mkv_rope(plan, one.expand(2, 9, 4, d), out=one.expand(2, 9, 4, d).clone()[:, :1].expand(2, 9, 4, d))


def test_rope_gradient(M):
    """<rope(x), g> = <x, transposed(g)>, and central differences of it, in fp32."""
    plan = M.mkv_rope_plan(64, rot_dim=48, scaling="yarn", factor=4.0, original=128)
    x, g = rnd((2, 5, 3, 64), F32, 1), rnd((2, 5, 3, 64), F32, 2)
    pos = torch.arange(10, dtype=torch.int32, device=DEV).view(2, 5) * 1000
    y, back = f64(M.mkv_rope(plan, x, pos)), f64(M.mkv_rope(plan, g, pos, transposed=True))
    n = x.numel()
    # every term within 12 u of a product of pairs' lengths (<= 2 mult |x| |g|), n of them
    size = np.linalg.norm(f64(x)) * np.linalg.norm(f64(g)) * plan.mult
    assert abs((y * f64(g)).sum() - (f64(x) * back).sum()) <= 2 * 12 * U * size * 2
    # the map is linear: a difference of any width is the derivative; width 1 in one element
    for i in (0, 130, 500, n - 1):
        e = torch.zeros(n, device=DEV)
        e[i] = 1.0
        e = e.view_as(x)
        d = (f64(M.mkv_rope(plan, x + e, pos)) - f64(M.mkv_rope(plan, x - e, pos))) / 2
        slope = (d * f64(g)).sum()
        # four rounded vectors of a pair: 12 u each times |x| + 1 <= 6, times |g| <= 6, twice
        assert abs(slope - back.reshape(-1)[i]) <= 4 * 12 * U * 36 * plan.mult


# ---- caches -------------------------------------------------------------------------------------

class Cache:
    """A cache with scattered pages; everything outside the sequences is NaN."""

    def __init__(self, M, dtype, lens, heads, dim, page, seed=0, spare=3, size=1.0, room=0):
        g = torch.Generator().manual_seed(seed)
        self.lens_list = list(lens)
        b = len(lens)
        per = max(1, -(-(max(list(lens) + [1]) + room) // page))
        n = b * per + spare
        table = torch.randperm(n, generator=g)[: b * per].view(b, per).to(torch.int32)
        # a table with a wider row stride and rubbish behind the pages in use
        wide = torch.full((b, per + 2), -77, dtype=torch.int32)
        wide[:, :per] = table
        for i, m in enumerate(lens):
            used = -(-(m + room) // page)
            wide[i, used:] = 2**30
        self.np_table = table.numpy()
        self.scales = [None, None]
        if dtype == E4M3:
            self.scales = [torch.rand(heads, generator=g) + 0.5 for _ in range(2)]
        self.pools = []
        dg = torch.Generator(device=DEV)
        dg.manual_seed(seed)
        held = (torch.arange(per * page).view(1, per, 1, page, 1) < torch.tensor(list(lens)).view(b, 1, 1, 1, 1)).to(DEV)
        for k in range(2):
            rows = torch.randn((b, per, heads, page, dim), generator=dg, device=DEV) * size
            if dtype == E4M3:
                rows = rows.clamp(-440, 440)
            x = torch.full((n, heads, page, dim), float("nan"), device=DEV)
            x[table.view(-1).long().to(DEV)] = torch.where(held, rows, float("nan")).flatten(0, 1)
            self.pools.append(x.to(dtype))
        self.table = wide.to(DEV)[:, :per]
        self.lens = torch.tensor(self.lens_list, dtype=torch.int32, device=DEV)
        self.dev_scales = [None if s is None else s.to(DEV) for s in self.scales]
        self.c = M.MkvPaged(*self.pools, self.table, *self.dev_scales)
        self.M = M

    def rows(self, i, n=None):
        n = self.lens_list[i] if n is None else n
        used = max(1, -(-n // self.pools[0].shape[2]))
        at = torch.from_numpy(self.np_table[i, :used]).long().to(DEV)
        pick = lambda x: x[at] if x.dtype != E4M3 else x.view(torch.uint8)[at].view(E4M3)
        return [P.gather(f64(pick(x)), range(used), n, None if s is None else s.numpy().astype(np.float64))
                for x, s in zip(self.pools, self.scales)]


def decode_check(cache, q, out, lse, acc, acc0, scale=None):
    d = q.shape[-1]
    for i in range(q.shape[0]):
        k, v = cache.rows(i)
        h, n, _ = k.shape
        qi = f64(q[i])
        want, wlse, mass, size = P.decode(qi, k, v, scale)
        g = qi.shape[0] // h
        s = d ** -0.5 if scale is None else scale
        err = np.array([s * (np.abs(k[j // g]) @ np.abs(qi[j])).max() if n else 0.0 for j in range(g * h)])
        err *= (d / 16 + 4) * 2.0**-22
        rel = 2 * err + 2.0**-16 + (n + 64) * U
        tol = rel[:, None] * size + HALF[out.dtype] * np.abs(want) + (2.0**-25 if out.dtype == F16 else 0)
        if cache.pools[0].dtype != BF16:
            tol += 2.0**-37 * np.abs(v).sum(1).repeat(g, 0)
        bad = np.abs(f64(out[i]) - want) > tol
        assert not bad.any(), (i, n, np.abs(f64(out[i]) - want).max())
        assert not np.isnan(f64(out[i])).any()
        if lse is not None:
            got = f64(lse[i])
            if n == 0:
                assert (got == -np.inf).all()
            else:
                assert (np.abs(got - wlse) <= err + (n + 64) * U + 2.0**-22 * np.abs(wlse) + 2.0**-21).all()
        if acc is not None:
            got, was = f64(acc[i]), f64(acc0[i])
            w = got[:, :n] - was[:, :n]
            r = rel.reshape(h, g).max(1)[:, None]
            assert (np.abs(w - mass) <= r * mass + U * np.abs(got[:, :n]) * 1.01 + 2.0**-100).all()
            assert (got[:, n:] == was[:, n:]).all()
    assert cache.c.check() == cache.M.MKV_OK


def decode_run(M, cache, heads, group, dim, qt, out_dtype=None, weights=True, seed=5, size=1.0, **kw):
    b = len(cache.lens_list)
    q = rnd((b, heads * group, dim), qt, seed, size)
    lse = torch.full((b, heads * group), 5.0, device=DEV)
    slots = max(cache.lens_list + [1, kw.get("max_len", 0)]) + 3
    acc = rnd((b, heads, slots), F32, seed + 1).abs() if weights else None
    acc0 = None if acc is None else acc.clone()
    if acc is not None:
        kw.setdefault("max_len", max(cache.lens_list + [1]))
    out = M.mkv_paged_decode(cache.c, q, cache.lens, lse=lse, acc=acc, out_dtype=out_dtype, **kw)
    decode_check(cache, q, out, lse, acc, acc0)
    return q, out, lse, acc


LENS = [0, 1, 2, 15, 16, 17, 47, 64, 65, 300]


@pytest.mark.parametrize("dtype,qt", [(F16, F16), (BF16, BF16), (E4M3, F16), (E4M3, BF16)])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("group", [1, 7, 16])
def test_decode_whole_streams(M, dtype, qt, dim, group):
    """Short streams in clusters of one or two CTAs: short sequences, an empty one, pages that end inside the work of a step."""
    for page in (16, 48):
        cache = Cache(M, dtype, LENS, 2, dim, page, seed=group)
        decode_run(M, cache, 2, group, dim, qt, out_dtype=F32 if group == 7 else None)


@pytest.mark.parametrize("dtype,qt", [(F16, F16), (BF16, BF16), (E4M3, BF16)])
@pytest.mark.parametrize("dim,group,page", [(64, 4, 16), (128, 4, 64), (128, 9, 48), (256, 8, 256), (256, 12, 32)])
@pytest.mark.parametrize("bound", [4097, 9000])
def test_decode_long_streams(M, dtype, qt, dim, group, page, bound):
    """Streams cut and joined: long and short ones, empty ones at both ends.  With a bound of 4097
    on 16 streams a cluster takes a stream, with 9000 the load is split over all streams."""
    cache = Cache(M, dtype, [0, 2500, 1, 0, 1100, 33, 4097, 0], 2, dim, page, seed=dim, room=bound - 4097)
    decode_run(M, cache, 2, group, dim, qt, out_dtype=F32, max_len=bound)
    decode_run(M, cache, 2, group, dim, qt, weights=False, seed=9, max_len=bound)


@pytest.mark.parametrize("heads,ctas", [(1, 8), (3, 4), (6, 2), (9, 1)])
def test_decode_sizes_of_cluster(M, heads, ctas):
    """8, 4, 2 and 1 CTAs a stream, with lengths that leave some of them without a token."""
    cache = Cache(M, F16, [1030, 1, 17, 0, 300, 129, 16, 500], heads, 64, 48, seed=heads)
    decode_run(M, cache, heads, 3, 64, F16, out_dtype=F32)


def test_decode_one_long_stream(M):
    """A single stream over all CTAs, and one KV head for 16 query heads."""
    cache = Cache(M, F16, [20011], 1, 64, 128, seed=1)
    decode_run(M, cache, 1, 16, 64, F16, out_dtype=F32)
    decode_run(M, cache, 1, 1, 64, F16)


def test_decode_many_sequences(M):
    """More sequences than the split kernel's prefix sums hold, and the most that they hold."""
    for b in (512, 513, 1025):
        lens = [(37 * i) % 2600 if i % 97 == 5 else i % 5 for i in range(b)]
        assert max(lens) > 2048
        cache = Cache(M, E4M3, lens, 1, 64, 256, seed=2, spare=0)
        decode_run(M, cache, 1, 2, 64, F16)


@pytest.mark.parametrize("size", [1e-6, 30.0, 2000.0])
def test_decode_small_and_large_scores(M, size):
    """Nearly uniform softmax, and one token that takes it all; scores past exp's range."""
    for dtype, qt in ((F16, F16), (BF16, BF16), (E4M3, F16)):
        cache = Cache(M, dtype, [1300, 40], 2, 128, 32, seed=3)
        decode_run(M, cache, 2, 4, 128, qt, out_dtype=F32, size=size)


def test_decode_equal_scores(M):
    """All scores equal: weights are exactly 1 / n each, also where 1 / n is below fp16's range."""
    n = 5000
    cache = Cache(M, F16, [n], 1, 64, 64, seed=4)
    q = torch.zeros((1, 4, 64), dtype=F16, device=DEV)
    acc = torch.zeros((1, 1, n), device=DEV)
    lse = torch.empty((1, 4), device=DEV)
    out = M.mkv_paged_decode(cache.c, q, cache.lens, lse=lse, acc=acc, out_dtype=F32, max_len=n)
    decode_check(cache, q, out, lse, acc, torch.zeros_like(acc))


def test_decode_strided_queries_scale_and_out(M):
    cache = Cache(M, BF16, [100, 1030], 3, 128, 16, seed=6)
    big = rnd((2, 20, 3, 128), BF16, 8)
    q = big[:, 2:14, 1]                          # 12 heads with a wider stride
    out = torch.empty((2, 12, 128), dtype=BF16, device=DEV)
    assert M.mkv_paged_decode(cache.c, q, cache.lens, out=out, scale=0.3) is out
    decode_check(cache, q, out, None, None, None, scale=float(np.float32(0.3)))
    ws = torch.empty(M.mkv_paged_decode_workspace(cache.c, 12), dtype=torch.uint8, device=DEV)
    again = M.mkv_paged_decode(cache.c, q.contiguous(), cache.lens, scale=0.3, workspace=ws)
    assert torch.equal(out, again)               # no atomics: the same bits
    with pytest.raises(M.MkvError, match="workspace"):
        M.mkv_paged_decode(cache.c, q, cache.lens, workspace=ws[: ws.numel() - 256])


def test_decode_lengths_and_pages_outside(M):
    """Bad lengths count as the nearest good one, a bad page's tokens as absent; both reported."""
    cache = Cache(M, F16, [70, 40, 1200], 2, 64, 16, seed=7)
    q = rnd((3, 4, 64), F16, 9)
    want = M.mkv_paged_decode(cache.c, q, torch.tensor([0, 40, 1200], dtype=torch.int32, device=DEV))
    assert cache.c.check() == M.MKV_OK
    zero = M.mkv_paged_decode(cache.c, q, torch.tensor([-5, 40, 1200], dtype=torch.int32, device=DEV))
    assert cache.c.check() == M.MKV_ERR_DEVICE_CHECK and cache.c.check() == M.MKV_OK
    assert (zero[0] == 0).all() and torch.equal(zero, want)
    # beyond the bound: as if 64 tokens were cached
    for bound in (64, 1100):
        lens = torch.tensor([bound + 1, 5, 2**31 - 1], dtype=torch.int32, device=DEV)
        few = torch.tensor([bound, 5, bound], dtype=torch.int32, device=DEV)
        cache.lens_list = few.tolist()
        cache2 = Cache(M, F16, [1200] * 3, 2, 64, 16, seed=8)
        got = M.mkv_paged_decode(cache2.c, q, lens, max_len=bound)
        assert cache2.c.check() == M.MKV_ERR_DEVICE_CHECK
        assert torch.equal(got, M.mkv_paged_decode(cache2.c, q, few, max_len=bound))
        assert cache2.c.check() == M.MKV_OK
    # pages 1 and 3 of sequence 2 are gone: the rest of its tokens are attended
    for bad in (-1, 2**31 - 1):
        cache3 = Cache(M, F16, [70, 40, 1200], 2, 64, 16, seed=7)
        cache3.table[2, 1] = bad
        cache3.table[2, 3] = bad
        acc = torch.zeros((3, 2, 1200), device=DEV)
        got = M.mkv_paged_decode(cache3.c, q, cache3.lens, acc=acc, out_dtype=F32)
        assert cache3.c.check() == M.MKV_ERR_DEVICE_CHECK
        k, v = cache3.rows(2)
        left = np.r_[0:16, 32:48, 64:1200]
        o, _, mass, size = P.decode(f64(q[2]), k[:, left], v[:, left])
        assert (np.abs(f64(got[2]) - o) <= 2.0**-12 * size).all()     # far inside: which tokens, not rounding
        a = f64(acc[2])
        assert (a[:, 16:32] == 0).all() and (a[:, 48:64] == 0).all() and (a[:, left] > 0).all()
    # every page of a sequence gone: an empty row
    cache3.table[1, :] = -9
    lse = torch.empty((3, 4), device=DEV)
    acc.zero_()
    got = M.mkv_paged_decode(cache3.c, q, cache3.lens, lse=lse, acc=acc)
    assert (got[1] == 0).all() and (lse[1] == -math.inf).all() and (acc[1] == 0).all()


def test_decode_nan_reaches_only_its_own(M):
    """A NaN or an infinity among live rows shows in its own stream's output and nowhere else."""
    cache = Cache(M, F16, [300, 1100], 2, 128, 16, seed=10)
    q = rnd((2, 8, 128), F16, 9)
    want = M.mkv_paged_decode(cache.c, q, cache.lens)
    k = cache.pools[0]
    k[int(cache.np_table[1, 2]), 1, 3, 5] = float("nan")
    got = M.mkv_paged_decode(cache.c, q, cache.lens)
    assert torch.isnan(got[1, 4:]).all() and torch.equal(got[0], want[0]) and torch.equal(got[1, :4], want[1, :4])


def test_decode_far_offsets(M):
    """Rows more than 2^32 bytes into a pool."""
    n, h, ps, d = 40000, 1, 256, 256
    pools = [torch.empty((n, h, ps, d), dtype=F16, device=DEV) for _ in range(2)]     # 5.2 GB each
    table = torch.tensor([[39999, 0, 20000, 32768]], dtype=torch.int32, device=DEV)
    rows = [rnd((4, h, ps, d), F16, 20 + i) for i in range(2)]
    for pool, r in zip(pools, rows):
        for j in range(4):
            pool[int(table[0, j])] = r[j]
    c = M.MkvPaged(*pools, table)
    q = rnd((1, 2, d), F16, 3)
    lens = torch.tensor([1024], dtype=torch.int32, device=DEV)
    got = M.mkv_paged_decode(c, q, lens)
    small = M.MkvPaged(*rows, torch.arange(4, dtype=torch.int32, device=DEV).view(1, 4))
    assert torch.equal(got, M.mkv_paged_decode(small, q, lens))
    # and written there
    k = rnd((1, h, d), F16, 4)
    slot = torch.tensor([5], dtype=torch.int32, device=DEV)
    M.mkv_paged_append(c, k, k, slot)
    assert torch.equal(pools[0][39999, 0, 5], k[0, 0]) and c.check() == M.MKV_OK


# ---- append -------------------------------------------------------------------------------------

@pytest.mark.parametrize("dtype,it", [(F16, F16), (BF16, BF16), (E4M3, F16), (E4M3, BF16)])
@pytest.mark.parametrize("dim,rot,interleaved", [(64, 64, False), (128, 128, True), (128, 32, False), (256, 8, True), (128, 0, False)])
def test_append(M, dtype, it, dim, rot, interleaved):
    h, hq, page = 3, 6, 48
    cache = Cache(M, dtype, [100, 7, 0, 55], h, dim, page, seed=1, room=60)
    n = 70
    g = torch.Generator().manual_seed(4)
    seq = torch.tensor([i % 3 for i in range(n)], dtype=torch.int32)
    slot = torch.tensor([(100, 7, 0)[i % 3] + i // 3 for i in range(n)], dtype=torch.int32)
    slot[10] = -1                                # padding
    pos = torch.randint(0, 100000, (n,), generator=g, dtype=torch.int32)
    fused = rnd((n, hq + 2 * h, dim), it, 5, 3.0)     # queries, keys, values of one projection
    if dtype == E4M3:
        fused[3, hq + 1, 2] = 5000.0             # saturates
    q, k, v = fused[:, :hq], fused[:, hq:hq + h], fused[:, hq + h:]
    slots = 170
    acc, meta = torch.ones((4, h, slots), device=DEV), torch.full((4, h, slots), -5, dtype=torch.int32, device=DEV)
    before = [x.clone() for x in cache.pools]
    plan = M.mkv_rope_plan(dim, rot_dim=rot, interleaved=interleaved) if rot else None
    q_out = M.mkv_paged_append(cache.c, k, v, slot.to(DEV), seq=seq.to(DEV), plan=plan, pos=pos.to(DEV), q=q,
                               acc=acc, pos_meta=meta)
    assert cache.c.check() == M.MKV_OK
    freq, _ = P.rope_frequencies(rot, 10000.0)
    turn = lambda x: P.rope(f64(x), pos.numpy(), freq, interleaved=interleaved) if rot else f64(x)
    if rot:
        rope_close(f64(q_out), turn(q), f64(q), rot, interleaved, 1.0, it)
    else:
        assert torch.equal(q_out, q)
    wk, wv = turn(k), f64(v)
    touched = [torch.zeros(x.shape[:3], dtype=torch.bool) for x in cache.pools]
    wa, wm = torch.ones((4, h, slots)), torch.full((4, h, slots), -5, dtype=torch.int32)
    for i in range(n):
        s, t = int(seq[i]), int(slot[i])
        if t < 0:
            continue
        page_i = int(cache.np_table[s, t // page])
        wa[s, :, t] = 0.0
        wm[s, :, t] = pos[i]
        for x, (pool, want, src) in enumerate(zip(cache.pools, (wk, wv), (k, v))):
            touched[x][page_i, :, t % page] = True
            got = f64(pool[page_i, :, t % page])
            if dtype != E4M3:
                if x == 0 and rot:
                    rope_close(got, want[i], f64(src[i]), rot, interleaved, 1.0, dtype)
                else:
                    assert (got == want[i]).all()
            else:
                sc = cache.scales[x].numpy().astype(np.float64)[:, None]
                y = np.clip(want[i] / sc, -448, 448)
                err = 12 * U * 2 * np.abs(f64(src[i])).max() / sc
                assert (np.abs(got - y) <= 2.0**-4 * np.abs(y) * (1 + 2.0**-4) + 2.0**-10 + err).all()
                assert np.abs(got).max() <= 448
    assert torch.equal(acc.cpu(), wa) and torch.equal(meta.cpu(), wm)
    for x, (pool, was) in enumerate(zip(cache.pools, before)):
        keep = ~touched[x].to(DEV)
        b8 = lambda z: z.view(torch.uint8)
        assert torch.equal(b8(pool)[keep], b8(was)[keep])


def test_append_outside_is_reported(M):
    cache = Cache(M, F16, [30, 30], 2, 64, 16, seed=1, room=2)
    before = [x.clone() for x in cache.pools]
    k = rnd((4, 2, 64), F16, 1)
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device=DEV)
    same = lambda: all(torch.equal(a.view(torch.int16), b.view(torch.int16)) for a, b in zip(cache.pools, before))
    for seq, slot in ((i32(2, -1, 9, 2**31 - 1), i32(0, 0, 0, 0)), (i32(0, 0, 0, 0), i32(32, 1000, 2**31 - 1, 48))):
        M.mkv_paged_append(cache.c, k, k, slot, seq=seq)
        assert cache.c.check() == M.MKV_ERR_DEVICE_CHECK and same()
    acc = torch.ones((2, 2, 20), device=DEV)      # shorter than the slot
    M.mkv_paged_append(cache.c, k, k, i32(20, 25, 31, 20), seq=i32(0, 0, 0, 1), acc=acc)
    assert cache.c.check() == M.MKV_ERR_DEVICE_CHECK and same() and (acc == 1).all()
    M.mkv_paged_append(cache.c, k, k, i32(-1, -1, -2, -2**31), seq=i32(0, 50, -1, 1))
    assert cache.c.check() == M.MKV_OK and same()     # padding is not an error
    with pytest.raises(M.MkvError):
        M.mkv_paged_append(cache.c, k, k, i32(1, 2, 3, 4))    # four tokens, two sequences, no seq


# ---- evict --------------------------------------------------------------------------------------

def evict_case(M, lens, heads, dim, page, budget, sink, recent, dtype=F16, seed=0, in_place=False,
               weights=None, max_len=0, pos=None, spare=3):
    b = len(lens)
    cache = Cache(M, dtype, lens, heads, dim, page, seed=seed, spare=spare)
    slots = max(max(lens) + 5, max_len)
    if max_len:                                  # a table with room for the bound
        room = torch.full((b, -(-max_len // page)), -1, dtype=torch.int32, device=DEV)
        room[:, : cache.table.shape[1]] = cache.table
        cache.c = M.MkvPaged(*cache.pools, room, *cache.dev_scales)
    g = torch.Generator().manual_seed(seed + 50)
    acc = torch.exp(3 * torch.randn((b, heads, slots), generator=g)) if weights is None else weights(b, heads, slots, g)
    if pos is None:
        pos = torch.rand((b, heads, slots), generator=g)
        for i, n in enumerate(lens):
            pos[i, :, n:] = 2.0
        pos = pos.argsort(-1).argsort(-1)
    pos = pos.to(torch.int32)
    nxt = torch.tensor(lens, dtype=torch.int32)
    before = [x.clone() for x in cache.pools]
    acc_d, pos_d, lens_d, nxt_d = (t.clone().to(DEV) for t in (acc, pos, torch.tensor(lens, dtype=torch.int32), nxt))
    kw = dict(sink=sink, recent=recent, max_len=max_len or max(max(lens), 1))
    if in_place:
        src = M.mkv_paged_evict(cache.c, acc_d, pos_d, lens_d, nxt_d, budget, **kw)
        acc_o, pos_o, lens_o = acc_d, pos_d, lens_d
    else:
        acc_o = torch.full((b, heads, budget + 2), -3.0, device=DEV)
        pos_o = torch.full((b, heads, budget + 2), -3, dtype=torch.int32, device=DEV)
        lens_o = torch.empty(b, dtype=torch.int32, device=DEV)
        src = M.mkv_paged_evict(cache.c, acc_d, pos_d, lens_d, nxt_d, budget, acc_out=acc_o, pos_out=pos_o,
                                lens_out=lens_o, **kw)
        assert torch.equal(acc_d.cpu().view(torch.int32), acc.view(torch.int32)) and torch.equal(pos_d.cpu(), pos)
        assert lens_d.tolist() == list(lens)
    assert cache.c.check() == M.MKV_OK
    assert lens_o.tolist() == [min(n, budget) for n in lens]
    src_c, acc_c, pos_c = src.cpu().numpy(), acc_o.cpu().numpy(), pos_o.cpu().numpy()
    idx = [torch.arange(x.shape[0] * x.shape[1] * x.shape[2]).view(x.shape[:3]) for x in before[:1]][0].numpy()
    want_row = idx.copy()                        # which old row every pool row must hold now
    for i, n in enumerate(lens):
        for h in range(heads):
            w = P.evict(acc[i, h, :n].numpy(), pos[i, h, :n].numpy(), int(nxt[i]), budget, sink, recent)
            assert (src_c[i, h, : len(w)] == w).all(), (i, h, n)
            assert (src_c[i, h, len(w):] == -1).all()
            assert np.array_equal(acc_c[i, h, : len(w)], acc[i, h].numpy()[w], equal_nan=True)
            assert (pos_c[i, h, : len(w)] == pos[i, h].numpy()[w]).all()
            rest = (acc[i, h].numpy(), pos[i, h].numpy()) if in_place else (np.float32(-3), -3)
            tail = [r[len(w):] if in_place else r for r in rest]
            assert np.array_equal(acc_c[i, h, len(w):], np.broadcast_to(tail[0], acc_c[i, h, len(w):].shape), equal_nan=True)
            assert (pos_c[i, h, len(w):] == tail[1]).all()
            for t, s in enumerate(w):
                if s != t:
                    want_row[cache.np_table[i, t // page], h, t % page] = idx[cache.np_table[i, s // page], h, s % page]
    rows = torch.from_numpy(want_row.reshape(-1)).to(DEV)
    for pool, was in zip(cache.pools, before):
        flat = lambda z: z.view(torch.uint8).reshape(rows.numel(), -1)
        assert torch.equal(flat(pool), flat(was)[rows])
    return cache


@pytest.mark.parametrize("dtype,dim", [(F16, 128), (BF16, 256), (E4M3, 64)])
@pytest.mark.parametrize("in_place", [False, True])
def test_evict(M, dtype, dim, in_place):
    for page, budget, sink, recent in ((16, 100, 4, 20), (48, 1, 0, 0), (64, 299, 0, 0), (32, 50, 20, 30), (16, 300, 1, 1)):
        evict_case(M, [300, 0, 1, 101, 100, 299, 33], 2, dim, page, budget, sink, recent, dtype, in_place=in_place,
                   seed=budget)


@pytest.mark.parametrize("name", ["ties", "zeros", "odd", "same", "close"])
@pytest.mark.parametrize("n", [90, 20000])
def test_evict_ties_and_odd_weights(M, name, n):
    def weights(b, h, s, g):
        r = torch.rand((b, h, s), generator=g)
        if name == "ties":
            return (r * 3).floor() + 1
        if name == "zeros":
            return torch.where(r < 0.9, torch.zeros(()), r)
        if name == "same":
            return torch.full((b, h, s), 0.25)
        if name == "close":                      # keys that differ in their last bits alone
            return (torch.full((b, h, s), 1.0).view(torch.int32) + (r * 5).int()).view(torch.float32)
        x = torch.tensor([float("nan"), -float("nan"), float("inf"), -float("inf"), -0.0, 0.0, -1.0, 1e-45, 1.0, 3.4e38])
        return x[(r * 10).long().clamp(max=9)]
    evict_case(M, [n, n // 2 + 1], 1, 64, 128, n // 3, 2, n // 16, weights=weights, seed=n, in_place=name == "odd")


@pytest.mark.parametrize("few", [1, 2, 4, 5])
def test_evict_a_few(M, few):
    """As many tokens over the budget as are found one by one, and one more; ties; one to eight CTAs;
    the tokens that leave below, at and behind the budget's end."""
    ties = lambda b, h, s, g: (torch.rand((b, h, s), generator=g) * 50).floor()
    same = lambda b, h, s, g: torch.full((b, h, s), 2.0)
    first = lambda b, h, s, g: torch.arange(s, dtype=torch.float32).expand(b, h, s).contiguous()
    last = lambda b, h, s, g: -first(b, h, s, g) + s + 1
    for w in (None, ties, same, first, last):
        evict_case(M, [96 + few, 97, 96, 3], 2, 64, 16, 96, 4, 10, weights=w, seed=few)
        evict_case(M, [few + 1, few + 1], 2, 64, 16, 1, 0, 0, weights=w, seed=few, in_place=True)
        evict_case(M, [4096 + few] * 2, 2, 64, 256, 4096, 4, 64, E4M3, weights=w, seed=few)
        evict_case(M, [16384 + few], 2, 64, 256, 16384, 0, 16384 - 2, E4M3, weights=w, seed=few)
        evict_case(M, [70000 + few], 1, 64, 256, 70000, 4, 64, E4M3, weights=w, seed=few)


def test_evict_sizes_of_cluster(M):
    """1, 2, 4 and 8 CTAs a stream; slices of 8 and 16 keys a thread, and longer ones."""
    evict_case(M, [8191, 4097], 1, 64, 256, 4096, 4, 100, E4M3, seed=1)
    evict_case(M, [8192] * 3, 8, 64, 256, 1000, 0, 999, E4M3, seed=2)
    evict_case(M, [16385] * 3 + [5], 8, 64, 256, 16384, 0, 0, E4M3, seed=3)
    evict_case(M, [16384] * 2, 8, 64, 256, 5000, 4, 100, E4M3, seed=10)
    evict_case(M, [40000, 33000, 20], 4, 64, 256, 30001, 4, 100, E4M3, seed=11)
    evict_case(M, [100000, 131072, 98765], 1, 64, 256, 7000, 0, 99, E4M3, seed=8)
    evict_case(M, [400001], 1, 64, 256, 3001, 4, 700, E4M3, seed=4)          # 8 slices of 50176
    evict_case(M, [400001], 1, 64, 256, 300001, 4, 700, E4M3, seed=4)        # most are kept
    evict_case(M, [50000, 45000] + [10] * 158, 1, 64, 256, 9000, 4, 700, E4M3, seed=5, spare=0)   # one CTA a stream
    # the long form by the bound alone, and many slots
    evict_case(M, [5000, 45, 9001] + [10] * 77, 1, 64, 256, 2000, 4, 700, E4M3, seed=6, spare=0, max_len=300000)
    evict_case(M, [2210000], 1, 64, 256, 5000, 4, 700, E4M3, seed=7)


@pytest.mark.parametrize("name", ["zeros", "same", "sampled"])
def test_evict_long_streams_that_mislead_the_sample(M, name):
    """Ties over a whole long stream; and large weights at just the slots that a bound is taken
    from (every 49th of 8 slices of 50176 slots), so that too few others reach it."""
    def weights(b, h, s, g):
        r = torch.rand((b, h, s), generator=g)
        if name == "zeros":
            return torch.where(r < 0.999, torch.zeros(()), r)
        if name == "same":
            return torch.full((b, h, s), 0.25)
        return torch.where(torch.arange(s) % 49 == 0, 100 + r, r)
    evict_case(M, [8 * 50176], 1, 64, 256, 20000, 4, 300, E4M3, weights=weights, seed=9)


def test_evict_protected_beyond_budget(M):
    """Positions that occur twice protect more tokens than the budget has: the lower slots stay."""
    pos = torch.zeros((1, 2, 205), dtype=torch.int32)
    pos[:, 1] = torch.arange(205) % 7
    evict_case(M, [200], 2, 64, 16, 32, 4, 10, pos=pos, seed=3)


def test_evict_budget_above_the_bound(M):
    """Nothing leaves; src says so for every slot, and the scratch does not grow with the budget."""
    evict_case(M, [200, 0, 63], 2, 64, 16, 1000, 4, 10, seed=3, in_place=True)
    cache = Cache(M, F16, [30], 1, 64, 16, seed=3)
    acc, pos = torch.rand((1, 1, 32), device=DEV), torch.arange(32, dtype=torch.int32, device=DEV).view(1, 1, 32)
    n = torch.tensor([30], dtype=torch.int32, device=DEV)
    ws = torch.empty(512, dtype=torch.uint8, device=DEV)
    src = M.mkv_paged_evict(cache.c, acc, pos, n, n, 5_000_000, workspace=ws)
    assert src[0, 0, :30].tolist() == list(range(30)) and (src[0, 0, 30:] == -1).all() and n.item() == 30


def test_evict_bad_pages_are_skipped(M):
    cache = Cache(M, F16, [64], 1, 64, 16, seed=2)
    acc = torch.arange(64, device=DEV, dtype=torch.float32).view(1, 1, 64)      # the last 32 are kept
    pos = torch.arange(64, device=DEV, dtype=torch.int32).view(1, 1, 64)
    n = torch.tensor([64], dtype=torch.int32, device=DEV)
    before = [x.clone() for x in cache.pools]
    cache.table[0, 3] = 2**31 - 1
    lens_out = torch.empty(1, dtype=torch.int32, device=DEV)
    src = M.mkv_paged_evict(cache.c, acc, pos, n, n, 32, lens_out=lens_out)
    assert src[0, 0].tolist() == list(range(32, 64)) and lens_out.item() == 32
    assert cache.c.check() == M.MKV_ERR_DEVICE_CHECK
    for pool, was in zip(cache.pools, before):
        t = cache.np_table[0]
        assert torch.equal(pool[int(t[0])], was[int(t[2])])                      # 32..47 arrived
        assert torch.equal(pool[int(t[1])], was[int(t[1])])                      # 48..63 have no page
    # a length beyond the bound counts as the bound
    cache = Cache(M, F16, [64], 1, 64, 16, seed=2)
    src = M.mkv_paged_evict(cache.c, acc, pos, torch.tensor([99], dtype=torch.int32, device=DEV), n, 32,
                            lens_out=lens_out, acc_out=torch.empty_like(acc), pos_out=torch.empty_like(pos))
    assert lens_out.item() == 32 and cache.c.check() == M.MKV_ERR_DEVICE_CHECK


# ---- together -----------------------------------------------------------------------------------

@pytest.mark.parametrize("dtype,it", [(F16, F16), (E4M3, BF16)])
def test_serving_loop(M, dtype, it):
    """A ragged prefill appended, then steps of append, decode with weights and eviction at a
    budget; every step against the oracle on the cache as it stands."""
    lens, h, hq, dim, page, budget = [130, 1, 64], 2, 8, 128, 16, 96
    cap = 160
    cache = Cache(M, dtype, [0, 0, 0], h, dim, page, seed=3, room=cap)
    plan = M.mkv_rope_plan(dim, base=500000.0, scaling="banded", factor=8.0, original=8192)
    acc, pos = torch.zeros((3, h, cap), device=DEV), torch.zeros((3, h, cap), dtype=torch.int32, device=DEV)
    n = sum(lens)
    seq = torch.cat([torch.full((m,), i) for i, m in enumerate(lens)]).to(torch.int32).to(DEV)
    slot = torch.cat([torch.arange(m) for m in lens]).to(torch.int32).to(DEV)
    M.mkv_paged_append(cache.c, rnd((n, h, dim), it, 1), rnd((n, h, dim), it, 2), slot, seq=seq, plan=plan,
                       acc=acc, pos_meta=pos)
    length = torch.tensor(lens, dtype=torch.int32, device=DEV)
    nxt = length.clone()
    for step in range(6):
        k, v, q = (rnd((3, x, dim), it, 10 * step + y) for y, x in enumerate((h, h, hq)))
        qr = M.mkv_paged_append(cache.c, k, v, length, plan=plan, pos=nxt, q=q, acc=acc, pos_meta=pos)
        length += 1
        nxt += 1
        acc0 = acc.clone()
        out = M.mkv_paged_decode(cache.c, qr, length, acc=acc, max_len=cap)
        cache.lens_list = length.tolist()
        decode_check(cache, qr, out, None, acc, acc0)
        a, p, m = acc.cpu().numpy().copy(), pos.cpu().numpy().copy(), length.tolist()
        src = M.mkv_paged_evict(cache.c, acc, pos, length, nxt, budget, sink=4, recent=16)
        for i in range(3):
            assert int(length[i]) == min(m[i], budget)
            for j in range(h):
                w = P.evict(a[i, j, : m[i]], p[i, j, : m[i]], int(nxt[i]), budget, 4, 16)
                assert (src[i, j, : len(w)].cpu().numpy() == w).all()
                held = pos[i, j, : len(w)].cpu().numpy()
                assert (held == p[i, j][w]).all() and len(set(held.tolist())) == len(w)
                assert set(range(max(0, int(nxt[i]) - 16), int(nxt[i]))) <= set(held.tolist())
    assert cache.c.check() == M.MKV_OK


def test_rope_feeds_the_compressed_cache(M):
    """Keys rotated into head-major order, compressed without loss of channels or tokens, and
    attended; the same keys in pages give the same attention."""
    b, t, h, hq, d = 1, 500, 2, 8, 128
    plan = M.mkv_rope_plan(d, base=500000.0)
    x, v = rnd((b, t, h, d), F16, 1), rnd((b, h, t, d), F16, 2)
    keys = torch.empty((b, h, t, d), dtype=F16, device=DEV)
    M.mkv_rope(plan, x, out=keys.transpose(1, 2))
    q = M.mkv_rope(plan, rnd((b, 1, hq, d), F16, 3), first_pos=t)[:, 0].contiguous()
    cfg = M.make_config(b, h, hq, t, 64, 128, 1.0, t)
    with M.Mkv(cfg) as m:
        m.compress(keys, v)
        dense = m.decode(q)
        torch.cuda.synchronize()
    page = 16
    per = -(-t // page)
    pools = [torch.zeros((per, h, page, d), dtype=F16, device=DEV) for _ in range(2)]
    c = M.MkvPaged(*pools, torch.arange(per, dtype=torch.int32, device=DEV).view(1, per))
    M.mkv_paged_append(c, keys[0].transpose(0, 1), v[0].transpose(0, 1),
                       torch.arange(t, dtype=torch.int32, device=DEV), seq=torch.zeros(t, dtype=torch.int32, device=DEV))
    paged = M.mkv_paged_decode(c, q, torch.tensor([t], dtype=torch.int32, device=DEV), out_dtype=F32)
    # the compressed cache holds rotated fp16 rows: half a step of fp16 on every element of keys
    # and values in another basis.  A score moves by at most 2^-11 scale |q| |k| (d), the output by
    # (2 d + 2^-11) times the largest value row's length.
    big = lambda z: float(z.float().norm(dim=-1).max())
    shift = 2.0**-11 * d ** -0.5 * big(q) * big(keys)
    assert (dense - paged).abs().max().item() <= (2 * shift + 2.0**-11) * big(v)


def test_streams_and_graphs(M):
    """On a side stream, captured and replayed with new inputs, two graphs with a workspace each."""
    cache = Cache(M, F16, [2000, 700], 2, 128, 64, seed=3, room=10)
    caches, graphs, outs, qs = [cache, Cache(M, F16, [1500, 3], 2, 128, 64, seed=4, room=10)], [], [], []
    plan = M.mkv_rope_plan(128)
    cap = 2010
    accs = [torch.zeros((2, 2, cap), device=DEV) for _ in caches]
    for x, acc in zip(caches, accs):
        q = torch.zeros((2, 8, 128), dtype=F16, device=DEV)
        pos = torch.arange(cap, dtype=torch.int32, device=DEV).expand(2, 2, cap).contiguous()
        kw = dict(acc=acc, max_len=min(x.c.capacity, cap))
        st = torch.cuda.Stream()
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):              # a first pass outside the capture
            qr = M.mkv_rope(plan, q.view(2, 1, 8, 128), first_pos=9)
            M.mkv_paged_decode(x.c, qr[:, 0], x.lens, **kw)
        torch.cuda.current_stream().wait_stream(st)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            qr = M.mkv_rope(plan, q.view(2, 1, 8, 128), first_pos=9)
            out = M.mkv_paged_decode(x.c, qr[:, 0], x.lens, **kw)
            lens_out = torch.empty(2, dtype=torch.int32, device=DEV)
            src = M.mkv_paged_evict(x.c, acc, pos, x.lens, x.lens, 600, recent=3, lens_out=lens_out,
                                    acc_out=torch.empty_like(acc), pos_out=torch.empty_like(pos))
        graphs.append(g)
        outs.append((out, src, lens_out))
        qs.append(q)
    want = []
    for i in range(2):
        qs[i].copy_(rnd((2, 8, 128), F16, 60 + i))
        accs[i].zero_()
        pools = [p.clone() for p in caches[i].pools]
        qr = M.mkv_rope(plan, qs[i].view(2, 1, 8, 128), first_pos=9)
        bound = min(caches[i].c.capacity, cap)    # the captured call's: the order of sums goes by it
        want.append((M.mkv_paged_decode(caches[i].c, qr[:, 0], caches[i].lens, max_len=bound), pools))
    torch.cuda.synchronize()
    sts = [torch.cuda.Stream(), torch.cuda.Stream()]
    for g, st in zip(graphs, sts):               # at the same time
        with torch.cuda.stream(st):
            g.replay()
    torch.cuda.synchronize()
    for i in range(2):
        assert torch.equal(outs[i][0], want[i][0])
        assert outs[i][2].tolist() == [min(n, 600) for n in caches[i].lens_list]
        total = accs[i].sum(-1).cpu().numpy()
        for j, n in enumerate(caches[i].lens_list):
            assert np.allclose(total[j], 4.0 if n else 0.0, rtol=2.0**-10)
    # an explicit stream, as an object and as an address
    st = torch.cuda.Stream()
    c3 = Cache(M, F16, [40, 1100], 2, 128, 64, seed=5)
    q = rnd((2, 8, 128), F16, 70)
    ref = M.mkv_paged_decode(c3.c, q, c3.lens)
    torch.cuda.synchronize()
    for s in (st, st.cuda_stream):
        got = M.mkv_paged_decode(c3.c, q, c3.lens, stream=s)
        st.synchronize()
        assert torch.equal(got, ref)


@pytest.mark.parametrize("bound", [600, 9000])
def test_graph_replays_with_other_lengths(M, bound):
    """A captured step (append, decode with weights, eviction) replayed after lengths, slots and
    queries changed gives what the eager calls give; in clusters and split over the streams."""
    lens = [500, 129, 128]
    caches = [Cache(M, F16, lens, 6, 64, 64, seed=5, room=bound - 500) for _ in range(2)]
    for a, b in zip(caches[0].pools, caches[1].pools):
        b.copy_(a)
    plan = M.mkv_rope_plan(64)
    state = []
    for _ in caches:
        state.append(dict(k=torch.zeros((3, 6, 64), dtype=F16, device=DEV), q=torch.zeros((3, 12, 64), dtype=F16, device=DEV),
                          slot=torch.zeros(3, dtype=torch.int32, device=DEV), lens=torch.zeros(3, dtype=torch.int32, device=DEV),
                          acc=torch.zeros((3, 6, bound), device=DEV), pos=torch.zeros((3, 6, bound), dtype=torch.int32, device=DEV),
                          lens_out=torch.zeros(3, dtype=torch.int32, device=DEV),
                          acc_out=torch.zeros((3, 6, 128), device=DEV), pos_out=torch.zeros((3, 6, 128), dtype=torch.int32, device=DEV),
                          src=torch.zeros((3, 6, 128), dtype=torch.int32, device=DEV), out=torch.zeros((3, 12, 64), dtype=F16, device=DEV)))

    def step(c, s):
        q = M.mkv_paged_append(c.c, s["k"], s["k"], s["slot"], plan=plan, q=s["q"], acc=s["acc"], pos_meta=s["pos"])
        M.mkv_paged_decode(c.c, q, s["lens"], out=s["out"], acc=s["acc"], max_len=bound)
        M.mkv_paged_evict(c.c, s["acc"], s["pos"], s["lens"], s["lens"], 128, sink=1, recent=8, acc_out=s["acc_out"],
                          pos_out=s["pos_out"], lens_out=s["lens_out"], src=s["src"], max_len=bound)

    s0 = state[0]
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        step(caches[0], s0)                      # nothing cached yet: lengths 0, token in slot 0
    torch.cuda.current_stream().wait_stream(st)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(caches[0], s0)
    for turn, now in enumerate(([500, 20, 3], [0, 1, 0], [137, 20, 2], [500, 129, 128])):
        for c, s in zip(caches, state):
            for a, b in zip(c.pools, Cache(M, F16, [500, 129, 128], 6, 64, 64, seed=5, room=bound - 500).pools):
                c.pools[0 if a is c.pools[0] else 1].copy_(torch.nan_to_num(b))
            s["k"].copy_(rnd((3, 6, 64), F16, 10 + turn))
            s["q"].copy_(rnd((3, 12, 64), F16, 20 + turn))
            s["lens"].copy_(torch.tensor(now, dtype=torch.int32))
            s["slot"].copy_(torch.tensor([max(0, n - 1) for n in now], dtype=torch.int32))
            s["acc"].copy_(rnd(s["acc"].shape, F32, 30 + turn).abs())
            s["pos"].copy_(torch.arange(bound, dtype=torch.int32))
            for k in ("acc_out", "pos_out"):
                s[k].zero_()
        g.replay()
        step(caches[1], state[1])
        torch.cuda.synchronize()
        for k in state[0]:
            assert torch.equal(state[0][k], state[1][k]), (turn, k)
        for a, b in zip(caches[0].pools, caches[1].pools):
            assert torch.equal(a, b), turn
        assert state[0]["lens_out"].tolist() == [min(n, 128) for n in now]
    assert all(c.c.check() == M.MKV_OK for c in caches)


def test_broadcast_positions_and_empty_calls(M):
    plan = M.mkv_rope_plan(64)
    x = rnd((3, 5, 2, 64), BF16, 1)
    row = torch.arange(5, dtype=torch.int32, device=DEV).view(1, 5) * 7
    assert torch.equal(M.mkv_rope(plan, x, row.expand(3, 5)), M.mkv_rope(plan, x, row.repeat(3, 1)))
    for shape in ((0, 5, 2, 64), (3, 0, 2, 64), (3, 5, 0, 64)):
        assert M.mkv_rope(plan, torch.empty(shape, dtype=F16, device=DEV)).shape == shape
    cache = Cache(M, F16, [0, 0], 2, 64, 16, seed=1)
    none = torch.empty((0, 2, 64), dtype=F16, device=DEV)
    M.mkv_paged_append(cache.c, none, none, torch.empty(0, dtype=torch.int32, device=DEV))
    # every sequence empty, in both forms of the kernel
    for cap in (1, 100):
        c = M.MkvPaged(*cache.pools, torch.full((2, cap), -1, dtype=torch.int32, device=DEV))
        q = rnd((2, 4, 64), F16, 2)
        lse = torch.zeros((2, 4), device=DEV)
        out = M.mkv_paged_decode(c, q, torch.zeros(2, dtype=torch.int32, device=DEV), lse=lse)
        assert (out == 0).all() and (lse == -math.inf).all() and c.check() == M.MKV_OK


def test_8_bit_cache_without_scales(M):
    """NULL scales stand for 1: the same bits as scales of 1, written and read."""
    n, one = 40, torch.ones(2, device=DEV)
    pools = [torch.zeros((4, 2, 16, 128), device=DEV).to(E4M3) for _ in range(4)]
    table = torch.arange(4, dtype=torch.int32, device=DEV).view(1, 4)
    a = M.MkvPaged(pools[0], pools[1], table)
    b = M.MkvPaged(pools[2], pools[3], table, k_scale=one, v_scale=one)
    k, v, q = rnd((n, 2, 128), F16, 1), rnd((n, 2, 128), F16, 2), rnd((1, 6, 128), F16, 3)
    i = torch.arange(n, dtype=torch.int32, device=DEV)
    outs = []
    for c in (a, b):
        M.mkv_paged_append(c, k, v, i, seq=torch.zeros_like(i))
        outs.append(M.mkv_paged_decode(c, q, torch.tensor([n], dtype=torch.int32, device=DEV)))
    for x, y in ((pools[0], pools[2]), (pools[1], pools[3])):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8)) and x.view(torch.uint8).any()
    assert torch.equal(*outs)
    assert torch.equal(pools[0].view(torch.uint8)[0, :, :16].transpose(0, 1),
                       k[:16].to(E4M3).view(torch.uint8))


def test_append_queries_in_place(M):
    cache = Cache(M, F16, [0] * 3, 2, 64, 16, seed=1, room=4)
    plan = M.mkv_rope_plan(64, interleaved=True)
    fused = rnd((3, 8, 64), F16, 4)
    i = torch.arange(3, dtype=torch.int32, device=DEV)
    k, v = fused[:, 4:6], fused[:, 6:]
    want = M.mkv_rope(plan, fused[:, :4].unsqueeze(1), i.view(3, 1))[:, 0]
    rest = fused[:, 4:].clone()
    q = fused[:, :4]
    assert M.mkv_paged_append(cache.c, k, v, torch.zeros_like(i), plan=plan, pos=i, q=q, q_out=q) is q
    assert torch.equal(q, want) and torch.equal(fused[:, 4:], rest)


def test_weights_with_default_bound(M):
    """acc shorter than the page table: it bounds the lengths; a longer sequence is reported."""
    cache = Cache(M, F16, [100, 37], 2, 64, 16, seed=6, room=500)
    q = rnd((2, 4, 64), F16, 1)
    acc = torch.zeros((2, 2, 100), device=DEV)
    out = M.mkv_paged_decode(cache.c, q, cache.lens, acc=acc)
    decode_check(cache, q, out, None, acc, torch.zeros_like(acc))
    cache2 = Cache(M, F16, [100, 37], 2, 64, 16, seed=6, room=500)
    M.mkv_paged_decode(cache2.c, q, cache2.lens, acc=torch.zeros((2, 2, 99), device=DEV))
    assert cache2.c.check() == M.MKV_ERR_DEVICE_CHECK


def test_calls_on_several_streams_at_once(M):
    """The same cache read by calls that overlap, each with its own workspace and outputs."""
    cache = Cache(M, BF16, [3000, 1, 900], 2, 128, 64, seed=12)
    qs = [rnd((3, 8, 128), BF16, 40 + i) for i in range(4)]
    want = [M.mkv_paged_decode(cache.c, q, cache.lens) for q in qs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in qs]
    for _ in range(5):
        got = [M.mkv_paged_decode(cache.c, q, cache.lens, stream=st) for q, st in zip(qs, streams)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_binding_checks(M):
    cache = Cache(M, F16, [40], 2, 64, 16, seed=5)
    q = rnd((1, 4, 64), F16, 1)
    with pytest.raises(TypeError):
        M.mkv_paged_decode(cache.c, q.float(), cache.lens)
    with pytest.raises(TypeError):
        M.mkv_paged_decode(cache.c, q, cache.lens.long())
    with pytest.raises(ValueError):
        M.mkv_paged_decode(cache.c, q, cache.lens.cpu())
    with pytest.raises(ValueError):
        M.mkv_paged_decode(cache.c, q[:, :, :32], cache.lens)
    with pytest.raises(M.MkvError, match="type"):
        M.mkv_paged_decode(cache.c, q.to(BF16), cache.lens)
    with pytest.raises(M.MkvError, match="n_q_heads"):
        M.mkv_paged_decode(cache.c, q[:, :3].contiguous(), cache.lens)
    with pytest.raises(TypeError):
        M.MkvPaged(cache.pools[0], cache.pools[1].float(), cache.table)
    with pytest.raises(ValueError):
        M.mkv_paged_append(cache.c, q[:, :2], q[:, :2], cache.lens, q_out=q)
    with pytest.raises(ValueError):
        M.mkv_paged_evict(cache.c, torch.zeros((1, 2, 48), device=DEV), torch.zeros((1, 2, 48), dtype=torch.int32, device=DEV),
                          cache.lens, cache.lens, 4, acc_out=torch.zeros((1, 2, 48), device=DEV))
