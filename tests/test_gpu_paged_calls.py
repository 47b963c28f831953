"""Calls of the paged cache that its documentation allows, beside those of test_gpu_paged.py:
views of one token or sequence, status words, handles made while a stream is busy, workspaces of
a stated size, sequences with a common prefix, captured first calls."""
import numpy as np
import pytest
import torch

from oracle import paged as P

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
F16, BF16, F32, E4M3 = torch.float16, torch.bfloat16, torch.float32, torch.float8_e4m3fn


@pytest.fixture(scope="module")
def M():
    from two_compressed_kv_gb300 import mkv
    return mkv


def f64(t):
    return t.detach().to(torch.float32).cpu().numpy().astype(np.float64)


def i32(*a):
    return torch.tensor(a, dtype=torch.int32, device=DEV)


def rnd(shape, dtype, seed, size=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * size).to(dtype).to(DEV)


def pages(n, heads, page, dim, dtype=F16, seed=0):
    return [rnd((n, heads, page, dim), F16, seed + i).to(dtype) for i in range(2)]


def test_strides_of_extents_of_1(M):
    """The unused stride of a single token, sequence or head may be anything."""
    pools, table = pages(4, 2, 16, 64), i32(2, 0, 3, 1).view(1, 4)
    c = M.MkvPaged(*pools, table)
    odd = lambda t, at, by: t.as_strided(t.shape, [by if i == at else s for i, s in enumerate(t.stride())])
    q, n = rnd((1, 8, 64), F16, 5), i32(50)
    assert torch.equal(M.mkv_paged_decode(c, odd(q, 0, 3), n), M.mkv_paged_decode(c, q, n))
    plan, outs = M.mkv_rope_plan(64), []
    k, v = rnd((1, 2, 64), F16, 6), rnd((1, 2, 64), F16, 7)
    for f in (lambda t: t, lambda t: odd(t, 0, 5)):
        for p in pools:
            p[1, :, 2:] = 0
        qr = M.mkv_paged_append(c, f(k), f(v), i32(50), plan=plan, q=f(q))
        outs.append([qr.clone()] + [p.clone() for p in pools])
    for a, b in zip(*outs):
        assert torch.equal(a, b)
    # one KV head and one query head
    pools = pages(2, 1, 16, 64, seed=9)
    c = M.MkvPaged(*pools, i32(0, 1).view(2, 1))
    q, n = rnd((2, 1, 64), F16, 5), i32(3, 16)
    assert torch.equal(M.mkv_paged_decode(c, odd(q, 1, 7), n), M.mkv_paged_decode(c, q, n))
    was = [p.clone() for p in pools]
    M.mkv_paged_append(c, odd(q, 1, 7), odd(q, 1, 9), i32(5, 6))
    for p, w in zip(pools, was):
        w[0, 0, 5], w[1, 0, 6] = q[0, 0], q[1, 0]
        assert torch.equal(p, w)
    assert c.check() == M.MKV_OK


def test_check_names_every_bit(M):
    """A wait that gave up (outputs undefined) is not hidden behind a page outside the cache."""
    c = M.MkvPaged(*pages(2, 1, 16, 64), i32(0, 1).view(1, 2))
    for bits, status, words in ((1, M.MKV_ERR_TIMEOUT, ["wait"]), (2, M.MKV_ERR_DEVICE_CHECK, ["page"]),
                                (3, M.MKV_ERR_TIMEOUT, ["wait", "page"])):
        c.status.fill_(bits)
        assert c.check() == status, bits
        assert all(w in M.mkv_last_error_string() for w in words)
        assert c.check() == M.MKV_OK


def test_status_word_is_ready_for_any_stream(M):
    """A handle made while its stream is busy: what a call on another stream reports stays."""
    pools, table = pages(2, 1, 16, 64), i32(0, 1).view(1, 2)
    k, slot = rnd((1, 1, 64), F16, 3), i32(1000)
    side = torch.cuda.Stream()
    first = M.MkvPaged(*pools, table)            # the kernel is loaded, which waits for the device
    M.mkv_paged_append(first, k, k, slot, stream=side)
    assert first.check() == M.MKV_ERR_DEVICE_CHECK
    torch.cuda._sleep(100_000_000)               # some 50 ms
    c = M.MkvPaged(*pools, table)
    M.mkv_paged_append(c, k, k, slot, stream=side)
    assert c.check() == M.MKV_ERR_DEVICE_CHECK and c.check() == M.MKV_OK


@pytest.mark.parametrize("batch,budget,max_len", [(2, 20, 0), (2, 20, 100), (3, 500, 60), (80, 100, 40000)])
def test_evict_workspace_of_the_stated_size(M, batch, budget, max_len):
    """Short and long forms, and a budget above the bound: the size given is enough and needed."""
    heads, page = 2, 256 if max_len > 1000 else 16
    cap = (max_len or 128) // page + 1
    pools = pages(2 * batch, heads, page, 64)
    table = torch.full((batch, cap), -1, dtype=torch.int32, device=DEV)
    table[:, :2] = torch.arange(2 * batch, dtype=torch.int32, device=DEV).view(batch, 2)
    c = M.MkvPaged(*pools, table)
    slots = max_len or c.capacity
    acc = torch.rand((batch, heads, slots), device=DEV)
    pos = torch.arange(slots, dtype=torch.int32, device=DEV).expand(batch, heads, slots).contiguous()
    lens = torch.full((batch,), min(2 * page, slots), dtype=torch.int32, device=DEV)
    size = M.mkv_paged_evict_workspace(c, budget, max_len=max_len)
    assert size > 0
    out = dict(acc_out=torch.empty_like(acc), pos_out=torch.empty_like(pos), lens_out=torch.empty_like(lens))
    want = M.mkv_paged_evict(c, acc, pos, lens, lens, budget, max_len=max_len, **out)
    ws = torch.empty(size, dtype=torch.uint8, device=DEV)
    assert torch.equal(want, M.mkv_paged_evict(c, acc, pos, lens, lens, budget, max_len=max_len, workspace=ws, **out))
    with pytest.raises(M.MkvError, match="workspace"):
        M.mkv_paged_evict(c, acc, pos, lens, lens, budget, max_len=max_len, workspace=ws[:-256], **out)
    with pytest.raises(M.MkvError, match="budget"):
        M.mkv_paged_evict_workspace(c, 0)
    assert c.check() == M.MKV_OK


@pytest.mark.parametrize("dtype", [F16, E4M3])
def test_common_prefix(M, dtype):
    """Three sequences over the same first pages: attention reads the shared pages; before
    eviction, which moves rows, all but one of the sequences get copies."""
    heads, page, dim, shared, budget = 2, 16, 64, 2, 40
    pools = pages(20, heads, page, dim, dtype, seed=3)
    lens = [70, 45, 33]
    table = i32(5, 9, 1, 2, 3, 5, 9, 4, -1, -1, 5, 9, 6, -1, -1).view(3, 5)
    c = M.MkvPaged(*pools, table)
    u8 = lambda p: p.view(torch.uint8) if dtype == E4M3 else p
    kept = lambda: [[f64(torch.cat(list(u8(p)[table[i, : -(-n // page)].long()].view(dtype)), 1)[:, :n])
                     for i, n in enumerate(lens)] for p in pools]
    K, V = kept()
    q, n = rnd((3, 4, dim), F16, 4), i32(*lens)
    out = f64(M.mkv_paged_decode(c, q, n, out_dtype=F32))
    for i in range(3):
        want, _, _, size = P.decode(f64(q[i]), K[i], V[i])
        assert (np.abs(out[i] - want) <= 2.0**-12 * size).all()
    # copies for sequences 1 and 2, then every head of every sequence keeps other tokens
    for i, new in ((1, (10, 11)), (2, (12, 13))):
        for j in range(shared):
            for p in pools:
                u8(p)[new[j]] = u8(p)[int(table[i, j])]
            table[i, j] = new[j]
    acc = torch.rand((3, heads, 80), generator=torch.Generator().manual_seed(8)).to(DEV)
    pos = torch.arange(80, dtype=torch.int32, device=DEV).expand(3, heads, 80).contiguous()
    a, p = acc.cpu().numpy().copy(), pos.cpu().numpy().copy()
    M.mkv_paged_evict(c, acc, pos, n, n.clone(), budget, sink=4, recent=8)
    assert c.check() == M.MKV_OK and n.tolist() == [min(m, budget) for m in lens]
    was, old, lens = (K, V), lens, n.tolist()
    for w, now in zip(was, kept()):
        for i in range(3):
            for h in range(heads):
                src = P.evict(a[i, h, : old[i]], p[i, h, : old[i]], old[i], budget, 4, 8)
                assert (now[i][h] == w[i][h][src]).all()


def test_captured_first_calls():
    """In a new process, the first call of every operator is one that a graph captures."""
    code = """
import torch
from two_compressed_kv_gb300 import mkv as M
dev = torch.device("cuda:0")
g = torch.Generator().manual_seed(1)
rnd = lambda *s: torch.randn(s, generator=g).half().to(dev)
i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device=dev)
pools = [rnd(8, 2, 16, 64) for _ in range(2)]
table = i32(*range(8)).view(2, 4)
c = M.MkvPaged(*pools, table)
plan = M.mkv_rope_plan(64)
k, q, slot, lens, nxt = rnd(2, 2, 64), rnd(2, 8, 64), i32(50, 30), i32(51, 31), i32(51, 31)
acc = torch.rand((2, 2, 64), generator=g).to(dev)
pos = torch.arange(64, dtype=torch.int32, device=dev).expand(2, 2, 64).contiguous()

def step(c, acc, pos, lens):
    r = M.mkv_rope(plan, q.view(2, 1, 8, 64), first_pos=7)
    a = M.mkv_paged_append(c, k, k, slot, plan=plan, q=q, acc=acc, pos_meta=pos)
    o = M.mkv_paged_decode(c, a, lens, acc=acc)
    s = M.mkv_paged_evict(c, acc, pos, lens, nxt, 20, sink=2, recent=5)
    return [r, a, o, s, acc, pos, lens]

other = [p.clone() for p in pools]
args = [t.clone() for t in (acc, pos, lens)]
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    got = step(c, acc, pos, lens)
graph.replay()
want = step(M.MkvPaged(*other, table), *args)
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(got + pools, want + other))
assert c.check() == M.MKV_OK
print("same")
"""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "same", r.stdout + r.stderr


def test_infinite_value_shows_in_its_channel_alone(M):
    """An infinity among a live token's values: that channel of its heads is not finite, all else is
    as it was; behind the sequence it changes nothing."""
    pools, table = pages(6, 2, 16, 64, seed=5), i32(4, 1, 0, 3, 2, 5).view(2, 3)
    c = M.MkvPaged(*pools, table)
    q, n = rnd((2, 8, 64), F16, 6), i32(40, 40)
    lse = [torch.empty((2, 8), device=DEV) for _ in range(2)]
    want = M.mkv_paged_decode(c, q, n, lse=lse[0])
    pools[1][5, :, 8:] = float("inf")            # slots 40 to 47 of sequence 1
    assert torch.equal(M.mkv_paged_decode(c, q, n, lse=lse[1]), want) and torch.equal(*lse)
    pools[1][3, 1, 2, 9] = float("-inf")         # slot 2 of sequence 1, head 1, channel 9
    got = M.mkv_paged_decode(c, q, n, lse=lse[1])
    assert torch.equal(*lse) and not torch.isfinite(got[1, 4:, 9]).any()
    got[1, 4:, 9] = want[1, 4:, 9]
    assert torch.equal(got, want)
