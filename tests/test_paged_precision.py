"""The precision of the paged attention's fp32 output: the kernel against the bound that
paged_precision derives, and, without a GPU, the bound against an emulation with and without
mistakes."""
import numpy as np
import pytest

import paged_precision as X


def to_bits(bits):
    return lambda x: X.round_to(x, bits)


CASES = [("plain", 4096, 128, 64), ("plain", 32768, 128, 600), ("long_run", 32768, 64, 4)]


@pytest.mark.parametrize("bits,parts", [(11, 2), (8, 3)])
@pytest.mark.parametrize("name,n,D,warps", CASES)
def test_emulation_holds_the_bound(name, n, D, warps, bits, parts):
    a = getattr(X, name)(n, D, 4, to_bits(bits))
    want = X.exact(*a)
    assert X.error(X.emulate(*a, bits, parts, warps=warps), want) <= X.BOUND
    assert X.error(X.emulate(*a, bits, parts, chains=2, warps=warps), want) <= X.BOUND_WIDE


@pytest.mark.parametrize("name,n,D,warps,bits,parts,kw", [
    (*CASES[0], 8, 2, {}), (*CASES[1], 8, 2, {}), (*CASES[0], 11, 1, {}), (*CASES[0], 8, 2, dict(chains=2)),
    (*CASES[2], 11, 2, dict(block_sums=False)), (*CASES[2], 8, 3, dict(block_sums=False))])
def test_planted_mistakes_exceed_it(name, n, D, warps, bits, parts, kw):
    a = getattr(X, name)(n, D, 4, to_bits(bits))
    assert X.error(X.emulate(*a, bits, parts, warps=warps, **kw), X.exact(*a)) > X.BOUND_WIDE


# ---- the kernel ---------------------------------------------------------------------------------

def run(build, n, D, heads, group, cache_type, batch=1, seed=0):
    """The first of `batch` sequences holds n tokens, the others none: (output, exact) of it."""
    import torch

    from two_compressed_kv_gb300 import mkv as M
    dev = torch.device("cuda:0")
    ct = getattr(torch, cache_type)
    qt = torch.float16 if cache_type == "float8_e4m3fn" else ct
    cast = lambda x, t: torch.from_numpy(np.asarray(x, dtype=np.float32)).to(t)
    fit = lambda x: cast(x, ct).float().numpy().astype(np.float64)
    page = 64
    per = -(-n // page)
    sets = [build(n, D, group, fit, seed=seed + h) for h in range(heads)]
    rows = lambda i: torch.stack([cast(s[i], torch.float32) for s in sets]).view(heads, per, page, D).transpose(0, 1)
    k, v = (rows(i).contiguous().to(ct).to(dev) for i in (1, 2))
    order = torch.randperm(per, generator=torch.Generator().manual_seed(1))
    pools = []
    for x in (k, v):
        pools.append(torch.empty_like(x))
        pools[-1].view(torch.uint8)[order.to(dev)] = x.view(torch.uint8)
    table = torch.full((batch, per), -1, dtype=torch.int32)
    table[0] = order
    c = M.MkvPaged(*pools, table.to(dev))
    q = torch.zeros((batch, heads * group, D), dtype=qt)
    q[0] = torch.cat([cast(s[0], qt) for s in sets])
    lens = torch.zeros(batch, dtype=torch.int32)
    lens[0] = n
    out = M.mkv_paged_decode(c, q.to(dev), lens.to(dev), out_dtype=torch.float32)
    assert c.check() == M.MKV_OK and not out[1:].any()
    return out[0].double().cpu().numpy(), np.concatenate([X.exact(*s) for s in sets])


TYPES = ["float16", "bfloat16", "float8_e4m3fn"]


@pytest.mark.gpu
@pytest.mark.parametrize("cache_type", TYPES)
@pytest.mark.parametrize("n,D,heads,group", [(4096, 64, 2, 4), (4096, 128, 2, 4), (32768, 128, 2, 4), (32768, 128, 4, 7),
                                             (4096, 128, 2, 12), (32768, 128, 1, 16), (4096, 256, 2, 4)])
def test_kernel_precision(cache_type, n, D, heads, group):
    """One CTA cluster a stream (4096) and the load split over all CTAs (32768)."""
    e = X.error(*run(X.plain, n, D, heads, group, cache_type))
    print(f"error {e:.2e}")
    assert e <= (X.BOUND if group <= 8 and D <= 128 else X.BOUND_WIDE)


@pytest.mark.gpu
@pytest.mark.parametrize("cache_type", TYPES)
@pytest.mark.parametrize("group", [4, 12])
def test_kernel_precision_of_long_runs(cache_type, group):
    """More sequences than the split takes: one CTA sums a whole stream, 512 blocks a warp."""
    e = X.error(*run(X.long_run, 32768, 64, 1, group, cache_type, batch=513))
    print(f"error {e:.2e}")
    assert e <= (X.BOUND if group <= 8 else X.BOUND_WIDE)
