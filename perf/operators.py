"""The paged-cache operators as measured: cases, inputs, plain forms and exact values.

Four operators of an uncompressed, paged key-value cache:

* rope    rotary positions of [batch, tokens, heads, head_dim] vectors
* append  new tokens' keys (rotated) and values written into cache pages
* decode  attention of one new token per sequence over its cached pages
* evict   a cache cut down to a budget by accumulated attention weight

`run` takes what `prepare` made through one operator: in elementary torch
operations where `own` is false, through the library's calls where it is true.
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32,
         "e4m3": torch.float8_e4m3fn}
SIZE = {"f16": 2, "bf16": 2, "f32": 4, "e4m3": 1}


def listed():
    return [
        # the queries of one decode step, batch 8, 32 heads, far positions
        dict(name="rope-step-b8", op="rope", type="f16", batch=8, tokens=1, heads=32, dim=128,
             rot=128, interleaved=False, scaling="none", transposed=False, head_major=False),
        # the keys of a 32K prefill, batch 4, from a projection's token-major order into the
        # head-major order that compression takes, frequencies scaled for a longer context
        dict(name="rope-prefill-32k-b4", op="rope", type="bf16", batch=4, tokens=32768, heads=8,
             dim=128, rot=128, interleaved=False, scaling="banded", transposed=False,
             head_major=True),
        # gradient of a partial, interleaved rotation in 32 bits, odd length
        dict(name="rope-grad-4099-part", op="rope", type="f32", batch=2, tokens=4099, heads=28,
             dim=96, rot=64, interleaved=True, scaling="yarn", transposed=True, head_major=False),
        # one decode step's tokens into their pages, batch 8, queries rotated in the same call
        dict(name="append-step-b8", op="append", type="f16", batch=8, tokens=1, kv_heads=8,
             group=4, dim=128, page=64, old=4096),
        # a ragged prefill of four prompts into an 8-bit cache
        dict(name="append-prefill-8k-e4m3", op="append", type="e4m3", batch=4, tokens=8191,
             kv_heads=8, group=4, dim=128, page=64, old=0),
        # a short conversation, one sequence: latency
        dict(name="decode-300-b1", op="decode", type="f16", batch=1, kv_heads=8, group=4, dim=128,
             page=16, ctx=300, ragged=False, weights=False, out="f16"),
        # one layer at 32K, batch 4, output in 32 bits
        dict(name="decode-32k-b4", op="decode", type="f16", batch=4, kv_heads=8, group=4, dim=128,
             page=64, ctx=32768, ragged=False, weights=False, out="f32"),
        # a serving batch of mixed lengths (one of them empty) over an 8-bit cache, 28 query heads
        dict(name="decode-mixed-b64-e4m3", op="decode", type="e4m3", batch=64, kv_heads=4, group=7,
             dim=128, page=48, ctx=16384, ragged=True, weights=False, out="bf16"),
        # one layer at 128K, batch 8, attention weights accumulated for eviction
        dict(name="decode-128k-b8-weights", op="decode", type="bf16", batch=8, kv_heads=8, group=4,
             dim=128, page=64, ctx=131072, ragged=False, weights=True, out="bf16"),
        # steady state: one token over the budget after every step
        dict(name="evict-step-b8", op="evict", type="f16", batch=8, kv_heads=8, dim=128, page=64,
             ctx=4097, budget=4096, sink=4, recent=256),
        # a 32K prefill cut to 2048 tokens
        dict(name="evict-32k-b4", op="evict", type="f16", batch=4, kv_heads=8, dim=128, page=64,
             ctx=32768, budget=2048, sink=4, recent=512),
        # a million-token sequence cut to 8192, 8-bit cache
        dict(name="evict-1m-b1-e4m3", op="evict", type="e4m3", batch=1, kv_heads=8, dim=128,
             page=128, ctx=1048576, budget=8192, sink=4, recent=1024),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "append", "decode", "decode", "evict"])
    if op == "rope":
        dim = rng.choice([64, 80, 96, 128, 128, 256])
        batch, heads = _log(rng, 1, 8), _log(rng, 1, 32)
        tokens = _log(rng, 1, 32768)
        tokens = max(1, min(tokens, (1 << 27) // (batch * heads * dim)))
        return dict(op=op, type=rng.choice(["f16", "bf16", "f32"]), batch=batch, tokens=tokens,
                    heads=heads, dim=dim, rot=rng.choice([dim, dim, dim // 2]),
                    interleaved=rng.random() < 0.5,
                    scaling=rng.choice(["none", "linear", "ntk", "yarn", "banded"]),
                    transposed=rng.random() < 0.3, head_major=rng.random() < 0.5)
    if op == "append":
        dim, batch = rng.choice([64, 128, 128, 256]), _log(rng, 1, 16)
        kv, group = rng.choice([1, 2, 4, 8]), rng.choice([1, 4, 7, 8])
        tokens = max(1, min(_log(rng, 1, 8192), (1 << 27) // (batch * kv * (group + 2) * dim)))
        return dict(op=op, type=rng.choice(["f16", "bf16", "e4m3"]), batch=batch, tokens=tokens,
                    kv_heads=kv, group=group, dim=dim, page=rng.choice([16, 32, 48, 64, 128]),
                    old=_log(rng, 1, 5000))
    if op == "decode":
        dim = rng.choice([64, 128, 128, 256])
        batch, kv = _log(rng, 1, 64), rng.choice([1, 2, 4, 8])
        ctx = min(_log(rng, 1, 131072), (1 << 29) // (batch * kv * dim))
        return dict(op=op, type=rng.choice(["f16", "bf16", "e4m3"]), batch=batch, kv_heads=kv,
                    group=rng.choice([1, 2, 3, 4, 7, 8, 12, 16]), dim=dim,
                    page=rng.choice([16, 32, 48, 64, 128, 256]), ctx=ctx,
                    ragged=rng.random() < 0.5, weights=rng.random() < 0.4,
                    out=rng.choice(["q", "q", "f32"]))
    dim = rng.choice([64, 128, 128, 256])
    batch, kv = _log(rng, 1, 16), rng.choice([1, 2, 4, 8])
    ctx = min(_log(rng, 64, 262144), (1 << 28) // (batch * kv * dim))
    budget = max(16, ctx - 1 if rng.random() < 0.3 else _log(rng, 16, ctx))
    return dict(op=op, type=rng.choice(["f16", "bf16", "e4m3"]), batch=batch, kv_heads=kv, dim=dim,
                page=rng.choice([16, 32, 48, 64, 128]), ctx=ctx, budget=budget,
                sink=min(4, budget // 4), recent=budget // 8)


# ---- inputs -----------------------------------------------------------------------------------

SCALINGS = {
    "none": dict(),
    "linear": dict(factor=4.0),
    "ntk": dict(factor=8.0),
    "yarn": dict(factor=16.0, original=8192, beta_fast=32.0, beta_slow=1.0),
    "banded": dict(factor=8.0, original=8192, low_freq=1.0, high_freq=4.0),
}
BASE = 500000.0


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _normal(shape, g, dtype):
    """Channels of falling size, as keys and values have them, in `dtype`; drawn in blocks."""
    x = torch.empty(shape, dtype=dtype, device=DEV)
    d = shape[-1]
    sigma = torch.exp(-torch.arange(d, device=DEV) / (0.5 * d)) * 2.0
    flat = x.view(-1, d)
    step = max(1, (1 << 26) // d)
    for i in range(0, flat.shape[0], step):
        part = flat[i:i + step]
        part.copy_(torch.randn(part.shape, generator=g, device=DEV) * sigma)
    return x


def _lens(case):
    """Cached tokens of each sequence: all `ctx`, or spread from 0 (only where there are several
    sequences) up to `ctx`."""
    b = case["batch"]
    if not case.get("ragged"):
        return [case["ctx"]] * b
    return [round(case["ctx"] * ((i * 0.6180339887) % 1.0) ** 2) if i else (0 if b > 1 else case["ctx"])
            for i in range(b - 1)] + [case["ctx"]]


def _q_type(case):
    return TYPES["bf16" if case["type"] == "e4m3" else case["type"]]


def _pages(case, rows, g, fill):
    """(key pages, value pages, page table, key scales, value scales) with room for `rows` tokens
    a sequence; the pages of a sequence lie scattered."""
    b, h, d, ps = case["batch"], case["kv_heads"], case["dim"], case["page"]
    per = -(-rows // ps)
    n = b * per + 3
    table = torch.randperm(n, generator=g, device=DEV)[: b * per].view(b, per).to(torch.int32)
    dtype = TYPES[case["type"]]
    made = _normal if fill else (lambda s, _, t: torch.zeros(s, device=DEV, dtype=t))
    pools = [made((n, h, ps, d), g, dtype) for _ in range(2)]
    scales = [None, None]
    if case["type"] == "e4m3":
        scales = [torch.rand(h, generator=g, device=DEV) * 0.5 + 0.5 for _ in range(2)]
    return (*pools, table, *scales)


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case=case)
    if case["op"] == "rope":
        b, t, h, d = (case[k] for k in ("batch", "tokens", "heads", "dim"))
        s["x"] = _normal((b, t, h, d), g, TYPES[case["type"]])
        s["pos"] = (torch.randint(0, 900000, (b, 1), generator=g, device=DEV)
                    + torch.arange(t, device=DEV)).to(torch.int32)
        shape = (b, h, t, d) if case["head_major"] else (b, t, h, d)
        out = torch.empty(shape, dtype=s["x"].dtype, device=DEV)
        s["out"] = out.transpose(1, 2) if case["head_major"] else out
    elif case["op"] == "append":
        b, n, h, d = (case[k] for k in ("batch", "tokens", "kv_heads", "dim"))
        # every prompt some tokens shorter than the one before; the batch is one list of tokens
        lens = [max(1, n - 97 * i) for i in range(b)]
        cap = case["old"] + n
        s["kp"], s["vp"], s["table"], s["ks"], s["vs"] = _pages(case, cap, g, False)
        s["k"], s["v"] = (_normal((sum(lens), h, d), g, _q_type(case)) for _ in range(2))
        s["q"] = _normal((sum(lens), h * case["group"], d), g, _q_type(case))
        s["seq"] = torch.cat([torch.full((m,), i) for i, m in enumerate(lens)]).to(DEV, torch.int32)
        s["slot"] = torch.cat([torch.arange(m) + case["old"] for m in lens]).to(DEV, torch.int32)
        s["pos"] = s["slot"] + 1000
        s["q_out"] = torch.empty_like(s["q"])
        s["acc"] = torch.rand((b, h, cap), generator=g, device=DEV)
        s["meta"] = torch.zeros((b, h, cap), dtype=torch.int32, device=DEV)
    elif case["op"] == "decode":
        b, h, d, gr = (case[k] for k in ("batch", "kv_heads", "dim", "group"))
        s["kp"], s["vp"], s["table"], s["ks"], s["vs"] = _pages(case, case["ctx"], g, True)
        s["lens"] = torch.tensor(_lens(case), dtype=torch.int32, device=DEV)
        # a query near one of the cached keys, so that the softmax has a peak
        page = torch.randint(0, s["kp"].shape[0], (b, h * gr), generator=g, device=DEV)
        at = torch.randint(0, case["page"], (b, h * gr), generator=g, device=DEV)
        head = torch.arange(h * gr, device=DEV) // gr
        base = s["kp"][page, head, at].float()
        s["q"] = (base + 0.5 * torch.randn(base.shape, generator=g, device=DEV)).to(_q_type(case))
        s["out"] = torch.empty(s["q"].shape, device=DEV,
                               dtype=s["q"].dtype if case["out"] == "q" else TYPES[case["out"]])
        s["lse"] = torch.empty((b, h * gr), device=DEV)
        s["acc"] = torch.zeros((b, h, case["ctx"]), device=DEV) if case["weights"] else None
    else:
        b, h, n = case["batch"], case["kv_heads"], case["ctx"]
        s["kp"], s["vp"], s["table"], s["ks"], s["vs"] = _pages(case, n, g, True)
        s["lens"] = torch.full((b,), n, dtype=torch.int32, device=DEV)
        # few tokens with most of the weight; some never attended at all (equal: ties)
        acc = torch.exp(3.0 * torch.randn((b, h, n), generator=g, device=DEV))
        s["acc"] = torch.where(torch.rand((b, h, n), generator=g, device=DEV) < 0.1, 0.0, acc)
        # slots hold tokens out of order once tokens have moved into holes
        order = torch.rand((b, h, n), generator=g, device=DEV).argsort(-1)
        s["pos"] = order.to(torch.int32)
        s["next"] = torch.full((b,), n, dtype=torch.int32, device=DEV)
        s["acc_out"], s["pos_out"] = (torch.zeros((b, h, case["budget"]), dtype=t, device=DEV)
                                      for t in (torch.float32, torch.int32))
        s["src"] = torch.empty((b, h, case["budget"]), dtype=torch.int32, device=DEV)
        s["lens_out"] = torch.empty((b,), dtype=torch.int32, device=DEV)
    if own:
        from two_compressed_kv_gb300 import mkv as M
        s["M"] = M
        if case["op"] == "rope":
            s["plan"] = M.mkv_rope_plan(case["dim"], rot_dim=case["rot"], base=BASE,
                                        interleaved=case["interleaved"], scaling=case["scaling"],
                                        **SCALINGS[case["scaling"]])
        elif case["op"] == "append":
            s["plan"] = M.mkv_rope_plan(case["dim"], base=BASE)
        if case["op"] != "rope":
            s["cache"] = M.MkvPaged(s["kp"], s["vp"], s["table"], k_scale=s["ks"], v_scale=s["vs"])
    elif case["op"] in ("rope", "append"):
        # the plain program keeps its frequencies too
        rot = case.get("rot", case["dim"])
        s["freq"], s["mult"] = _frequencies(rot, case.get("scaling", "none"))
    return s


def _frequencies(rot, scaling):
    """Angle per position of each pair, in 64 bits, and the factor on the rotated vector."""
    p = SCALINGS[scaling]
    i = torch.arange(rot // 2, dtype=torch.float64, device=DEV)
    f = torch.pow(torch.tensor(BASE, dtype=torch.float64, device=DEV), -2.0 * i / rot)
    if scaling == "linear":
        return f / p["factor"], 1.0
    if scaling == "ntk":
        base = BASE * p["factor"] ** (rot / (rot - 2))
        return torch.pow(torch.tensor(base, dtype=torch.float64, device=DEV), -2.0 * i / rot), 1.0
    if scaling == "yarn":
        at = lambda turns: rot * math.log(p["original"] / (turns * 2 * math.pi)) / (2 * math.log(BASE))
        lo = max(0.0, math.floor(at(p["beta_fast"])))
        hi = min(rot - 1.0, math.ceil(at(p["beta_slow"])))
        ramp = ((i - lo) / max(hi - lo, 0.001)).clamp(0.0, 1.0)
        return f * (1 - ramp) + f / p["factor"] * ramp, 0.1 * math.log(p["factor"]) + 1.0
    if scaling == "banded":
        turns = p["original"] * f / (2 * math.pi)
        keep = ((turns - p["low_freq"]) / (p["high_freq"] - p["low_freq"])).clamp(0.0, 1.0)
        return f * keep + f / p["factor"] * (1 - keep), 1.0
    return f, 1.0


# ---- one pass ---------------------------------------------------------------------------------

def run(s):
    op = s["case"]["op"]
    if own:
        return {"rope": _own_rope, "append": _own_append, "decode": _own_decode,
                "evict": _own_evict}[op](s)
    return {"rope": _plain_rope, "append": _plain_append, "decode": _plain_decode,
            "evict": _plain_evict}[op](s)


def _own_rope(s):
    return s["M"].mkv_rope(s["plan"], s["x"], s["pos"], out=s["out"],
                           transposed=s["case"]["transposed"])


def _own_append(s):
    s["M"].mkv_paged_append(s["cache"], s["k"], s["v"], s["slot"], seq=s["seq"], plan=s["plan"],
                            pos=s["pos"], q=s["q"], q_out=s["q_out"], acc=s["acc"],
                            pos_meta=s["meta"])
    return s["kp"], s["vp"], s["q_out"], s["acc"], s["meta"]


def _own_decode(s):
    s["M"].mkv_paged_decode(s["cache"], s["q"], s["lens"], out=s["out"], lse=s["lse"],
                            acc=s["acc"])
    return s["out"], s["lse"], s["acc"]


def _own_evict(s):
    c = s["case"]
    s["M"].mkv_paged_evict(s["cache"], s["acc"], s["pos"], s["lens"], s["next"], c["budget"],
                           sink=c["sink"], recent=c["recent"], acc_out=s["acc_out"],
                           pos_out=s["pos_out"], lens_out=s["lens_out"], src=s["src"])
    return s["src"], s["lens_out"], s["acc_out"], s["pos_out"], s["kp"], s["vp"]


def _rotate(x, pos, freq, mult, rot, interleaved, transposed):
    """x [..., heads, dim] in 32 bits, pos [...]: rotated by angles that are formed in 64 bits."""
    angle = (pos.double().unsqueeze(-1) * freq).unsqueeze(-2)
    cos, sin = (torch.cos(angle) * mult).float(), (torch.sin(angle) * mult).float()
    if transposed:
        sin = -sin
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2)
    else:
        a, b = x[..., : rot // 2], x[..., rot // 2:rot]
        turned = torch.cat((a * cos - b * sin, a * sin + b * cos), -1)
    return torch.cat((turned, x[..., rot:]), -1)


def _plain_rope(s):
    c = s["case"]
    y = _rotate(s["x"].float(), s["pos"], s["freq"], s["mult"], c["rot"], c["interleaved"],
                c["transposed"])
    s["out"].copy_(y)
    return s["out"]


def _bits(x):
    """8-bit values as bytes, which indexing takes; others as they are."""
    return x.view(torch.uint8) if x.dtype == TYPES["e4m3"] else x


def _plain_append(s):
    c = s["case"]
    ps, dim = c["page"], c["dim"]
    k = _rotate(s["k"].float(), s["pos"], s["freq"], s["mult"], dim, False, False)
    v = s["v"].float()
    s["q_out"].copy_(_rotate(s["q"].float(), s["pos"], s["freq"], s["mult"], dim, False, False))
    if s["ks"] is not None:
        k = (k / s["ks"].unsqueeze(-1)).clamp(-448.0, 448.0)
        v = (v / s["vs"].unsqueeze(-1)).clamp(-448.0, 448.0)
    slot, seq = s["slot"].long(), s["seq"].long()
    page = s["table"][seq, slot // ps].long()
    heads = torch.arange(c["kv_heads"], device=DEV).unsqueeze(0)
    at = (page.unsqueeze(1), heads, (slot % ps).unsqueeze(1))
    _bits(s["kp"]).index_put_(at, _bits(k.to(s["kp"].dtype)))
    _bits(s["vp"]).index_put_(at, _bits(v.to(s["vp"].dtype)))
    s["acc"][seq, :, slot] = 0.0
    s["meta"][seq, :, slot] = s["pos"].unsqueeze(1)
    return s["kp"], s["vp"], s["q_out"], s["acc"], s["meta"]


def _rows(pool, table, n, scale=None, dtype=torch.float32):
    """The first n cached rows of every sequence, [batch, heads, n, dim], as the values they stand for."""
    b, per = table.shape
    _, h, ps, d = pool.shape
    x = _bits(pool)[table.long()].view(pool.dtype).to(dtype)
    x = x.permute(0, 2, 1, 3, 4).reshape(b, h, per * ps, d)[:, :, :n]
    return x if scale is None else x * scale.to(dtype).view(1, h, 1, 1)


def _plain_decode(s):
    c = s["case"]
    b, h, d, gr, n = (c[k] for k in ("batch", "kv_heads", "dim", "group", "ctx"))
    k = _rows(s["kp"], s["table"], n, s["ks"])
    score = torch.matmul(s["q"].float().view(b, h, gr, d), k.transpose(-1, -2)) / math.sqrt(d)
    del k
    live = torch.arange(n, device=DEV) < s["lens"].view(b, 1, 1, 1)
    score = torch.where(live, score, -math.inf)
    top = score.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)     # an empty sequence has no highest score
    p = torch.exp(score - top)
    total = p.sum(-1, keepdim=True)
    p = torch.where(total > 0, p / total, 0.0)
    out = torch.matmul(p, _rows(s["vp"], s["table"], n, s["vs"]))
    s["out"].copy_(out.view(b, h * gr, d))
    s["lse"].copy_((top + torch.log(total)).view(b, h * gr))
    if s["acc"] is not None:
        s["acc"] += p.sum(2)
    return s["out"], s["lse"], s["acc"]


def _plain_evict(s):
    c = s["case"]
    b, h, n, m, ps = c["batch"], c["kv_heads"], c["ctx"], c["budget"], c["page"]
    held = torch.arange(n, device=DEV) < s["lens"].view(b, 1, 1)
    safe = (s["pos"] < c["sink"]) | (s["pos"] >= (s["next"].view(b, 1, 1) - c["recent"]))
    key = torch.where(safe, math.inf, s["acc"])
    key = torch.where(held, key, -1.0)
    best = torch.sort(key, dim=-1, descending=True, stable=True).indices[..., :m]
    keep = torch.zeros((b, h, n), dtype=torch.bool, device=DEV).scatter_(-1, best, True) & held
    below = torch.arange(n, device=DEV) < m
    hole, mover = ~keep & below & held, keep & ~below
    # the i-th hole takes the i-th kept token from behind the budget
    rank = torch.cumsum(hole, -1) - 1
    movers = torch.sort(torch.where(mover, torch.arange(n, device=DEV), n), -1).values
    src = torch.where(hole, torch.gather(movers, -1, rank.clamp(min=0)), torch.arange(n, device=DEV))
    src = torch.where(held, src, -1)[..., :m]
    at = src.clamp(min=0)
    s["src"].copy_(src)
    s["lens_out"].copy_(s["lens"].clamp(max=m))
    s["acc_out"].copy_(torch.gather(s["acc"], -1, at))
    s["pos_out"].copy_(torch.gather(s["pos"], -1, at))
    bi, hi, to = torch.nonzero(hole[..., :m], as_tuple=True)
    table = s["table"].long()
    of = src[bi, hi, to]
    put = (table[bi, to // ps], hi, to % ps)
    get = (table[bi, of // ps], hi, of % ps)
    for pool in (_bits(s["kp"]), _bits(s["vp"])):
        pool.index_put_(put, pool[get])
    return s["src"], s["lens_out"], s["acc_out"], s["pos_out"], s["kp"], s["vp"]


# ---- what a pass cannot do without ------------------------------------------------------------

def work(case):
    op, es = case["op"], SIZE[case["type"]]
    if op == "rope":
        rows = case["batch"] * case["tokens"]
        n = rows * case["heads"] * case["dim"]
        return {"bytes": 2 * n * es + 4 * rows, "flops": 3 * rows * case["heads"] * case["rot"]}
    if op == "append":
        rows = sum(max(1, case["tokens"] - 97 * i) for i in range(case["batch"]))
        kv = rows * case["kv_heads"] * case["dim"]
        return {"bytes": kv * 2 * (2 + es) + 2 * kv * case["group"] * 2
                + rows * (12 + 8 * case["kv_heads"]), "flops": 3 * kv * (1 + case["group"])}
    if op == "decode":
        tokens = sum(_lens(case)) * case["kv_heads"]
        heads = case["batch"] * case["kv_heads"] * case["group"]
        out = 4 if case["out"] == "f32" else 2
        return {"bytes": 2 * tokens * case["dim"] * es + heads * (case["dim"] * (2 + out) + 4)
                + (8 * tokens if case["weights"] else 0),
                "flops": 4 * tokens * case["group"] * case["dim"]}
    streams, n, m = case["batch"] * case["kv_heads"], case["ctx"], case["budget"]
    m = min(n, m)
    moved = m * (n - m) / n     # what a random choice of m tokens has behind slot m
    return {"bytes": streams * (8 * n + 12 * m + moved * 4 * case["dim"] * es), "flops": streams * n}


# ---- 64 bits ----------------------------------------------------------------------------------

def exact(case, seed):
    was = globals()["own"]
    globals()["own"] = False
    try:
        s = prepare(case, seed)
    finally:
        globals()["own"] = was
    return {"rope": _exact_rope, "append": _exact_append, "decode": _exact_decode,
            "evict": _exact_evict}[case["op"]](s)


def _exact_turn(x, pos, rot, scaling, interleaved, back):
    """Each pair as a complex number, times e^(i theta)."""
    p, half = SCALINGS[scaling], rot // 2
    speeds, mult = [], 1.0
    for i in range(half):
        f = math.exp(-2.0 * i / rot * math.log(BASE))
        if scaling == "linear":
            f = f / p["factor"]
        elif scaling == "ntk":
            f = math.exp(-2.0 * i / rot * (math.log(BASE) + rot / (rot - 2) * math.log(p["factor"])))
        elif scaling == "yarn":
            first, last = (rot * math.log(p["original"] / (2 * math.pi * p[k])) / (2 * math.log(BASE))
                           for k in ("beta_fast", "beta_slow"))
            first, last = max(0, math.floor(first)), min(rot - 1, math.ceil(last))
            part = min(1.0, max(0.0, (i - first) / max(0.001, last - first)))
            f = f + (f / p["factor"] - f) * part
            mult = 1.0 + 0.1 * math.log(p["factor"])
        elif scaling == "banded":
            wave = 2 * math.pi / f
            if wave > p["original"] / p["low_freq"]:
                f = f / p["factor"]
            elif wave >= p["original"] / p["high_freq"]:
                part = (p["original"] / wave - p["low_freq"]) / (p["high_freq"] - p["low_freq"])
                f = (1 - part) * f / p["factor"] + part * f
        speeds.append(f)
    theta = pos.double()[..., None, None] * torch.tensor(speeds, dtype=torch.float64, device=DEV)
    z = torch.polar(torch.full_like(theta, mult), -theta if back else theta)
    y = x.double()
    if interleaved:
        w = torch.view_as_complex(y[..., :rot].reshape(*y.shape[:-1], half, 2).contiguous()) * z
        turned = torch.view_as_real(w).flatten(-2)
    else:
        w = torch.complex(y[..., :half], y[..., half:rot]) * z
        turned = torch.cat((w.real, w.imag), -1)
    return torch.cat((turned, y[..., rot:]), -1)


def _exact_rope(s):
    c = s["case"]
    return _exact_turn(s["x"], s["pos"], c["rot"], c["scaling"], c["interleaved"], c["transposed"])


def _exact_append(s):
    c = s["case"]
    ps, h = c["page"], c["kv_heads"]
    k = _exact_turn(s["k"], s["pos"], c["dim"], "none", False, False)
    q = _exact_turn(s["q"], s["pos"], c["dim"], "none", False, False)
    v = s["v"].double()
    if s["ks"] is not None:
        k, v = (torch.clamp(x / f.double()[:, None], -448, 448) for x, f in ((k, s["ks"]), (v, s["vs"])))
    kp, vp = (torch.zeros(s["kp"].shape, dtype=torch.float64, device=DEV) for _ in range(2))
    acc, seq, slot = s["acc"].double(), s["seq"].long(), s["slot"].long()
    row = s["table"].long()[seq, slot // ps] * (h * ps) + slot % ps
    for i in range(h):
        kp.view(-1, c["dim"])[row + i * ps] = k[:, i]
        vp.view(-1, c["dim"])[row + i * ps] = v[:, i]
        acc[seq, i, slot] = 0.0
    return kp, vp, q, acc, None


def _exact_decode(s):
    c = s["case"]
    b, h, d, gr, n = (c[k] for k in ("batch", "kv_heads", "dim", "group", "ctx"))
    out = torch.zeros((b, h * gr, d), dtype=torch.float64, device=DEV)
    lse = torch.full((b, h * gr), -math.inf, dtype=torch.float64, device=DEV)
    acc = torch.zeros((b, h, n), dtype=torch.float64, device=DEV)
    for i, m in enumerate(_lens(c)):
        if m == 0:
            continue
        k = _rows(s["kp"], s["table"][i:i + 1], m, s["ks"], torch.float64)[0]
        v = _rows(s["vp"], s["table"][i:i + 1], m, s["vs"], torch.float64)[0]
        z = torch.einsum("hgd,htd->hgt", s["q"][i].double().view(h, gr, d), k) * d ** -0.5
        norm = torch.logsumexp(z, -1)
        w = torch.exp(z - norm[..., None])
        out[i] = torch.einsum("hgt,htd->hgd", w, v).reshape(h * gr, d)
        lse[i] = norm.reshape(h * gr)
        acc[i, :, :m] = w.sum(1)
    return out, lse, acc if c["weights"] else None


def _exact_evict(s):
    c = s["case"]
    m, ps, table = c["budget"], c["page"], s["table"].long()
    kp, vp = ((x.view(torch.uint8) if c["type"] == "e4m3" else x).clone() for x in (s["kp"], s["vp"]))
    acc, pos, lens = s["acc"].cpu(), s["pos"].cpu(), s["lens"].tolist()
    acc_out = torch.zeros(s["acc_out"].shape, dtype=torch.float64)
    for b, n in enumerate(lens):
        for h in range(c["kv_heads"]):
            a, p = acc[b, h, :n].double(), pos[b, h, :n]
            safe = (p < c["sink"]) | (p >= n - c["recent"])
            rest = torch.nonzero(~safe).flatten()
            rest = rest[torch.sort(-a[rest], stable=True).indices][: max(0, m - int(safe.sum()))]
            keep = torch.zeros(n, dtype=torch.bool)
            keep[torch.cat((torch.nonzero(safe).flatten(), rest))] = True
            to, of = torch.nonzero(~keep[:m]).flatten(), torch.nonzero(keep[m:]).flatten() + m
            to = to[: len(of)]
            a[to] = a[of]
            acc_out[b, h, : min(n, m)] = a[:m]
            t, f = to.to(DEV), of.to(DEV)
            for x in (kp, vp):
                x[table[b, t // ps], h, t % ps] = x[table[b, f // ps], h, f % ps]
    view = (lambda x: x.view(TYPES["e4m3"]).double()) if c["type"] == "e4m3" else (lambda x: x.double())
    return None, None, acc_out.to(DEV), None, view(kp), view(vp)
