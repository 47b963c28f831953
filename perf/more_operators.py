"""Operators around the two caches as measured: cases, inputs, plain forms and exact values.

* multi    rotary positions with several axes of [batch, tokens, heads, head_dim] vectors
* norm     RMS norms of query and key heads and their rotation in one pass, and the gradients
* prefill  attention of a prompt over itself or over cached tokens and itself: causal, prefix,
           window and document masks, scores capped by a tanh, a bias that falls with distance
* attend   attention of several new tokens a sequence (a chain, or a tree of drafts) over the
           pages of a cache, with the same treatment of scores

`run` takes what `prepare` made through one operator: in elementary torch
operations where `own` is false, through the library's calls where it is true.
"""
import math
import random

import torch

own = False

DEV = "cuda"
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32,
         "e4m3": torch.float8_e4m3fn}
SIZE = {"f16": 2, "bf16": 2, "f32": 4, "e4m3": 1}
BASE = 500000.0
EPS = 1e-6


def listed():
    return [
        # queries of a prompt with pictures: time, height and width, pairs dealt in blocks
        dict(name="multi-image-16k-b2", op="multi", type="bf16", batch=2, tokens=16384, heads=28,
             dim=128, sections="16,24,24", order="blocks", restart=False, interleaved=False,
             transposed=False),
        # gradient of the rotation of a vision tower's heads by row and column, odd sizes
        dict(name="multi-grid-grad-4099", op="multi", type="f32", batch=3, tokens=4099, heads=16,
             dim=80, sections="20,20", order="cyclic", restart=True, interleaved=True,
             transposed=True),
        # the new token of 8 sequences: latency
        dict(name="norm-step-b8", op="norm", type="bf16", batch=8, tokens=1, heads=32, kv_heads=8,
             dim=128, axes=1, grad=False),
        # queries and keys of a prompt, views of one projection's output
        dict(name="norm-prefill-8k-b4", op="norm", type="bf16", batch=4, tokens=8192, heads=32,
             kv_heads=8, dim=128, axes=1, grad=False),
        # a training step's way back, three axes, odd length
        dict(name="norm-grad-4099-b4", op="norm", type="bf16", batch=4, tokens=4099, heads=16,
             kv_heads=16, dim=128, axes=3, grad=True),
        # a short question: latency
        dict(name="prefill-77-b1", op="prefill", type="f16", batch=1, heads=32, kv_heads=8,
             dim=128, tokens=77, cached=0, causal=True, window=0, prefix=0, docs=0, ragged=False,
             cap=0.0, bias=False),
        # ordinary prompts, 32 query heads over 8
        dict(name="prefill-8k-b4", op="prefill", type="bf16", batch=4, heads=32, kv_heads=8,
             dim=128, tokens=8192, cached=0, causal=True, window=0, prefix=0, docs=0, ragged=False,
             cap=0.0, bias=False),
        # documents packed into one row, capped scores, 28 query heads over 4
        dict(name="prefill-16k-docs-cap", op="prefill", type="bf16", batch=1, heads=28, kv_heads=4,
             dim=128, tokens=16381, cached=0, causal=True, window=0, prefix=0, docs=5,
             ragged=False, cap=50.0, bias=False),
        # a padded batch over cached tokens, prefix seen both ways, bias by distance, heads of 64
        dict(name="prefill-ragged-prefix-bias", op="prefill", type="f16", batch=8, heads=12,
             kv_heads=12, dim=64, tokens=1531, cached=500, causal=True, window=0, prefix=300,
             docs=0, ragged=True, cap=0.0, bias=True),
        # a few drafts after a short conversation: latency
        dict(name="tree-300-b1", op="attend", type="f16", batch=1, kv_heads=8, group=4, dim=128,
             page=16, ctx=300, new=16, tree=True, ragged=False, window=0, cap=0.0, bias=False),
        # 64 drafts a sequence over 32K tokens
        dict(name="tree-32k-b4", op="attend", type="bf16", batch=4, kv_heads=8, group=4, dim=128,
             page=64, ctx=32768, new=64, tree=True, ragged=False, window=0, cap=0.0, bias=False),
        # single tokens of a serving batch over an 8-bit cache of mixed lengths, capped scores
        dict(name="single-mixed-b32-e4m3-cap", op="attend", type="e4m3", batch=32, kv_heads=4,
             group=4, dim=256, page=48, ctx=16384, new=1, tree=False, ragged=True, window=4096,
             cap=30.0, bias=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["multi", "norm", "norm", "prefill", "prefill", "prefill", "attend", "attend"])
    if op == "multi":
        dim = rng.choice([64, 80, 96, 128, 128, 256])
        pairs, axes = rng.choice([dim, dim, dim // 2]) // 2, rng.choice([2, 3, 3])
        cut = sorted(rng.sample(range(1, pairs), axes - 1))
        batch, heads = _log(rng, 1, 8), _log(rng, 1, 32)
        tokens = max(1, min(_log(rng, 1, 32768), (1 << 26) // (batch * heads * dim)))
        return dict(op=op, type=rng.choice(["f16", "bf16", "f32"]), batch=batch, tokens=tokens,
                    heads=heads, dim=dim,
                    sections=",".join(str(b - a) for a, b in zip([0] + cut, cut + [pairs])),
                    order=rng.choice(["blocks", "cyclic"]), restart=rng.random() < 0.4,
                    interleaved=rng.random() < 0.4, transposed=rng.random() < 0.3)
    if op == "norm":
        dim, grad = rng.choice([64, 80, 96, 128, 128, 256]), rng.random() < 0.5
        kv = _log(rng, 1, 16)
        heads, batch = kv * rng.choice([1, 2, 4, 7]), _log(rng, 1, 8)
        tokens = max(1, min(_log(rng, 1, 16384), (1 << 25) // (batch * (heads + kv) * dim)))
        return dict(op=op, type=rng.choice(["f16", "bf16", "bf16", "f32"]), batch=batch,
                    tokens=tokens, heads=heads, kv_heads=kv, dim=dim, axes=rng.choice([1, 1, 3]),
                    grad=grad)
    if op == "prefill":
        dim, kv = rng.choice([64, 128, 128, 256]), rng.choice([1, 2, 4, 8])
        heads, batch = kv * rng.choice([1, 3, 4, 7, 8]), _log(rng, 1, 8)
        cached = rng.choice([0, 0, _log(rng, 1, 8192)])
        most = 10**12 / (batch * heads * dim)
        tokens = _log(rng, 1, 16384)
        while tokens > 1 and tokens * (tokens + cached) > most:
            tokens = tokens * 2 // 3
        causal, total = rng.random() < 0.8, tokens + cached
        return dict(op=op, type=rng.choice(["f16", "bf16", "bf16"]), batch=batch, heads=heads,
                    kv_heads=kv, dim=dim, tokens=tokens, cached=cached, causal=causal,
                    window=rng.choice([0, 0, _log(rng, 16, 4096)]),
                    prefix=rng.choice([0, 0, 1 + total // 3]) if causal else 0,
                    docs=rng.choice([0, 0, 4]), ragged=rng.random() < 0.3,
                    cap=rng.choice([0.0, 0.0, 20.0, 50.0]), bias=rng.random() < 0.25)
    dim, kv = rng.choice([64, 128, 128, 256]), rng.choice([1, 2, 4, 8])
    batch = _log(rng, 1, 32)
    ctx = max(1, min(_log(rng, 16, 131072), (1 << 27) // (batch * kv * dim)))
    new = min(_log(rng, 1, 64), ctx)
    return dict(op=op, type=rng.choice(["f16", "bf16", "e4m3"]), batch=batch, kv_heads=kv,
                group=rng.choice([1, 2, 4, 7, 8]), dim=dim, page=rng.choice([16, 32, 48, 64, 128]),
                ctx=ctx, new=new, tree=rng.random() < 0.6, ragged=rng.random() < 0.4,
                window=rng.choice([0, 0, 0, 1024]), cap=rng.choice([0.0, 0.0, 30.0]),
                bias=rng.random() < 0.25)


# ---- inputs -----------------------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _normal(shape, g, dtype):
    """Channels of falling size, as queries, keys and values have them, in `dtype`."""
    x = torch.empty(shape, dtype=dtype, device=DEV)
    d = shape[-1]
    sigma = torch.exp(-torch.arange(d, device=DEV) / (0.5 * d)) * 2.0
    flat = x.view(-1, d)
    step = max(1, (1 << 26) // d)
    for i in range(0, flat.shape[0], step):
        part = flat[i:i + step]
        part.copy_(torch.randn(part.shape, generator=g, device=DEV) * sigma)
    return x


def _spread(n, most, least=0):
    """n lengths from `least` to `most`, unequal; the last is `most`."""
    at = lambda i: least + round((most - least) * ((i * 0.6180339887) % 1.0) ** 2)
    return [at(i) for i in range(n - 1)] + [most]


def _prompt_lens(case):
    """(queries, keys) of each sequence."""
    b, t = case["batch"], case["tokens"]
    q = _spread(b, t, min(1, t)) if case["ragged"] else [t] * b
    return q, [n + case["cached"] for n in q]


def _ends(case):
    """Where the documents of a row of keys end: unequal shares, the first the longest."""
    n, parts = case["tokens"] + case["cached"], case["docs"]
    share = [parts - i + 0.5 for i in range(parts)]
    return [round(n * sum(share[:i + 1]) / sum(share)) for i in range(parts)]


def _new_lens(case):
    """(cached tokens with the new ones, new tokens) of each sequence."""
    b, n, m = case["batch"], case["ctx"], case["new"]
    if not case["ragged"]:
        return [n] * b, [m] * b
    lens = _spread(b, n)
    return lens, [min(1 + (m + 5 * i) % m, lens[i]) for i in range(b)]


def _slopes(heads):
    return [2.0 ** (-8.0 * (i + 1) / heads) for i in range(heads)]


def _sections(case):
    """Pairs of each axis."""
    return [int(n) for n in case["sections"].split(",")]


def _axes_positions(b, t, axes, g):
    """Text positions, then pictures of rows and columns: [axes, batch, tokens]."""
    i = torch.arange(t, device=DEV)
    start = torch.randint(0, 30000, (b, 1), generator=g, device=DEV)
    grid = torch.stack((i // 1024, i // 32 % 32, i % 32))[:axes].unsqueeze(1)
    lone = (i < t // 4).expand(axes, b, t)
    return torch.where(lone, i.expand(axes, b, t), t // 4 + grid).add(start).to(torch.int32)


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case=case)
    op = case["op"]
    if op == "multi":
        b, t, h, d = (case[k] for k in ("batch", "tokens", "heads", "dim"))
        s["x"] = _normal((b, t, h, d), g, TYPES[case["type"]])
        s["pos"] = _axes_positions(b, t, len(_sections(case)), g)
        s["out"] = torch.empty_like(s["x"])
        s["pairs"] = _pairs(_sections(case), case["order"], case["restart"])
    elif op == "norm":
        b, t, h, kv, d = (case[k] for k in ("batch", "tokens", "heads", "kv_heads", "dim"))
        # one projection's output: the heads of queries, keys and values of a token in a row
        proj = _normal((b, t, h + 2 * kv, d), g, TYPES[case["type"]])
        s["q"], s["k"] = proj[:, :, :h], proj[:, :, h:h + kv]
        s["qw"], s["kw"] = (1.0 + 0.2 * torch.randn(d, generator=g, device=DEV) for _ in range(2))
        s["pos"] = _axes_positions(b, t, case["axes"], g)
        s["sections"] = (d // 2,) if case["axes"] == 1 else (d // 2 - 2 * (d // 6), d // 6, d // 6)
        s["pairs"] = _pairs(s["sections"], "blocks", False)
        if case["grad"]:
            s["dq"], s["dk"] = (_normal((b, t, n, d), g, proj.dtype) for n in (h, kv))
        s["q_out"], s["k_out"] = (torch.empty((b, t, n, d), dtype=proj.dtype, device=DEV)
                                  for n in (h, kv))
    elif op == "prefill":
        b, t, h, kv, d = (case[k] for k in ("batch", "tokens", "heads", "kv_heads", "dim"))
        dtype, n = TYPES[case["type"]], t + case["cached"]
        proj = _normal((b, n, 2 * kv, d), g, dtype)
        s["k"], s["v"] = proj[:, :, :kv], proj[:, :, kv:]
        # a query near one of the keys, so that the softmax has a peak
        at = torch.randint(0, n, (b, t, 1, 1), generator=g, device=DEV)
        near = torch.gather(s["k"], 1, at.expand(b, t, kv, d)).repeat_interleave(h // kv, 2)
        s["q"] = near.add(_normal((b, t, h, d), g, dtype)).mul_(0.7)
        s["out"] = torch.zeros_like(s["q"])
        ql, kl = _prompt_lens(case)
        s["ql"], s["kl"] = (torch.tensor(x, dtype=torch.int32, device=DEV) if case["ragged"]
                            else None for x in (ql, kl))
        s["prefix"] = (torch.full((b,), case["prefix"], dtype=torch.int32, device=DEV)
                       if case["prefix"] else None)
        s["docs"] = None
        if case["docs"]:
            ends = torch.tensor(_ends(case), device=DEV)
            s["docs"] = (torch.arange(n, device=DEV).unsqueeze(-1) >= ends).sum(-1).to(
                torch.int32).expand(b, n).contiguous()
        s["slopes"] = torch.tensor(_slopes(h), device=DEV) if case["bias"] else None
    else:
        b, h, gr, d, m = (case[k] for k in ("batch", "kv_heads", "group", "dim", "new"))
        ps, dtype = case["page"], TYPES[case["type"]]
        per = -(-case["ctx"] // ps)
        n = b * per + 3
        s["table"] = torch.randperm(n, generator=g, device=DEV)[:b * per].view(b, per).to(torch.int32)
        s["kp"], s["vp"] = (_normal((n, h, ps, d), g, dtype) for _ in range(2))
        s["ks"], s["vs"] = ((torch.rand(h, generator=g, device=DEV) * 0.5 + 0.5 for _ in range(2))
                            if case["type"] == "e4m3" else (None, None))
        lens, new = _new_lens(case)
        s["lens"], s["new"] = (torch.tensor(x, dtype=torch.int32, device=DEV) for x in (lens, new))
        page = torch.randint(0, n, (b, m, h * gr), generator=g, device=DEV)
        at = torch.randint(0, ps, (b, m, h * gr), generator=g, device=DEV)
        base = s["kp"][page, torch.arange(h * gr, device=DEV) // gr, at].float()
        qt = torch.bfloat16 if case["type"] == "e4m3" else dtype
        s["q"] = (0.7 * base + torch.randn(base.shape, generator=g, device=DEV)).to(qt)
        s["out"] = torch.zeros_like(s["q"])
        s["lse"] = torch.zeros((b, m, h * gr), device=DEV)
        s["slopes"] = torch.tensor(_slopes(h * gr), device=DEV) if case["bias"] else None
        s["tree"] = None
        if case["tree"]:
            # every draft hangs on one before it, mostly on a recent one
            rng, rows = random.Random(seed), []
            for _ in range(b):
                seen = []
                for i in range(m):
                    up = 0 if i == 0 else seen[max(0, i - 1 - int(rng.random() ** 2 * 8))]
                    seen.append(up | 1 << i)
                rows.append([x - (1 << 64) if x >> 63 else x for x in seen])
            s["tree"] = torch.tensor(rows, dtype=torch.int64, device=DEV)
    if own:
        from two_compressed_kv_gb300 import mkv as M
        s["M"] = M
        if op == "multi":
            s["plan"] = M.mkv_rope_axes_plan(
                case["dim"], _sections(case), order=case["order"], restart=case["restart"],
                base=BASE, interleaved=case["interleaved"])
        elif op == "norm":
            s["plan"] = M.mkv_rope_axes_plan(case["dim"], s["sections"], base=BASE)
        elif op == "attend":
            s["cache"] = M.MkvPaged(s["kp"], s["vp"], s["table"], k_scale=s["ks"], v_scale=s["vs"])
    return s


def _pairs(sections, order, restart):
    """(axis, frequency in 64 bits) of each pair."""
    axis = []
    if order == "blocks":
        for a, n in enumerate(sections):
            axis += [a] * n
    else:
        left = list(sections)
        while any(left):
            for a in range(len(left)):
                if left[a]:
                    axis.append(a)
                    left[a] -= 1
    total, seen, freq = len(axis), [0] * len(sections), []
    for i, a in enumerate(axis):
        freq.append(BASE ** (-seen[a] / sections[a]) if restart else BASE ** (-i / total))
        seen[a] += 1
    return (torch.tensor(axis, device=DEV),
            torch.tensor(freq, dtype=torch.float64, device=DEV))


# ---- one pass ---------------------------------------------------------------------------------

def run(s):
    op = s["case"]["op"]
    if own:
        return {"multi": _own_multi, "norm": _own_norm, "prefill": _own_prefill,
                "attend": _own_attend}[op](s)
    return {"multi": _plain_multi, "norm": _plain_norm, "prefill": _plain_prefill,
            "attend": _plain_attend}[op](s)


def _own_multi(s):
    return s["M"].mkv_rope_multi(s["plan"], s["x"], s["pos"], out=s["out"],
                                 transposed=s["case"]["transposed"])


def _own_norm(s):
    M = s["M"]
    if s["case"]["grad"]:
        return M.mkv_norm_rope_grad(s["plan"], s["dq"], s["q"], s["qw"], s["pos"], dk=s["dk"],
                                    k=s["k"], k_weight=s["kw"], eps=EPS, dq_out=s["q_out"],
                                    dk_out=s["k_out"])
    return M.mkv_norm_rope(s["plan"], s["q"], s["qw"], s["pos"], k=s["k"], k_weight=s["kw"],
                           eps=EPS, q_out=s["q_out"], k_out=s["k_out"])


def _own_prefill(s):
    c = s["case"]
    return s["M"].mkv_prefill(s["q"], s["k"], s["v"], out=s["out"], causal=c["causal"],
                              window=c["window"], prefix=s["prefix"], docs=s["docs"],
                              q_lens=s["ql"], kv_lens=s["kl"], cap=c["cap"], slopes=s["slopes"])


def _own_attend(s):
    c = s["case"]
    s["M"].mkv_paged_attend(s["cache"], s["q"], s["lens"], tree=s["tree"], new_lens=s["new"],
                            out=s["out"], lse=s["lse"], max_len=c["ctx"], window=c["window"],
                            cap=c["cap"], slopes=s["slopes"])
    return s["out"], s["lse"]


def _turn(x, pos, pairs, interleaved, back):
    """x [..., heads, dim] in 32 bits, pos [axes, ...]: angles formed in 64 bits."""
    axis, freq = pairs
    angle = (pos.double()[axis].movedim(0, -1) * freq).unsqueeze(-2)
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    if back:
        sin = -sin
    rot = 2 * freq.numel()
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        turned = torch.cat((a * cos - b * sin, a * sin + b * cos), -1)
    return torch.cat((turned, x[..., rot:]), -1)


def _plain_multi(s):
    c = s["case"]
    s["out"].copy_(_turn(s["x"].float(), s["pos"], s["pairs"], c["interleaved"], c["transposed"]))
    return s["out"]


def _plain_norm(s):
    if not s["case"]["grad"]:
        one = lambda x, w, out: out.copy_(_turn(_unit(x)[0] * w, s["pos"], s["pairs"], False, False))
        return one(s["q"], s["qw"], s["q_out"]), one(s["k"], s["kw"], s["k_out"])

    def back(dy, x, w, out):
        n, r = _unit(x)
        u = _turn(dy.float(), s["pos"], s["pairs"], False, True)
        e = u * w
        out.copy_(r * (e - n * (e * n).mean(-1, keepdim=True)))
        return out, (u * n).sum((0, 1, 2))

    dq, dqw = back(s["dq"], s["q"], s["qw"], s["q_out"])
    dk, dkw = back(s["dk"], s["k"], s["kw"], s["k_out"])
    return dq, dk, dqw, dkw


def _unit(x):
    """Heads divided by their root mean square, and the factor that did it."""
    x = x.float()
    r = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
    return x * r, r


def _softmax_times(score, live, v):
    """(weights times values, ln of the sum of exp) with zeros and -inf where no key is live."""
    score = torch.where(live, score, -math.inf)
    top = score.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = torch.exp(score - top)
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v)
    return torch.where(total > 0, o / total, 0.0), (top + torch.log(total)).squeeze(-1)


def _visible(c, s, b, p, j):
    """Which keys j [n] of sequence b the queries at places p [t, 1] of the keys see."""
    live = j < (c["tokens"] + c["cached"] if s["kl"] is None else s["kl"][b])
    if c["causal"]:
        before = j <= p
        live = live & (before if s["prefix"] is None else before | (j < s["prefix"][b]))
    if c["window"]:
        live = live & (p - j < c["window"])
        live = live if c["causal"] else live & (j - p < c["window"])
    if s["docs"] is not None:
        live = live & (p >= 0) & (s["docs"][b][p.clamp(0, s["docs"].shape[1] - 1)] == s["docs"][b])
    return live


def _plain_prefill(s):
    c = s["case"]
    t, n, h, kv, d = (c["tokens"], c["tokens"] + c["cached"], c["heads"], c["kv_heads"], c["dim"])
    i, j = torch.arange(t, device=DEV).unsqueeze(-1), torch.arange(n, device=DEV)
    for b in range(c["batch"]):      # one sequence's scores at a time
        p = i + (c["cached"] if s["ql"] is None else s["kl"][b] - s["ql"][b])
        q = s["q"][b].float().view(t, kv, h // kv, d).permute(1, 2, 0, 3)
        k, v = (x[b].float().transpose(0, 1).unsqueeze(1) for x in (s["k"], s["v"]))
        score = torch.matmul(q, k.transpose(-1, -2)) / math.sqrt(d)
        if c["cap"]:
            score = torch.tanh(score / c["cap"]) * c["cap"]
        if s["slopes"] is not None:
            score = score - s["slopes"].view(kv, -1, 1, 1) * (p - j).abs()
        o = _softmax_times(score, _visible(c, s, b, p, j), v)[0]
        o = o.permute(2, 0, 1, 3).reshape(t, h, d).to(s["out"].dtype)
        s["out"][b].copy_(o if s["ql"] is None
                          else torch.where(i.unsqueeze(-1) < s["ql"][b], o, s["out"][b]))
    return s["out"]


def _rows(pool, table, n, scale, dtype):
    """The first n cached rows of every sequence, [batch, heads, n, dim], as the values they stand for."""
    b, per = table.shape
    _, h, ps, d = pool.shape
    x = (pool.view(torch.uint8) if pool.dtype == TYPES["e4m3"] else pool)[table.long()]
    x = x.view(pool.dtype).to(dtype).permute(0, 2, 1, 3, 4).reshape(b, h, per * ps, d)[:, :, :n]
    return x if scale is None else x * scale.to(dtype).view(1, h, 1, 1)


def _tree_view(s):
    """(places of the drafts [b, m], place of every key [b, n], which keys a draft sees [b, m, n])."""
    c = s["case"]
    m, n = c["new"], c["ctx"]
    i, j = torch.arange(m, device=DEV), torch.arange(n, device=DEV)
    new, lens = s["new"].long().unsqueeze(-1), s["lens"].long().unsqueeze(-1)
    base = lens - new
    if s["tree"] is None:
        sees = (i <= i.unsqueeze(-1)).expand(c["batch"], m, m)
    else:
        sees = (s["tree"].unsqueeze(-1) >> i & 1).bool()
    sees = sees & (i < new).unsqueeze(1)
    depth = (sees & (i != i.unsqueeze(-1))).sum(-1)
    draft = (j - base).clamp(0, m - 1)                       # which draft lies in a slot
    place = torch.where(j < base, j, base + torch.gather(depth, 1, draft))
    live = torch.gather(sees, 2, draft.unsqueeze(1).expand(-1, m, -1))
    live = (live | (j < base).unsqueeze(1)) & (j < lens).unsqueeze(1)
    at = base + depth
    if c["window"]:
        live = live & (at.unsqueeze(-1) - place.unsqueeze(1) < c["window"])
    return at, place, live


def _plain_attend(s):
    c = s["case"]
    b, h, gr, d, m, n = (c[k] for k in ("batch", "kv_heads", "group", "dim", "new", "ctx"))
    at, place, live = _tree_view(s)
    k = _rows(s["kp"], s["table"], n, s["ks"], torch.float32)
    q = s["q"].float().view(b, m, h, gr, d).permute(0, 2, 3, 1, 4).reshape(b, h, gr * m, d)
    score = (torch.matmul(q, k.transpose(-1, -2)) / math.sqrt(d)).view(b, h, gr, m, n)
    del k
    if c["cap"]:
        score = torch.tanh(score / c["cap"]) * c["cap"]
    if s["slopes"] is not None:
        far = (at.unsqueeze(-1) - place.unsqueeze(1)).abs()
        score = score - s["slopes"].view(1, h, gr, 1, 1) * far.view(b, 1, 1, m, n)
    v = _rows(s["vp"], s["table"], n, s["vs"], torch.float32).unsqueeze(2)
    o, lse = _softmax_times(score, live.view(b, 1, 1, m, n), v)
    there = (torch.arange(m, device=DEV) < s["new"].unsqueeze(-1)).unsqueeze(-1)
    o = o.permute(0, 3, 1, 2, 4).reshape(b, m, h * gr, d).to(s["out"].dtype)
    s["out"].copy_(torch.where(there.unsqueeze(-1), o, s["out"]))
    s["lse"].copy_(torch.where(there, lse.permute(0, 3, 1, 2).reshape(b, m, h * gr), s["lse"]))
    return s["out"], s["lse"]


# ---- what a pass cannot do without ------------------------------------------------------------

def _seen(case):
    """Pairs of a query and a key that it sees, over all sequences, for one head."""
    total = 0
    for b, (nq, nk) in enumerate(zip(*_prompt_lens(case))):
        p = torch.arange(nq) + nk - nq
        lo, hi = torch.zeros_like(p), torch.full_like(p, nk)
        if case["causal"]:
            hi = torch.clamp(p + 1, min=min(case["prefix"], nk))
        if case["window"]:
            lo = torch.clamp(p - case["window"] + 1, min=0)
            hi = hi if case["causal"] else torch.minimum(hi, p + case["window"])
        if case["docs"]:
            ends = torch.tensor([0] + _ends(case))
            d = (p.unsqueeze(-1) >= ends[1:]).sum(-1)
            lo, hi = torch.maximum(lo, ends[d]), torch.minimum(hi, ends[d + 1])
        total += int((hi - lo).clamp(min=0).sum())
    return total


def work(case):
    op, es = case["op"], SIZE[case["type"]]
    if op == "multi":
        rows = case["batch"] * case["tokens"]
        n = rows * case["heads"] * case["dim"]
        return {"bytes": 2 * n * es + 4 * rows * len(_sections(case)),
                "flops": 6 * rows * case["heads"] * sum(_sections(case))}
    if op == "norm":
        rows = case["batch"] * case["tokens"]
        n = rows * (case["heads"] + case["kv_heads"]) * case["dim"]
        return {"bytes": n * es * (3 if case["grad"] else 2) + 4 * rows * case["axes"]
                + case["dim"] * (16 if case["grad"] else 8),
                "flops": n * (14 if case["grad"] else 7)}
    if op == "prefill":
        ql, kl = _prompt_lens(case)
        return {"bytes": 2 * es * case["dim"] * (sum(ql) * case["heads"] + sum(kl) * case["kv_heads"]),
                "flops": 4 * case["dim"] * case["heads"] * _seen(case)}
    lens, new = _new_lens(case)
    reach = [min(n, case["window"] + m) if case["window"] else n for n, m in zip(lens, new)]
    heads = sum(new) * case["kv_heads"] * case["group"]
    pairs = sum(r * m for r, m in zip(reach, new))
    return {"bytes": 2 * sum(reach) * case["kv_heads"] * case["dim"] * es
            + heads * (case["dim"] * 4 + 4),
            "flops": 4 * pairs * case["kv_heads"] * case["group"] * case["dim"]}


# ---- 64 bits ----------------------------------------------------------------------------------

def exact(case, seed):
    was = globals()["own"]
    globals()["own"] = False
    try:
        s = prepare(case, seed)
    finally:
        globals()["own"] = was
    if case["op"] == "prefill":
        full = case["batch"] * case["heads"] * case["tokens"] * (case["tokens"] + case["cached"])
        if full * case["dim"] > 1.5e12:      # some seconds of 64-bit products
            return None
    return {"multi": _exact_multi, "norm": _exact_norm, "prefill": _exact_prefill,
            "attend": _exact_attend}[case["op"]](s)


def _exact_spin(x, pos, sections, order, restart, interleaved, back):
    """Each pair as a complex number, times e^(i theta), theta of the pair's own axis."""
    half = sum(sections)
    owner = [a for a, n in enumerate(sections) for _ in range(n)]
    if order == "cyclic":
        # the k-th pair of axis a comes after the pairs of every axis in k full turns
        owner = [a for _, a in sorted((k, a) for a, n in enumerate(sections) for k in range(n))]
    theta = torch.empty((*pos.shape[1:], half), dtype=torch.float64, device=DEV)
    for i, a in enumerate(owner):
        part = owner[:i].count(a) / sections[a] if restart else i / half
        theta[..., i] = pos[a].double() * math.exp(-part * math.log(BASE))
    z = torch.polar(torch.ones_like(theta), -theta if back else theta).unsqueeze(-2)
    y = x.double()
    if interleaved:
        w = torch.view_as_complex(y[..., :2 * half].reshape(*y.shape[:-1], half, 2).contiguous()) * z
        turned = torch.view_as_real(w).flatten(-2)
    else:
        w = torch.complex(y[..., :half], y[..., half:2 * half]) * z
        turned = torch.cat((w.real, w.imag), -1)
    return torch.cat((turned, y[..., 2 * half:]), -1)


def _exact_multi(s):
    c = s["case"]
    return _exact_spin(s["x"], s["pos"], _sections(c), c["order"], c["restart"], c["interleaved"],
                       c["transposed"])


def _exact_norm(s):
    spin = lambda x, back: _exact_spin(x, s["pos"], s["sections"], "blocks", False, False, back)
    if not s["case"]["grad"]:
        one = lambda x, w: spin(x.double() / (x.double().pow(2).mean(-1, keepdim=True) + EPS).sqrt()
                                * w.double(), False)
        return one(s["q"], s["qw"]), one(s["k"], s["kw"])

    def back(dy, x, w):
        x, d = x.double(), x.shape[-1]
        size = (x.pow(2).mean(-1, keepdim=True) + EPS).sqrt()
        u = spin(dy, True)
        along = (u * w.double() * x).sum(-1, keepdim=True)
        return u * w.double() / size - x * along / (d * size ** 3), (u * x / size).flatten(0, 2).sum(0)

    (dq, dqw), (dk, dkw) = back(s["dq"], s["q"], s["qw"]), back(s["dk"], s["k"], s["kw"])
    return dq, dk, dqw, dkw


def _exact_prefill(s):
    c = s["case"]
    t, h, kv, d = (c[k] for k in ("tokens", "heads", "kv_heads", "dim"))
    out = torch.zeros((c["batch"], t, h, d), dtype=torch.float64, device=DEV)
    docs = None
    if c["docs"]:
        docs = torch.bucketize(torch.arange(t + c["cached"], device=DEV),
                               torch.tensor(_ends(c), device=DEV), right=True)
    for b, (nq, nk) in enumerate(zip(*_prompt_lens(c))):
        p = torch.arange(nk - nq, nk, device=DEV)[:, None]
        j = torch.arange(nk, device=DEV)[None]
        shut = torch.zeros((nq, nk), dtype=torch.bool, device=DEV)
        if c["causal"]:
            shut |= (j > p) & (j >= c["prefix"])
        if c["window"]:
            shut |= j <= p - c["window"]
            if not c["causal"]:
                shut |= j >= p + c["window"]
        if docs is not None:
            shut |= docs[nk - nq:nk, None] != docs[None, :nk]
        for i in range(h):
            z = (s["q"][b, :nq, i].double() @ s["k"][b, :nk, i * kv // h].double().T) * d ** -0.5
            if c["cap"]:
                z = c["cap"] * torch.tanh(z / c["cap"])
            if c["bias"]:
                z -= float(torch.tensor(_slopes(h)[i])) * (p - j).abs()
            z[shut] = -math.inf
            w = torch.softmax(z, -1)
            w[shut.all(-1)] = 0.0
            out[b, :nq, i] = w @ s["v"][b, :nk, i * kv // h].double()
    return out


def _exact_attend(s):
    c = s["case"]
    h, gr, d = (c[k] for k in ("kv_heads", "group", "dim"))
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device=DEV)
    lse = torch.zeros(s["lse"].shape, dtype=torch.float64, device=DEV)
    slope = torch.tensor(_slopes(h * gr)).double().to(DEV).view(h, gr, 1)
    for b, (n, m) in enumerate(zip(*_new_lens(c))):
        if m == 0:
            continue
        k, v = (_rows(pool, s["table"][b:b + 1], n, scale, torch.float64)[0]
                for pool, scale in ((s["kp"], s["ks"]), (s["vp"], s["vs"])))
        base = n - m
        seen = [[j for j in range(m) if (j <= i if s["tree"] is None else int(s["tree"][b, i]) >> j & 1)]
                for i in range(m)]
        place = list(range(base)) + [base + sum(j != i for j in seen[i]) for i in range(m)]
        at = torch.tensor(place, device=DEV)
        for i in range(m):
            z = torch.einsum("hgd,htd->hgt", s["q"][b, i].double().view(h, gr, d), k) * d ** -0.5
            if c["cap"]:
                z = c["cap"] * torch.tanh(z / c["cap"])
            if c["bias"]:
                z = z - slope * (place[base + i] - at).abs()
            shut = torch.ones(n, dtype=torch.bool, device=DEV)
            shut[:base] = False
            shut[[base + j for j in seen[i]]] = False
            if c["window"]:
                shut |= place[base + i] - at >= c["window"]
            z[..., shut] = -math.inf
            norm = torch.logsumexp(z, -1)
            out[b, i] = torch.einsum("hgt,htd->hgd", torch.exp(z - norm[..., None]), v).reshape(h * gr, d)
            lse[b, i] = norm.reshape(h * gr)
    return out, lse
