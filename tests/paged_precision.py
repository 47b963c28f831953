"""What an fp32 output of the paged attention must hold to, and an emulation of its arithmetic in
which the mistakes that the bound is there for can be planted.

Errors are RMS over a call's outputs, relative to the outputs' own RMS, against 64 bits.

The bound (scores of size 1, D = 128, u = 2^-24).  A token's weight is off, independently of the
others', by
  1.9e-7  the exponent's argument, below 16: steps of 2^-20, evenly spread, times ln 2;
  1.4e-7  exp2 within 2^-22, evenly spread;
  1.4e-7  fp16 weights as two parts of 11 bits, 2^-22 (three bf16 parts: 2^-26);
  2.7e-7  the score: 8 matrix steps in chains of 2, sums of up to 32 products of size sqrt(32) < 8,
          each cut off by up to 2^-22 of 8, evenly spread, times scale = 128^-1/2;
in all 3.9e-7, and an output sum p v by the same share of itself, as the v are independent too.
What all outputs share (the sum of the weights, a block's products cut off by 2^-23, sums of blocks
and joins rounded to nearest, some sqrt(N / 3) 2.5e-8 for N blocks a warp, averaged over the warps)
adds 1 to 2e-7: 4.3e-7 for both.  Taken: 1.7 times that, 3/4 of 2^-20.  More than 8 heads a group
go in chains of 4 (64 products of size 8 < 16: 5.5e-7 for the score, 6.3e-7 in all): twice it.

Against that stand, as `emulate` shows: weights of a bf16 cache in two parts, 2.2e-6, fp16 weights in
one, 2e-4 (`plain`); blocks summed by the matrix steps themselves, which cut every sum off towards
zero, N / 4 2^-23 of a sum that grows evenly over N blocks: 1 to 3e-5 for 512 (`long_run`).  Scores in
one chain instead of four are too near to tell (4.3e-7 for 3.3e-7)."""
import numpy as np

BOUND = 0.75 * 2.0**-20
BOUND_WIDE = 2 * BOUND           # 9 to 16 heads a group


def round_to(x, bits):
    """x to `bits` significant bits, to nearest even (fp16 without its range: 11; bf16: 8; fp32: 24)."""
    m, e = np.frexp(np.asarray(x, dtype=np.float64))
    return np.ldexp(np.rint(np.ldexp(m, bits)), e - bits)


def cut(x):
    """x to 24 significant bits, towards zero: a matrix step's result."""
    m, e = np.frexp(np.asarray(x, dtype=np.float64))
    return np.ldexp(np.trunc(np.ldexp(m, 24)), e - 24)


def f32(x):
    return np.asarray(x, dtype=np.float64).astype(np.float32).astype(np.float64)


def exact(q, k, v, scale):
    """q [heads, D], k, v [n, D] of one KV head in 64 bits."""
    z = scale * (q @ k.T)
    p = np.exp(z - z.max(1, keepdims=True))
    return (p @ v) / p.sum(1, keepdims=True)


def error(got, want):
    return float(np.sqrt(np.mean((got - want) ** 2) / np.mean(want**2)))


def emulate(q, k, v, scale, bits, parts, chains=4, block_sums=True, warps=32):
    """One KV head's attention as the kernel computes it: blocks of 16 tokens dealt to warps, scores
    in `chains` chains of 16-channel matrix steps, weights in `parts` parts of `bits` bits, blocks'
    products by themselves and added with rounding to nearest (block_sums) or in one long chain."""
    g, D = q.shape
    n = len(k)
    sc = f32(scale * 1.4426950408889634)
    steps = [q[:, i:i + 16] @ k[:, i:i + 16].T for i in range(0, D, 16)]
    part = [np.zeros((g, n)) for _ in range(chains)]
    for i, s in enumerate(steps):
        part[i % chains] = cut(part[i % chains] + s)
    while len(part) > 1:
        part = [f32(a + b) for a, b in zip(part[::2], part[1::2])]
    s = part[0]
    tops, sums, outs = [], [], []
    blocks = -(-n // 16)
    for w in range(min(warps, blocks)):
        m, l, o = np.full(g, -np.inf), np.zeros(g), np.zeros((g, D))
        for j in range(w, blocks, warps):
            t = slice(16 * j, min(n, 16 * j + 16))
            top = np.maximum(m, s[:, t].max(1))
            with np.errstate(invalid="ignore"):
                move = ~((s[:, t].max(1) - m) * sc <= 3)
            new = np.where(move, top, m)
            f = np.where(move & np.isfinite(m), f32(np.exp2(f32((m - new) * sc))), np.where(move, 0.0, 1.0))
            l, o, m = f32(l * f), f32(o * f[:, None]), new
            ref = f32(12 - f32(m * sc))
            x = f32(np.exp2(f32(s[:, t] * sc + ref[:, None])))
            l = f32(l + x.sum(1))
            left, ps = x, []
            for _ in range(parts):
                ps.append(round_to(left, bits))
                left = left - ps[-1]
            if block_sums:
                acc = np.zeros((g, D))
                for p in reversed(ps):
                    acc = cut(acc + p @ v[t])
                o = f32(o + acc)
            else:
                for p in reversed(ps):
                    o = cut(o + p @ v[t])
        tops.append(f32(m * sc)), sums.append(l), outs.append(o)
    top = np.max(tops, 0)
    f = [np.exp2(t - top) for t in tops]
    return sum(o * a[:, None] for o, a in zip(outs, f)) / sum(l * a for l, a in zip(sums, f))[:, None]


# ---- inputs: q [heads, D], k, v [n, D], scale; `fit` rounds to the values of a type -------------

def plain(n, D, heads, fit, seed=0):
    """Scores of size 1, values of both signs."""
    rng = np.random.default_rng(seed)
    q, k, v = (rng.standard_normal(s) for s in ((heads, D), (n, D), (n, D)))
    return fit(q), fit(k), fit(v), D**-0.5


def long_run(n, D, heads, fit, seed=0):
    """Values around 1: sums that grow evenly over all blocks."""
    q, k, v, scale = plain(n, D, heads, fit, seed)
    return q, k, fit(1 + v / 16), scale
