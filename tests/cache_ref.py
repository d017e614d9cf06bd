"""Plain 64-bit forms of the paged cache's operators, and how far a kernel's result may
be from them. CPU tensors throughout; nothing of the library.

Rotation. The angle is exact to 2^-32 of a turn, then rounded to fp32 (half a unit of 2^-24
of half a turn at most, pi 2^-25 radians); cosine and sine are off by 2 units of 2^-24 at most. Together
under 2^-22. Two products and their sum in fp32 add 3 2^-24 of each term. So a rotated value is within
2^-21 factor (|a| + |b|) of its own, before it is rounded.

E4M3 rows. q = E4M3(src / s): the nearest of E4M3's values, so q s is within half a step of
src: 2^-4 |src| or, below E4M3's normal range, 2^-10 s; the quotient's and the scale's own
roundings add 2^-22 |src|.

Attention. S is a sum of D products, within D 2^-22 of the sum of their sizes (the bound of grouped
products); beside E4M3 rows a bf16 q has 11 bits and an exponent a head: it loses 2^-24 of the
head's largest |q| at most, for each value. The factors of S and the difference from the
running maximum, in units of log2 p, add 2^-22 of |x| each, exp2 2^-21 of p. So p is within d of
itself, d = all these, and the quotient of two sums within 2 d of the sum of p |v|, A. p's parts keep
2^-18 of it (bf16, two), 2^-22 (fp16, two) or 2^-12 (fp16, one), and 2^-24 of the largest w = p times scale
for each row where they are fp16. A tensor core's instruction adds 16 products
and the accumulator, each cut to a unit of 2^-23 of the running magnitude: 17 of
them for every 16 tokens and part, in a quarter of the warps' tokens each."""
import math

import torch

from group_ref import check, gen, rounding, step  # noqa: F401

E4M3 = torch.float8_e4m3fn
BF16, F16, F64 = torch.bfloat16, torch.float16, torch.float64


def turns(R, base=10000.0, seed=None):
    """Frequencies of R/2 pairs in 2^-64 of a turn: powers of a base, or any 64 bits."""
    if seed is not None:
        return torch.randint(-(1 << 63), (1 << 63) - 1, (R // 2,), generator=gen(seed))
    return torch.tensor([int(base ** (-2 * i / R) / (2 * math.pi) * 2.0 ** 64) for i in range(R // 2)], dtype=torch.int64)


def rope(x, positions, freqs, layout="half", factor=1.0, inverse=False):
    """(rotated heads [T, H, D], how far from them fp32 may be before rounding)."""
    R, h = 2 * len(freqs), len(freqs)
    whole = 1 << 64
    part = [[(p * f) % whole / whole for f in freqs.tolist()] for p in positions.tolist()]
    angle = 2 * math.pi * torch.tensor(part, dtype=F64).view(len(positions), 1, h) * (-1 if inverse else 1)
    y, tol = x.double().clone(), torch.zeros_like(x, dtype=F64)
    at = torch.arange(h)
    first, second = (at, at + h) if layout == "half" else (2 * at, 2 * at + 1)
    a, b = y[..., first].clone(), y[..., second].clone()
    factor = float(torch.tensor(factor, dtype=torch.float32))
    y[..., first], y[..., second] = factor * (a * angle.cos() - b * angle.sin()), factor * (a * angle.sin() + b * angle.cos())
    size = 2.0 ** -21 * abs(factor) * (a.abs() + b.abs())
    tol[..., first], tol[..., second] = size, size
    return y, tol


def fp8(v):
    return v.view(E4M3).double()


def quantised(rows, tol=0.0):
    """(values, tolerance) that E4M3 rows with a scale each may stand for."""
    s = rows.abs().amax(-1, keepdim=True) / 448
    return rows, rows.abs() * (2.0 ** -4 + 2.0 ** -20) + s * 2.0 ** -10 + 2 * torch.as_tensor(tol)


def pool(kind, pages, heads, P, D, dtype, seed, order="head"):
    """A cache with random rows: k, v [pages, heads, P, D] and their scales (or None)."""
    r = gen(seed)
    out = []
    for _ in range(2):
        shape = (pages, heads, P, D) if order == "head" else (pages, P, heads, D)
        t = torch.randn(shape, generator=r)
        t = t.to(dtype) if kind == "none" else (t * 100).clamp(-448, 448).to(E4M3).view(torch.uint8)
        out.append(t if order == "head" else t.transpose(1, 2))
    scales = [0.005 + 0.02 * torch.rand(pages, heads, P, generator=r) if kind != "none" else None for _ in range(2)]
    return out[0], out[1], scales[0], scales[1]


def rows_at(cache, scale, page, place):
    """Rows [n, heads, D] in 64 bits."""
    v = cache[page, :, place]
    return v.double() if scale is None else fp8(v) * scale[page, :, place].double().unsqueeze(-1)


def tokens(b, table, lengths, window, pages, P):
    """The tokens of sequence b that are not masked."""
    n = min(max(int(lengths[b]), 0), table.shape[1] * P)
    t = torch.arange(max(0, n - window) if window else 0, n)
    page = table[b, t // P].long()
    ok = (page >= 0) & (page < pages)
    return page[ok], (t % P)[ok]


def attention(q, k, v, ks, vs, table, lengths, scale=None, window=0, sinks=None):
    """(out, its tolerance, lse, its tolerance) in 64 bits."""
    B, Hq, D = q.shape
    pages, heads, P, _ = k.shape
    g = Hq // heads
    scale = float(torch.tensor(D ** -0.5 if scale is None else scale, dtype=torch.float32))
    out, tol = torch.zeros(B, Hq, D, dtype=F64), torch.zeros(B, Hq, D, dtype=F64)
    lse, ltol = torch.full((B, Hq), -math.inf, dtype=F64), torch.zeros(B, Hq, dtype=F64)
    parts, kept, floor = {(False, BF16): (2, 2.0 ** -18, 0.0), (False, F16): (2, 2.0 ** -22, 2.0 ** -24), (True, BF16): (1, 2.0 ** -12, 2.0 ** -24),
                          (True, F16): (2, 2.0 ** -22, 2.0 ** -24)}[(ks is not None, q.dtype)]
    for b in range(B):
        page, place = tokens(b, table, lengths, window, pages, P)
        n = len(page)
        if n == 0:
            if sinks is not None:
                lse[b], ltol[b] = sinks.double(), 2.0 ** -21 * sinks.double().abs()
            continue
        kk, vv = rows_at(k, ks, page, place).transpose(0, 1), rows_at(v, vs, page, place).transpose(0, 1)   # [heads, n, D]
        sc = torch.ones(heads, n, dtype=F64) if vs is None else vs[page, :, place].double().T
        qq = q[b].double().view(heads, g, D)
        x = scale * (qq @ kk.transpose(1, 2))
        size = abs(scale) * (qq.abs() @ kk.abs().transpose(1, 2))
        off = D * 2.0 ** -22 * size
        if ks is not None and q.dtype == BF16:
            off = off + abs(scale) * 2.0 ** -24 * qq.abs().amax(-1, keepdim=True) * kk.abs().sum(-1).unsqueeze(1)
        m = x.amax(-1, keepdim=True)
        sink = None if sinks is None else sinks.double().view(heads, g, 1)
        if sink is not None:
            m = torch.maximum(m, sink)
        p = (x - m).exp()
        total = p.sum(-1, keepdim=True) + (0 if sink is None else (sink - m).exp())
        d = off + 4 * 2.0 ** -22 * (x.abs() + m.abs()) * 1.4427 + 2.0 ** -21
        p = p / total
        # what a token's own error can do: its p, and its share of the sum
        dm = (p * d).sum(-1, keepdim=True) + (n / 32 + 64) * 2.0 ** -24
        A = p @ vv.abs()
        o = p @ vv
        t = (p * d) @ vv.abs() + dm * A + kept * A + ((n / 64 + 8) * 17 * parts) * 2.0 ** -23 * A
        w = p * sc.unsqueeze(1)
        t = t + 2 * floor * w.amax(-1, keepdim=True) * (vv.abs() / sc.clamp(min=2.0 ** -140).unsqueeze(-1)).sum(1).unsqueeze(1)
        out[b], tol[b] = o.reshape(Hq, D), t.reshape(Hq, D)
        lse[b] = (m + total.log()).reshape(Hq)
        ltol[b] = (dm + 2.0 ** -21 * (m + total.log()).abs() + 2.0 ** -21).reshape(Hq)
    tol = tol + rounding(out.abs() + tol, q.dtype)
    return out, tol, lse, ltol


def off_by_rounding(got, ref):
    """The size of got - ref over that of one rounding to got's type: a step's error spread evenly over half of it on both sides."""
    return float((got.double() - ref).square().mean().sqrt() / (step(ref, got.dtype).square() / 12).mean().sqrt())


def table_of(lengths, P, width=None, seed=0, spare=3):
    """Pages in any order for sequences of these lengths, -1 behind them; (table [B, width], pages of the cache)."""
    need = [-(-max(0, n) // P) for n in lengths]
    width = max(need + [0]) if width is None else width
    ids = torch.randperm(sum(need) + spare, generator=gen(seed)).to(torch.int32)
    table, at = torch.full((len(lengths), width), -1, dtype=torch.int32), 0
    for b, n in enumerate(need):
        table[b, :n] = ids[at:at + n]
        at += n
    return table, len(ids)
