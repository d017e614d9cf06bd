"""Plain 64-bit forms of the ragged-group operators, and how far a kernel's
result may be from them. CPU tensors throughout; nothing of the library.

Tolerances. A product of two stored values (8 or 11 significant bits at most)
is exact in fp32. A tensor core adds the products of one instruction and the
accumulator after aligning them to the largest, so that each of them loses at
most one unit of 2^-23 of the running magnitude, which is at most A = sum of
|terms|; fp32 additions one by one lose half of that. So a sum of K products
is within K 2^-22 A (twice the bound, for the additions that join partial
sums). The result is rounded once, by at most eps/2 of its type relative to
the value (and half its smallest subnormal)."""
import torch

E4M3 = torch.float8_e4m3fn
UNIT = {"mxfp8": 32, "block128": 128, "per_token": 16, "none": 8}


def gen(seed):
    return torch.Generator().manual_seed(seed)


def rounding(value, dtype):
    """Largest rounding error of `value` (64 bits) to `dtype`."""
    f = torch.finfo(dtype)
    return value.abs() * (f.eps / 2) + f.tiny * f.eps / 2


def group_rows(ids, groups):
    """offsets, rows, slots of ids [T, k] by going through them one by one."""
    T, k = ids.shape
    flat = ids.flatten().tolist()
    of = [[i for i, v in enumerate(flat) if v == g] for g in range(groups)] if groups * len(flat) < 1 << 22 else None
    if of is None:
        of = [[] for _ in range(groups)]
        for i, v in enumerate(flat):
            if 0 <= v < groups:
                of[v].append(i)
    offsets, rows, slots = [0], [], [-1] * len(flat)
    for g in range(groups):
        for i in of[g]:
            slots[i] = len(rows)
            rows.append(i // k)
        offsets.append(len(rows))
    rows += [-1] * (len(flat) - len(rows))
    as32 = lambda v: torch.tensor(v, dtype=torch.int32)  # noqa: E731
    return as32(offsets), as32(rows), as32(slots).view(T, k)


def ranges(offsets, S):
    """The slot ranges that offsets stand for, held to [0, S] and ascending."""
    out, prev = [], 0
    o = offsets.tolist()
    for g in range(len(o) - 1):
        lo = min(max(o[g], prev), S)
        out.append((lo, min(max(o[g + 1], lo), S)))
        prev = lo
    return out


def operands(fmt, X, G, N, K, seed, dtype=torch.bfloat16):
    """x, x_scale, w, w_scale (row-major, [G, N, K/32] for MXFP8) of a format."""
    r = gen(seed)
    if fmt == "none":
        return torch.randn(X, K, generator=r).to(dtype), None, (torch.randn(G, N, K, generator=r) / 8).to(dtype), None
    q = lambda *s: (torch.randn(*s, generator=r) * 100).clamp(-448, 448).to(E4M3).view(torch.uint8)  # noqa: E731
    x, w = q(X, K), q(G, N, K)
    if fmt == "mxfp8":
        return (x, torch.randint(117, 123, (X, K // 32), generator=r).to(torch.uint8), w,
                torch.randint(112, 116, (G, N, K // 32), generator=r).to(torch.uint8))
    if fmt == "block128":
        return (x, torch.rand(X, K // 128, generator=r) * 0.01 + 0.005, w,
                torch.rand(G, -(-N // 128), K // 128, generator=r) * 1e-3 + 1e-4)
    return x, torch.rand(X, 1, generator=r) * 0.01 + 0.005, w, torch.rand(G, N, generator=r) * 1e-3 + 1e-4


def swizzled(codes):
    """[G, N, B] E8M0 codes -> [G, N up to 128, B up to 4] holding 512-byte tiles:
    row r, column b of a 128 x 4 tile at byte (r % 32) * 16 + (r // 32) * 4 + b."""
    G, N, B = codes.shape
    Np, Bp = -(-N // 128) * 128, -(-B // 4) * 4
    full = torch.zeros(G, Np, Bp, dtype=torch.uint8)
    full[:, :N, :B] = codes
    out = torch.zeros(G, Np // 128, Bp // 4, 512, dtype=torch.uint8)
    r = torch.arange(128).view(-1, 1)
    b = torch.arange(4).view(1, -1)
    at = ((r % 32) * 16 + (r // 32) * 4 + b).flatten()
    for t in range(Np // 128):
        for c in range(Bp // 4):
            out[:, t, c, at] = full[:, t * 128:(t + 1) * 128, c * 4:(c + 1) * 4].reshape(G, -1)
    return out.view(G, Np, Bp)


def values(fmt, q, scale, N=None):
    """What stored rows stand for, in 64 bits. q [.., W, K]."""
    if fmt == "none":
        return q.double()
    v = q.view(E4M3).double()
    if fmt == "mxfp8":
        return v * (2.0 ** (scale.double() - 127)).repeat_interleave(32, -1)
    if fmt == "block128":
        s = scale.double().repeat_interleave(128, -1)
        return v * (s if N is None else s.repeat_interleave(128, -2)[..., :N, :])
    return v * (scale.double() if N is None else scale.double().unsqueeze(-1))


def grouped_gemm(fmt, x, xs, w, ws, offsets, rows, S, out, dtype):
    """(result, tolerance) in 64 bits; `out` gives what slots of no group keep."""
    G, N, K = w.shape
    res, tol = out.double().clone(), torch.zeros(S, N, dtype=torch.float64)
    xv = values(fmt, x, xs)
    for g, (a, b) in enumerate(ranges(offsets, S)):
        if a == b:
            continue
        r = torch.arange(a, b) if rows is None else rows[a:b].long()
        there = (r >= 0) & (r < x.shape[0])
        xr = torch.where(there[:, None], xv[r.clamp(0, max(0, x.shape[0] - 1))], 0.0) if x.shape[0] else torch.zeros(b - a, K, dtype=torch.float64)
        wv = values(fmt, w[g], None if ws is None else ws[g], N)
        res[a:b] = xr @ wv.T
        tol[a:b] = K * 2.0 ** -22 * (xr.abs() @ wv.abs().T) + rounding(res[a:b], dtype)
    return res, tol


def combine(y, slots, weights, dtype):
    T, k = slots.shape
    res, mag = torch.zeros(T, y.shape[1], dtype=torch.float64), torch.zeros(T, y.shape[1], dtype=torch.float64)
    for j in range(k):
        s = slots[:, j].long()
        ok = (s >= 0) & (s < y.shape[0])
        if not ok.any():
            continue
        c = 1.0 if weights is None else weights[ok, j, None].double()
        res[ok] += c * y[s[ok]].double()
        mag[ok] += (c * y[s[ok]].double()).abs()
    return res, (k + 1) * 2.0 ** -23 * mag + rounding(res, dtype)


def lora(x, a, b, y, offsets, rows, slots, scaling, S):
    """(result, tolerance). The factor v may be split into two 16-bit parts on its
    way through a tensor core: 2^-16 of |v| is lost at most (two bf16 parts of 8
    bits each), and for fp16 2^-20 of the row's largest |v|."""
    T, K = x.shape
    G, R, _ = a.shape
    res, tol = y.double().clone(), torch.zeros_like(y, dtype=torch.float64)
    for g, (lo, hi) in enumerate(ranges(offsets, S)):
        t = [(s if rows is None else int(rows[s])) for s in range(lo, hi)]
        t = [v for s, v in zip(range(lo, hi), t) if rows is None or (0 <= v < T and int(slots[v]) == s)]
        if not t:
            continue
        t = torch.tensor(t)
        xv, av, bv = x[t].double(), a[g].double(), b[g].double()
        c = 1.0 if scaling is None else float(scaling[g])
        v = xv @ av.T
        ev = K * 2.0 ** -22 * (xv.abs() @ av.abs().T) + 2.0 ** -16 * v.abs()
        if x.dtype == torch.float16:
            ev = ev + 2.0 ** -20 * v.abs().amax(1, keepdim=True)
        d = v @ bv.T
        res[t] = y[t].double() + c * d
        tol[t] = abs(c) * (ev @ bv.abs().T + R * 2.0 ** -22 * (v.abs() @ bv.abs().T)) + 2.0 ** -22 * (y[t].double().abs() + (c * d).abs())
        tol[t] += rounding(res[t].abs() + tol[t], y.dtype)
    return res, tol


def check(got, ref, tol, what=""):
    got = got.double()
    bad = ~((got - ref).abs() <= tol)
    if bad.any():
        at = bad.nonzero()[0].tolist()
        i = tuple(at)
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} off, first at {at}: {got[i]} for {ref[i]} (may be {tol[i]} off)")


# ------------------------------------------------------------------ precision of long sums
#
# The bound above grows with K for each element and cannot tell fp32 sums from
# sums kept in 11 bits once K is some thousands. Over many elements the sums
# can be told apart by how often the one rounding at the end goes the other
# way: a value whose error before it is d crosses a boundary, one of which lies
# in every step of the type, with probability |d| / step.
#
# d of fp32 sums: M = sqrt(sum of terms^2) is the size of the running sum of K
# terms of random sign. Each product loses at most a unit of 2^-23 M, with a
# random sign, together sqrt(K / 3) 2^-23 M; the accumulator, cut once an
# instruction of 16 products at least, loses half a unit each time in one
# direction, K / 16 2^-24 times the mean 2/3 M. Up to K = 8192 these are 2^-17.3
# and 2^-15.6 of M; 4 sqrt(K) 2^-23 M, 2^-14.5 there, is more than twice both.

def step(value, dtype):
    """The distance of `dtype`'s values at `value` (64 bits)."""
    f = torch.finfo(dtype)
    return f.eps * torch.exp2(torch.floor(torch.log2(value.abs().clamp(min=f.tiny))))


def spread(fmt, x, xs, w, ws, offsets, rows, S):
    """sqrt of the sum of the squared terms of every result of grouped_gemm; rows inside x."""
    G, N, K = w.shape
    out = torch.zeros(S, N, dtype=torch.float64)
    xv = values(fmt, x, xs)
    for g, (a, b) in enumerate(ranges(offsets, S)):
        if a < b:
            xr = xv[torch.arange(a, b) if rows is None else rows[a:b].long()]
            out[a:b] = ((xr ** 2) @ (values(fmt, w[g], None if ws is None else ws[g], N) ** 2).T).sqrt()
    return out


def misrounded(got, res):
    """The share of `got` that is not the 64-bit result rounded to its type."""
    return float((got != res.to(got.dtype)).double().mean())


def misrounded_limit(res, size, K, dtype):
    """What fp32 sums leave of it: the mean chance, and four standard deviations of a count of as many."""
    p = (4 * K ** 0.5 * 2.0 ** -23 * size / step(res, dtype)).clamp(max=1).mean()
    return float(p + 4 * (p / res.numel()).sqrt() + 1 / res.numel())


# ------------------------------------------------------------------ adapters whose v takes all of fp32

def exact_lora(T, R, N, K, dtype, seed):
    """x, a, b of one adapter for which every v takes 23 bits and every sum on
    the way is exact in fp32, and the 64-bit result (of y = 0): v of a pair of
    ranks differ in their last bits alone, and b takes the difference.

    x holds three digits of 7 bits, 2^8 apart, so that v = d0 + 2^-8 e1 d1 +
    2^-16 e2 d2 with e of 0 and 1 from a; all terms are multiples of 2^-16 and
    all sums below 2^7. The last two ranks have the largest |v|, 2^12 times the
    others', and nothing of it reaches y."""
    r = gen(seed)
    x = torch.zeros(T, K, dtype=torch.float64)
    at = torch.randperm(K, generator=r)[:3]
    x[:, at[0]] = torch.randint(64, 96, (T,), generator=r).double()
    x[:, at[1]] = torch.randint(64, 128, (T,), generator=r).double() * 2.0 ** -8
    x[:, at[2]] = (2 * torch.randint(32, 64, (T,), generator=r) + 1).double() * 2.0 ** -16
    a = torch.zeros(R, K, dtype=torch.float64)
    a[:, at[0]] = 1
    a[:, at[1]] = torch.randint(0, 2, (R // 2,), generator=r).double().repeat_interleave(2)
    a[0::2, at[2]] = 1                                   # of a pair, the second lacks the last digit
    a[-2:] *= 2.0 ** 12
    sign = torch.randint(-1, 2, (N, R // 2), generator=r).double()
    sign[:, -1] = 0
    b = torch.stack([sign, -sign], -1).view(N, R)
    res = (x @ a.T) @ b.T
    x, a, b = (t.to(dtype) for t in (x, a[None], b[None]))
    return x, a, b, res
