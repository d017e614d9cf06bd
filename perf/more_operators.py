"""A paged key-value cache between the library's rows: the cases that are measured, their plain
forms in elementary torch operations and their definitions in 64 bits.

Four operators:
  rope    rotary positions on heads, two orders of pairs, part of a head, scaled for long contexts
  write   rotated keys, and values, into the cache's rows (16 bits, or E4M3 with a scale a row), queries rotated beside them
  read    rows of the cache back as 16-bit values
  attend  attention of one new token a sequence over its pages

A row is one head of one token. A cache holds [pages, heads, page size, D]; slot = page * page size + place in it.
"""
import math

import torch

own = False

DEV = "cuda"
BF16, F16, F32, F64 = torch.bfloat16, torch.float16, torch.float32, torch.float64
E4M3 = torch.float8_e4m3fn


def listed():
    return [
        # Queries of a decode step of 64 requests, where latency counts; contexts up to 131072.
        {"name": "rope 64x32x128", "op": "rope", "T": 64, "H": 32, "D": 128, "R": 128, "layout": "half", "far": 131072, "stretch": 1.0, "dtype": "bf16"},
        # A prefill batch, half of each head rotated in interleaved pairs, a context stretched to a million.
        {"name": "rope 16384x40x128 r64", "op": "rope", "T": 16384, "H": 40, "D": 128, "R": 64, "layout": "interleaved", "far": 1 << 20, "stretch": 32.0, "dtype": "fp16"},
        # A decode step's new rows: q rotated, k rotated and written, v written, from one fused projection.
        {"name": "write 64 bf16", "op": "write", "fmt": "none", "T": 64, "Hq": 32, "Hkv": 8, "D": 128, "R": 128, "layout": "half", "far": 131072, "stretch": 1.0,
         "P": 16, "order": "head", "dtype": "bf16", "skipped": 0.0},
        # A prefill batch's rows quantised as they are written, and read back for the batch's own attention.
        {"name": "write+read 8192 fp8", "op": "write", "fmt": "per_token", "T": 8192, "Hq": 32, "Hkv": 8, "D": 128, "R": 128, "layout": "half", "far": 131072, "stretch": 16.0,
         "P": 64, "order": "head", "dtype": "bf16", "skipped": 0.0},
        # A padded batch of odd size into a cache that keeps a token's heads side by side.
        {"name": "write 4099x2x80 fp16", "op": "write", "fmt": "none", "T": 4099, "Hq": 14, "Hkv": 2, "D": 80, "R": 32, "layout": "half", "far": 32768, "stretch": 1.0,
         "P": 16, "order": "token", "dtype": "fp16", "skipped": 0.1},
        # A short prefix of a quantised cache, for one request's next chunk; some slots are not there.
        {"name": "read 777x4x192 fp8", "op": "read", "fmt": "per_token", "S": 777, "Hkv": 4, "D": 192, "P": 16, "order": "head", "dtype": "fp16", "skipped": 0.05},
        # The prefix of a long request, for a library's prompt attention.
        {"name": "read 131072x8x128 fp8", "op": "read", "fmt": "per_token", "S": 131072, "Hkv": 8, "D": 128, "P": 64, "order": "head", "dtype": "bf16", "skipped": 0.0},
        # One request early in its answer: the smallest call of a serving loop.
        {"name": "attend 1x700 bf16", "op": "attend", "fmt": "none", "B": 1, "L": 700, "least": 1.0, "Hq": 32, "Hkv": 8, "D": 128, "P": 16, "order": "head", "dtype": "bf16",
         "window": 0, "sinks": False, "empty": 0.0},
        # A decode batch of unlike requests, some of its rows padding.
        {"name": "attend 64x4096 bf16", "op": "attend", "fmt": "none", "B": 64, "L": 4096, "least": 0.05, "Hq": 32, "Hkv": 8, "D": 128, "P": 16, "order": "head", "dtype": "bf16",
         "window": 0, "sinks": False, "empty": 0.05},
        # Long contexts on a quantised cache: the largest, bound by reading it.
        {"name": "attend 8x131072 fp8", "op": "attend", "fmt": "per_token", "B": 8, "L": 131072, "least": 0.7, "Hq": 64, "Hkv": 8, "D": 128, "P": 64, "order": "head", "dtype": "bf16",
         "window": 0, "sinks": False, "empty": 0.0},
        # A layer with a window of 128 tokens and a sink a head: little to read of long sequences.
        {"name": "attend 96x8192 window", "op": "attend", "fmt": "none", "B": 96, "L": 8192, "least": 0.01, "Hq": 64, "Hkv": 8, "D": 64, "P": 16, "order": "token", "dtype": "bf16",
         "window": 128, "sinks": True, "empty": 0.0},
        # Odd sizes: seven queries a head, a narrow head, pages that no tile fits.
        {"name": "attend 33x5001 fp8 odd", "op": "attend", "fmt": "per_token", "B": 33, "L": 5001, "least": 0.0, "Hq": 21, "Hkv": 3, "D": 80, "P": 20, "order": "head", "dtype": "fp16",
         "window": 0, "sinks": False, "empty": 0.1},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("rope", "write", "write", "read", "attend", "attend", "attend", "attend"))
    fmt = rng.choice(("none", "per_token"))
    D = rng.choice((64, 80, 96, 112, 128, 128, 192, 256))
    R = 16 * rng.randint(1, D // 16)
    turn = {"R": R, "layout": rng.choice(("half", "interleaved")), "far": _log(rng, 1000, 1 << 20), "stretch": rng.choice((1.0, 8.0))}
    page = {"P": rng.choice((1, 8, 16, 16, 20, 32, 64, 128)), "order": rng.choice(("head", "token")), "dtype": rng.choice(("bf16", "fp16"))}
    if op == "rope":
        return {"op": op, "T": _log(rng, 1, 16384), "H": rng.randint(1, 40), "D": D if D < 192 else 128, **turn, "R": min(R, 128 if D >= 192 else D), "dtype": page["dtype"]}
    if op == "write":
        Hkv = rng.randint(1, 8)
        return {"op": op, "fmt": fmt, "T": _log(rng, 1, 8192), "Hq": Hkv * rng.randint(1, 8), "Hkv": Hkv, "D": D, **turn, **page, "skipped": rng.choice((0.0, 0.1))}
    if op == "read":
        return {"op": op, "fmt": fmt, "S": _log(rng, 1, 65536), "Hkv": rng.randint(1, 8), "D": D, **page, "skipped": rng.choice((0.0, 0.1))}
    Hkv, B = rng.randint(1, 8), _log(rng, 1, 128)
    return {"op": op, "fmt": fmt, "B": B, "L": min(_log(rng, 1, 131072), max(1, 196608 // B)), "least": rng.choice((0.0, 0.5, 1.0)), "Hq": Hkv * rng.choice((1, 2, 3, 4, 5, 7, 8, 16)),
            "Hkv": Hkv, "D": D, **page, "window": rng.choice((0, 0, 100, 1024)), "sinks": rng.random() < 0.3, "empty": rng.choice((0.0, 0.1))}


def _dtype(name):
    return {"bf16": BF16, "fp16": F16}[name]


# ------------------------------------------------------------------------------------ inputs


def _frequencies(R, stretch, base=500000.0, trained=8192, fast=32.0, slow=1.0):
    """Radians a position of the R/2 pairs, slow pairs stretched for a context longer than the trained one, and the factor on the result that goes with it."""
    inv = [base ** (-2 * i / R) for i in range(R // 2)]
    if stretch == 1.0:
        return inv, 1.0
    at = lambda turns: R * math.log(trained / (turns * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
    lo, hi = max(0, math.floor(at(fast))), min(R - 1, math.ceil(at(slow)))
    slowness = [min(1.0, max(0.0, (i - lo) / max(hi - lo, 0.001))) for i in range(R // 2)]
    return [f * (1 - s) + f / stretch * s for f, s in zip(inv, slowness)], 0.1 * math.log(stretch) + 1


def _turns(inv):
    """The same in 2^-64 of a turn, as an operator takes them."""
    return torch.tensor([int(f / (2 * math.pi) * 2.0 ** 64) for f in inv], dtype=torch.int64, device=DEV)


def _angles(s, gen):
    c = s["case"]
    inv, s["factor"] = _frequencies(c["R"], c["stretch"])
    s["inv"], s["turns"] = torch.tensor(inv, dtype=F64, device=DEV), _turns(inv)
    s["positions"] = torch.randint(0, c["far"], (c["T"],), generator=gen, device=DEV)


def _normal(gen, shape, dtype, scale=1.0):
    return torch.randn(shape, dtype=dtype, generator=gen, device=DEV).mul_(scale)


def _pool(gen, c, pages):
    """A cache of `pages` pages with what earlier requests have left in it, [pages, heads, page size, D]."""
    shape = (pages, c["Hkv"], c["P"], c["D"])
    laid = shape if c["order"] == "head" else (pages, c["P"], c["Hkv"], c["D"])
    pool = {}
    for name in ("k", "v"):
        t = _normal(gen, laid, _dtype(c["dtype"]))
        if c["fmt"] != "none":
            t = t.mul_(100).clamp_(-448, 448).to(E4M3).view(torch.uint8)
        pool[name] = t if c["order"] == "head" else t.transpose(1, 2)
        pool[name + "_scale"] = 0.01 * (1 + torch.rand(shape[:3], generator=gen, device=DEV)) if c["fmt"] != "none" else None
    return pool


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    c, s = case, {"case": case}
    op = c["op"]
    if op == "rope":
        _angles(s, gen)
        s["x"] = _normal(gen, (c["T"], c["H"], c["D"]), _dtype(c["dtype"]))
        return s
    if op in ("write", "read"):
        n = c["T"] if op == "write" else c["S"]
        step = op == "write" and n <= 256
        pages = (n if step else -(-n // c["P"])) + 7
        s.update(_pool(gen, c, pages))
        order = torch.randperm(pages, generator=gen, device=DEV)
        if step:                                                     # a token of each request, in the last page that it has
            slots = order[:n] * c["P"] + torch.randint(0, c["P"], (n,), generator=gen, device=DEV)
        else:                                                        # pages in any order, a request's tokens side by side in them
            slots = (order[:, None] * c["P"] + torch.arange(c["P"], device=DEV)).flatten()[:n]
        s["slots"] = torch.where(torch.rand(n, generator=gen, device=DEV) < c["skipped"], -1, slots).to(torch.int32)
        if op == "write":
            _angles(s, gen)
            qkv = _normal(gen, (n, c["Hq"] + 2 * c["Hkv"], c["D"]), _dtype(c["dtype"]))
            s["q"], s["new_k"], s["new_v"] = qkv.split((c["Hq"], c["Hkv"], c["Hkv"]), dim=1)
        return s
    B, L, P = c["B"], c["L"], c["P"]
    some = c["least"] + (1 - c["least"]) * torch.rand(B, generator=gen, device=DEV)
    lengths = (some * L).ceil().clamp(min=1).to(torch.int32)
    s["lengths"] = torch.where(torch.rand(B, generator=gen, device=DEV) < c["empty"], 0, lengths)
    width = -(-L // P)
    s.update(_pool(gen, c, B * width))
    table = torch.randperm(B * width, generator=gen, device=DEV).to(torch.int32).view(B, width)
    s["pages"] = torch.where(torch.arange(width, device=DEV) * P < s["lengths"][:, None], table, -1)
    s["q"] = _normal(gen, (B, c["Hq"], c["D"]), _dtype(c["dtype"]), 2.0)
    s["sinks"] = _normal(gen, (c["Hq"],), F32) if c["sinks"] else None
    s["scale"] = 1 / math.sqrt(c["D"])
    return s


# ------------------------------------------------------------------------------------ plain forms


def _turned(x, s):
    """Rotated rows [T, H, D], in 32 bits (the angles of far positions in 64)."""
    c = s["case"]
    R, h = c["R"], c["R"] // 2
    angle = s["positions"].double()[:, None] * s["inv"]
    cos, sin = ((t * s["factor"]).float().unsqueeze(1) for t in (angle.cos(), angle.sin()))
    x = x.float()
    a, b = (x[..., :h], x[..., h:R]) if c["layout"] == "half" else (x[..., 0:R:2], x[..., 1:R:2])
    u, w = a * cos - b * sin, a * sin + b * cos
    y = torch.cat((u, w), -1) if c["layout"] == "half" else torch.stack((u, w), -1).flatten(-2)
    return torch.cat((y, x[..., R:]), -1)


def _rows(pool, scale, slots, P):
    """The values of a cache's rows at slots, [S, heads, D] in 32 bits."""
    page, place = slots.long().clamp(min=0) // P, slots.long().clamp(min=0) % P
    v = pool.transpose(1, 2)[page, place]
    if scale is not None:
        return v.view(E4M3).float() * scale.transpose(1, 2)[page, place].unsqueeze(-1)
    return v.float()


def _plain_read(s):
    c = s["case"]
    there = (s["slots"] >= 0).view(-1, 1, 1)
    out = [torch.where(there, _rows(s[n], s[n + "_scale"], s["slots"], c["P"]), 0.0).to(_dtype(c["dtype"])) for n in ("k", "v")]
    return {"k": out[0], "v": out[1]}


def _put(pool, scale, rows, slots, P):
    """Rows [T, heads, D] of 32 bits into the cache at slots, rounded once."""
    at = (slots >= 0).nonzero().flatten()
    page, place = slots[at].long() // P, slots[at].long() % P
    rows = rows[at]
    if scale is not None:
        sc = rows.abs().amax(-1, keepdim=True) / 448
        rows = torch.where(sc > 0, rows / sc, 0.0).clamp(-448, 448).to(E4M3).view(torch.uint8)
        scale.transpose(1, 2)[page, place] = sc.squeeze(-1)
    pool.transpose(1, 2)[page, place] = rows.to(pool.dtype)


def _plain_write(s):
    c = s["case"]
    q = _turned(s["q"], s).to(s["q"].dtype)
    _put(s["k"], s["k_scale"], _turned(s["new_k"], s), s["slots"], c["P"])
    _put(s["v"], s["v_scale"], s["new_v"].float(), s["slots"], c["P"])
    return {"q": q, **({"k": s["k"], "v": s["v"]} if c["fmt"] == "none" else _plain_read(s))}


def _plain_attend(s):
    c = s["case"]
    B, g = c["B"], c["Hq"] // c["Hkv"]
    pages = s["pages"].long().clamp(min=0)
    values = lambda n: (s[n][pages].view(E4M3).float() * s[n + "_scale"][pages].unsqueeze(-1)  # noqa: E731
                        if s[n + "_scale"] is not None else s[n][pages].float()).transpose(1, 2).flatten(2, 3)   # [B, heads, tokens, D]
    t = torch.arange(pages.shape[1] * c["P"], device=DEV)
    n = s["lengths"].unsqueeze(1)
    there = (t < n) & ((t >= n - c["window"]) if c["window"] else True)
    q = s["q"].float().view(B, c["Hkv"], g, c["D"])
    x = torch.matmul(q, values("k").transpose(2, 3)) * s["scale"]
    x = torch.where(there[:, None, None], x, -math.inf)
    m = x.amax(-1, keepdim=True)
    if s["sinks"] is not None:
        sink = s["sinks"].view(1, c["Hkv"], g, 1)
        m = torch.maximum(m, sink)
    p = torch.exp(x - torch.where(m > -math.inf, m, 0.0))
    total = p.sum(-1, keepdim=True) + (torch.exp(sink - m) if s["sinks"] is not None else 0.0)
    out = torch.matmul(p, values("v")) / torch.where(total > 0, total, 1.0)
    return {"out": out.view(B, c["Hq"], c["D"]).to(s["q"].dtype), "lse": (m + torch.log(total)).view(B, c["Hq"])}


def run(state):
    s, c = state, state["case"]
    op = c["op"]
    if own:
        import swiglu_fp8_activation_gb300 as sgq
        if op == "rope":
            return sgq.rope(s["x"], s["positions"], s["turns"], layout=c["layout"], factor=s["factor"])
        scales = {"fmt": c["fmt"], "k_scale": s["k_scale"], "v_scale": s["v_scale"]}
        if op == "attend":
            out, lse = sgq.paged_attention(s["q"], s["k"], s["v"], s["pages"], s["lengths"], scale=s["scale"], window=c["window"], sinks=s["sinks"], lse=True, **scales)
            return {"out": out, "lse": lse}
        if op == "read":
            k, v = sgq.cache_read(s["k"], s["v"], s["slots"], dtype=_dtype(c["dtype"]), **scales)
            return {"k": k, "v": v}
        q = sgq.cache_write(s["new_k"], s["new_v"], s["k"], s["v"], s["slots"], q=s["q"], positions=s["positions"], freqs=s["turns"], layout=c["layout"], factor=s["factor"], **scales)
        if c["fmt"] == "none":
            return {"q": q, "k": s["k"], "v": s["v"]}
        k, v = sgq.cache_read(s["k"], s["v"], s["slots"], dtype=_dtype(c["dtype"]), **scales)
        return {"q": q, "k": k, "v": v}
    return {"rope": lambda s: _turned(s["x"], s).to(s["x"].dtype), "write": _plain_write, "read": _plain_read, "attend": _plain_attend}[op](s)


# ------------------------------------------------------------------------------------ definitions in 64 bits


def _rotation(x, s):
    """Every pair as a complex number, times factor e^(i position frequency)."""
    c, y = s["case"], x.double().clone()
    R, h = c["R"], c["R"] // 2
    at = torch.arange(h, device=DEV)
    first, second = (at, at + h) if c["layout"] == "half" else (2 * at, 2 * at + 1)
    z = torch.complex(y[..., first], y[..., second])
    z = z * torch.polar(torch.full_like(s["inv"], s["factor"]).expand(c["T"], h), s["positions"].double().outer(s["inv"])).unsqueeze(1)
    y[..., first], y[..., second] = z.real, z.imag
    return y


def _quantised(rows):
    """What E4M3 rows with one 32-bit scale, a 448th of the largest value, stand for: the nearest value of each, even digits where two are as near.
    The scale and the quotient by it are 32-bit values by definition."""
    sc = (rows.abs().amax(-1, keepdim=True) / 448).float().double()
    v = torch.where(sc > 0, rows / sc, 0.0).float().double()
    step = 2.0 ** (torch.frexp(v).exponent.double() - 4).clamp(min=-9)
    return ((v / step).round() * step).clamp(-448, 448) * sc


def exact(case, seed):
    s, c = prepare(case, seed), case
    op = c["op"]
    if op == "rope":
        return _rotation(s["x"], s)
    if op == "write":
        out = {"q": _rotation(s["q"], s)}
        slots = s["slots"].long()
        for name, rows in (("k", _rotation(s["new_k"], s)), ("v", s["new_v"].double())):
            if c["fmt"] == "none":
                full = s[name].double()
                t = (slots >= 0).nonzero().flatten()
                full[slots[t] // c["P"], :, slots[t] % c["P"]] = rows[t]
                out[name] = full
            else:
                out[name] = _quantised(rows) * (slots >= 0).view(-1, 1, 1)
        return out
    if op == "read":
        out = {}
        for name in ("k", "v"):
            rows = torch.zeros(c["S"], c["Hkv"], c["D"], dtype=F64, device=DEV)
            t = (s["slots"] >= 0).nonzero().flatten()
            page, place = s["slots"][t].long() // c["P"], s["slots"][t].long() % c["P"]
            for h in range(c["Hkv"]):
                v = s[name][:, h][page, place]
                rows[t, h] = v.double() if c["fmt"] == "none" else v.view(E4M3).double() * s[name + "_scale"][:, h][page, place].double()[:, None]
            out[name] = rows
        return out
    g = c["Hq"] // c["Hkv"]
    out = torch.zeros(c["B"], c["Hq"], c["D"], dtype=F64, device=DEV)
    lse = torch.full((c["B"], c["Hq"]), -math.inf, dtype=F64, device=DEV)
    lengths = s["lengths"].tolist()
    for b, n in enumerate(lengths):
        lo = max(0, n - c["window"]) if c["window"] else 0
        t = torch.arange(lo, n, device=DEV)
        page, place = s["pages"][b].long()[t // c["P"]], t % c["P"]
        for h in range(c["Hkv"]):
            k, v = ((s[m][:, h][page, place].double() if c["fmt"] == "none" else
                     s[m][:, h][page, place].view(E4M3).double() * s[m + "_scale"][:, h][page, place].double()[:, None]) for m in ("k", "v"))
            heads = slice(h * g, (h + 1) * g)
            x = s["scale"] * (s["q"][b, heads].double() @ k.T)
            if s["sinks"] is not None:
                x = torch.cat((x, s["sinks"][heads].double()[:, None]), 1)
                v = torch.cat((v, torch.zeros(1, c["D"], dtype=F64, device=DEV)))
            if x.shape[1]:
                lse[b, heads] = torch.logsumexp(x, 1)
                out[b, heads] = torch.softmax(x, 1) @ v
    return {"out": out, "lse": lse}


# ------------------------------------------------------------------------------------ what a pass cannot do without


def work(case):
    c = case
    if c["op"] == "rope":
        n = c["T"] * c["H"]
        return {"bytes": 4 * n * c["D"] + 8 * c["T"], "flops": 3 * n * c["R"]}
    row = 2 * c["D"] if c["fmt"] == "none" else c["D"] + 4
    if c["op"] == "write":
        n = 2 * c["T"] * c["Hkv"] * (1 - c["skipped"])
        moved = 4 * c["T"] * c["Hq"] * c["D"] + n * (2 * c["D"] + row) + 12 * c["T"]
        if c["fmt"] != "none":
            moved += n * row + 4 * c["T"] * c["Hkv"] * c["D"]
        return {"bytes": moved, "flops": 3 * c["T"] * (c["Hq"] + c["Hkv"]) * c["R"] + 2 * n * c["D"]}
    if c["op"] == "read":
        n = 2 * c["S"] * c["Hkv"]
        return {"bytes": n * (1 - c["skipped"]) * row + 2 * n * c["D"] + 4 * c["S"], "flops": n * c["D"]}
    mean = c["L"] * (1 + c["least"]) / 2
    if c["window"]:                                                  # of lengths spread evenly from least * L to L
        lo, w = c["least"] * c["L"], c["window"]
        mean = w if lo >= w else (mean if c["L"] <= w else ((w * w - lo * lo) / 2 + (c["L"] - w) * w) / max(1e-9, c["L"] - lo))
    tokens = c["B"] * (1 - c["empty"]) * mean
    return {"bytes": 2 * tokens * c["Hkv"] * row + 4 * c["B"] * c["Hq"] * (c["D"] + 1) + 4 * tokens / c["P"], "flops": 4 * tokens * c["Hq"] * c["D"]}
