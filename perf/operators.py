"""The ragged products that read the library's rows, and what stands around them: the cases that
are measured, their plain forms in elementary torch operations and their definitions in 64 bits.

Four operators:
  group    group ids of tokens -> offsets, token of every slot in group order, slot of every id
  gemm     matrix products grouped by expert: out[s] = x[rows[s]] . w[g]^T, FP8 (three formats) or 16 bits
  combine  the weighted sum of the k expert rows of every token
  lora     low-rank adapters of many requests, added in place to a shared projection's output
"""
import math

import torch

own = False

DEV = "cuda"
BF16, F16, F32, F64 = torch.bfloat16, torch.float16, torch.float32, torch.float64
E4M3 = torch.float8_e4m3fn
#: Multiple that the contraction's length has in each format.
UNIT = {"mxfp8": 32, "block128": 128, "per_token": 16, "bf16": 8, "fp16": 8}


def listed():
    return [
        # One decode step of 64 requests, 8 of 128 experts each: the routing of a layer, where latency counts.
        {"name": "group 64x8 of 128", "op": "group", "T": 64, "k": 8, "G": 128, "dropped": 0.0},
        # The routing of a 16384-token prefill batch, with some ids that another rank's experts own (-1).
        {"name": "group 16384x8 of 160", "op": "group", "T": 16384, "k": 8, "G": 160, "dropped": 0.05},
        # Gate-and-up product of one request's token: the smallest call of a serving loop, bound by eight experts' weights.
        {"name": "gemm mxfp8 decode 1x8", "op": "gemm", "fmt": "mxfp8", "T": 1, "k": 8, "G": 64, "N": 1536, "K": 6144, "gather": True},
        # Gate-and-up product of a decode batch of 64: nearly every expert has a few rows, bound by reading all weights.
        {"name": "gemm mxfp8 decode 64x8", "op": "gemm", "fmt": "mxfp8", "T": 64, "k": 8, "G": 64, "N": 4096, "K": 4096, "gather": True},
        # Gate-and-up product of a prefill batch: the largest, bound by the tensor cores.
        {"name": "gemm mxfp8 prefill 8192x4", "op": "gemm", "fmt": "mxfp8", "T": 8192, "k": 4, "G": 32, "N": 4096, "K": 6144, "gather": True},
        # Down product of a 1x128-quantised activation on block-scaled weights, a chunk of a prefill.
        {"name": "gemm block128 2048x8", "op": "gemm", "fmt": "block128", "T": 2048, "k": 8, "G": 32, "N": 4096, "K": 1536, "gather": False},
        # Per-token rows on per-channel weights at odd sizes: a ragged batch, widths that fill no tile.
        {"name": "gemm per_token 333x3 odd", "op": "gemm", "fmt": "per_token", "T": 333, "k": 3, "G": 7, "N": 1544, "K": 2096, "gather": True},
        # 16-bit experts of an unquantised layer.
        {"name": "gemm bf16 4096x2", "op": "gemm", "fmt": "bf16", "T": 4096, "k": 2, "G": 8, "N": 4096, "K": 2048, "gather": True},
        # The end of an expert layer in a decode step.
        {"name": "combine 64x8 x4096", "op": "combine", "T": 64, "k": 8, "N": 4096, "dtype": "bf16", "dropped": 0.0},
        # The end of an expert layer in a prefill batch; some rows were other ranks' to compute.
        {"name": "combine 8192x8 x6144", "op": "combine", "T": 8192, "k": 8, "N": 6144, "dtype": "bf16", "dropped": 0.05},
        # A decode step of 64 requests on 32 adapters beside an output projection.
        {"name": "lora 64 of 32 r16", "op": "lora", "T": 64, "L": 32, "R": 16, "K": 4096, "N": 4096, "dtype": "bf16", "dropped": 0.1},
        # A prefill batch of 8 requests beside a gate-and-up projection, a rank that fills a tile.
        {"name": "lora 8192 of 8 r64", "op": "lora", "T": 8192, "L": 8, "R": 64, "K": 4096, "N": 8192, "dtype": "bf16", "dropped": 0.0},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("group", "gemm", "gemm", "gemm", "combine", "lora", "lora"))
    if op == "group":
        return {"op": op, "T": _log(rng, 1, 16384), "k": rng.randint(1, 8), "G": rng.randint(1, 320), "dropped": rng.choice((0.0, 0.1, 1.0))}
    if op == "combine":
        return {"op": op, "T": _log(rng, 1, 8192), "k": rng.randint(1, 8), "N": 8 * _log(rng, 8, 768), "dtype": rng.choice(("bf16", "fp16")), "dropped": rng.choice((0.0, 0.1))}
    if op == "lora":
        return {"op": op, "T": _log(rng, 1, 8192), "L": _log(rng, 1, 32), "R": 8 * rng.randint(1, 16), "K": 8 * _log(rng, 32, 512), "N": 8 * _log(rng, 32, 512),
                "dtype": rng.choice(("bf16", "fp16")), "dropped": rng.choice((0.0, 0.3))}
    fmt = rng.choice(tuple(UNIT))
    G = _log(rng, 1, 48)
    return {"op": op, "fmt": fmt, "T": _log(rng, 1, 4096), "k": rng.randint(1, min(8, G)), "G": G, "N": 8 * _log(rng, 8, 320),
            "K": UNIT[fmt] * max(1, _log(rng, 128, 4096) // UNIT[fmt]), "gather": rng.random() < 0.5}


def _dtype(name):
    return {"bf16": BF16, "fp16": F16}[name]


# ------------------------------------------------------------------------------------ inputs


def _route(gen, T, k, G):
    """k different groups of G for each token, some groups in more demand than others."""
    want = torch.randn(T, G, generator=gen, device=DEV) + 0.7 * torch.randn(1, G, generator=gen, device=DEV)
    return want.topk(min(k, G), dim=1).indices.to(torch.int32)


def _order(ids, G):
    """Offsets, token of every slot and slot of every id, for inputs that a grouping before the call has left."""
    n, k = ids.numel(), ids.shape[1]
    key = torch.where((ids >= 0) & (ids < G), ids, G).reshape(-1).long()
    order = torch.sort(key, stable=True).indices
    offsets = torch.searchsorted(key[order], torch.arange(G + 1, device=DEV)).to(torch.int32)
    rows = torch.where(key[order] < G, order // k, -1).to(torch.int32)
    slots = torch.empty(n, dtype=torch.int64, device=DEV)
    slots[order] = torch.arange(n, device=DEV)
    slots = torch.where(key < G, slots, -1).to(torch.int32).reshape(ids.shape)
    return offsets, rows, slots


def _drop(gen, ids, p):
    return torch.where(torch.rand(ids.shape, generator=gen, device=DEV) < p, -1, ids) if p else ids


def _fp8(gen, shape):
    """E4M3 bytes of rows that were scaled to use the format's range, as a quantiser leaves them."""
    return torch.randn(shape, dtype=BF16, generator=gen, device=DEV).mul_(100).clamp_(-448, 448).to(E4M3).view(torch.uint8)


def _normal(gen, shape, dtype, scale):
    return torch.randn(shape, dtype=dtype, generator=gen, device=DEV).mul_(scale)


def _swizzled(codes):
    """E8M0 codes [G, N, B] in the 512-byte tiles that a block-scaled product reads, [G, N up to 128, B up to 4]."""
    G, N, B = codes.shape
    Np, Bp = -(-N // 128) * 128, -(-B // 4) * 4
    full = torch.zeros(G, Np, Bp, dtype=torch.uint8, device=DEV)
    full[:, :N, :B] = codes
    tiles = full.view(G, Np // 128, 4, 32, Bp // 4, 4).permute(0, 1, 4, 3, 2, 5)
    return tiles.reshape(G, Np, Bp).contiguous()


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    c, s = case, {"case": case}
    if c["op"] == "group":
        s["ids"] = _drop(gen, _route(gen, c["T"], c["k"], c["G"]), c["dropped"])
        return s
    if c["op"] == "combine":
        T, k, N = c["T"], c["k"], c["N"]
        slots = torch.randperm(T * k, generator=gen, device=DEV).to(torch.int32).reshape(T, k)
        s["slots"] = _drop(gen, slots, c["dropped"])
        s["y"] = _normal(gen, (T * k, N), _dtype(c["dtype"]), 1.0)
        s["weights"] = torch.rand(T, k, generator=gen, device=DEV) / k
        return s
    if c["op"] == "lora":
        T, L, R, K, N, dt = c["T"], c["L"], c["R"], c["K"], c["N"], _dtype(c["dtype"])
        # a request's tokens follow one another in a prefill batch; a decode batch has one token of each
        per = max(1, T // (2 * L)) if T > 256 else 1
        ids = torch.randint(0, L, (-(-T // per),), generator=gen, device=DEV).to(torch.int32)
        ids = _drop(gen, ids, c["dropped"]).repeat_interleave(per)[:T].reshape(T, 1).contiguous()
        s["offsets"], s["rows"], s["slots"] = _order(ids, L)
        s["x"] = _normal(gen, (T, K), dt, 1.0)
        s["a"] = _normal(gen, (L, R, K), dt, 1.0 / math.sqrt(K))
        s["b"] = _normal(gen, (L, N, R), dt, 0.02)
        s["y"] = _normal(gen, (T, N), dt, 1.0)
        s["scaling"] = torch.rand(L, generator=gen, device=DEV) + 0.5
        s["most"] = max(1, int((s["offsets"][1:] - s["offsets"][:-1]).max()))   # a plan of the plain form alone
        return s
    fmt, T, k, G, N, K = c["fmt"], c["T"], c["k"], c["G"], c["N"], c["K"]
    s["offsets"], rows, _ = _order(_route(gen, T, k, G), G)
    s["most"] = int((s["offsets"][1:] - s["offsets"][:-1]).max())
    s["rows"] = rows if c["gather"] else None
    X = T if c["gather"] else T * k
    if fmt in ("bf16", "fp16"):
        s["x"] = _normal(gen, (X, K), _dtype(fmt), 1.0)
        s["w"] = _normal(gen, (G, N, K), _dtype(fmt), 1.0 / math.sqrt(K))
        s["xs"] = s["ws"] = s["ws_laid"] = None
    else:
        s["x"], s["w"] = _fp8(gen, (X, K)), _fp8(gen, (G, N, K))
        if fmt == "mxfp8":
            s["xs"] = torch.randint(118, 122, (X, K // 32), generator=gen, device=DEV).to(torch.uint8)
            s["ws"] = torch.randint(112, 115, (G, N, K // 32), generator=gen, device=DEV).to(torch.uint8)
            s["ws_laid"] = _swizzled(s["ws"])
        elif fmt == "block128":
            s["xs"] = 0.01 * (1 + torch.rand(X, K // 128, generator=gen, device=DEV))
            s["ws_laid"] = s["ws"] = 1e-4 * (1 + torch.rand(G, -(-N // 128), K // 128, generator=gen, device=DEV))
        else:
            s["xs"] = 0.01 * (1 + torch.rand(X, 1, generator=gen, device=DEV))
            s["ws_laid"] = s["ws"] = 1e-4 * (1 + torch.rand(G, N, generator=gen, device=DEV))
    s["out"] = torch.zeros(T * k, N, dtype=F16 if fmt == "fp16" else BF16, device=DEV)
    return s


# ------------------------------------------------------------------------------------ plain forms


def _values(q, scale, fmt):
    """The values that stored rows [.., W, K] stand for, in 32 bits; the scales fit the rows' last axes."""
    if fmt in ("bf16", "fp16"):
        return q.float()
    v = q.view(E4M3).float()
    if fmt == "mxfp8":
        by = torch.exp2(scale.float() - 127)
        return (v.unflatten(-1, (-1, 32)) * by.unsqueeze(-1)).flatten(-2)
    if fmt == "block128":
        return (v.unflatten(-1, (-1, 128)) * scale.unsqueeze(-1)).flatten(-2)
    return v * scale


def _weights(s):
    c = s["case"]
    if c["fmt"] == "block128":
        return _values(s["w"], s["ws"].repeat_interleave(128, dim=1)[:, :c["N"]], "block128")
    if c["fmt"] == "per_token":
        return _values(s["w"], s["ws"].unsqueeze(-1), "per_token")
    return _values(s["w"], s["ws"], c["fmt"])


def _padded(offsets, most):
    """Slots of each group side by side, [G, most], and which of them there are."""
    at = offsets[:-1].long().unsqueeze(1) + torch.arange(most, device=DEV)
    there = at < offsets[1:].long().unsqueeze(1)
    return torch.where(there, at, 0), there


def _plain_group(s):
    ids, G = s["ids"], s["case"]["G"]
    offsets, rows, slots = _order(ids, G)
    return {"offsets": offsets, "rows": rows, "slots": slots}


def _plain_gemm(s):
    c = s["case"]
    at, there = _padded(s["offsets"], s["most"])
    rows = at if s["rows"] is None else s["rows"].long()[at]
    x = _values(s["x"], s["xs"], c["fmt"])[rows]
    d = torch.bmm(x, _weights(s).transpose(1, 2))
    s["out"][at[there]] = d[there].to(s["out"].dtype)
    return s["out"]


def _plain_combine(s):
    slots = s["slots"].long()
    w = torch.where(slots >= 0, s["weights"], 0.0)
    y = s["y"][slots.clamp(min=0)].float()
    return (y * w.unsqueeze(-1)).sum(1).to(s["y"].dtype)


def _plain_lora(s):
    at, there = _padded(s["offsets"], s["most"])
    rows = s["rows"].long()[at]
    x = s["x"][torch.where(there, rows, 0)].float()
    v = torch.bmm(x, s["a"].float().transpose(1, 2))
    d = torch.bmm(v, s["b"].float().transpose(1, 2)) * s["scaling"].view(-1, 1, 1)
    to = rows[there]
    s["y"][to] = (s["y"][to].float() + d[there]).to(s["y"].dtype)
    return s["y"]


def run(state):
    s, op = state, state["case"]["op"]
    if own:
        import swiglu_fp8_activation_gb300 as sgq
        c = s["case"]
        if op == "group":
            offsets, rows, slots = sgq.group_rows(s["ids"], c["G"])
            return {"offsets": offsets, "rows": rows, "slots": slots}
        if op == "combine":
            return sgq.combine_rows(s["y"], s["slots"], s["weights"])
        if op == "lora":
            return sgq.lora_add(s["x"], s["a"], s["b"], s["y"], s["offsets"], rows=s["rows"], slots=s["slots"], scaling=s["scaling"])
        fmt = "none" if c["fmt"] in ("bf16", "fp16") else c["fmt"]
        return sgq.grouped_gemm(s["x"], s["w"], s["offsets"], fmt=fmt, x_scale=s["xs"], w_scale=s["ws_laid"], rows=s["rows"], out=s["out"])
    return {"group": _plain_group, "gemm": _plain_gemm, "combine": _plain_combine, "lora": _plain_lora}[op](s)


# ------------------------------------------------------------------------------------ definitions in 64 bits


def exact(case, seed):
    s, c = prepare(case, seed), case
    if c["op"] == "group":
        ids = s["ids"].flatten().tolist()
        k, G = c["k"] if c["k"] < c["G"] else c["G"], c["G"]
        members = [[] for _ in range(G)]
        for i, g in enumerate(ids):
            if 0 <= g < G:
                members[g].append(i)
        offsets, rows, slots = [0], [], [-1] * len(ids)
        for m in members:
            for i in m:
                slots[i] = len(rows)
                rows.append(i // k)
            offsets.append(len(rows))
        rows += [-1] * (len(ids) - len(rows))
        as32 = lambda v: torch.tensor(v, dtype=torch.int32)  # noqa: E731
        return {"offsets": as32(offsets), "rows": as32(rows), "slots": as32(slots).view(-1, k)}
    if c["op"] == "combine":
        out = torch.zeros(c["T"], c["N"], dtype=F64, device=DEV)
        for j in range(c["k"]):
            slot = s["slots"][:, j].long()
            t = (slot >= 0).nonzero().flatten()
            out[t] += s["weights"][t, j, None].double() * s["y"][slot[t]].double()
        return out
    off = s["offsets"].tolist()
    if c["op"] == "lora":
        y = s["y"].double()
        for g in range(c["L"]):
            t = s["rows"][off[g]:off[g + 1]].long()
            if len(t):
                y[t] += s["scaling"][g].double() * ((s["x"][t].double() @ s["a"][g].double().T) @ s["b"][g].double().T)
        return y
    out = torch.zeros(c["T"] * c["k"], c["N"], dtype=F64, device=DEV)
    fmt, K = c["fmt"], c["K"]
    fp8 = fmt in UNIT and fmt not in ("bf16", "fp16")
    block = {"mxfp8": 32, "block128": 128}.get(fmt, K)
    for g in range(c["G"]):
        a, b = off[g], off[g + 1]
        if a == b:
            continue
        r = torch.arange(a, b, device=DEV) if s["rows"] is None else s["rows"][a:b].long()
        x, w = s["x"][r], s["w"][g]
        x, w = (x.view(E4M3).double(), w.view(E4M3).double()) if fp8 else (x.double(), w.double())
        if fp8:
            xs, ws = s["xs"][r].double(), s["ws"][g].double()
            if fmt == "mxfp8":
                xs, ws = 2.0 ** (xs - 127), 2.0 ** (ws - 127)
            elif fmt == "block128":
                ws = ws[torch.arange(c["N"], device=DEV) // 128]
            else:
                ws = ws[:, None]
            x, w = x * xs.repeat_interleave(block, 1), w * ws.repeat_interleave(block, 1)
        out[a:b] = x @ w.T
    return out


# ------------------------------------------------------------------------------------ what a pass cannot do without


def work(case):
    c = case
    if c["op"] == "group":
        n = c["T"] * min(c["k"], c["G"])
        return {"bytes": 12 * n + 4 * (c["G"] + 1), "flops": 0}
    if c["op"] == "combine":
        n = c["T"] * c["k"]
        return {"bytes": 2 * c["N"] * (n * (1 - c["dropped"]) + c["T"]) + 8 * n, "flops": 2 * n * c["N"] * (1 - c["dropped"])}
    if c["op"] == "lora":
        T, L, R, K, N = c["T"] * (1 - c["dropped"]), c["L"], c["R"], c["K"], c["N"]
        requests = T if c["T"] <= 256 else min(T, 2 * L)
        used = L * (1 - (1 - 1 / L) ** requests)
        return {"bytes": 2 * (T * K + 2 * T * N + used * R * (K + N)) + 8 * T, "flops": 2 * T * R * (K + N)}
    S, G, N, K = c["T"] * c["k"], c["G"], c["N"], c["K"]
    used = G * (1 - (1 - c["k"] / G) ** c["T"])
    X = c["T"] if c["gather"] else S
    wide = 2 if c["fmt"] in ("bf16", "fp16") else 1
    x_scale, w_scale = {"mxfp8": (K / 32, N * K / 32), "block128": (K / 32, N * K / 4096), "per_token": (4, 4 * N)}.get(c["fmt"], (0, 0))
    return {"bytes": used * (N * K * wide + w_scale) + X * (K * wide + x_scale) + 2 * S * N + 4 * S, "flops": 2 * S * N * K}
