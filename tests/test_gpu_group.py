"""GPU parity of the ragged-group operators (include/sgq_group.h) against
plain 64-bit forms (group_ref.py, with the tolerances derived there): every
format and type, ragged and empty groups, odd widths, rows out of range,
offsets out of order, guard bands around every output, other streams, graph
replay, and an expert layer run end to end."""
import contextlib
import math

import pytest
import torch

import group_ref as ref
import swiglu_fp8_activation_gb300 as sgq
from swiglu_fp8_activation_gb300 import binding

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
GUARD = 4096


@pytest.fixture(autouse=True, scope="module")
def no_wait_ran_out():
    yield
    assert sgq.wait_timeouts() == 0


@contextlib.contextmanager
def planned_for(sms):
    binding.set_sm_budget(sms)
    try:
        yield
    finally:
        binding.set_sm_budget(0)


def guarded(shape, dtype):
    """A tensor inside a buffer of 0xFF bytes, and a function that checks the bytes around it."""
    n = math.prod(shape) * torch.empty((), dtype=dtype).element_size()
    raw = torch.full((n + 2 * GUARD,), 0xFF, dtype=torch.uint8, device=DEV)
    t = raw[GUARD:GUARD + n].view(dtype).view(shape)

    def untouched():
        assert (raw[:GUARD] == 0xFF).all() and (raw[GUARD + n:] == 0xFF).all(), "bytes written outside the output"
    return t, untouched


def cuda(*ts):
    return [None if t is None else t.to(DEV) for t in ts]


def sizes_to_offsets(sizes, lead=0):
    return torch.cumsum(torch.tensor([lead] + list(sizes)), 0).to(torch.int32)


# ------------------------------------------------------------------ group_rows

ROWS = [(0, 1, 4), (1, 1, 1), (1, 8, 64), (3, 2, 5), (33, 3, 7), (64, 8, 128), (100, 1, 1024), (511, 8, 160), (1000, 7, 1), (5000, 4, 33),
        (20000, 8, 256), (131072, 3, 1000)]


@pytest.mark.parametrize("dtype", [torch.int32, torch.int64])
@pytest.mark.parametrize("T,k,G", ROWS)
def test_group_rows(T, k, G, dtype):
    ids = torch.randint(-2, G + 1, (T, k), generator=ref.gen(T + k)).to(dtype)
    if dtype == torch.int64 and T:
        ids[T // 2] = (1 << 32) + 0            # its low half is a group
    want = ref.group_rows(ids, G)
    o, uo = guarded((G + 1,), torch.int32)
    r, ur = guarded((T * k,), torch.int32)
    s, us = guarded((T, k), torch.int32)
    got = sgq.group_rows(ids.to(DEV), G, offsets_out=o, rows_out=r, slots_out=s)
    for name, a, b in zip(("offsets", "rows", "slots"), got, want):
        assert torch.equal(a.cpu(), b), name
    uo(), ur(), us()


@pytest.mark.parametrize("T,k", [(1, 1), (40, 2), (9000, 4)])
@pytest.mark.parametrize("what", ["one group", "all dropped", "last group"])
def test_group_rows_skewed(T, k, what):
    G = 12
    ids = torch.full((T, k), {"one group": 5, "all dropped": -1, "last group": G - 1}[what], dtype=torch.int32)
    for a, b in zip(sgq.group_rows(ids.to(DEV), G), ref.group_rows(ids, G)):
        assert torch.equal(a.cpu(), b)


@pytest.mark.parametrize("n", [8192, 8193, 16384, 16385, 262144, 262145])
@pytest.mark.parametrize("G", [40, 200, 1000])
def test_group_rows_at_the_steps_of_its_plan(n, G):
    """Where the number of CTAs changes, and where a lane's ids no longer stay in registers; replayed from a graph."""
    ids = torch.randint(-1, G, (n,), generator=ref.gen(n + G)).to(torch.int32)
    order = torch.argsort(torch.where(ids < 0, G, ids), stable=True)
    kept = int((ids >= 0).sum())
    rows = torch.where(torch.arange(n) < kept, order, -1).to(torch.int32)
    slots = torch.empty(n, dtype=torch.int32)
    slots[order] = torch.where(torch.arange(n) < kept, torch.arange(n), -1).to(torch.int32)
    offsets = torch.cat([torch.zeros(1, dtype=torch.int64), torch.bincount(ids[ids >= 0], minlength=G).cumsum(0)]).to(torch.int32)
    dids = ids.to(DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, r, s = sgq.group_rows(dids, G)
    graph.replay()
    for got, want in ((o, offsets), (r, rows), (s, slots)):
        assert torch.equal(got.cpu(), want)


def test_group_rows_of_a_vector():
    ids = torch.tensor([2, -1, 0, 2], dtype=torch.int64, device=DEV)
    o, r, s = sgq.group_rows(ids, 3)
    assert o.tolist() == [0, 1, 1, 3] and r.tolist() == [2, 0, 3, -1] and s.tolist() == [1, -1, 0, 2]


# ------------------------------------------------------------------ grouped_gemm

def run_gemm(fmt, sizes, N, K, *, dtype=torch.bfloat16, lead=0, tail=0, gather=None, seed=0, offsets=None, x_rows=None):
    """grouped_gemm against the plain form; gather: a [S] row index, or None."""
    off = sizes_to_offsets(sizes, lead) if offsets is None else offsets
    G = off.numel() - 1
    S = lead + sum(sizes) + tail
    X = x_rows if x_rows is not None else (S if gather is None else max(1, S // 2))
    x, xs, w, ws = ref.operands(fmt, X, G, N, K, seed, dtype)
    rows = gather(S, X) if gather is not None else None
    out, untouched = guarded((S, N), dtype)
    before = out.cpu()
    res, tol = ref.grouped_gemm(fmt, x, xs, w, ws, off, rows, S, torch.zeros(S, N), dtype)
    covered = torch.zeros(S, dtype=torch.bool)
    for a, b in ref.ranges(off, S):
        covered[a:b] = True
    dx, dxs, dw, doff, drows = cuda(x, xs, w, off, rows)
    dws = None if ws is None else (ref.swizzled(ws) if fmt == "mxfp8" else ws).to(DEV)
    got = sgq.grouped_gemm(dx, dw, doff, fmt=fmt, x_scale=dxs, w_scale=dws, rows=drows, out=out)
    torch.cuda.synchronize()
    assert got is out
    cpu = out.cpu()
    assert torch.equal(cpu[~covered].view(torch.int16), before[~covered].view(torch.int16)), "a slot of no group was written"
    ref.check(cpu[covered], res[covered], tol[covered], f"{fmt} {sizes} N={N} K={K}")
    untouched()
    again = torch.zeros_like(out)
    sgq.grouped_gemm(dx, dw, doff, fmt=fmt, x_scale=dxs, w_scale=dws, rows=drows, out=again)
    assert torch.equal(again.cpu()[covered].view(torch.int16), cpu[covered].view(torch.int16)), "two runs differ"
    return cpu


FMTS = ["mxfp8", "block128", "per_token", "none"]
SHAPES = [  # group sizes, N, K in units of the format
    ([1], 8, 1), ([1], 128, 4), ([3, 0, 2], 136, 3), ([0, 0, 5], 64, 9), ([17, 1, 0, 33], 264, 5), ([128], 128, 16),
    ([129, 127], 384, 8), ([200, 3, 61], 520, 13), ([0], 64, 2), ([300], 1000, 6), ([1] * 40, 256, 40), ([64] * 6, 640, 33),
]


@pytest.mark.parametrize("sizes,N,units", SHAPES, ids=str)
@pytest.mark.parametrize("fmt", FMTS)
def test_grouped_gemm(fmt, sizes, N, units):
    run_gemm(fmt, sizes, N, units * ref.UNIT[fmt])


@pytest.mark.parametrize("fmt", FMTS)
def test_grouped_gemm_fp16(fmt):
    run_gemm(fmt, [5, 0, 130, 31], 264, 6 * ref.UNIT[fmt] if fmt != "none" else 200, dtype=torch.float16)


def some_rows(S, X):
    return torch.randint(0, X, (S,), generator=ref.gen(S)).to(torch.int32)


def wild_rows(S, X):
    r = some_rows(S, X)
    r[::3] = torch.tensor([-1, X, -(1 << 31), (1 << 31) - 1], dtype=torch.int32)[torch.arange(len(r[::3])) % 4]
    return r


@pytest.mark.parametrize("sizes", [[1], [7, 0, 3], [140, 20, 300], [2] * 70], ids=str)
@pytest.mark.parametrize("fmt", FMTS)
def test_grouped_gemm_gathers_rows(fmt, sizes):
    run_gemm(fmt, sizes, 200, 6 * ref.UNIT[fmt], gather=some_rows)


@pytest.mark.parametrize("fmt", FMTS)
def test_grouped_gemm_reads_rows_outside_as_zeros(fmt):
    run_gemm(fmt, [40, 9, 150], 136, 5 * ref.UNIT[fmt], gather=wild_rows)


@pytest.mark.parametrize("fmt", FMTS)
def test_grouped_gemm_without_rows_of_x(fmt):
    run_gemm(fmt, [5, 3], 64, 2 * ref.UNIT[fmt], gather=lambda S, X: torch.zeros(S, dtype=torch.int32), x_rows=0)


@pytest.mark.parametrize("fmt", FMTS)
def test_grouped_gemm_slots_of_no_group(fmt):
    run_gemm(fmt, [20, 0, 70], 136, 4 * ref.UNIT[fmt], lead=3, tail=45)


@pytest.mark.parametrize("offsets", [[-7, 20, 12, 60, 1 << 30], [50, 10, 90, 90, 3], [0, 0, 0, 0, 0], [-(1 << 31), 2, -1, 70, (1 << 31) - 1]])
@pytest.mark.parametrize("fmt", FMTS)
def test_grouped_gemm_holds_offsets_inside(fmt, offsets):
    run_gemm(fmt, [64], 72, 3 * ref.UNIT[fmt], offsets=torch.tensor(offsets, dtype=torch.int32))


def test_grouped_gemm_many_groups():
    run_gemm("mxfp8", [(7 * i) % 5 for i in range(1024)], 64, 64)


@pytest.mark.parametrize("fmt", FMTS)
def test_grouped_gemm_long_products(fmt):
    run_gemm(fmt, [3, 18], 40, 8192)


@pytest.mark.parametrize("fmt", FMTS)
def test_grouped_gemm_single_tokens_wide(fmt):
    run_gemm(fmt, [1, 0, 1, 1], 2048, 1024)


@pytest.mark.parametrize("K", [1024, 1152, 2688, 4480])
@pytest.mark.parametrize("sizes,N", [([1], 72), ([31], 136), ([2, 0, 33], 264), ([0, 0], 128)], ids=str)
@pytest.mark.parametrize("gather", [None, wild_rows], ids=["rows in order", "rows outside"])
@pytest.mark.parametrize("fmt", FMTS)
def test_grouped_gemm_few_tiles_and_long_products(fmt, gather, sizes, N, K):
    """Few enough tiles that the CTAs of a cluster share one, in pieces of K of unlike lengths."""
    run_gemm(fmt, sizes, N, K, gather=gather, lead=1, tail=2)
    if fmt in ("none", "per_token"):
        run_gemm(fmt, sizes, N, K + 16, gather=gather, dtype=torch.float16)


@pytest.mark.parametrize("fmt", FMTS)
def test_grouped_gemm_many_rows(fmt):
    run_gemm(fmt, [700, 1, 1300, 0, 255], 512, 512)


@pytest.mark.parametrize("sizes,N,units", [([300], 256, 4), ([257, 0, 140, 500], 136, 5), ([130, 400, 1], 264, 9), ([1000, 16, 33], 640, 33)], ids=str)
@pytest.mark.parametrize("gather", [None, some_rows, wild_rows], ids=["rows in order", "gathered", "rows outside"])
@pytest.mark.parametrize("fmt", FMTS)
def test_grouped_gemm_large_groups(fmt, sizes, N, units, gather):
    """Planned for two multiprocessors, so that the widest tiles (pairs of CTAs, but
    for 1x128) run, each CTA many of them; then for the device's own count."""
    for sms in (2, 0):
        with planned_for(sms):
            run_gemm(fmt, sizes, N, units * ref.UNIT[fmt] if fmt != "none" else units * 24, gather=gather, lead=2, tail=5)


@pytest.mark.parametrize("fmt", FMTS)
def test_grouped_gemm_large_groups_long_products(fmt):
    for sms in (2, 0):
        with planned_for(sms):
            run_gemm(fmt, [290, 31], 384, 6144, gather=some_rows)


@pytest.mark.parametrize("mean", [20, 50, 100, 200])
@pytest.mark.parametrize("gather", [None, some_rows], ids=["rows in order", "gathered"])
@pytest.mark.parametrize("fmt", FMTS)
def test_grouped_gemm_many_tiles_a_cta(fmt, gather, mean):
    """Every width of tile, three CTAs (or one pair) walking over all of them."""
    sizes = [mean, 0, mean // 3, 2 * mean + 1, 1, mean + 7]
    with planned_for(3):
        run_gemm(fmt, sizes, 392, 11 * ref.UNIT[fmt] if fmt != "none" else 264, gather=gather, tail=3)
        if fmt != "block128":
            run_gemm(fmt, sizes, 128, 2 * ref.UNIT[fmt], gather=gather, dtype=torch.float16)


def test_grouped_gemm_padding_of_w_scale_is_not_read_into_the_result():
    """Codes behind N and behind K/32 in the scales' padding hold NaN codes (255)."""
    sizes, N, K = [9, 200], 72, 96
    off = sizes_to_offsets(sizes)
    x, xs, w, ws = ref.operands("mxfp8", 209, 2, N, K, 3)
    laid, real = ref.swizzled(ws), ref.swizzled(torch.full_like(ws, 1))
    laid[real == 0] = 255
    res, tol = ref.grouped_gemm("mxfp8", x, xs, w, ws, off, None, 209, torch.zeros(209, N), torch.bfloat16)
    dx, dxs, dw, doff, dws = cuda(x, xs, w, off, laid)
    ref.check(sgq.grouped_gemm(dx, dw, doff, fmt="mxfp8", x_scale=dxs, w_scale=dws).cpu(), res, tol)


def test_grouped_gemm_extreme_scales():
    """E8M0 codes 0 and 254, whose product of scales is 1 or leaves the range of 32 bits' normal numbers."""
    N, K = 64, 128
    off = sizes_to_offsets([8])
    x, xs, w, ws = ref.operands("mxfp8", 8, 1, N, K, 4)
    xs[:], ws[:] = 254, 0
    res, tol = ref.grouped_gemm("mxfp8", x, xs, w, ws, off, None, 8, torch.zeros(8, N), torch.bfloat16)
    dx, dxs, dw, doff, dws = cuda(x, xs, w, off, ref.swizzled(ws))
    ref.check(sgq.grouped_gemm(dx, dw, doff, fmt="mxfp8", x_scale=dxs, w_scale=dws).cpu(), res, tol)


def test_grouped_gemm_keeps_a_nan_row_to_itself():
    sizes, N, K = [30, 34], 136, 256
    off = sizes_to_offsets(sizes)
    for fmt in FMTS:
        x, xs, w, ws = ref.operands(fmt, 64, 2, N, K, 5)
        res, tol = ref.grouped_gemm(fmt, x, xs, w, ws, off, None, 64, torch.zeros(64, N), torch.bfloat16)
        if fmt == "none":
            x[29] = float("nan")
        else:
            x[29] = 0x7F
        dx, dxs, dw, doff = cuda(x, xs, w, off)
        dws = None if ws is None else (ref.swizzled(ws) if fmt == "mxfp8" else ws).to(DEV)
        got = sgq.grouped_gemm(dx, dw, doff, fmt=fmt, x_scale=dxs, w_scale=dws).cpu()
        assert got[29].isnan().all()
        keep = torch.arange(64) != 29
        ref.check(got[keep], res[keep], tol[keep], fmt)


def test_grouped_gemm_scales_at_any_address():
    """x_scale is a byte tensor of MXFP8 codes: no alignment is asked of it, whatever its rows' length."""
    for K in (96, 512, 640, 1024):
        off = sizes_to_offsets([9, 31])
        x, xs, w, ws = ref.operands("mxfp8", 40, 2, 72, K, K)
        res, tol = ref.grouped_gemm("mxfp8", x, xs, w, ws, off, None, 40, torch.zeros(40, 72), torch.bfloat16)
        dx, dw, doff, dws = cuda(x, w, off, ref.swizzled(ws))
        for shift in (1, 4, 8, 13):
            raw = torch.zeros(xs.numel() + 16, dtype=torch.uint8, device=DEV)
            at = raw[shift:shift + xs.numel()].view(xs.shape)
            at.copy_(xs)
            ref.check(sgq.grouped_gemm(dx, dw, doff, x_scale=at, w_scale=dws).cpu(), res, tol, f"K={K} shift={shift}")


@pytest.mark.parametrize("sms", [1, 7, 64, 1000])
def test_planned_for_other_counts_of_multiprocessors(sms):
    with planned_for(sms):
        for fmt in FMTS:
            run_gemm(fmt, [300, 1, 77], 264, 1152, gather=some_rows)
            run_gemm(fmt, [3, 0, 1], 136, 3584)
        run_lora(mixed(300, 3), 3, 40, 520, 264)
        run_lora(mixed(700, 3), 3, 104, 264, 1032, torch.float16)
        run_lora(mixed(30, 9), 9, 16, 520, 264)


def test_offsets_past_32_bits():
    """Outputs and inputs of more than 2^31 elements: the rows at their ends."""
    N = 4096
    S = (1 << 31) // N + 3000
    x = torch.randn(S, 8, generator=ref.gen(1)).to(torch.bfloat16).to(DEV)
    w = torch.randn(2, N, 8, generator=ref.gen(2)).to(torch.bfloat16).to(DEV)
    off = torch.tensor([0, S - 700, S], dtype=torch.int32, device=DEV)
    out = sgq.grouped_gemm(x, w, off, fmt="none")
    for lo, hi, g in ((S - 900, S - 700, 0), (S - 700, S, 1)):
        want = x[lo:hi].double() @ w[g].double().T
        mag = x[lo:hi].double().abs() @ w[g].double().abs().T
        ref.check(out[lo:hi].cpu(), want.cpu(), (8 * 2.0 ** -22 * mag).cpu() + ref.rounding(want.cpu(), torch.bfloat16))
    slots = torch.randint(S - 2000, S, (64, 3), generator=ref.gen(3)).to(torch.int32)
    got = sgq.combine_rows(out, slots.to(DEV))
    low = S - 2000
    res, tol = ref.combine(out[low:].cpu(), slots - low, None, torch.bfloat16)
    ref.check(got.cpu(), res, tol)
    # lora_add on the same rows, some of the last ones with an adapter
    ids = torch.full((S,), -1, dtype=torch.int32)
    ids[-300:] = torch.randint(-1, 2, (300,), generator=ref.gen(4)).to(torch.int32)
    a = torch.randn(2, 16, 8, generator=ref.gen(5)).to(torch.bfloat16)
    b = torch.randn(2, N, 16, generator=ref.gen(6)).to(torch.bfloat16)
    o, r, s = sgq.group_rows(ids.to(DEV), 2)
    before = out[-400:].cpu()
    sgq.lora_add(x, a.to(DEV), b.to(DEV), out, o, rows=r, slots=s)
    o2, r2, s2 = ref.group_rows(ids[-400:].view(-1, 1), 2)
    res, tol = ref.lora(x[-400:].cpu(), a, b, before, o2, r2, s2.view(-1), None, 400)
    ref.check(out[-400:].cpu(), res, tol)


def test_empty_calls():
    i = lambda *s: torch.zeros(*s, dtype=torch.int32, device=DEV)  # noqa: E731
    b = lambda *s: torch.ones(*s, dtype=torch.bfloat16, device=DEV)  # noqa: E731
    assert sgq.grouped_gemm(b(3, 64), b(2, 32, 64), i(3), fmt="none", rows=i(0)).shape == (0, 32)
    assert sgq.grouped_gemm(b(0, 64), b(2, 32, 64), i(3), fmt="none").shape == (0, 32)
    assert sgq.combine_rows(b(3, 64), i(0, 2)).shape == (0, 64)
    y = b(4, 32)
    assert (sgq.lora_add(b(4, 64), b(2, 8, 64), b(2, 32, 8), y, i(3), rows=i(0), slots=i(4) - 1) == 1).all()
    assert sgq.lora_add(b(0, 64), b(2, 8, 64), b(2, 32, 8), b(0, 32), i(3)).shape == (0, 32)
    o, r, s = sgq.group_rows(i(0, 3), 5)
    assert (o == 0).all() and r.shape == (0,) and s.shape == (0, 3)


# ------------------------------------------------------------------ combine_rows

@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("T,k,S,N", [(1, 1, 1, 8), (5, 8, 40, 1032), (64, 8, 512, 4096), (33, 3, 10, 64), (300, 20, 77, 1024), (2, 1, 0, 16), (1000, 9, 9000, 136)])
def test_combine(T, k, S, N, dtype):
    r = ref.gen(T * k + N)
    y = torch.randn(S, N, generator=r).to(dtype)
    slots = torch.randint(-1, S + 1, (T, k), generator=r).to(torch.int32)
    slots[0, 0] = (1 << 31) - 1
    weights = torch.randn(T, k, generator=r)
    for w in (weights, None):
        res, tol = ref.combine(y, slots, w, dtype)
        out, untouched = guarded((T, N), dtype)
        dy, ds, dw = cuda(y, slots, w)
        sgq.combine_rows(dy, ds, dw, out=out)
        ref.check(out.cpu(), res, tol)
        untouched()


def test_combine_does_not_use_the_weight_or_rows_of_a_slot_outside():
    y = torch.full((3, 64), float("nan"), dtype=torch.bfloat16)
    y[1] = 2
    slots = torch.tensor([[1, -1], [3, -1]], dtype=torch.int32)
    w = torch.tensor([[0.5, float("nan")], [float("inf"), float("nan")]])
    out = sgq.combine_rows(*cuda(y, slots, w)).cpu()
    assert (out[0] == 1).all() and (out[1] == 0).all()


# ------------------------------------------------------------------ lora_add

def run_lora(ids, G, R, K, N, dtype=torch.bfloat16, scaled=True, seed=0, sorted_rows=False, tamper=None):
    T = len(ids)
    r = ref.gen(seed)
    x = torch.randn(T, K, generator=r).to(dtype)
    a = (torch.randn(G, R, K, generator=r) / math.sqrt(K)).to(dtype)
    b = (torch.randn(G, N, R, generator=r) * 0.1).to(dtype)
    y = torch.randn(T, N, generator=r).to(dtype)
    scaling = torch.randn(G, generator=r) if scaled else None
    offsets, rows, slots = ref.group_rows(torch.tensor(ids, dtype=torch.int32).view(T, 1), G)
    slots = slots.view(-1)
    if sorted_rows:
        rows = slots = None
    if tamper:
        tamper(offsets, rows, slots)
    res, tol = ref.lora(x, a, b, y, offsets, rows, slots, scaling, T)
    out, untouched = guarded((T, N), dtype)
    out.copy_(y)
    ws, ws_untouched = guarded((sgq.lora_workspace_bytes(T, G, R),), torch.uint8)
    dx, da, db, doff, drows, dslots, dc = cuda(x, a, b, offsets, rows, slots, scaling)
    got = sgq.lora_add(dx, da, db, out, doff, rows=drows, slots=dslots, scaling=dc, workspace=ws)
    assert got is out
    ref.check(out.cpu(), res, tol, f"T={T} R={R} K={K} N={N}")
    same = (res == y.double()).all(1) & (tol == 0).all(1)
    assert torch.equal(out.cpu()[same].view(torch.int16), y[same].view(torch.int16))
    untouched(), ws_untouched()
    return int(same.sum())


def mixed(T, G, seed=0, none=0.2):
    r = ref.gen(seed)
    ids = torch.randint(0, G, (T,), generator=r)
    return torch.where(torch.rand(T, generator=r) < none, -1, ids).tolist()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("R", [8, 16, 24, 64, 104, 128])
def test_lora_ranks(R, dtype):
    run_lora(mixed(70, 4), 4, R, 264, 520, dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("R", [8, 24, 56, 128])
def test_lora_ranks_few_slots_an_adapter(R, dtype):
    G = 90 * R // 128 + 1                                           # few enough slots an adapter
    run_lora(mixed(90, G), G, R, 520, 1032, dtype)
    run_lora([3] * 40 + mixed(20, 6), 60, R, 136, 520, dtype)       # 40 slots of one, few on average
    run_lora(mixed(5, 6), 6, R, 4104, 8200, dtype)


@pytest.mark.parametrize("T,G,K,N", [(1, 1, 8, 8), (1, 5, 1024, 2048), (2, 2, 4096, 72), (64, 32, 512, 512), (65, 64, 136, 1032), (333, 3, 1000, 264),
                                     (600, 7, 256, 4096), (1500, 2, 2048, 128)])
def test_lora_shapes(T, G, K, N):
    run_lora(mixed(T, G), G, 16, K, N)
    run_lora(mixed(T, G, 1), G, 40, K, N, torch.float16, scaled=False)


def test_lora_rows_of_a_prefill_batch():
    assert run_lora([1] * 200 + [-1] * 50 + [0] * 300 + [1] * 33, 3, 32, 256, 384) == 50


def test_lora_without_adapters_leaves_y():
    assert run_lora([-1] * 40, 3, 16, 64, 64) == 40


def test_lora_sorted_rows_need_no_index():
    run_lora([0] * 30 + [1] * 2 + [3] * 100, 4, 16, 128, 256, sorted_rows=True)


def test_lora_passes_over_slots_that_disagree():
    def tamper(offsets, rows, slots):
        rows[3] = rows[4]           # one token in two slots: its own slot alone counts
        rows[10] = 1 << 30
        rows[11] = -3
        slots[int(rows[20])] = 21
    assert run_lora(mixed(64, 3, none=0.0), 3, 16, 128, 192, tamper=tamper) == 4


def test_lora_holds_offsets_inside():
    def tamper(offsets, rows, slots):
        offsets[0], offsets[2], offsets[3], offsets[4] = -4, 90, 40, 1 << 30
    run_lora(mixed(64, 4, none=0.0), 4, 24, 128, 192, tamper=tamper)


def test_lora_large_factors_fp16():
    """Factors v near and beyond the range of fp16, which y still holds: nothing overflows on the way."""
    T, R, K, N = 20, 16, 512, 64
    r = ref.gen(9)
    x = (torch.randn(T, K, generator=r) * 200).half()
    a = (torch.randn(1, R, K, generator=r) * 30).half()
    b = (torch.randn(1, N, R, generator=r) * 1e-3).half()
    y = torch.zeros(T, N).half()
    offsets = torch.tensor([0, T], dtype=torch.int32)
    scaling = torch.tensor([1e-1])
    res, tol = ref.lora(x, a, b, y, offsets, None, None, scaling, T)
    dx, da, db, dy, do, dc = cuda(x, a, b, y, offsets, scaling)
    ref.check(sgq.lora_add(dx, da, db, dy, do, scaling=dc).cpu(), res, tol)


# ------------------------------------------------------------------ streams, graphs, chains

def test_other_stream_and_its_allocations():
    st = torch.cuda.Stream()
    ids = torch.randint(0, 9, (500, 2), generator=ref.gen(2)).to(torch.int32)
    dids = ids.to(DEV)
    y = torch.randn(1000, 64, generator=ref.gen(3)).to(torch.bfloat16).to(DEV)
    torch.cuda.synchronize()
    with pytest.raises(sgq.SgqError):
        sgq.combine_rows(y, dids.cpu())
    o, r, s = sgq.group_rows(dids, 9, stream=st)
    out = sgq.combine_rows(y, s, stream=st)
    st.synchronize()
    want = ref.group_rows(ids, 9)
    assert torch.equal(o.cpu(), want[0]) and torch.equal(r.cpu(), want[1]) and torch.equal(s.cpu(), want[2])
    res, tol = ref.combine(y.cpu(), want[2], None, torch.bfloat16)
    ref.check(out.cpu(), res, tol)
    assert torch.cuda.current_stream() == torch.cuda.default_stream()


class Layer:
    """An expert layer with adapters beside its gate-and-up product's input norm, as a program would run it."""

    def __init__(self, T, H, I, E, k, seed):
        r = torch.Generator(device=DEV).manual_seed(seed)
        rn = lambda *s, scale=1.0: (torch.randn(*s, generator=r, device=DEV) * scale).to(torch.bfloat16)  # noqa: E731
        self.T, self.E, self.k = T, E, k
        self.x, self.res, self.nw = rn(T, H), rn(T, H), rn(H, scale=0.1)
        self.ids = torch.stack([torch.randperm(E, generator=r, device=DEV)[:k] for _ in range(T)])
        self.weights = torch.rand(T, k, generator=r, device=DEV)
        up, down = rn(E * 2 * I, H, scale=H ** -0.5), rn(E * H, I, scale=I ** -0.5)
        self.q1, self.s1 = sgq.quantize_fp8(up, fmt="mxfp8", scale_layout="swizzled")
        self.q2, self.s2 = sgq.quantize_fp8(down, fmt="mxfp8", scale_layout="swizzled")
        self.r1, self.r2 = sgq.quantize_fp8(up, fmt="mxfp8")[1], sgq.quantize_fp8(down, fmt="mxfp8")[1]
        self.H, self.I = H, I
        self.ad = torch.randint(-1, 3, (T,), generator=r, device=DEV).to(torch.int32)
        self.la, self.lb = rn(3, 16, H, scale=H ** -0.5), rn(3, H, 16, scale=0.1)

    def run(self):
        H, I, E = self.H, self.I, self.E
        q, s, normed, _ = sgq.rmsnorm_add_quant(self.x, self.nw, residual_in=self.res, residual_out=torch.empty_like(self.res), normed=True)
        off, rows, slots = sgq.group_rows(self.ids, E)
        gu = sgq.grouped_gemm(q, self.q1.view(E, 2 * I, H), off, x_scale=s, w_scale=self.s1.view(E, 2 * I, -1), rows=rows)
        aq, asc = sgq.swiglu_quant(gu)
        y = sgq.grouped_gemm(aq, self.q2.view(E, H, I), off, x_scale=asc, w_scale=self.s2.view(E, H, -1))
        out = sgq.combine_rows(y, slots, self.weights)
        aoff, arows, aslots = sgq.group_rows(self.ad, 3)
        sgq.lora_add(normed, self.la, self.lb, out, aoff, rows=arows, slots=aslots)
        return q, s, normed, off, rows, slots, gu, aq, asc, y, out

    def check(self, r):
        """Each step's result against the plain form of what the step before it left."""
        q, s, normed, off, rows, slots, gu, aq, asc, y, out = [t.cpu() for t in r]
        E, H, I, T = self.E, self.H, self.I, self.T
        for a, b in zip((off, rows, slots), ref.group_rows(self.ids.cpu(), E)):
            assert torch.equal(a, b)
        S = T * self.k
        w1 = self.q1.cpu().view(E, 2 * I, H), self.r1.cpu().view(E, 2 * I, -1)
        w2 = self.q2.cpu().view(E, H, I), self.r2.cpu().view(E, H, -1)
        ref.check(gu, *ref.grouped_gemm("mxfp8", q, s, *w1, off, rows, S, torch.zeros(S, 2 * I), torch.bfloat16), "gate and up")
        ref.check(y, *ref.grouped_gemm("mxfp8", aq, asc, *w2, off, None, S, torch.zeros(S, H), torch.bfloat16), "down")
        res, tol = ref.combine(y, slots, self.weights.cpu(), torch.bfloat16)
        ao, ar, asl = ref.group_rows(self.ad.cpu().view(-1, 1), 3)
        base = res.to(torch.bfloat16)
        lres, ltol = ref.lora(normed, self.la.cpu(), self.lb.cpu(), base, ao, ar, asl.view(-1), None, T)
        # base may be the neighbour of the kernel's rounding: one step of bf16
        ref.check(out, lres, ltol + tol + base.double().abs() * 2.0 ** -7, "layer")


@pytest.mark.parametrize("T,H,I,E,k", [(1, 256, 128, 4, 2), (24, 512, 256, 8, 2), (200, 384, 128, 5, 3)])
def test_expert_layer(T, H, I, E, k):
    m = Layer(T, H, I, E, k, T)
    r = m.run()
    torch.cuda.synchronize()
    m.check(r)


def test_expert_layer_in_a_graph_and_two_streams():
    m = Layer(40, 256, 128, 6, 2, 1)
    want = [t.clone() for t in m.run()]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = m.run()
    for _ in range(3):
        for t in got:
            t.view(-1).view(torch.uint8).fill_(0xAB)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    # other inputs in the captured buffers
    m.x.copy_(torch.randn(40, 256, generator=ref.gen(8)).to(torch.bfloat16))
    m.ids.copy_(torch.stack([torch.randperm(6, generator=ref.gen(i))[:2] for i in range(40)]))
    graph.replay()
    torch.cuda.synchronize()
    m.check(got)
    # two streams at once
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    layers = [Layer(60 + i, 256, 128, 6, 2, 5 + i) for i in range(2)]
    torch.cuda.synchronize()
    outs = [None, None]
    for _ in range(4):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                outs[i] = layers[i].run()
    torch.cuda.synchronize()
    for m, r in zip(layers, outs):
        m.check(r)


def test_many_calls_on_several_streams():
    """Calls of every form at once on four streams, each equal, bit for bit, to the same call alone."""
    calls = []                                   # (name, function that makes its outputs)

    def gemm(fmt, sizes, N, K, gather, seed):
        off = sizes_to_offsets(sizes)
        S, G = sum(sizes), len(sizes)
        x, xs, w, ws = ref.operands(fmt, S, G, N, K, seed)
        dx, dxs, dw, doff = cuda(x, xs, w, off)
        dws = None if ws is None else (ref.swizzled(ws) if fmt == "mxfp8" else ws).to(DEV)
        rows = some_rows(S, S).to(DEV) if gather else None
        calls.append((f"{fmt} {sizes}", lambda: sgq.grouped_gemm(dx, dw, doff, fmt=fmt, x_scale=dxs, w_scale=dws, rows=rows)))

    for i, fmt in enumerate(FMTS):
        gemm(fmt, [1, 0, 2], 264, 4096, True, i)                  # a cluster a tile
        gemm(fmt, [9, 17, 3, 0, 30] * 8, 1024, 512, i % 2 == 0, i)       # narrow tiles
        gemm(fmt, [1500, 900], 2048, 512, i % 2 == 1, i)                 # pairs of CTAs, or the widest tiles
    for T, G, R, N in ((40, 20, 16, 1032), (900, 3, 64, 2048), (500, 2, 128, 520)):
        r = ref.gen(T)
        x, y = torch.randn(T, 512, generator=r).to(torch.bfloat16).to(DEV), torch.randn(T, N, generator=r).to(torch.bfloat16).to(DEV)
        a, b = torch.randn(G, R, 512, generator=r).to(torch.bfloat16).to(DEV), torch.randn(G, N, R, generator=r).to(torch.bfloat16).to(DEV)
        o, rows, slots = sgq.group_rows(torch.tensor(mixed(T, G), dtype=torch.int32, device=DEV), G)
        calls.append((f"lora {T}", lambda x=x, a=a, b=b, y=y, o=o, rows=rows, slots=slots:
                      sgq.lora_add(x, a, b, y.clone(), o, rows=rows, slots=slots)))
    ids = torch.randint(-1, 200, (9000, 4), generator=ref.gen(5)).to(torch.int32).to(DEV)
    calls.append(("group_rows", lambda: sgq.group_rows(ids, 200)[1]))
    torch.cuda.synchronize()
    alone = []
    for _, f in calls:
        alone.append(f())
        torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(4)]
    for turn in range(6):
        got = []
        for i in range(4 * len(calls)):
            name, f = calls[(i * 5 + turn) % len(calls)]
            with torch.cuda.stream(streams[i % 4]):
                got.append(((i * 5 + turn) % len(calls), f()))
        torch.cuda.synchronize()
        for k, t in got:
            assert torch.equal(t.view(torch.uint8), alone[k].view(torch.uint8)), calls[k][0]


@pytest.mark.parametrize("seed", range(40))
def test_random_calls(seed):
    """Shapes, formats, indices and plans drawn at random."""
    import random
    r = random.Random(1000 + seed)
    sms = r.choice((0, 0, 1, 3, 20))
    with planned_for(sms):
        fmt = r.choice(FMTS)
        unit = ref.UNIT[fmt]
        sizes = [r.choice((0, 1, r.randint(0, 40), r.randint(0, 400))) for _ in range(r.randint(1, 9))]
        run_gemm(fmt, sizes, 8 * r.randint(1, 80), unit * r.randint(1, max(1, 2600 // unit)), seed=seed,
                 gather=r.choice((None, some_rows, wild_rows)), lead=r.choice((0, 3)), tail=r.choice((0, 50)),
                 dtype=r.choice((torch.bfloat16, torch.float16)))
        T, G = r.choice((1, r.randint(1, 40), r.randint(1, 900))), r.randint(1, 40)
        run_lora(mixed(T, G, seed, r.choice((0.0, 0.5))), G, 8 * r.randint(1, 16), 8 * r.randint(1, 200), 8 * r.randint(1, 200),
                 r.choice((torch.bfloat16, torch.float16)), scaled=r.random() < 0.7, seed=seed)
