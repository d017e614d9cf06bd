"""GPU parity of the paged cache's operators (include/sgq_cache.h) against plain
64-bit forms (cache_ref.py, with the tolerances derived there): every format and
type, head widths, groups and page sizes, lengths around every border, windows, sinks, strides, masked rows
that hold NaN, guard bands around every output, shares of few and many CTAs, other streams, graph
replay, and prompts and steps run end to end."""
import contextlib
import math

import pytest
import torch

import cache_ref as ref
import swiglu_fp8_activation_gb300 as sgq
from swiglu_fp8_activation_gb300 import binding

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
GUARD = 4096
BF16, F16 = torch.bfloat16, torch.float16
KINDS = [("none", BF16), ("none", F16), ("per_token", BF16), ("per_token", F16)]


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
    """On the device, with the same strides."""
    out = []
    for t in ts:
        if t is None:
            out.append(None)
            continue
        d = torch.empty_strided(t.shape, t.stride(), dtype=t.dtype, device=DEV)
        out.append(d.copy_(t))
    return out


# ------------------------------------------------------------------ rope

ROPE = [(1, 1, 16, 16), (1, 5, 64, 32), (3, 1, 128, 128), (7, 3, 72, 48), (33, 2, 256, 256), (64, 32, 128, 64), (700, 2, 80, 80), (2500, 3, 40, 16), (5000, 1, 64, 64)]


@pytest.mark.parametrize("T,H,D,R", ROPE)
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_rope(T, H, D, R, layout, dtype):
    x = torch.randn(T, H, D, generator=ref.gen(T + D)).to(dtype)
    pos = torch.randint(0, 1 << 20, (T,), generator=ref.gen(R)).to(torch.int32 if T % 2 else torch.int64)
    freqs = ref.turns(R)
    for factor, inverse in ((1.0, False), (1.3, True)):
        want, tol = ref.rope(x, pos, freqs, layout, factor, inverse)
        out, untouched = guarded((T, H, D), dtype)
        got = sgq.rope(*cuda(x, pos, freqs), layout=layout, factor=factor, inverse=inverse, out=out)
        assert got is out
        ref.check(out.cpu(), want, tol + ref.rounding(want.abs() + tol, dtype), f"{layout} {factor}")
        assert torch.equal(out.cpu()[..., R:], x[..., R:])
        untouched()


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rope_at_far_and_negative_positions_with_any_frequencies(layout):
    pos = torch.tensor([0, 1, -1, (1 << 31) - 1, -(1 << 31), (1 << 62) + 12345, -(1 << 62) - 1, 999999937], dtype=torch.int64)
    x = torch.randn(len(pos), 2, 64, generator=ref.gen(0)).to(F16)
    freqs = ref.turns(64, seed=4)
    want, tol = ref.rope(x, pos, freqs, layout)
    ref.check(sgq.rope(*cuda(x, pos, freqs), layout=layout).cpu(), want, tol + ref.rounding(want.abs() + tol, F16))


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rope_turns_back(layout):
    """Its inverse is its gradient: against differences of the 64-bit form, and <y, R x> = <R^-1 y, x>."""
    T, H, D, R, f = 5, 2, 32, 16, 1.25
    r = ref.gen(3)
    x, dy = torch.randn(T, H, D, generator=r).to(F16), torch.randn(T, H, D, generator=r).to(F16)
    pos, freqs = torch.randint(0, 5000, (T,), generator=r), ref.turns(R)
    dx = sgq.rope(*cuda(dy, pos, freqs), layout=layout, factor=f, inverse=True).cpu()
    _, tol = ref.rope(dy, pos, freqs, layout, f, True)
    loss = lambda v: (ref.rope(v, pos, freqs, layout, f)[0] * dy.double()).sum()  # noqa: E731
    for i in range(0, T * H * D, 7):
        e = torch.zeros(T * H * D, dtype=torch.float64)
        e[i] = 0.5
        e = e.view(T, H, D)
        slope = (loss(x.double() + e) - loss(x.double() - e)).item()
        got, t = dx.flatten()[i].item(), tol.flatten()[i].item()
        assert abs(got - slope) <= t + abs(slope) * 2.0 ** -11 + 2.0 ** -25 + 1e-12


def test_rope_in_place_in_a_projection():
    """q and k side by side in one projection's rows, each turned where it stands; the rest stays."""
    T, Hq, Hk, D = 37, 4, 2, 64
    qkv = torch.randn(T, (Hq + 2 * Hk) * D, generator=ref.gen(1)).to(BF16)
    pos, freqs = torch.arange(T), ref.turns(64)
    d, dp, df = cuda(qkv, pos, freqs)
    heads = d.view(T, -1, D)
    q, k = heads[:, :Hq], heads[:, Hq:Hq + Hk]
    assert sgq.rope(q, dp, df, out=q) is q
    sgq.rope(k, dp, df, out=k)
    want, tol = ref.rope(qkv.view(T, -1, D)[:, :Hq + Hk], pos, freqs)
    ref.check(heads[:, :Hq + Hk].cpu(), want, tol + ref.rounding(want.abs() + tol, BF16))
    assert torch.equal(heads[:, Hq + Hk:].cpu(), qkv.view(T, -1, D)[:, Hq + Hk:])
    # from one part of the rows into another
    out = sgq.rope(heads[:, Hq + Hk:], dp, df, out=heads[:, Hq:Hq + Hk])
    want, tol = ref.rope(qkv.view(T, -1, D)[:, Hq + Hk:], pos, freqs)
    ref.check(out.cpu(), want, tol + ref.rounding(want.abs() + tol, BF16))


def test_rope_of_a_part_of_each_head():
    """The last 64 of 192 columns, by a view."""
    x = torch.randn(50, 3, 192, generator=ref.gen(2)).to(BF16)
    pos, freqs = torch.arange(50) * 1000, ref.turns(64)
    d, dp, df = cuda(x, pos, freqs)
    part = d[..., 128:]
    sgq.rope(part, dp, df, layout="interleaved", out=part)
    want, tol = ref.rope(x[..., 128:], pos, freqs, "interleaved")
    ref.check(d[..., 128:].cpu(), want, tol + ref.rounding(want.abs() + tol, BF16))
    assert torch.equal(d[..., :128].cpu(), x[..., :128])


# ------------------------------------------------------------------ cache_write, cache_read

WRITE = [(1, 1, 1, 16, 16, 16), (5, 4, 2, 64, 64, 1), (64, 8, 8, 128, 128, 16), (33, 7, 1, 80, 32, 20), (300, 6, 3, 256, 128, 64), (701, 2, 2, 96, 48, 3), (2000, 16, 4, 48, 16, 128)]


@pytest.mark.parametrize("T,Hq,H,D,R,P", WRITE)
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("fmt,dtype", KINDS)
@pytest.mark.parametrize("order", ["head", "token"])
def test_cache_write_and_read(T, Hq, H, D, R, P, layout, fmt, dtype, order):
    r = ref.gen(T + D)
    pages = -(-T // P) + 2
    k, v, ks, vs = ref.pool(fmt, pages, H, P, D, dtype, 5, order)
    slots = torch.randperm(pages * P, generator=r)[:T].to(torch.int32 if T % 2 else torch.int64)
    slots[::5] = torch.tensor([-1, pages * P, -(1 << 31), (1 << 31) - 1])[torch.arange(len(slots[::5])) % 4].to(slots.dtype)
    qkv = torch.randn(T, Hq + 2 * H, D, generator=r).to(dtype)
    qkv[T // 2, Hq] = 0                                               # a row of zeros
    pos, freqs, factor = torch.randint(0, 100000, (T,), generator=r), ref.turns(R), 1.2
    dk, dv, dks, dvs, dslots, dqkv, dpos, dfreqs = cuda(k, v, ks, vs, slots, qkv, pos, freqs)
    q, nk, nv = dqkv.split((Hq, H, H), 1)
    out, untouched = guarded((T, Hq, D), dtype)
    got = sgq.cache_write(nk, nv, dk, dv, dslots, fmt=fmt, k_scale=dks, v_scale=dvs, q=q, q_out=out, positions=dpos, freqs=dfreqs, layout=layout, factor=factor)
    assert got is out
    untouched()
    assert torch.equal(dqkv.cpu(), qkv)
    wq, tq = ref.rope(qkv[:, :Hq], pos, freqs, layout, factor)
    ref.check(out.cpu(), wq, tq + ref.rounding(wq.abs() + tq, dtype), "q")
    wk, tk = ref.rope(qkv[:, Hq:Hq + H], pos, freqs, layout, factor)
    wv, tv = qkv[:, Hq + H:].double(), torch.zeros(T, H, D, dtype=torch.float64)
    ok = (slots >= 0) & (slots < pages * P)
    page, place = slots[ok].long() // P, slots[ok].long() % P
    back = sgq.cache_read(dk, dv, dslots, fmt=fmt, k_scale=dks, v_scale=dvs, dtype=dtype)
    for name, old, new, scale, oldscale, (w, t), rows in (("k", k, dk.cpu(), None if dks is None else dks.cpu(), ks, (wk, tk), back[0].cpu()),
                                                          ("v", v, dv.cpu(), None if dvs is None else dvs.cpu(), vs, (wv, tv), back[1].cpu())):
        stored = ref.rows_at(new, scale, page, place)
        if fmt == "none":
            ref.check(stored, w[ok], t[ok] + (ref.rounding(w.abs() + t, dtype)[ok] if name == "k" else 0), name)
        else:
            w8, t8 = ref.quantised(w[ok], t[ok])
            ref.check(stored, w8, t8, name)
            ref.check(scale[page, :, place], w[ok].abs().amax(-1) / 448, w[ok].abs().amax(-1) / 448 * 2.0 ** -23 + t[ok].amax(-1) / 448 + 2.0 ** -149, name + "_scale")
        want = torch.zeros(T, H, D, dtype=torch.float64)
        want[ok] = stored
        ref.check(rows, want, ref.rounding(want, dtype) if fmt != "none" else torch.zeros_like(want), name + " read")
        # rows at other slots stay as they are
        touched = torch.zeros(pages, P, dtype=torch.bool)
        touched[page, place] = True
        bits = lambda c: c.transpose(1, 2).contiguous().view(torch.uint8)[~touched]  # noqa: E731
        assert torch.equal(bits(old), bits(new)), name
        if scale is not None:
            assert torch.equal(oldscale.transpose(1, 2)[~touched], scale.transpose(1, 2)[~touched])


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("T,H,D", [(3, 2, 128), (200, 5, 80), (1500, 1, 256), (9, 3, 16)])
def test_rows_are_quantize_fp8s(T, H, D, dtype):
    """Without rotation the codes and scales of a row are quantize_fp8's, byte for byte: at any size, zeros and subnormal scales too."""
    x = torch.randn(2, T, H, D, generator=ref.gen(D)) * torch.exp2(torch.randint(-14, 14, (2, T, H, 1), generator=ref.gen(1)).float())
    if dtype == BF16:
        x[:, 0] *= 2.0 ** -118
    x[:, -1, 0] = 0
    x = x.to(dtype).to(DEV)
    k, v = torch.empty(2, T, H, 1, D, dtype=torch.uint8, device=DEV)
    ks, vs = torch.empty(2, T, H, 1, device=DEV)
    assert sgq.cache_write(x[0], x[1], k, v, torch.arange(T, device=DEV), fmt="per_token", k_scale=ks, v_scale=vs) is None
    for rows, codes, scale in ((x[0], k, ks), (x[1], v, vs)):
        q, s = sgq.quantize_fp8(rows.reshape(T * H, D), fmt="per_token")
        assert torch.equal(codes.view(T * H, D), q) and torch.equal(scale.view(T * H, 1), s)


@pytest.mark.parametrize("fmt", ["none", "per_token"])
def test_halves_of_each_page(fmt):
    """k and v as the halves of one tensor's pages; q rotated in place in the projection."""
    pages, H, P, D, T = 6, 2, 16, 64, 40
    both = torch.zeros(pages, 2, H, P, D, dtype=BF16 if fmt == "none" else torch.uint8, device=DEV)
    k, v = both[:, 0], both[:, 1]
    ks, vs = (None, None) if fmt == "none" else torch.zeros(2, pages, H, P, device=DEV)
    qkv = torch.randn(T, 8 + 2 * H, D, generator=ref.gen(0)).to(BF16)
    d, pos, freqs = cuda(qkv, torch.arange(T), ref.turns(64))
    q, nk, nv = d.split((8, H, H), 1)
    slots = torch.arange(T, device=DEV, dtype=torch.int32) + 3
    assert sgq.cache_write(nk, nv, k, v, slots, fmt=fmt, k_scale=ks, v_scale=vs, q=q, q_out=q, positions=pos, freqs=freqs) is q
    assert torch.equal(d[:, 8:].cpu(), qkv[:, 8:])
    want, tol = ref.rope(qkv, torch.arange(T), ref.turns(64))
    ref.check(q.cpu(), want[:, :8], (tol + ref.rounding(want.abs() + tol, BF16))[:, :8])
    gk, gv = sgq.cache_read(k, v, slots, fmt=fmt, k_scale=ks, v_scale=vs)
    wk, tk = (want[:, 8:8 + H], tol[:, 8:8 + H]) if fmt == "none" else ref.quantised(want[:, 8:8 + H], tol[:, 8:8 + H])
    ref.check(gk.cpu(), wk, tk + ref.rounding(wk.abs() + tk, BF16))
    wv, tv = (qkv[:, 8 + H:].double(), torch.zeros(T, H, D)) if fmt == "none" else ref.quantised(qkv[:, 8 + H:].double())
    ref.check(gv.cpu(), wv, tv + (ref.rounding(wv.abs() + tv, BF16) if fmt != "none" else 0))


def test_cache_read_names_a_slot_often_and_in_any_type():
    k, v, ks, vs = ref.pool("per_token", 5, 3, 8, 48, BF16, 2)
    slots = torch.tensor([3, 3, -1, 39, 0, 40, 3, 1 << 40])
    for dtype in (BF16, F16):
        gk, gv = sgq.cache_read(*cuda(k, v, slots), fmt="per_token", k_scale=ks.to(DEV), v_scale=vs.to(DEV), dtype=dtype)
        for got, c, s in ((gk, k, ks), (gv, v, vs)):
            want = torch.zeros(8, 3, 48, dtype=torch.float64)
            ok = (slots >= 0) & (slots < 40)
            want[ok] = ref.rows_at(c, s, slots[ok] // 8, slots[ok] % 8)
            ref.check(got.cpu(), want, ref.rounding(want, dtype))
    only, untouched = guarded((8, 3, 48), BF16)
    sgq.cache_read(*cuda(k, v, slots), fmt="per_token", k_scale=ks.to(DEV), v_scale=vs.to(DEV), k_out=only)
    untouched()


# ------------------------------------------------------------------ paged_attention

def attend(fmt, dtype, lengths, heads, group, D, P, *, order="head", window=0, sinks=False, scale=None, width=None, seed=0, spread=1.0, change=None,
           cache=None, norm=False):
    """paged_attention against the plain form, with guard bands; every row that is masked or not in use holds NaN."""
    B, Hq = len(lengths), heads * group
    table, pages = ref.table_of(lengths, P, width, seed)
    k, v, ks, vs = ref.pool(fmt, pages, heads, P, D, dtype, seed, order) if cache is None else cache(pages)
    q = (torch.randn(B, Hq, D, generator=ref.gen(seed + 9)) * spread).to(dtype)
    n = torch.tensor(lengths, dtype=torch.int32)
    if change:
        table, n = change(table, n)
    used = torch.zeros(pages, P, dtype=torch.bool)
    for b in range(B):
        used[ref.tokens(b, table, n, window, pages, P)] = True
    for t, s in ((k, ks), (v, vs)):
        if s is None:
            t.transpose(1, 2)[~used] = math.nan
        else:
            t.transpose(1, 2)[~used] = 0x7F
            s.transpose(1, 2)[~used] = math.nan
    sk = torch.randn(Hq, generator=ref.gen(seed + 3)) * 2 if sinks else None
    want, tol, wl, tl = ref.attention(q, k, v, ks, vs, table, n, scale, window, sk)
    what = f"{fmt} {dtype} {lengths} H={heads}x{group} D={D} P={P} window={window}"
    none = wl == -math.inf
    # the table as it is, and one for long sequences, which CTAs share (a window's items are short all the same)
    room = 0
    for wide in (table, torch.nn.functional.pad(table, (0, -(-60000 // P)), value=-1)) if int(n.max()) <= table.shape[1] * P else (table,):
        out, uo = guarded((B, Hq, D), dtype)
        lse, ul = guarded((B, Hq), torch.float32)
        room = sgq.attention_workspace_bytes(fmt, B, Hq, heads, D, wide.shape[1], P, window)
        ws, uw = guarded((room,), torch.uint8)
        dq, dk, dv, dks, dvs, dt, dn, dsk = cuda(q, k, v, ks, vs, wide, n, sk)
        kw = dict(fmt=fmt, k_scale=dks, v_scale=dvs, scale=scale, window=window, sinks=dsk)
        got = sgq.paged_attention(dq, dk, dv, dt, dn, out=out, lse=lse, workspace=ws, **kw)
        torch.cuda.synchronize()
        assert got[0] is out and got[1] is lse
        uo(), ul(), uw()
        ref.check(out.cpu(), want, tol, what)
        assert (lse.cpu()[none] == -math.inf).all()
        ref.check(lse.cpu()[~none], wl[~none], tl[~none], what + " lse")
        again = sgq.paged_attention(dq, dk, dv, dt, dn, **kw)
        assert torch.equal(again.view(torch.int16), out.view(torch.int16)), "two runs differ"
        if norm:
            assert ref.off_by_rounding(out.cpu(), want) < 1.1
    assert room or window or wide is table
    return out.cpu(), want


BORDERS = [0, 1, 2, 15, 16, 17, 31, 33, 63, 64, 65, 80, 127, 128, 129, 191, 193, 300]


@pytest.mark.parametrize("fmt,dtype", KINDS)
@pytest.mark.parametrize("D", [16, 48, 64, 80, 128, 192, 256])
@pytest.mark.parametrize("P", [1, 16, 20])
def test_attention_at_every_border(fmt, dtype, D, P):
    attend(fmt, dtype, BORDERS, 2, 4, D, P, seed=D + P)


@pytest.mark.parametrize("fmt,dtype", KINDS)
@pytest.mark.parametrize("group", [1, 2, 3, 7, 8, 9, 16, 17, 40])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_attention_groups(fmt, dtype, group, D):
    attend(fmt, dtype, [130, 0, 1, 77], 3, group, D, 16, seed=group)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("D", [8, 24, 72, 136, 248])
def test_attention_of_16_bit_heads_of_odd_widths(dtype, D):
    attend("none", dtype, [100, 3, 0, 64], 2, 5, D, 8, seed=D)


@pytest.mark.parametrize("fmt,dtype", KINDS)
@pytest.mark.parametrize("window", [1, 2, 16, 63, 64, 65, 100, 1000])
@pytest.mark.parametrize("sinks", [False, True])
def test_attention_windows_and_sinks(fmt, dtype, window, sinks):
    attend(fmt, dtype, BORDERS, 2, 3, 64, 16, window=window, sinks=sinks, seed=window)


@pytest.mark.parametrize("fmt,dtype", KINDS)
@pytest.mark.parametrize("order", ["head", "token"])
@pytest.mark.parametrize("P", [1, 3, 8, 16, 48, 64, 256])
def test_attention_orders_and_pages(fmt, dtype, order, P):
    attend(fmt, dtype, [5, 257, 64, 0, 1000], 3, 4, 128, P, order=order, seed=P)


@pytest.mark.parametrize("fmt,dtype", KINDS)
@pytest.mark.parametrize("sms", [1, 2, 3, 7, 152])
def test_attention_shares(fmt, dtype, sms):
    """Few CTAs walk over many items, many share one item; sequences of no token at the ends and between."""
    with planned_for(sms):
        attend(fmt, dtype, [0, 0, 700, 1, 0, 64, 65, 3000, 0, 129, 0], 2, 4, 128, 16, seed=sms)
        attend(fmt, dtype, [4000], 1, 8, 64, 16, seed=sms)
        attend(fmt, dtype, [0], 1, 1, 64, 16, width=3, seed=sms)


@pytest.mark.parametrize("fmt,dtype", KINDS)
@pytest.mark.parametrize("D", [64, 128, 256])
def test_attention_long_sequences_are_summed_in_32_bits(fmt, dtype, D):
    """Two q heads' worth of spread and none: the error is that of the one rounding at the end."""
    attend(fmt, dtype, [20000, 12345], 2, 8, D, 64, seed=D, norm=True)
    attend(fmt, dtype, [9001], 2, 16, D, 32, seed=D, spread=4.0, norm=True)


@pytest.mark.parametrize("fmt,dtype", KINDS)
@pytest.mark.parametrize("D", [64, 128, 256])
def test_attention_long_windows(fmt, dtype, D):
    """Windows of many tiles, that begin anywhere in one."""
    attend(fmt, dtype, [20001, 9000, 8999, 17], 1, 8, D, 16, window=9000, sinks=True, seed=D)


@pytest.mark.parametrize("fmt,dtype", KINDS)
@pytest.mark.parametrize("P,lengths", [(4096, [4096, 4097, 100]), (65536, [5000]), (2048, [1])])
def test_attention_large_pages(fmt, dtype, P, lengths):
    attend(fmt, dtype, lengths, 1, 2, 64, P, seed=P)


@pytest.mark.parametrize("fmt,dtype", KINDS)
@pytest.mark.parametrize("P", [16, 5])
def test_attention_of_a_part_of_each_row(fmt, dtype, P):
    """Heads that lie in the first columns of wider rows, of every second page; one query for all sequences."""
    def part(pages):
        k, v, ks, vs = ref.pool(fmt, 2 * pages, 2, P, 96, dtype, 0)
        return (*(t[::2, :, :, :80] for t in (k, v)), *(t if t is None else t[::2].contiguous() for t in (ks, vs)))
    attend(fmt, dtype, [200, 0, 77], 2, 3, 80, P, cache=part)
    table, pages = ref.table_of([200, 0, 77], P)
    k, v, ks, vs = part(pages)
    q = torch.randn(1, 6, 80, generator=ref.gen(0)).to(dtype)
    n = torch.tensor([200, 0, 77], dtype=torch.int32)
    want, tol, _, _ = ref.attention(q.expand(3, -1, -1), k, v, ks, vs, table, n)
    dq, dk, dv, dks, dvs, dt, dn = cuda(q, k, v, ks, vs, table, n)
    ref.check(sgq.paged_attention(dq.expand(3, -1, -1), dk, dv, dt, dn, fmt=fmt, k_scale=dks, v_scale=dvs).cpu(), want, tol)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("P", [16, 64])
def test_attention_scales_on_any_4_bytes(dtype, P):
    """Scales that no 16-byte copy can bring, of k, of v or of both."""
    lengths = [200, 0, 77, 64]
    table, pages = ref.table_of(lengths, P)
    k, v, ks, vs = ref.pool("per_token", pages, 2, P, 80, dtype, 0)
    q = torch.randn(4, 6, 80, generator=ref.gen(0)).to(dtype)
    n = torch.tensor(lengths, dtype=torch.int32)
    want, tol, _, _ = ref.attention(q, k, v, ks, vs, table, n)
    dq, dk, dv, dt, dn = cuda(q, k, v, table, n)
    for at_k, at_v in ((1, 0), (0, 3), (2, 2)):
        sk, sv = (torch.full((s.numel() + 4,), math.nan, device=DEV) for s in (ks, vs))
        sk, sv = sk[at_k:at_k + ks.numel()].view(ks.shape), sv[at_v:at_v + vs.numel()].view(vs.shape)
        sk.copy_(ks), sv.copy_(vs)
        ref.check(sgq.paged_attention(dq, dk, dv, dt, dn, fmt="per_token", k_scale=sk, v_scale=sv).cpu(), want, tol)


@pytest.mark.parametrize("fmt,dtype", KINDS)
@pytest.mark.parametrize("heads", [1, 3])
@pytest.mark.parametrize("sinks", [False, True])
def test_attention_of_a_padded_batch(fmt, dtype, heads, sinks):
    """Most sequences, or all of them, are empty: their rows are zeros, whoever writes them."""
    attend(fmt, dtype, [0] * 9 + [700] + [0] * 25 + [65, 1] + [0] * 12 + [3000], heads, 2, 64, 16, sinks=sinks)
    attend(fmt, dtype, [0] * 400 + [700] + [0] * 100 + [300, 1], heads, 9, 48, 16, sinks=sinks)
    attend(fmt, dtype, [0] * 200, heads, 8, 128, 16, width=3, sinks=sinks)


@pytest.mark.parametrize("fmt,dtype", KINDS)
def test_attention_many_sequences(fmt, dtype):
    attend(fmt, dtype, [(7 * i) % 40 for i in range(1500)], 1, 2, 64, 16, seed=1)
    with planned_for(5):
        attend(fmt, dtype, [(11 * i) % 150 for i in range(333)], 2, 1, 64, 8, seed=2)


@pytest.mark.parametrize("fmt,dtype", KINDS)
def test_attention_lengths_outside_and_wild_pages(fmt, dtype):
    """Lengths are held to the table's width, pages outside the cache mask their tokens."""
    def wild(table, n):
        table = table.clone()
        table[0, 1], table[1, 0], table[2, 2], table[3, :] = 1 << 20, -5, (1 << 31) - 1, -(1 << 31)
        n = n.clone()
        n[4], n[5] = -3, (1 << 31) - 1
        return table, n
    attend(fmt, dtype, [100, 90, 300, 50, 40, 320, 17], 2, 4, 80, 16, change=wild, sinks=True)
    attend(fmt, dtype, [100, 90, 300, 50, 40, 320, 17], 2, 4, 80, 16, change=wild)


@pytest.mark.parametrize("fmt,dtype", KINDS)
def test_attention_shares_pages(fmt, dtype):
    """A prefix that all sequences share."""
    def shared(table, n):
        table = table.clone()
        table[:, :5] = table[0, :5]
        return table, n
    attend(fmt, dtype, [100, 90, 300, 81], 2, 4, 64, 16, change=shared)


@pytest.mark.parametrize("fmt,dtype", KINDS)
@pytest.mark.parametrize("spread", [0.0, 30.0])
def test_attention_flat_and_peaked(fmt, dtype, spread):
    """Equal logits, and logits hundreds apart, rising and falling along the sequence: the maximum moves often."""
    def rising(pages):
        k, v, ks, vs = ref.pool(fmt, pages, 2, 16, 64, dtype, 0)
        size = torch.linspace(0.05, 2.0, pages).view(-1, 1, 1, 1)
        k = (k.float() * size).to(dtype) if fmt == "none" else k
        return k, v, ks if ks is None else ks * size.squeeze(-1), vs
    attend(fmt, dtype, [600, 40, 333], 2, 4, 64, 16, spread=spread, cache=rising)


@pytest.mark.parametrize("dtype", [BF16, F16])
def test_attention_where_scales_differ_widely(dtype):
    """Rows of zeros with a scale of 0, rows that differ by 2^20 in size, and a first row that has all the
    weight and a small value."""
    def rows(pages):
        k, v, ks, vs = ref.pool("per_token", pages, 2, 16, 64, dtype, 0)
        vs = vs * torch.exp2(torch.randint(-20, 1, vs.shape, generator=ref.gen(4)).float())
        k[0], ks[0], v[1], vs[1] = 0, 0.0, 0, 0.0
        return k, v, ks, vs
    attend("per_token", dtype, [600, 40, 333], 2, 4, 64, 16, cache=rows)
    for low, high in ((-90, -85), (30, 35)):
        def scaled(pages, low=low, high=high):
            k, v, ks, vs = ref.pool("per_token", pages, 2, 16, 64, dtype, 0)
            return k, v, ks, torch.exp2(torch.randint(low, high, vs.shape, generator=ref.gen(4)).float())
        if dtype == BF16:
            attend("per_token", dtype, [200, 40], 2, 4, 64, 16, cache=scaled)


def test_attention_bf16_q_of_any_size_beside_fp8_rows():
    """A head of zeros, heads 2^60 apart, a head with one large value."""
    B, Hq, D = 3, 8, 64
    table, pages = ref.table_of([100, 17, 64], 16)
    k, v, ks, vs = ref.pool("per_token", pages, 2, 16, D, BF16, 0)
    q = torch.randn(B, Hq, D, generator=ref.gen(0))
    q[:, 0], q[:, 1], q[:, 5], q[0, 2, 7] = 0, q[:, 1] * 2.0 ** -60, q[:, 5] * 2.0 ** -126, 300.0
    q = q.to(BF16)
    n = torch.tensor([100, 17, 64], dtype=torch.int32)
    want, tol, wl, tl = ref.attention(q, k, v, ks, vs, table, n)
    out, lse = sgq.paged_attention(*cuda(q, k, v, table, n), fmt="per_token", k_scale=ks.to(DEV), v_scale=vs.to(DEV), lse=True)
    ref.check(out.cpu(), want, tol)
    ref.check(lse.cpu(), wl, tl)


@pytest.mark.parametrize("fmt,dtype", KINDS)
def test_attention_strided_queries_and_halves_of_pages(fmt, dtype):
    lengths, H, g, D, P = [100, 0, 260], 2, 4, 64, 16
    table, pages = ref.table_of(lengths, P)
    k, v, ks, vs = ref.pool(fmt, pages, H, P, D, dtype, 1)
    qkv = torch.randn(3, H * g + 2 * H, D, generator=ref.gen(2)).to(dtype)
    n = torch.tensor(lengths, dtype=torch.int32)
    both = torch.stack((k, v), 1).to(DEV)
    d, dt, dn, dks, dvs = cuda(qkv, table, n, ks, vs)
    out = sgq.paged_attention(d[:, :H * g], both[:, 0], both[:, 1], dt, dn, fmt=fmt, k_scale=dks, v_scale=dvs)
    want, tol, _, _ = ref.attention(qkv[:, :H * g], k, v, ks, vs, table, n)
    ref.check(out.cpu(), want, tol)


@pytest.mark.parametrize("fmt", ["none", "per_token"])
def test_attention_beyond_32_bit_offsets(fmt):
    """A cache whose last pages begin behind 2^32 bytes, read, written and attended there."""
    H, P, D = 8, 16, 256
    pages = (1 << 32) // (H * P * D * (2 if fmt == "none" else 1)) + 40
    dt = BF16 if fmt == "none" else torch.uint8
    k, v = (torch.zeros(pages, H, P, D, dtype=dt, device=DEV) for _ in range(2))
    ks, vs = (None, None) if fmt == "none" else torch.zeros(2, pages, H, P, device=DEV)
    n = 200
    table = torch.arange(pages - 13, pages, dtype=torch.int32).view(1, 13)
    slots = (table.view(-1, 1).long() * P + torch.arange(P)).flatten()[:n]
    rows = torch.randn(2, n, H, D, generator=ref.gen(0)).to(BF16)
    dk, dv, dslots, dtable = cuda(rows[0], rows[1], slots, table)
    sgq.cache_write(dk, dv, k, v, dslots, fmt=fmt, k_scale=ks, v_scale=vs)
    gk, gv = sgq.cache_read(k, v, dslots, fmt=fmt, k_scale=ks, v_scale=vs)
    for got, x in ((gk, rows[0]), (gv, rows[1])):
        w, t = (x.double(), torch.zeros(1)) if fmt == "none" else ref.quantised(x.double())
        ref.check(got.cpu(), w, t + (ref.rounding(w.abs() + t, BF16) if fmt != "none" else torch.zeros(1)))
    q = torch.randn(1, 16, D, generator=ref.gen(1)).to(BF16)
    dn = torch.tensor([n], dtype=torch.int32, device=DEV)
    out = sgq.paged_attention(q.to(DEV), k, v, dtable, dn, fmt=fmt, k_scale=ks, v_scale=vs)
    last = slice(pages - 13, pages)
    cpu = [None if t is None else t[last].cpu() for t in (k, v, ks, vs)]
    want, tol, _, _ = ref.attention(q, *cpu, torch.arange(13, dtype=torch.int32).view(1, 13), torch.tensor([n]))
    ref.check(out.cpu(), want, tol)


# ------------------------------------------------------------------ calls

@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rows_that_pass_l2_by(layout):
    """Large calls ask for rows ahead: the same rows as in pieces."""
    T, Hq, H, D = 7001, 32, 4, 128
    r = torch.Generator(device=DEV).manual_seed(0)
    qkv = torch.randn(T, Hq + 2 * H, D, generator=r, device=DEV).to(BF16)
    assert 2 * qkv.numel() * 2 > 128 << 20
    slots = torch.randperm(T, generator=r, device=DEV)
    positions = torch.randint(0, 1 << 30, (T,), generator=r, device=DEV)
    freqs = ref.turns(64).to(DEV)
    pieces = [slice(0, 1), slice(1, 2048), slice(2048, 5000), slice(5000, T)]
    whole = sgq.rope(qkv, positions, freqs, layout=layout)
    assert torch.equal(whole, torch.cat([sgq.rope(qkv[p], positions[p], freqs, layout=layout) for p in pieces]))
    for fmt in ("none", "per_token"):
        def cache():
            k, v = (torch.zeros(T // 16 + 1, H, 16, D, dtype=BF16 if fmt == "none" else torch.uint8, device=DEV) for _ in range(2))
            ks, vs = (None, None) if fmt == "none" else torch.zeros(2, *k.shape[:3], device=DEV)
            return k, v, ks, vs

        def put(c, p):
            d = qkv[p]
            return sgq.cache_write(d[:, Hq:Hq + H], d[:, Hq + H:], c[0], c[1], slots[p], fmt=fmt, k_scale=c[2], v_scale=c[3], q=d[:, :Hq],
                                   positions=positions[p], freqs=freqs, layout=layout)
        one, many = cache(), cache()
        q = put(one, slice(0, T))
        assert torch.equal(q, torch.cat([put(many, p) for p in pieces])) and torch.equal(q, whole[:, :Hq])
        assert all(a is None or torch.equal(a, b) for a, b in zip(one, many))


def test_calls_of_no_rows():
    k, v, _, _ = ref.pool("none", 2, 2, 16, 64, BF16, 0)
    dk, dv = cuda(k, v)
    none = torch.empty(0, 2, 64, dtype=BF16, device=DEV)
    idx = torch.empty(0, dtype=torch.int32, device=DEV)
    freqs = ref.turns(64).to(DEV)
    assert sgq.rope(none, idx, freqs).shape == (0, 2, 64)
    assert sgq.cache_write(none, none, dk, dv, idx, q=none, positions=idx, freqs=freqs).shape == (0, 2, 64)
    assert sgq.cache_read(dk, dv, idx)[0].shape == (0, 2, 64)
    assert sgq.paged_attention(none, dk, dv, idx.view(0, 1).expand(0, 3).contiguous(), idx).shape == (0, 2, 64)
    out, lse = sgq.paged_attention(torch.ones(3, 4, 64, dtype=BF16, device=DEV), dk, dv, torch.empty(3, 0, dtype=torch.int32, device=DEV),
                                   torch.full((3,), 7, dtype=torch.int32, device=DEV), lse=True)
    assert (out == 0).all() and (lse == -math.inf).all()
    assert torch.equal(dk.cpu(), k)


@pytest.mark.parametrize("fmt,dtype", KINDS)
def test_a_graph_follows_lengths_tables_and_slots(fmt, dtype):
    """A captured decode step, replayed over inputs that change between replays; two graphs, a workspace each."""
    B, H, g, D, P, width = 5, 2, 4, 64, 16, 12
    r = ref.gen(0)
    k, v, ks, vs = ref.pool(fmt, B * width, H, P, D, dtype, 3)
    dk, dv, dks, dvs = cuda(k, v, ks, vs)
    table = torch.randperm(B * width, generator=r).to(torch.int32).view(B, width)
    dt = table.to(DEV)
    freqs = ref.turns(64)
    dfreqs = freqs.to(DEV)
    qkv = torch.zeros(B, H * g + 2 * H, D, dtype=dtype, device=DEV)
    q, nk, nv = qkv.split((H * g, H, H), 1)
    pos, slots, n = (torch.zeros(B, dtype=d, device=DEV) for d in (torch.int64, torch.int64, torch.int32))

    def a_step():
        turned = sgq.cache_write(nk, nv, dk, dv, slots, fmt=fmt, k_scale=dks, v_scale=dvs, q=q, positions=pos, freqs=dfreqs)
        return sgq.paged_attention(turned, dk, dv, dt, n, fmt=fmt, k_scale=dks, v_scale=dvs, window=100), turned
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        n.fill_(1)
        a_step()
        st.synchronize()
        graphs = []
        for _ in range(2):
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=st):
                graphs.append((graph, *a_step()))
        st.synchronize()
        for turn in range(6):
            at = torch.randint(0, width * P, (B,), generator=r)
            new = torch.randn(B, H * g + 2 * H, D, generator=r).to(dtype)
            graph, out, turned = graphs[turn % 2]
            qkv.copy_(new), pos.copy_(at), n.copy_(at + 1)
            slots.copy_(table[torch.arange(B), at // P].long() * P + at % P)
            graph.replay()
            st.synchronize()
            want, tol, _, _ = ref.attention(turned.cpu(), dk.cpu(), dv.cpu(), None if ks is None else dks.cpu(), None if vs is None else dvs.cpu(), table, at + 1, window=100)
            ref.check(out.cpu(), want, tol, f"turn {turn}")
            wq, tq = ref.rope(new[:, :H * g], at, freqs)
            ref.check(turned.cpu(), wq, tq + ref.rounding(wq.abs() + tq, dtype))


def test_calls_at_once_on_streams():
    """Long and short calls of every format on four streams, each of them right."""
    cases = []
    for i, (fmt, dtype) in enumerate(KINDS):
        lengths = [3000 + 100 * i, 0, 17]
        table, pages = ref.table_of(lengths, 16, seed=i)
        k, v, ks, vs = ref.pool(fmt, pages, 2, 16, 128, dtype, i)
        q = torch.randn(3, 16, 128, generator=ref.gen(i)).to(dtype)
        n = torch.tensor(lengths, dtype=torch.int32)
        want = ref.attention(q, k, v, ks, vs, table, n)
        cases.append((cuda(q, k, v, table, n), dict(fmt=fmt, k_scale=cuda(ks)[0], v_scale=cuda(vs)[0]), want))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    outs = [[] for _ in cases]
    for _ in range(10):
        for i, (args, kw, _) in enumerate(cases):
            outs[i].append(sgq.paged_attention(*args, **kw, stream=streams[i]))
    torch.cuda.synchronize()
    for got, (_, _, (want, tol, _, _)) in zip(outs, cases):
        ref.check(got[0].cpu(), want, tol)
        assert all(torch.equal(got[0], o) for o in got)


@pytest.mark.parametrize("fmt,dtype", KINDS)
def test_a_prompt_then_steps(fmt, dtype):
    """A prompt written in two chunks, read back as a library's attention would, then six steps, against dense
    attention in 64 bits on what the cache holds."""
    H, g, D, P, R = 2, 3, 80, 16, 32
    freqs, factor = sgq.rope_frequencies(R, 10000.0, scaling="yarn", stretch=4.0, trained=64, device=DEV)
    pages = torch.randperm(9, generator=ref.gen(0)).to(torch.int32)[:5]
    table = pages.view(1, 5).to(DEV)
    shape = (9, H, P, D)
    k, v = (torch.zeros(shape, dtype=dtype if fmt == "none" else torch.uint8, device=DEV) for _ in range(2))
    ks, vs = (None, None) if fmt == "none" else torch.zeros(2, *shape[:3], device=DEV)
    kw = dict(fmt=fmt, k_scale=ks, v_scale=vs)
    place = lambda t: pages[t // P].long() * P + t % P  # noqa: E731
    r = ref.gen(7)
    keys, values = [], []

    def put(t0, n):
        qkv = torch.randn(n, H * g + 2 * H, D, generator=r).to(dtype)
        t = torch.arange(t0, t0 + n)
        d = qkv.to(DEV)
        q = sgq.cache_write(d[:, H * g:H * g + H], d[:, H * g + H:], k, v, place(t).to(DEV), q=d[:, :H * g], positions=t.to(DEV), freqs=freqs, factor=factor, **kw)
        keys.append(ref.rope(qkv[:, H * g:H * g + H], t, freqs.cpu(), factor=factor))
        values.append(qkv[:, H * g + H:].double())
        return q
    put(0, 33), put(33, 20)
    for i in range(6):
        q = put(53 + i, 1)
        n = 54 + i
        t = torch.arange(n)
        gk, gv = sgq.cache_read(k, v, place(t).to(DEV), dtype=dtype, **kw)
        wk, tk = torch.cat([a for a, _ in keys]), torch.cat([b for _, b in keys])
        wv, tv = torch.cat(values), torch.zeros(1)
        if fmt != "none":
            (wk, tk), (wv, tv) = ref.quantised(wk, tk), ref.quantised(wv)
        ref.check(gk.cpu(), wk, tk + ref.rounding(wk.abs() + tk, dtype))
        ref.check(gv.cpu(), wv, tv + (ref.rounding(wv.abs() + tv, dtype) if fmt != "none" else torch.zeros(1)))
        out = sgq.paged_attention(q, k, v, table, torch.tensor([n], dtype=torch.int32, device=DEV), **kw)
        cpu = [None if x is None else x.cpu() for x in (k, v, ks, vs)]
        want, tol, _, _ = ref.attention(q.cpu(), *cpu, table.cpu(), torch.tensor([n]))
        ref.check(out.cpu(), want, tol)


def test_an_attention_layers_step_in_fp8():
    """norm -> FP8 projection -> cache_write -> paged_attention -> FP8 rows -> projection: each step's rows are the next one's."""
    B, hidden, H, g, D, P = 6, 256, 2, 4, 64, 16
    r = ref.gen(0)
    width = (H * g + 2 * H) * D
    x = torch.randn(B, hidden, generator=r).to(BF16).to(DEV)
    w1 = (torch.randn(width, hidden, generator=r) / 16).to(BF16).to(DEV)
    w2 = (torch.randn(hidden, H * g * D, generator=r) / 22).to(BF16).to(DEV)
    one = torch.tensor([0, B], dtype=torch.int32, device=DEV)
    q8, s8, _, _ = sgq.rmsnorm_add_quant(x, torch.zeros(hidden, dtype=BF16, device=DEV), fmt="per_token")
    w8, ws = sgq.quantize_fp8(w1, fmt="per_token")
    qkv = sgq.grouped_gemm(q8, w8.view(1, width, hidden), one, fmt="per_token", x_scale=s8, w_scale=ws.view(1, width)).view(B, -1, D)
    lengths = torch.tensor([20, 1, 64, 33, 7, 80])
    table, pages = ref.table_of(lengths.tolist(), P)
    k, v, ks, vs = cuda(*ref.pool("per_token", pages, H, P, D, BF16, 1))
    at = lengths - 1
    slots = (table[torch.arange(B), at // P].long() * P + at % P).to(DEV)
    freqs, _ = sgq.rope_frequencies(D, 10000.0, device=DEV)
    kw = dict(fmt="per_token", k_scale=ks, v_scale=vs)
    q = sgq.cache_write(qkv[:, H * g:H * g + H], qkv[:, H * g + H:], k, v, slots, q=qkv[:, :H * g], positions=at.to(DEV), freqs=freqs, **kw)
    out = sgq.paged_attention(q, k, v, table.to(DEV), lengths.to(torch.int32).to(DEV), **kw)
    want, tol, _, _ = ref.attention(q.cpu(), k.cpu(), v.cpu(), ks.cpu(), vs.cpu(), table, lengths)
    ref.check(out.cpu(), want, tol)
    wk, tk = ref.quantised(*ref.rope(qkv[:, H * g:H * g + H].cpu(), at, freqs.cpu()))
    gk, _ = sgq.cache_read(k, v, slots, **kw)
    ref.check(gk.cpu(), wk, tk + ref.rounding(wk.abs() + tk, BF16))
    o8, os_ = sgq.quantize_fp8(out.view(B, H * g * D), fmt="per_token")
    v8, vs8 = sgq.quantize_fp8(w2, fmt="per_token")
    y = sgq.grouped_gemm(o8, v8.view(1, hidden, -1), one, fmt="per_token", x_scale=os_, w_scale=vs8.view(1, hidden))
    ov, wv = ref.fp8(o8.cpu()) * os_.cpu().double(), ref.fp8(v8.cpu()) * vs8.cpu().double()
    ref.check(y.cpu(), ov @ wv.T, H * g * D * 2.0 ** -22 * (ov.abs() @ wv.abs().T) + ref.rounding(ov @ wv.T, BF16))
